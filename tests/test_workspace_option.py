"""The option that limits the workspace's blocks."""
import pytest

import decode_attention_output_gb300 as da
from test_abi import lib  # noqa: F401


def test_default_and_range(lib):  # noqa: F811
    assert da.decode_attn_get_option("workspace_mib") == 0
    for bad in (-1, (1 << 20) + 1):
        with pytest.raises(da.DecodeAttnError):
            da.decode_attn_set_option("workspace_mib", bad)
        assert da.decode_attn_get_option("workspace_mib") == 0
    da.decode_attn_set_option("workspace_mib", 1 << 20)
    assert da.decode_attn_get_option("workspace_mib") == 1 << 20
    da.decode_attn_set_option("workspace_mib", 0)
