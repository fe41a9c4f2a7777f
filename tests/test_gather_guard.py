"""The bounds-checked build's guard on the rows that decode_attn_chunk lays out: of a buffer that is said to end a row early no byte of
that row is written, and the error word tells. (The buffer has the row: nothing is written past memory.)"""
import ctypes
import os
import subprocess

import pytest
import torch

from decode_attention_output_gb300 import build
from test_bounds_checked import BOUNDS_BIT, DEV, _checked_library  # noqa: F401

pytestmark = pytest.mark.gpu

HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.fixture(scope="module")
def one_tile(tmp_path_factory, _checked_library):  # noqa: F811
    path, checked = str(tmp_path_factory.mktemp("guard") / "gather_guard.so"), build.lib_path(checked=True)
    subprocess.run([build.nvcc(), *build.ARCH, "-std=c++17", "-Xcompiler", "-fPIC", "-shared", f"-I{build.INCLUDE}", f"-I{build.CSRC}",
                    os.path.join(HERE, "gather_guard.cu"), checked, "-Xlinker", f"-rpath={os.path.dirname(checked)}", "-o", path], check=True)
    fn = ctypes.CDLL(path).gather_one_tile
    fn.argtypes = [ctypes.c_void_p] * 9 + [ctypes.c_int, ctypes.c_int64, ctypes.c_void_p]
    return fn


@pytest.mark.parametrize("kv8", [False, True])
@pytest.mark.parametrize("rows", [128, 127, 1])
def test_rows_past_the_end_are_reported_and_not_written(one_tile, kv8, rows):
    g = torch.Generator().manual_seed(5)
    tokens = torch.randint(-8, 9, (2, 128, 128), generator=g).float()  # exact in both kinds
    pools = [t.view(8, 1, 16, 128).to(DEV).to(torch.float8_e4m3fn if kv8 else torch.bfloat16) for t in tokens]
    scales = torch.ones((8, 1, 2, 16), device=DEV)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
    c, lens, table, err = i32([0, 1]), i32([128]), i32([list(range(8))]), i32([0])
    outs = [torch.full((128, 128), 77.0, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    status = one_tile(*(t.data_ptr() for t in (*pools, scales, c, lens, table, *outs, err)), int(kv8), rows * 128,
                      torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    assert status == 0 and int(err) == (0 if rows == 128 else BOUNDS_BIT)
    for out, t in zip(outs, tokens):
        assert torch.equal(out[:rows].float().cpu(), t[:rows])
        assert (out[rows:] == 77.0).all()
