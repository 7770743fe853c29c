"""Workspaces of dspark_markov_grad, which a program keeps for the largest of its calls."""
import ctypes

import pytest

pytest.importorskip("torch")


@pytest.fixture(scope="module")
def size():
    from speculative_decoding_dspark_gb300 import build
    try:
        build.nvcc()
    except RuntimeError:
        pytest.skip("nvcc not available")
    f = ctypes.CDLL(build.build()).dspark_workspace_size
    f.restype, f.argtypes = ctypes.c_size_t, [ctypes.c_int] * 7 + [ctypes.c_uint]
    return lambda V, rank, rows: f(6, 0, 0, V, rank, rows, 1, 0)


@pytest.mark.parametrize("V,rank", [(64, 64), (8000, 64), (32000, 256), (129280, 512), (151936, 512), (1 << 22, 320)])
def test_more_rows_take_no_less(size, V, rank):
    """What holds a call of many rows holds one of fewer."""
    last = 0
    for rows in [*range(0, 1300), *range(1300, 20000, 61), 1 << 18, 1 << 19]:
        now = size(V, rank, rows)
        assert now >= last, rows
        last = now
