"""A wait of the attention kernels that runs out: the call ends soon after the limit and reports DSPARK_ERR_TIMEOUT, whatever
work its CTAs still had before them, and the next call is as good as ever.

The library's test injection keeps the queries of every item from being complete, so the products wait for them until the
limit of 2 s; all other warps wait for the products, on one another or far ahead of them."""
import time

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

from test_gpu_attention import B, attend, attention_case  # noqa: E402,F401

LIMIT_S = 2.0


@pytest.mark.parametrize("n,kv_len,page,hq,hkv,d,shared", [
    ([1], [0], 16, 1, 1, 64, None),
    ([8] * 60, [700] * 60, 16, 8, 2, 128, None),          # many items to a CTA, four copies of each row
    ([8] * 60, [700] * 60, 12, 8, 2, 64, None),           # rows gathered one by one
    ([40], [60000], 16, 8, 1, 128, None),                 # two tiles over dozens of blocks to a CTA
    ([5] * 20, [1024 + 50] * 20, 16, 16, 2, 64, 1024),
])
def test_a_wait_that_runs_out(B, n, kv_len, page, hq, hkv, d, shared):
    q, kc, vc, table, cu = attention_case(41, n, kv_len, page, hq, hkv, d)
    groups = None
    if shared:
        table[:, :shared // page] = table[0, :shared // page]
        groups = ([0, len(n)], [shared])
    want, wz, status = attend(B, q, kc, vc, table, kv_len, cu, groups=groups)
    assert status == 0
    assert B.dspark_set_fault_injection(B.DSPARK_INJECT_ATTENTION_QUERIES) == 0
    try:
        start = time.monotonic()
        _, _, status = attend(B, q, kc, vc, table, kv_len, cu, groups=groups)
        took = time.monotonic() - start
    finally:
        assert B.dspark_set_fault_injection(0) == B.DSPARK_INJECT_ATTENTION_QUERIES
    assert status == B.DSPARK_ERR_TIMEOUT
    assert LIMIT_S <= took < LIMIT_S + 1.0
    out, z, status = attend(B, q, kc, vc, table, kv_len, cu, groups=groups)
    assert status == 0 and torch.equal(out, want) and torch.equal(z, wz)


def test_the_limit_of_the_grid_waits_is_not_theirs(B):
    """A short limit for the grid-wide waits leaves the attention's alone."""
    q, kc, vc, table, cu = attention_case(42, [3, 200], [20000, 50], 16, 8, 2, 128)
    want, _, status = attend(B, q, kc, vc, table, [20000, 50], cu)
    assert status == 0
    B.dspark_set_wait_limit_ns(1)
    try:
        out, _, status = attend(B, q, kc, vc, table, [20000, 50], cu)
    finally:
        B.dspark_set_wait_limit_ns(0)
    assert status == 0 and torch.equal(out, want)
    assert np.isfinite(out.float().cpu().numpy()).all()
