"""Values that are not finite, in keys that a row does see: the channels that hold them become what the definition
makes of them, and every other channel of every row stays within its tolerance (attention_reference.py derives it)."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

import attention_reference as A  # noqa: E402
from test_gpu_attention import B, attend, attention_case, close  # noqa: E402,F401

INF, NAN = float("inf"), float("nan")


def check(B, case, kv_len, full=False, groups=None):
    """The call on (q, k_cache, v_cache, table, cu) against the definition, channel by channel."""
    q, kc, vc, table, cu = case
    out, z, status = attend(B, q, kc, vc, table, kv_len, cu, full, groups)
    assert status == 0
    ref, lse, tol, ztol = A.attention(q, kc, vc, table, kv_len, cu, float(np.float32(q.shape[2] ** -0.5)), full)
    got, finite = out.double().cpu(), torch.isfinite(ref)
    assert bool((~finite).any())  # (the case has some)
    odd, want = got[~finite], ref[~finite]
    wrong = ~((odd == want) | (torch.isnan(odd) & torch.isnan(want)))
    assert not bool(wrong.any()), ("not finite", int(wrong.sum()), odd[wrong][:4], want[wrong][:4])
    close(got[finite], ref[finite], tol[finite], "finite channels")
    close(z, lse, ztol, "lse")


def share(table, starts, shared, page):
    for g in range(len(shared)):
        for r in range(starts[g], starts[g + 1]):
            table[r, :shared[g] // page] = table[starts[g], :shared[g] // page]


def put(vc, table, r, pos, channel, x):
    page = vc.shape[2]
    vc[int(table[r, pos // page]), :, pos % page, channel] = x


@pytest.mark.parametrize("shared", [0, 192])
@pytest.mark.parametrize("requests,n,keys,page,hq,hkv,d", [
    (128, 8, 300, 16, 8, 2, 128),   # 32 rows a key head, many items to a CTA
    (128, 8, 300, 12, 4, 1, 64),    # the same of pages that end anywhere
    (100, 8, 400, 16, 16, 2, 64),   # 64 rows: one tile
    (100, 11, 500, 10, 8, 1, 128),  # 88 rows
    (40, 40, 500, 16, 8, 2, 128),   # 160 rows: two tiles over each block
    (40, 40, 500, 24, 8, 2, 64),
    (5, 300, 700, 16, 4, 1, 128),   # several items, whose rows end in several blocks
    (3, 300, 700, 7, 8, 1, 64),
])
def test_values_of_late_rows(B, requests, n, keys, page, hq, hkv, d, shared):
    """One channel of the value of a late row, or of several: rows before it see nothing of it, rows from it on do."""
    shared -= shared % page
    rng = np.random.default_rng(requests + d)
    rows = [n - int(x) for x in rng.integers(0, 3, requests)]
    kv_len = [shared + int(x) for x in rng.integers(0, keys, requests)]
    case = attention_case(requests, rows, kv_len, page, hq, hkv, d, peak=1.0)
    _, _, vc, table, _ = case
    groups = None
    if shared:
        groups = ([0, requests // 2, requests], [shared, shared])
        share(table, *groups, page)
    for r in range(requests):
        for i in sorted({rows[r] - 1 - r % 3, rows[r] // 2, rows[r] // 5}):
            put(vc, table, r, kv_len[r] + i, (7 * r + 5 * i) % d, (INF, -INF, INF, NAN)[(r + i) % 4])
    check(B, case, kv_len, groups=groups)


@pytest.mark.parametrize("full", [False, True])
@pytest.mark.parametrize("n,kv_len,page,hq,hkv,d", [
    ([1], [300], 16, 8, 2, 128),                     # one token: 4 rows a key head
    ([8, 1, 3], [900, 130, 5000], 16, 8, 2, 64),     # up to 32 rows, blocks of both tiles, pieces that are joined
    ([8, 5], [900, 260], 10, 4, 1, 128),
    ([40, 90], [300, 1000], 16, 4, 1, 64),           # 160 and 360 rows
    ([9], [700], 12, 4, 1, 128),                     # 36 rows: one tile
])
def test_values_that_all_rows_see(B, n, kv_len, page, hq, hkv, d, full):
    """Infinities and NaN in the history, in keys of every quarter of a block."""
    case = attention_case(29, n, kv_len, page, hq, hkv, d, peak=1.0)
    for r in range(len(n)):
        for pos, channel, x in ((3, 5, INF), (40, 6, -INF), (70, 7, INF), (100, 8, -INF), (kv_len[r] // 128 * 128 - 5, 9, INF),
                                (64, 10, NAN), (1, 11, INF), (33, 11, -INF)):
            put(case[2], case[3], r, pos, channel, x)
    check(B, case, kv_len, full)


def test_values_of_a_shared_part(B):
    n, page, hq, hkv, d = [8, 1, 4, 0, 2], 16, 8, 2, 128
    kv_len = [512 + 40, 512, 512 + 300, 512, 512 + 7]
    case = attention_case(30, n, kv_len, page, hq, hkv, d, peak=1.0)
    groups = ([0, 5], [512])
    share(case[3], *groups, page)
    put(case[2], case[3], 0, 17, 3, INF)
    put(case[2], case[3], 0, 300, 4, -INF)
    put(case[2], case[3], 2, 520, 5, INF)
    check(B, case, kv_len, groups=groups)
