"""GPU parity of the attention step: dspark_qk_norm_rope, dspark_kv_append, dspark_verify_attention and
dspark_prefix_attention against their 64-bit definitions (attention_reference.py, whose docstring derives the
tolerances).  Outputs and workspaces lie between guard bytes."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

import attention_reference as A  # noqa: E402
import parity_helpers as H  # noqa: E402

BF16, F32 = torch.bfloat16, torch.float32
DEVICE_INPUT = -6


@pytest.fixture(scope="module")
def B():
    from speculative_decoding_dspark_gb300 import build
    build.build()
    from speculative_decoding_dspark_gb300 import binding
    return binding


def normal(seed, shape, dtype, scale=1.0):
    g = torch.Generator("cuda")
    g.manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def close(got, ref, tol, what):
    got = got.double().cpu()
    err = (got - ref).abs()
    bad = ~(err <= tol)
    assert not bool(bad.any()), (what, int(bad.sum()), float((err / tol).nan_to_num(1e9).max()))


def freqs(rot):
    return torch.tensor([10000.0 ** (-2.0 * i / rot) for i in range(rot // 2)], device="cuda")


# ------------------------------------------------------------------------------------------- heads
@pytest.mark.parametrize("rows,hq,hkv,d,rot,pairs,dt,out", [
    (1, 32, 8, 128, 128, False, BF16, BF16), (3, 4, 4, 64, 64, True, BF16, BF16), (7, 5, 1, 80, 64, False, F32, BF16),
    (13, 2, 1, 256, 256, False, F32, F32), (2, 16, 2, 128, 48, True, BF16, F32), (5, 3, 1, 8, 0, False, BF16, BF16),
    (300, 1, 1, 64, 48, False, F32, F32), (9, 48, 8, 192, 112, False, BF16, BF16), (1, 1, 1, 16, 16, True, F32, F32),
])
def test_norm_rope(B, rows, hq, hkv, d, rot, pairs, dt, out):
    G = H.Guarded()
    qkv = normal(rows, (rows, hq + 2 * hkv, d), dt, 3.0)
    q, k = qkv[:, :hq], qkv[:, hq:hq + hkv]  # views: rows lie apart
    wq, wk = normal(1, (d,), dt), normal(2, (d,), dt)
    pos = i32(np.random.default_rng(rows).integers(0, 1 << 20, rows))
    f = freqs(rot) if rot else None
    qo, ko = G.out((rows, hq, d), out, 7), G.out((rows, hkv, d), out, 7)
    status = G.out((1,), torch.int32, 0)
    B.dspark_qk_norm_rope(q, k, wq, wk, 1e-6, pos if rot else None, f, qo, ko, interleaved=pairs, dev_status=status)
    torch.cuda.synchronize()
    G.check()
    assert int(status.item()) == 0
    for x, w, y in ((q, wq, qo), (k, wk, ko)):
        ref, size = A.heads(x, w, float(np.float32(1e-6)), pos, f, pairs)
        close(y, ref, A.heads_tol(ref, size, out), "heads")


def test_norm_rope_in_place_without_a_weight_and_bad_position(B):
    rows, hq, hkv, d = 6, 8, 2, 128
    qkv = normal(3, (rows, hq + hkv, d), BF16)
    before = qkv.clone()
    q, k = qkv[:, :hq], qkv[:, hq:]
    wq, pos, f, status = normal(4, (d,), BF16), i32([5, 0, -1, 7, 70000, 2]), freqs(d), i32([0])
    B.dspark_qk_norm_rope(q, k, wq, None, 1e-5, pos, f, q, k, dev_status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == DEVICE_INPUT
    good = [0, 1, 3, 4, 5]
    assert bool(torch.isnan(qkv[2]).all())
    for x, w, y in ((before[:, :hq], wq, q), (before[:, hq:], None, k)):
        ref, size = A.heads(x[good], w, float(np.float32(1e-5)), pos[good], f, False)
        close(y[good], ref, A.heads_tol(ref, size, BF16), "in place")


def append_case(seed, n, kv_len, page, hkv, d, dt):
    rng = np.random.default_rng(seed)
    cu = np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
    table, pool = A.pages_for(rng, kv_len, cu, page)
    kc, vc = normal(seed, (pool, hkv, page, d), dt), normal(seed + 1, (pool, hkv, page, d), dt)
    return cu, table, kc, vc


@pytest.mark.parametrize("n,kv_len,page,hq,hkv,d,rot,pairs,dt,out", [
    ([1], [0], 16, 4, 1, 64, 64, False, BF16, BF16),
    ([3, 0, 8, 1], [15, 4, 0, 300], 16, 32, 8, 128, 128, False, BF16, BF16),
    ([0, 0, 40, 0], [9, 0, 7, 0], 7, 6, 2, 64, 48, True, F32, BF16),
    ([5, 2], [1, 100000], 1, 2, 2, 128, 64, True, BF16, F32),
    ([17] * 40, list(range(40)), 10, 0, 2, 80, 80, False, F32, F32),
])
def test_kv_append(B, n, kv_len, page, hq, hkv, d, rot, pairs, dt, out):
    cu, table, kc, vc = append_case(sum(n), n, kv_len, page, hkv, d, out)
    rows = int(cu[-1]) + 3  # three rows of padding past the last request
    G = H.Guarded()
    gk, gv = G.out(kc.shape, out, 0), G.out(vc.shape, out, 0)
    gk.copy_(kc), gv.copy_(vc)
    qkv = normal(9, (rows, hq + 2 * hkv, d), dt, 2.0)
    q, k, v = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
    wq, wk, f = normal(5, (d,), dt), normal(6, (d,), dt), freqs(rot)
    qo = G.out((rows, hq, d), out, 7) if hq else None
    status = G.out((1,), torch.int32, 0)
    B.dspark_kv_append(q if hq else None, k, v, wq, wk, 1e-6, f, i32(cu), i32(kv_len), i32(table), gk, gv, qo,
                       interleaved=pairs, dev_status=status)
    torch.cuda.synchronize()
    G.check()
    assert int(status.item()) == 0
    pos, ids, slots = [], [], []
    for r in range(len(n)):
        for i in range(n[r]):
            p = kv_len[r] + i
            pos.append(p), ids.append(int(table[r, p // page])), slots.append(p % page)
    live, pos = int(cu[-1]), torch.tensor(pos)
    eps = float(np.float32(1e-6))
    ref, size = A.heads(k[:live], wk, eps, pos, f, pairs)
    close(gk[ids, :, slots], ref, A.heads_tol(ref, size, out), "keys")
    assert torch.equal(gv[ids, :, slots], v[:live].to(out))
    if hq:
        ref, size = A.heads(q[:live], wq, eps, pos, f, pairs)
        close(qo[:live], ref, A.heads_tol(ref, size, out), "queries")
        assert bool((qo[live:] == 7).all())
    kc[ids, :, slots], vc[ids, :, slots] = gk[ids, :, slots], gv[ids, :, slots]
    assert torch.equal(gk, kc) and torch.equal(gv, vc)  # nothing else was touched


def test_kv_append_bad_pages_and_lengths(B):
    """A missing page, a page past the pool, a position past max_blocks, a negative length: those rows write nothing."""
    n, kv_len, page, hq, hkv, d = [2, 2, 2, 2, 2], [3, 3, 3, 12, 5], 4, 4, 2, 64
    cu, table, kc, vc = append_case(1, n, kv_len, page, hkv, d, BF16)
    table = table[:, :3].copy()                # request 3's positions 12 and 13 are past max_blocks
    table[0, 1], table[1, 1] = -1, kc.shape[0]  # the second row of requests 0 and 1
    kv_len[4] = -1
    rows = int(cu[-1])
    G = H.Guarded()
    gk, gv = G.out(kc.shape, BF16, 0), G.out(vc.shape, BF16, 0)
    gk.copy_(kc), gv.copy_(vc)
    qo, status = G.out((rows, hq, d), BF16, 7), G.out((1,), torch.int32, 0)
    q, k, v = normal(1, (rows, hq, d), BF16), normal(2, (rows, hkv, d), BF16), normal(3, (rows, hkv, d), BF16)
    B.dspark_kv_append(q, k, v, None, None, 1e-6, None, i32(cu), i32(kv_len), i32(table), gk, gv, qo,
                       dev_status=status)
    torch.cuda.synchronize()
    G.check()
    assert int(status.item()) == DEVICE_INPUT
    good = [(0, 0, 3), (2, 1, 3), (4, 2, 3), (5, 2, 4)]  # (row, request, position)
    for row in range(rows):
        if row in [g[0] for g in good]:
            assert torch.equal(qo[row], q[row])
        else:
            assert bool(torch.isnan(qo[row]).all()), row
    for row, r, p in good:
        at = (int(table[r, p // page]), slice(None), p % page)
        assert torch.equal(gk[at], k[row]) and torch.equal(gv[at], v[row])
        kc[at], vc[at] = k[row], v[row]
    assert torch.equal(gk, kc) and torch.equal(gv, vc)


def test_heads_on_another_stream_and_in_a_graph(B):
    n, kv_len, page, hq, hkv, d = [3, 5], [20, 0], 16, 4, 2, 128
    cu, table, kc, vc = append_case(3, n, kv_len, page, hkv, d, BF16)
    qkv, w, f = normal(4, (8, hq + 2 * hkv, d), BF16), normal(5, (d,), BF16), freqs(d)
    q, k, v = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
    lens, status = i32(kv_len), i32([0])
    args = [i32(cu), lens, i32(table)]

    def run(stream=None):
        c = [kc.clone(), vc.clone(), torch.zeros(8, hq, d, dtype=BF16, device="cuda")]
        torch.cuda.synchronize()
        B.dspark_kv_append(q, k, v, w, w, 1e-6, f, *args, *c, dev_status=status, stream=stream)
        torch.cuda.synchronize()
        return c

    want = run()
    assert all(torch.equal(a, b) for a, b in zip(want, run(torch.cuda.Stream())))
    c = [kc.clone(), vc.clone(), torch.zeros_like(want[2])]
    lens.zero_()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        B.dspark_kv_append(q, k, v, w, w, 1e-6, f, *args, *c, dev_status=status)
    lens.copy_(i32(kv_len))
    g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, c)) and int(status.item()) == 0


# --------------------------------------------------------------------------------------- attention
def attention_case(seed, n, kv_len, page, hq, hkv, d, shared=0, peak=3.0):
    rng = np.random.default_rng(seed)
    cu = np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
    table, pool = A.pages_for(rng, kv_len, cu, page, shared)
    kc, vc = normal(seed, (pool, hkv, page, d), BF16), normal(seed + 1, (pool, hkv, page, d), BF16)
    # whatever lies past a request's last position is not to be seen
    unused = np.ones((pool, page), bool)
    for r in range(len(n)):
        for p in range(int(kv_len[r]) + n[r]):
            unused[table[r, p // page], p % page] = False
    mask = torch.tensor(unused, device="cuda")[:, None, :, None]
    kc.masked_fill_(mask, float("nan"))
    vc.masked_fill_(mask, float("nan"))
    q = normal(seed + 2, (int(cu[-1]), hq, d), BF16, peak)
    return q, kc, vc, table, cu


def attend(B, q, kc, vc, table, kv_len, cu, full=False, groups=None, lse=True, stream=None, ws=None, scale=None):
    """(out, lse, status) of the call, every buffer guarded; groups: (group_start, shared_len)."""
    rows, hq, d = q.shape
    G = H.Guarded()
    out = G.out((rows, hq, d), BF16, 7)
    z = G.out((rows, hq), F32, 7) if lse else None
    status = G.out((1,), torch.int32, 0)
    n_groups = 0 if groups is None else len(groups[1])
    need = B.dspark_attention_workspace_size(len(kv_len), n_groups, rows, hq, kc.shape[1], d)
    ws = G.workspace(need) if ws is None else ws
    args = [q, kc, vc, i32(table), i32(kv_len), i32(cu)]
    more = dict(lse=z, full_block=full, ws=ws, dev_status=status, stream=stream)
    scale = d ** -0.5 if scale is None else scale
    torch.cuda.synchronize()
    if groups is None:
        B.dspark_verify_attention(*args, scale, out, **more)
    else:
        B.dspark_prefix_attention(*args, i32(groups[0]), i32(groups[1]), scale, out, **more)
    torch.cuda.synchronize()
    G.check()
    return out, z, int(status.item())


def check_attention(B, seed, n, kv_len, page, hq, hkv, d, full=False, groups=None, shared=0, peak=3.0):
    q, kc, vc, table, cu = attention_case(seed, n, kv_len, page, hq, hkv, d, shared, peak)
    out, z, status = attend(B, q, kc, vc, table, kv_len, cu, full, groups)
    assert status == 0
    ref, lse, tol, ztol = A.attention(q, kc, vc, table, kv_len, cu, float(np.float32(d ** -0.5)), full)
    close(out, ref, tol, "out")
    close(z, lse, ztol, "lse")
    return q, kc, vc, table, cu, out, z


@pytest.mark.parametrize("full", [False, True])
@pytest.mark.parametrize("n,kv_len,page,hq,hkv,d", [
    ([1], [0], 16, 1, 1, 64),                                # one key
    ([1], [777], 16, 32, 8, 128),
    ([1, 1, 1], [127, 128, 129], 16, 4, 2, 64),              # around a block's edge
    ([2, 0, 5, 1, 0], [0, 40, 125, 1000, 3], 7, 8, 8, 128),  # empty requests, pages that end inside a tile
    ([8] * 9, [0, 1, 31, 32, 33, 200, 255, 256, 511], 1, 24, 8, 64),
    ([17, 3], [250, 1], 100, 16, 2, 128),                    # 136 rows a key head: more than one tile
    ([40], [90], 64, 16, 1, 64),                             # a prompt's rows, 640 a key head
    ([150], [0], 256, 2, 1, 128),                            # no history
    ([1], [300], 16, 128, 1, 64),                            # the largest group
])
def test_attention(B, n, kv_len, page, hq, hkv, d, full):
    check_attention(B, 11, n, kv_len, page, hq, hkv, d, full)


@pytest.mark.parametrize("d,hq,hkv", [(128, 8, 2), (64, 4, 4)])
def test_attention_long(B, d, hq, hkv):
    """Few rows and many keys: the work of an item is split and joined again."""
    check_attention(B, 5, [3, 1], [20011, 9000], 16, hq, hkv, d)


@pytest.mark.parametrize("full", [False, True])
@pytest.mark.parametrize("page,hq,hkv,d", [(8, 8, 2, 128), (24, 16, 1, 64), (40, 4, 4, 128), (48, 16, 2, 64), (1000, 8, 1, 128)])
def test_attention_boxes_that_overrun(B, page, hq, hkv, d, full):
    """Pages of several boxes, whose last one holds slots past the last key (not a number, as all unused ones)."""
    check_attention(B, 31, [1, 2, 9, 17, 3, 0, 1], [0, 6, 119, 230, 381, 9, 1000], page, hq, hkv, d, full)


@pytest.mark.parametrize("full", [False, True])
@pytest.mark.parametrize("seed,requests,rows,keys,page,hq,hkv,d", [
    (1, 60, 9, 700, 16, 8, 2, 64), (2, 40, 40, 500, 12, 16, 2, 64), (3, 25, 20, 1500, 32, 32, 2, 128),
    (4, 90, 3, 300, 5, 4, 4, 128), (5, 12, 70, 2000, 64, 4, 1, 128),
])
def test_ragged_batches(B, seed, requests, rows, keys, page, hq, hkv, d, full):
    """Items of one and two tiles after another, cut anywhere."""
    rng = np.random.default_rng(seed)
    n = [int(x) for x in rng.integers(0, rows + 1, requests)]
    kv_len = [int(x) for x in rng.integers(0, keys, requests)]
    check_attention(B, seed, n, kv_len, page, hq, hkv, d, full)


def test_more_requests_than_threads(B):
    rng = np.random.default_rng(7)
    n, kv_len = [int(x) for x in rng.integers(0, 3, 1300)], [int(x) for x in rng.integers(0, 40, 1300)]
    check_attention(B, 7, n, kv_len, 16, 2, 1, 64)


def test_more_groups_than_threads(B):
    """Every request a group of its own, some of them without a shared part."""
    rng = np.random.default_rng(8)
    R = 700
    n = [int(x) for x in rng.integers(0, 3, R)]
    shared = [16 * int(x) for x in rng.integers(0, 4, R)]
    kv_len = [shared[r] + int(rng.integers(0, 40)) for r in range(R)]
    check_attention(B, 9, n, kv_len, 16, 4, 2, 64, groups=(list(range(R + 1)), shared))


@pytest.mark.parametrize("n,kv_len,page,hq,hkv,d", [([700], [100], 16, 8, 2, 128), ([513, 1, 300], [0, 600, 77], 12, 4, 1, 64)])
def test_prompts(B, n, kv_len, page, hq, hkv, d):
    """Many tiles of rows, each of which sees other keys."""
    check_attention(B, 19, n, kv_len, page, hq, hkv, d)


@pytest.mark.parametrize("page", [16, 20])
@pytest.mark.parametrize("d", [64, 128])
def test_two_tiles_over_a_long_history(B, page, d):
    """320 rows to a key head, whose two items are cut into dozens of pieces."""
    check_attention(B, 13, [20], [30011], page, 16, 1, d)


@pytest.mark.parametrize("scale", [0.0, 1e-4, 1.0])
def test_scales(B, scale):
    n, kv_len, page, hq, hkv, d = [3, 5], [400, 77], 16, 8, 2, 128
    q, kc, vc, table, cu = attention_case(17, n, kv_len, page, hq, hkv, d)
    out, z, status = attend(B, q, kc, vc, table, kv_len, cu, scale=scale)
    assert status == 0
    ref, lse, tol, ztol = A.attention(q, kc, vc, table, kv_len, cu, float(np.float32(scale)), False)
    close(out, ref, tol, "out")
    close(z, lse, ztol, "lse")


@pytest.mark.parametrize("peak", [0.0, 0.05, 40.0])
def test_attention_flat_and_peaked(B, peak):
    """Equal scores, and scores hundreds apart whose running maximum keeps moving."""
    check_attention(B, 6, [2, 6], [700, 300], 16, 8, 2, 128, peak=peak)


@pytest.mark.parametrize("full", [False, True])
@pytest.mark.parametrize("starts,shared,page,hq,hkv,d", [
    ([0, 5], [256], 16, 8, 2, 128), ([0, 5], [96], 32, 8, 8, 64), ([0, 5], [1008], 7, 4, 1, 128),
    ([0, 0, 5, 5], [64, 512, 32], 16, 16, 2, 64), ([0, 2, 5], [0, 512], 16, 8, 2, 128), ([0, 1, 2, 3, 4, 5], [512] * 5, 64, 2, 2, 64),
])
def test_prefix(B, starts, shared, page, hq, hkv, d, full):
    n, own = [3, 1, 8, 0, 2], [0, 5, 130, 40, 300]
    group = [max(g for g in range(len(shared)) if starts[g] <= r and (starts[g] < starts[g + 1])) for r in range(5)]
    kv_len = [shared[group[r]] + own[r] for r in range(5)]
    # one pool in which all requests share the longest prefix: every group's is a part of it
    top = min([max(shared)] + [shared[group[r]] for r in range(5) if shared[group[r]]] or [0])
    q, kc, vc, table, cu = attention_case(3, n, kv_len, page, hq, hkv, d, 0)
    for g in range(len(shared)):
        for r in range(starts[g], starts[g + 1]):
            table[r, :shared[g] // page] = table[starts[g], :shared[g] // page]
    out, z, status = attend(B, q, kc, vc, table, kv_len, cu, full, (starts, shared))
    assert status == 0 and top >= 0
    ref, lse, tol, ztol = A.attention(q, kc, vc, table, kv_len, cu, float(np.float32(d ** -0.5)), full)
    close(out, ref, tol, "out")
    close(z, lse, ztol, "lse")


def test_prefix_many_rows(B):
    """A group of more rows than one tile holds, and one whose requests have no rows at all."""
    n, shared, page = [8] * 30 + [0, 0], 640, 16
    kv_len = [shared + 3 * r for r in range(30)] + [shared, shared]
    check_attention(B, 8, n, kv_len, page, 16, 2, 128, groups=([0, 30, 32], [shared, shared]), shared=shared)


@pytest.mark.parametrize("page,hq,hkv,d", [(16, 8, 1, 64), (25, 16, 2, 128)])
def test_prefix_cut_into_pieces(B, page, hq, hkv, d):
    """Groups of one and several tiles over long shared parts, requests with and without rows of their own."""
    rng = np.random.default_rng(page)
    n = [int(x) for x in rng.integers(0, 12, 24)]
    shared = [page * 150, page * 31]
    kv_len = [shared[r >= 20] + int(rng.integers(0, 300)) for r in range(24)]
    q, kc, vc, table, cu = attention_case(14, n, kv_len, page, hq, hkv, d)
    for r in range(24):
        table[r, :shared[r >= 20] // page] = table[20 * (r >= 20), :shared[r >= 20] // page]
    out, z, status = attend(B, q, kc, vc, table, kv_len, cu, groups=([0, 20, 24], shared))
    assert status == 0
    ref, lse, tol, ztol = A.attention(q, kc, vc, table, kv_len, cu, float(np.float32(d ** -0.5)), False)
    close(out, ref, tol, "out")
    close(z, lse, ztol, "lse")


def test_same_bits_twice_and_without_lse(B):
    q, kc, vc, table, cu = attention_case(2, [8, 1, 5], [3000, 50, 9001], 16, 8, 2, 128)
    kv = [3000, 50, 9001]
    a, z, _ = attend(B, q, kc, vc, table, kv, cu)
    for _ in range(3):
        b, _, _ = attend(B, q, kc, vc, table, kv, cu, lse=False)
        assert torch.equal(a, b)
    # a workspace full of another call's leftovers changes nothing
    ws = torch.full((B.dspark_attention_workspace_size(3, 0, 14, 8, 2, 128),), 0xFF, dtype=torch.uint8, device="cuda")
    b, z2, _ = attend(B, q, kc, vc, table, kv, cu, ws=ws)
    assert torch.equal(a, b) and torch.equal(z, z2)


def test_values_of_unseen_rows_have_no_influence(B):
    """NaN and infinities in the keys and values of a request's last rows reach those rows alone."""
    n, kv_len, page, hq, hkv, d = [6, 3], [123, 60], 16, 8, 2, 64
    q, kc, vc, table, cu = attention_case(4, n, kv_len, page, hq, hkv, d)
    ref, lse, tol, ztol = A.attention(q, kc, vc, table, kv_len, cu, float(np.float32(d ** -0.5)), False)
    for r, i, x in ((0, 4, float("nan")), (0, 5, float("inf")), (1, 2, float("-inf"))):
        p = kv_len[r] + i
        vc[int(table[r, p // page]), :, p % page, ::3] = x
        kc[int(table[r, p // page]), 0, p % page] = x
    out, z, status = attend(B, q, kc, vc, table, kv_len, cu)
    assert status == 0
    clean = [0, 1, 2, 3, 6, 7]
    close(out[clean], ref[clean], tol[clean], "out")
    close(z[clean], lse[clean], ztol[clean], "lse")
    assert bool(torch.isnan(out[4][:, ::3]).all())  # a row does see its own


def test_values_of_unseen_rows_across_tiles(B):
    """The same where a request's rows fill several tiles and blocks."""
    n, kv_len, page, hq, hkv, d = [140], [20], 16, 4, 1, 128
    q, kc, vc, table, cu = attention_case(4, n, kv_len, page, hq, hkv, d)
    ref, lse, tol, ztol = A.attention(q, kc, vc, table, kv_len, cu, float(np.float32(d ** -0.5)), False)
    p = kv_len[0] + 100
    vc[int(table[0, p // page]), :, p % page] = float("nan")
    out, z, _ = attend(B, q, kc, vc, table, kv_len, cu)
    close(out[:100], ref[:100], tol[:100], "out")
    close(z, lse, ztol, "lse")
    assert bool(torch.isnan(out[100:]).all())


@pytest.mark.parametrize("groups", [None, ([0, 3, 5], [32, 0])])
def test_bad_requests_are_reported(B, groups):
    """A page id outside the pool, a negative length, positions past max_blocks: NaN rows for those requests alone."""
    n, kv_len, page, hq, hkv, d = [2, 3, 1, 4, 2], [40, 50, 300, 33, 100], 16, 4, 2, 64
    q, kc, vc, table, cu = attention_case(9, n, kv_len, page, hq, hkv, d)
    if groups:
        for r in range(3):
            table[r, :2] = table[0, :2]
    good = A.attention(q, kc, vc, table, kv_len, cu, float(np.float32(d ** -0.5)), False)
    t, kv = table.copy(), list(kv_len)
    t[1, 3] = kc.shape[0]
    t[4, 6] = -1
    kv[2] = t.shape[1] * page
    out, z, status = attend(B, q, kc, vc, t, kv, cu, groups=groups)
    assert status == DEVICE_INPUT
    rows = [0, 1] + list(range(6, 10))
    close(out[rows], good[0][rows], good[2][rows], "out")
    close(z[rows], good[1][rows], good[3][rows], "lse")
    bad = [2, 3, 4, 5, 10, 11]
    assert bool(torch.isnan(out[bad]).all()) and bool(torch.isnan(z[bad]).all())
    kv = list(kv_len)
    kv[3] = -1
    out, z, status = attend(B, q, kc, vc, table, kv, cu, groups=groups)
    assert status == DEVICE_INPUT and bool(torch.isnan(out[6:10]).all())
    close(out[:6], good[0][:6], good[2][:6], "out")


@pytest.mark.parametrize("starts,shared", [([0, 5], [48]), ([0, 5], [24]), ([0, 5], [-16]), ([0, 2, 4], [16, 16]),
                                           ([1, 5], [16]), ([0, 7, 5], [16, 16])])
def test_bad_groups_are_reported(B, starts, shared):
    """More shared than a request holds, a length inside a page or below zero, groups that are not 0 .. R."""
    n, kv_len, page, hq, hkv, d = [2, 3, 1, 4, 2], [40, 50, 60, 33, 100], 16, 4, 2, 64
    q, kc, vc, table, cu = attention_case(9, n, kv_len, page, hq, hkv, d)
    out, z, status = attend(B, q, kc, vc, table, kv_len, cu, groups=(starts, shared))
    assert status == DEVICE_INPUT
    assert bool(torch.isnan(out).all()) and bool(torch.isnan(z).all())


@pytest.mark.parametrize("cu", [[1, 3, 6], [0, 9, 6], [0, 3, 60]])
def test_bad_rows_are_reported(B, cu):
    q, kc, vc, table, _ = attention_case(9, [3, 3], [40, 50], 16, 4, 2, 64)
    out, z, status = attend(B, q, kc, vc, table, [40, 50], cu)
    assert status == DEVICE_INPUT and bool(torch.isnan(out).all())


def test_rows_past_the_last_request_are_not_touched(B):
    q, kc, vc, table, cu = attention_case(12, [2, 3], [40, 500], 16, 4, 2, 64)
    q = torch.cat([q, q])
    for groups in (None, ([0, 2], [0])):
        out, z, status = attend(B, q, kc, vc, table, [40, 500], cu, groups=groups)
        assert status == 0
        assert bool((out[5:] == 7).all()) and bool((z[5:] == 7).all())


def test_offsets_past_32_bits(B):
    """Pages whose elements lie beyond 2^31, written by the append and read back by the attention."""
    hkv, page, d, hq = 2, 16, 128, 4
    pool = (1 << 31) // (hkv * page * d) + 40
    kc = torch.empty((pool, hkv, page, d), dtype=BF16, device="cuda")
    vc = torch.empty_like(kc)
    kv_len, n = [0, 0], [300, 20]
    cu = np.array([0, 300, 320], np.int32)
    table = np.full((2, 20), -1, np.int32)
    table[0, :19] = pool - 1 - np.arange(19)
    table[1, :2] = [3, pool - 25]
    q, k, v = normal(1, (320, hq, d), BF16), normal(2, (320, hkv, d), BF16), normal(3, (320, hkv, d), BF16)
    qo, status = torch.empty_like(q), i32([0])
    B.dspark_kv_append(q, k, v, None, None, 1e-6, None, i32(cu), i32(kv_len), i32(table), kc, vc, qo,
                       dev_status=status)
    torch.cuda.synchronize()
    assert torch.equal(qo, q) and torch.equal(kc[pool - 1, :, 0], k[0]) and torch.equal(vc[pool - 25, :, 3], v[319])
    out, z, st = attend(B, qo, kc, vc, table, kv_len, cu)
    assert st == 0 and int(status.item()) == 0
    ref, lse, tol, ztol = A.attention(qo, kc, vc, table, kv_len, cu, float(np.float32(d ** -0.5)), False)
    close(out, ref, tol, "out")
    close(z, lse, ztol, "lse")


def test_other_stream_and_graph(B):
    """The calls follow the stream they are given and can be captured; a replay sees new lengths and rows."""
    n, kv_len, page, hq, hkv, d = [3, 1], [200, 90], 16, 8, 2, 128
    q, kc, vc, table, cu = attention_case(21, n, kv_len, page, hq, hkv, d)
    want, wz, _ = attend(B, q, kc, vc, table, kv_len, cu, groups=([0, 2], [0]))
    side = torch.cuda.Stream()
    got, gz, _ = attend(B, q, kc, vc, table, kv_len, cu, groups=([0, 2], [0]), stream=side)
    assert torch.equal(want, got) and torch.equal(wz, gz)
    out, z, status = torch.empty_like(q), torch.empty(4, hq, device="cuda"), i32([0])
    ws = B.workspace(B.dspark_attention_workspace_size(2, 0, 4, hq, hkv, d))
    args = [q, kc, vc, i32(table), i32([1, 1]), i32(cu)]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        B.dspark_verify_attention(*args, d ** -0.5, out, lse=z, ws=ws, dev_status=status)
    args[4].copy_(i32(kv_len))
    for _ in range(2):
        out.fill_(0)
        g.replay()
    torch.cuda.synchronize()
    want, wz, _ = attend(B, q, kc, vc, table, kv_len, cu)
    assert int(status.item()) == 0 and torch.equal(out, want) and torch.equal(z, wz)


def test_binding_refusals(B):
    q, kc, vc, table, cu = attention_case(1, [1], [5], 16, 4, 2, 64)
    ws = B.workspace(B.dspark_attention_workspace_size(1, 0, 1, 4, 2, 64))
    args = [q, kc, vc, i32(table), i32([5]), i32(cu)]
    with pytest.raises(TypeError):
        B.dspark_verify_attention(q.float(), *args[1:], 1.0, torch.empty_like(q), ws=ws)
    with pytest.raises(ValueError):
        B.dspark_verify_attention(*args, 1.0, torch.empty_like(q)[:, :2], ws=ws)
    with pytest.raises(ValueError):
        B.dspark_verify_attention(q, kc[:, :, :, ::2], *args[2:], 1.0, torch.empty_like(q), ws=ws)
    with pytest.raises(B.DSparkError):
        B.dspark_verify_attention(*args, 1.0, torch.empty_like(q), ws=ws[:16])
    with pytest.raises(ValueError):
        B.dspark_qk_norm_rope(q[:, :, ::2], q[:, :, ::2], None, None, 0.0, None, None, q, q)
