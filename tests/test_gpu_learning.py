"""GPU parity of dspark_token_logprobs, dspark_distill_loss and dspark_markov_grad against their 64-bit definitions
(learning_reference.py, whose docstring derives the tolerances).  Outputs and workspaces lie between guard bytes."""
import time

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

import learning_reference as L  # noqa: E402
import parity_helpers as H  # noqa: E402

BF16, F32, I32 = torch.bfloat16, torch.float32, torch.int32
INF, NAN = float("inf"), float("nan")
DEVICE_INPUT = -6


@pytest.fixture(scope="module")
def B():
    from speculative_decoding_dspark_gb300 import build
    build.build()
    from speculative_decoding_dspark_gb300 import binding
    return binding


def generator(seed):
    g = torch.Generator("cuda")
    g.manual_seed(seed)
    return g


def normal(seed, shape, scale=1.0):
    return torch.randn(shape, generator=generator(seed), device="cuda") * scale


def i32(x):
    return torch.tensor(np.asarray(x), dtype=I32, device="cuda")


def rows_of(x, dtype, offset, gap):
    """x as rows that begin `offset` elements behind a boundary and lie `gap` elements further apart than they are long."""
    rows, V = x.shape
    buf = torch.full((offset + rows * (V + gap) + 16,), NAN, dtype=dtype, device="cuda")
    y = buf.as_strided((rows, V), (V + gap, 1), offset)
    y.copy_(x)
    return y


def close(got, ref, tol, what):
    got = got.double()
    special = ~ref.isfinite()
    same = torch.where(ref.isnan(), got.isnan(), got == ref)
    assert bool(same[special].all()), (what, "not finite", int((~same[special]).sum()))
    err = (got - ref).abs()[~special]
    bad = ~(err <= tol[~special])
    assert not bool(bad.any()), (what, int(bad.sum()), float((err / tol[~special]).nan_to_num(1e9).max()))


# ------------------------------------------------------------------------------------- log probabilities
def logprobs(B, x, tokens, T, top, cu=None, fill=7, stream=None):
    rows = x.shape[0]
    G = H.Guarded()
    lp, lse, ent = (G.out((rows,), F32, fill) for _ in range(3))
    ids = G.out((rows, top), I32, fill) if top else None
    val = G.out((rows, top), F32, fill) if top else None
    status = G.out((1,), I32, 0)
    torch.cuda.synchronize()
    B.dspark_token_logprobs(x, tokens, T, lp, lse, ent, ids, val, cu_seqlens=cu, dev_status=status, stream=stream)
    torch.cuda.synchronize()
    G.check()
    return lp, lse, ent, ids, val, int(status.item())


def check_logprobs(B, x, tokens, T, top):
    lp, lse, ent, ids, val, status = logprobs(B, x, tokens, T, top)
    assert status == 0
    ref, tol = L.logprobs(x, tokens, T, top)
    for got, r, t, what in zip((lp, lse, ent), ref, tol, ("logprob", "lse", "entropy")):
        close(got, r, t, what)
    if top:
        assert torch.equal(ids.long(), ref[3])
        close(val, ref[4], tol[3], "top_logprobs")


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("rows,V,top,T,offset,gap", [
    (1, 1, 1, 1.0, 0, 0), (1, 1, 128, 1.0, 1, 0), (2, 2, 3, 0.5, 1, 3), (5, 3, 1, 1.0, 0, 0), (4, 7, 20, 2.0, 3, 1),
    (3, 8, 8, 1.0, 0, 0), (3, 9, 5, 1.0, 7, 0), (7, 100, 128, 1.0, 0, 5), (300, 257, 20, 0.7, 1, 0), (3, 1000, 0, 1.0, 0, 0),
    (6, 1023, 128, 1.0, 2, 2), (6, 1024, 128, 1.0, 0, 0), (2, 2047, 128, 1.3, 0, 0), (5, 4096, 64, 1.0, 0, 8),
    (4, 4097, 1, 1.0, 0, 0), (9, 32000, 20, 1.0, 0, 0), (3, 50001, 128, 0.8, 5, 0), (2, 129280, 20, 1.0, 0, 0),
    (1, 151936, 5, 1.0, 0, 0), (40, 151936, 20, 1.0, 0, 0), (700, 8192, 5, 1.0, 0, 0), (1, 262147, 128, 1.0, 1, 0),
    (1, 1 << 22, 50, 1.0, 0, 0),
])
def test_logprobs(B, dtype, rows, V, top, T, offset, gap):
    x = rows_of(normal(V + rows, (rows, V), 3.0), dtype, offset, gap)
    tokens = torch.randint(0, V, (rows,), generator=generator(1), device="cuda", dtype=I32)
    check_logprobs(B, x, tokens, T, top)


def test_logprobs_without_tokens_or_lists(B):
    x = normal(3, (5, 777), 2.0)
    lse = torch.empty(5, device="cuda")
    B.dspark_token_logprobs(x, None, 1.0, None, lse)
    ref, tol = L.logprobs(x, None, 1.0, 0)
    close(lse, ref[1], tol[1], "lse")
    got = torch.full((5,), 3.0, device="cuda")
    tokens = i32([0, 1, 2, 3, 4])
    B.dspark_token_logprobs(x, tokens, 1.0, got)
    ref, tol = L.logprobs(x, tokens, 1.0, 0)
    close(got, ref[0], tol[0], "logprob")
    B.dspark_token_logprobs(x, None, 1.0, got)
    assert bool((got == 0).all())


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("kind", ["equal", "few", "rising", "falling", "thread", "zeros", "masked", "lowest", "peak", "steps", "window"])
@pytest.mark.parametrize("V,top", [(5000, 128), (70001, 128), (70001, 3), (300, 20), (151936, 1)])
def test_logprobs_orders(B, dtype, kind, V, top):
    """Values that come in orders and in numbers that a list of candidates is not made for."""
    v = torch.arange(V, device="cuda", dtype=F32)
    g = generator(V)
    x = {
        "equal": lambda: torch.full((V,), -1.5, device="cuda"),
        "few": lambda: torch.randint(0, 3, (V,), generator=g, device="cuda").float(),
        "rising": lambda: v / V * 9,
        "falling": lambda: -v / V * 9,
        "thread": lambda: torch.where((v % 2048) < 8, 9 - v / V, -v / V),  # the best all with one thread
        "zeros": lambda: torch.where(v % 2 == 0, 0.0, -0.0),
        "masked": lambda: torch.where(v % 97 == 5, v % 13, -INF),
        "lowest": lambda: torch.where(v % 97 == 5, v % 13, float(torch.finfo(dtype).min)),
        "peak": lambda: torch.where(v == V // 2, 80.0, -30.0 + v / V),
        "steps": lambda: torch.floor(v / 1100) % 7,
        "window": lambda: torch.where((v > 0.6 * V) & (v < 0.65 * V), torch.randn(V, generator=g, device="cuda"), -INF),
    }[kind]()
    x = torch.stack([x, x.flip(0), x.roll(V // 3)]).to(dtype)
    check_logprobs(B, x, i32([0, V - 1, V // 2]), 1.0, top)


def test_logprobs_all_lowest(B):
    """A mask of the type's lowest value that leaves nothing: finite, so every token is as likely as the next."""
    for dtype in (F32, BF16):
        x = torch.full((2, 4096), float(torch.finfo(dtype).min), device="cuda").to(dtype)
        lp, lse, ent, ids, val, status = logprobs(B, x, i32([5, 9]), 1.0, 4)
        assert status == 0 and ids.tolist() == [[0, 1, 2, 3]] * 2
        # logf and the sum of 4096 equal terms (exact): one step of 8.3 each for the logarithm and its rounding
        for got, want in ((lp, -np.log(4096)), (ent, np.log(4096)), (val, -np.log(4096))):
            assert float((got.double() - want).abs().max()) <= 4 * 2.0 ** -24 * 8.4


def test_logprobs_rows_without_a_value(B):
    x = normal(5, (9, 3001), 2.0)
    x[1] = -INF
    x[2, 17] = NAN
    x[3, 2999] = INF
    x[4, 0] = NAN
    x[5, 3000] = NAN
    x[6, 1:] = -INF
    good = [0, 6, 7, 8]
    tokens = i32([3, 3, 3, 3, 3, 3, 0, -1, 3])
    lp, lse, ent, ids, val, status = logprobs(B, x, tokens, 1.0, 5)
    assert status == DEVICE_INPUT
    for n in (1, 2, 3, 4, 5):
        assert lp[n].isnan() and lse[n].isnan() and ent[n].isnan() and (ids[n] == -1).all() and val[n].isnan().all(), n
    assert lp[7] == 0 and lse[7] == 0 and ent[7] == 0 and (ids[7] == -1).all() and (val[7] == -INF).all()
    assert lp[6] == 0 and ent[6] == 0 and ids[6].tolist() == [0, -1, -1, -1, -1]
    ref, tol = L.logprobs(x[good], tokens[good].clamp(min=0), 1.0, 5)
    for n, at in enumerate(good):
        if at != 7:
            close(lp[at], ref[0][n], tol[0][n], "logprob")
            assert torch.equal(ids[at].long(), ref[3][n])


def test_logprobs_bad_token(B):
    x = normal(6, (3, 640))
    lp, lse, ent, ids, val, status = logprobs(B, x, i32([639, 640, 2 ** 31 - 1]), 1.0, 2)
    assert status == DEVICE_INPUT and lp[1:].isnan().all() and lse[1:].isnan().all() and (ids[1:] == -1).all()
    assert lp[0].isfinite() and (ids[0] >= 0).all()


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("n,width,rows", [([3, 0, 1, 8, 2], 8, 14), ([1], 1, 1), ([4, 4, 4], 2, 20), ([0, 0, 5], 6, 9)])
def test_logprobs_packed(B, dtype, n, width, rows):
    """Tokens beside cu_seqlens, as a verify leaves them: -1 behind each request's last, rows behind the last request."""
    V = 4099
    cu = np.concatenate([[0], np.cumsum(n)])
    x = normal(rows, (rows, V), 3.0).to(dtype)
    rng = np.random.default_rng(7)
    tokens = rng.integers(0, V, (len(n), width)).astype(np.int32)
    for r, m in enumerate(n):
        tokens[r, max(1, m - 1):] = -1  # the last row is not asked for
    x[int(cu[-1]):] = NAN
    flat = np.full(rows, -1)
    for r, m in enumerate(n):
        for j in range(min(m, width)):
            flat[cu[r] + j] = tokens[r, j]
            if tokens[r, j] < 0:
                x[int(cu[r]) + j] = NAN  # not read
    lp, lse, ent, ids, val, status = logprobs(B, x, i32(tokens), 0.7, 6, cu=i32(cu))
    assert status == 0
    asked = np.nonzero(flat >= 0)[0]
    ref, tol = L.logprobs(x[asked], i32(flat[asked]), 0.7, 6)
    for got, r, t in zip((lp, lse, ent, val), (ref[0], ref[1], ref[2], ref[4]), tol):
        close(got[asked], r, t, "packed")
    assert torch.equal(ids[asked].long(), ref[3])
    for row in range(rows):
        if row >= cu[-1]:
            assert lp[row] == 7 and lse[row] == 7 and ent[row] == 7 and (ids[row] == 7).all() and (val[row] == 7).all()
        elif flat[row] < 0:
            assert lp[row] == 0 and lse[row] == 0 and ent[row] == 0 and (ids[row] == -1).all() and (val[row] == -INF).all()


@pytest.mark.parametrize("cu,good", [([1, 2, 4], [1]), ([0, 3, 2], [0]), ([0, 2, 7], [0]), ([0, -1, 3], []), ([0, 2, 2 ** 31 - 1], [0])])
def test_logprobs_bad_lengths(B, cu, good):
    x = normal(8, (6, 515))
    lp, _, _, _, _, status = logprobs(B, x, i32(np.zeros((2, 3))), 1.0, 0, cu=i32(cu))
    assert status == DEVICE_INPUT
    expect = torch.zeros(6, dtype=torch.bool)
    for r in good:
        expect[cu[r]:cu[r + 1]] = True
    assert torch.equal((lp != 7).cpu(), expect)


def test_logprobs_of_a_verify(B):
    """The tokens a verify emits and the probabilities it saw: exp(logprob) of the drafts it kept is its p_tok."""
    w, d = H.cycle_inputs("varlen_verify", R=17, V=8192, gamma=5, rank=64, w_sigma=0.2)
    from speculative_decoding_dspark_gb300 import inputs
    g = H.gpu_draft(d, 0.7, 2)
    l = inputs.verify_lengths(w)
    target = H.dev(inputs.pack_rows(inputs.target_full(w, d["U"]), l))
    cu = H.dev(inputs.cu_from_lengths(l))
    R, gamma = l.size, 5
    n_acc, out, p_tok = (torch.empty(R, dtype=I32, device="cuda"), torch.empty(R, gamma + 1, dtype=I32, device="cuda"),
                         torch.zeros(R, gamma, device="cuda"))
    rows = target.shape[0]
    ws = B.workspace(B.dspark_workspace_size(B.DSPARK_OP_VERIFY, R, gamma, target.shape[1], 0, rows))
    B.dspark_verify(target, cu, g["y_dev"], g["q_logits_dev"], g["q_lse_dev"], g["q_tok_dev"], H.dev(d["seeds"]), 2, 0.7, rows,
                    n_acc, out, p_tok, ws)
    lp, _, _, ids, val, status = logprobs(B, target, out, 0.7, 8, cu=cu)
    assert status == 0
    for r in range(R):
        n = int(n_acc[r])
        for j in range(n + 1):
            row = int(cu[r]) + j
            ref, tol = L.logprobs(target[row:row + 1], out[r, j:j + 1], 0.7, 8)
            close(lp[row:row + 1], ref[0], tol[0], "emitted")
            if j < n:
                # each is off by its own error: of lp, and of the verify's 2^(t - lse) alike
                assert abs(float(lp[row].exp()) / float(p_tok[r, j]) - 1) <= 2 * float(tol[0]) + 2.0 ** -20
        for j in range(n + 1, int(l[r]) + 1):
            assert lp[int(cu[r]) + j] == 0


# ------------------------------------------------------------------------------------------ distillation
def distill(B, x, ids, value, T, grad=None, weight=None, rest=False, in_place=False, gap=0, offset=0):
    rows, V = x.shape
    G = H.Guarded()
    loss = G.out((rows,), F32, 7)
    status = G.out((1,), I32, 0)
    g = x if in_place else None if grad is None else rows_of(torch.zeros(rows, V, device="cuda"), grad, offset, gap)
    torch.cuda.synchronize()
    B.dspark_distill_loss(x, ids, value, T, loss, grad=g, row_weight=weight, rest=rest, dev_status=status)
    torch.cuda.synchronize()
    G.check()
    if g is not None and gap and not in_place:
        between = g.as_strided((rows, gap), (V + gap, 1), offset + V)
        assert bool(between.isnan().all())
    return loss, g, int(status.item())


def teacher_of(seed, x, top, T=1.0):
    z = (0.6 * x.float() + normal(seed, x.shape, 2.4)) / T
    best, ids = z.topk(top, dim=1)
    return ids.to(I32), best - z.logsumexp(1, keepdim=True)


def check_distill(B, x, ids, value, T, grad, weight=None, rest=False, in_place=False, gap=0, offset=0):
    ref, tol = L.distill(x, ids, value, T, weight, rest, grad)
    loss, g, status = distill(B, x, ids, value, T, grad, weight, rest, in_place, gap, offset)
    assert status == 0
    close(loss, ref[0], tol[0], "loss")
    if g is not None:
        close(g, ref[1], tol[1], "grad")


SHAPES = [
    (1, 1, 1, 1.0, 0, 0), (2, 2, 1, 1.0, 1, 0), (3, 3, 3, 0.5, 1, 1), (5, 7, 4, 1.0, 3, 0), (4, 8, 8, 1.0, 0, 0), (3, 9, 2, 2.0, 0, 7),
    (6, 100, 100, 1.0, 5, 3), (7, 513, 128, 1.0, 0, 0), (200, 1001, 20, 0.7, 0, 0), (3, 4096, 64, 1.0, 0, 8), (5, 32003, 33, 1.0, 1, 2),
    (2, 50001, 128, 2.0, 7, 0), (3, 129280, 128, 1.0, 0, 0), (2, 151936, 20, 1.0, 0, 0), (1, 151937, 1, 1.0, 1, 0),
]


@pytest.mark.parametrize("rest", [False, True])
@pytest.mark.parametrize("dtype,grad", [(F32, None), (F32, F32), (F32, BF16), (BF16, None), (BF16, F32), (BF16, BF16)])
@pytest.mark.parametrize("rows,V,top,T,offset,gap", SHAPES)
def test_distill(B, rest, dtype, grad, rows, V, top, T, offset, gap):
    x = rows_of(normal(V, (rows, V), 3.0), dtype, offset, gap)
    ids, value = teacher_of(V + 1, x, top, T)
    if rows > 2:
        ids[1, top // 2:] = -1  # fewer tokens than places
        ids[2] = -1
    weight = None if rows % 2 else torch.linspace(-1.0, 2.0, rows, device="cuda")
    check_distill(B, x, ids, value, T, grad, weight, rest, gap=gap, offset=offset)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("rows,V,top", [(3, 9, 3), (4, 4097, 20), (2, 151936, 64), (3, 600001, 16)])
def test_distill_in_place(B, dtype, rows, V, top):
    """Rows that give way to their gradient; the longest do not stay in shared memory."""
    for rest in (False, True):
        x = rows_of(normal(V, (rows, V), 3.0), dtype, 1, 2)
        ids, value = teacher_of(5, x, top)
        weight = torch.tensor([0.5, 0.0, 1.0, 2.0][:rows], device="cuda")
        check_distill(B, x, ids, value, 1.0, dtype, weight, rest, in_place=True)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_distill_long_rows(B, dtype):
    V = 1 << 22
    x = normal(1, (1, V), 3.0).to(dtype)
    ids, value = teacher_of(2, x, 128)
    for grad in (None, F32, BF16):
        check_distill(B, x, ids, value, 1.0, grad, rest=True)


@pytest.mark.parametrize("grad", [F32, BF16])
@pytest.mark.parametrize("rest", [False, True])
def test_distill_sure_and_masked(B, rest, grad):
    """A drafter that is sure of a listed token, of one that is not, one with a mask of -inf or of the type's lowest value
    over the rest, over listed tokens, and a teacher that knows one token only."""
    V = 2000
    x = normal(11, (8, V), 1.0)
    x[0, 5] = 60.0
    x[1, 900] = 200.0
    x[2, 10:] = -INF
    x[3, 10:] = torch.finfo(F32).min
    x[4, 7] = -INF
    x[5] = torch.finfo(F32).min
    x[6, :] *= 40.0
    ids = i32([list(range(10))] * 8)
    value = torch.log_softmax(normal(12, (8, 10)), 1) - 0.3
    value[7] = -INF
    value[7, 3] = 0.0
    check_distill(B, x, ids, value, 1.0, grad, rest=rest)


@pytest.mark.parametrize("rest", [False, True])
def test_distill_large_teacher_values(B, rest):
    """Logits instead of log probabilities (renormalised), and a teacher whose listed mass is all there is."""
    x = normal(13, (4, 900), 2.0)
    ids, value = teacher_of(14, x, 6)
    value = value + (0.0 if rest else 300.0)
    if rest:
        value = value - value.logsumexp(1, keepdim=True)
    check_distill(B, x, ids, value, 1.0, F32, rest=rest)


def test_distill_rows_without_a_value(B):
    V, top = 3001, 6
    x = normal(15, (14, V), 2.0)
    ids, value = teacher_of(16, x, top)
    weight = torch.ones(14, device="cuda")
    x[0, 100] = NAN
    x[1, 0] = INF
    x[2] = -INF
    x[3, int(ids[3, 2])] = NAN
    ids[4, 1] = V
    ids[5, 3] = ids[5, 0]
    ids[6, :2] = 0  # twice, before the first boundary or in the first piece
    ids[7, 4:] = V - 1  # twice, at the row's end
    value[8, 0] = NAN
    value[9, 0] = INF
    weight[10] = INF
    weight[11] = NAN
    bad = list(range(12))
    weight[12] = 0.0
    x[12, 4] = NAN  # not read
    for rest in (False, True):
        for grad in (None, F32, BF16):
            for y in (x, rows_of(x, BF16, 3, 0)):
                loss, g, status = distill(B, y, ids, value, 1.0, grad, weight, rest)
                assert status == DEVICE_INPUT
                assert loss[bad].isnan().all() and loss[12] == 0 and loss[13].isfinite(), (loss, rest)
                if grad is not None:
                    assert g[bad].isnan().all() and (g[12] == 0).all() and g[13].isfinite().all()
    # too much mass for a number
    value[13] = 100.0
    loss, g, status = distill(B, x[13:], ids[13:], value[13:], 1.0, F32, None, True)
    assert status == DEVICE_INPUT and loss.isnan().all() and g.isnan().all()


@pytest.mark.parametrize("in_place", [False, True])
def test_distill_rows_without_weight(B, in_place):
    """Rows of weight 0, alone and among others, at every alignment: not read, their gradient zero and nothing beside it."""
    for V in (1, 5, 1027, 40003):
        for weights in ([0.0] * 6, [0.0, 1.0, 0.0, 0.0, 2.0, -0.0]):
            for dtype in (F32, BF16):
                x = rows_of(normal(V, (6, V)), dtype, 3, 5)
                weight = torch.tensor(weights, device="cuda")
                ids, value = teacher_of(1, x, 1)
                ref, tol = L.distill(x, ids, value, 1.0, weight, False, dtype)
                x[weight == 0] = NAN
                loss, g, status = distill(B, x, ids, value, 1.0, dtype, weight, False, in_place, gap=0 if in_place else 5, offset=3)
                assert status == 0
                close(loss, ref[0], tol[0], "loss")
                close(g, ref[1], tol[1], "grad")


def test_distill_more_places_than_tokens(B):
    x = normal(19, (3, 3), 2.0)
    ids = i32([[2, -1, -7, 0, -1, -1, -1, 1], [-1] * 8, [-1] * 7 + [1]])
    value = torch.full((3, 8), NAN, device="cuda")  # (beside no token a value says nothing)
    value[0, [0, 3, 7]] = torch.tensor([0.2, 0.3, 0.5], device="cuda").log()
    value[2, 7] = -0.1
    for rest in (False, True):
        clean = torch.where(ids >= 0, value, torch.zeros_like(value))
        ref, tol = L.distill(x, ids, clean, 1.0, None, rest, F32)
        loss, g, status = distill(B, x, ids, value, 1.0, F32, None, rest)
        assert status == 0
        close(loss, ref[0], tol[0], "loss")
        close(g, ref[1], tol[1], "grad")


def test_distill_gradient_is_the_slope(B):
    """Against differences of the operator's own loss, in steps that the loss resolves."""
    V, h = 40, 0.05
    x = normal(17, (1, V), 1.0)
    ids, value = teacher_of(18, x, 5)
    for rest in (False, True):
        _, g, _ = distill(B, x, ids, value, 0.8, F32, None, rest)
        moved = x.repeat(2 * V, 1)
        for v in range(V):
            moved[2 * v, v] += h
            moved[2 * v + 1, v] -= h
        loss, _, _ = distill(B, moved, ids.repeat(2 * V, 1), value.repeat(2 * V, 1), 0.8, None, None, rest)
        slope = (loss[0::2] - loss[1::2]).double() / (2 * h)
        # h^2 / 6 of a third derivative below 8 / T^3 each for the row and the rest, and two losses' error (below 1e-5) over 2h
        assert float((slope - g[0].double()).abs().max()) <= h * h / 6 * 16 / 0.8 ** 3 + 1e-5 / h


# ------------------------------------------------------------------------------ the Markov factors' gradient
def markov_case(seed, rows, V, rank, gap=0):
    g = rows_of(normal(seed, (rows, V), 0.01) + (torch.rand(rows, V, generator=generator(seed), device="cuda") < 0.01) * 1.0,
                BF16, 0, gap)
    W1, W2 = (normal(seed + k, (V, rank), 0.05).to(BF16) for k in (1, 2))
    prev = torch.randint(-1, max(1, min(V, rows // 2 + 1)), (rows,), generator=generator(seed), device="cuda", dtype=I32)
    return g, prev, W1, W2


def markov(B, g, prev, W1, W2, accumulate=False, want=(True, True), start=(0.0, 0.0)):
    rows, V = g.shape
    rank = W1.shape[1]
    G = H.Guarded()
    gp = G.out((rows, rank), F32, 7)
    d1, d2 = (G.out((V, rank), F32, start[k]) if want[k] else None for k in (0, 1))
    status = G.out((1,), I32, 0)
    ws = G.workspace(B.dspark_workspace_size(B.DSPARK_OP_MARKOV_GRAD, 0, 0, V, rank, rows))
    torch.cuda.synchronize()
    B.dspark_markov_grad(g, prev, W1, W2, gp, dW1=d1, dW2=d2, accumulate=accumulate, ws=ws, dev_status=status)
    torch.cuda.synchronize()
    G.check()
    return gp, d1, d2, int(status.item())


@pytest.mark.parametrize("rows,V,rank,gap", [
    (1, 8, 64, 0), (1, 64, 128, 0), (3, 72, 64, 8), (7, 1000, 320, 0), (63, 128, 192, 0), (64, 136, 256, 0), (65, 4096, 448, 16),
    (127, 4104, 512, 0), (128, 8192, 512, 0), (129, 8200, 64, 0), (300, 5000, 384, 0), (1100, 640, 128, 0), (2500, 1032, 512, 0),
    (896, 32000, 512, 0), (2, 151936, 512, 0), (33, 129280, 256, 0),
])
def test_markov_grad(B, rows, V, rank, gap):
    g, prev, W1, W2 = markov_case(rows + V, rows, V, rank, gap)
    gp, d1, d2, status = markov(B, g, prev, W1, W2, start=(7.0, 9.0))
    assert status == 0
    ref, tol = L.markov(g, prev, W1, W2)
    close(gp, ref[0], tol[0], "grad_prev")
    seen = torch.zeros(V, dtype=torch.bool, device="cuda")
    seen[prev[prev >= 0].long()] = True
    close(d1[seen], ref[1][seen], tol[1][seen], "dW1")
    assert bool((d1[~seen] == 7.0).all())
    close(d2, ref[2], tol[2], "dW2")


@pytest.mark.parametrize("rows,V,rank", [(5, 72, 64), (200, 4104, 320), (1500, 1000, 512)])
def test_markov_grad_accumulates(B, rows, V, rank):
    g, prev, W1, W2 = markov_case(5, rows, V, rank)
    gp, d1, d2, status = markov(B, g, prev, W1, W2, True, start=(0.5, -2.0))
    assert status == 0
    ref, tol = L.markov(g, prev, W1, W2, torch.full((V, rank), 0.5, device="cuda"), torch.full((V, rank), -2.0, device="cuda"))
    close(gp, ref[0], tol[0], "grad_prev")
    close(d1, ref[1], tol[1], "dW1")
    close(d2, ref[2], tol[2], "dW2")


@pytest.mark.parametrize("want", [(False, False), (True, False), (False, True)])
def test_markov_grad_in_part(B, want):
    g, prev, W1, W2 = markov_case(6, 70, 2000, 128)
    all_of = markov(B, g, prev, W1, W2)
    some = markov(B, g, prev, W1, W2, want=want)
    for a, b in zip(all_of[:3], some[:3]):
        assert b is None or torch.equal(a, b)


@pytest.mark.parametrize("rows,V,rank", [(40, 640, 64), (150, 4104, 320)])
def test_markov_grad_bad_token(B, rows, V, rank):
    """Tokens that are none: their rows give nothing, and what stands in them is not seen."""
    g, prev, W1, W2 = markov_case(7, rows, V, rank)
    prev[3], prev[17], prev[rows - 1] = V, 2 ** 31 - 1, -5
    seen = g.clone()
    seen[[3, 17, rows - 1]] = 0
    g[3], g[17, 5], g[rows - 1] = NAN, INF, -INF
    gp, d1, d2, status = markov(B, g, prev, W1, W2)
    assert status == DEVICE_INPUT
    ref, tol = L.markov(seen, prev, W1, W2)
    close(gp, ref[0], tol[0], "grad_prev")
    close(d1, ref[1], tol[1], "dW1")
    close(d2, ref[2], tol[2], "dW2")


def test_markov_grad_no_rows(B):
    V, rank = 640, 64
    g, W = torch.empty(0, V, dtype=BF16, device="cuda"), torch.zeros(V, rank, dtype=BF16, device="cuda")
    prev = torch.empty(0, dtype=I32, device="cuda")
    _, d1, d2, _ = markov(B, g, prev, W, W, start=(3.0, 3.0))
    assert (d1 == 3).all() and (d2 == 0).all()
    _, d1, d2, _ = markov(B, g, prev, W, W, True, start=(3.0, 3.0))
    assert (d1 == 3).all() and (d2 == 3).all()


@pytest.mark.parametrize("rows,V,rank", [(5, 640, 64), (300, 4104, 512)])
def test_markov_grad_wait_that_runs_out(B, rows, V, rank):
    """Operands that are never complete: the call ends soon after the limit of 2 s for each of its two products, reports the
    timeout, and the next call is as good as ever."""
    g, prev, W1, W2 = markov_case(8, rows, V, rank)
    want = markov(B, g, prev, W1, W2)
    assert want[3] == 0
    assert B.dspark_set_fault_injection(B.DSPARK_INJECT_MARKOV_OPERANDS) == 0
    try:
        start = time.monotonic()
        _, _, _, status = markov(B, g, prev, W1, W2)
        took = time.monotonic() - start
    finally:
        assert B.dspark_set_fault_injection(0) == B.DSPARK_INJECT_MARKOV_OPERANDS
    assert status == B.DSPARK_ERR_TIMEOUT and 4.0 <= took < 6.0
    again = markov(B, g, prev, W1, W2)
    assert again[3] == 0 and all(torch.equal(a, b) for a, b in zip(again[:3], want[:3]))


@pytest.mark.parametrize("same", [True, False])
def test_markov_grad_equal_tokens(B, same):
    """One token before every row; the rows' sums go to one row of dW1."""
    rows, V, rank = 700, 264, 128
    g, prev, W1, W2 = markov_case(9, rows, V, rank)
    prev.fill_(V - 1) if same else prev.copy_(torch.arange(rows, device="cuda") % 3 * 100)
    gp, d1, d2, status = markov(B, g, prev, W1, W2)
    assert status == 0
    ref, tol = L.markov(g, prev, W1, W2)
    close(gp, ref[0], tol[0], "grad_prev")
    close(d1, ref[1], tol[1], "dW1")
    close(d2, ref[2], tol[2], "dW2")


def test_markov_grad_no_tokens(B):
    """No row has a token before it: nothing to learn, whatever stands in the rows."""
    rows, V, rank = 200, 1000, 64
    g, prev, W1, W2 = markov_case(10, rows, V, rank)
    prev.fill_(-1)
    g[:130] = NAN
    gp, d1, d2, status = markov(B, g, prev, W1, W2, start=(3.0, 3.0))
    assert status == 0 and (gp == 0).all() and (d1 == 3).all() and (d2 == 0).all()


def markov_holds(B, g, prev, W1, W2, status=0, accumulate=False, start=(0.0, 0.0), seen=None):
    """The three outputs against their definitions; `seen`: the gradient without what must not be seen."""
    V, rank = W1.shape
    gp, d1, d2, got = markov(B, g, prev, W1, W2, accumulate, start=start)
    assert got == status
    base = [torch.full((V, rank), x if accumulate else 0.0, device="cuda") for x in start]
    ref, tol = L.markov(g if seen is None else seen, prev, W1, W2, *base)
    there = torch.zeros(V, dtype=torch.bool, device="cuda")
    there[prev[(prev >= 0) & (prev < V)].long()] = True
    close(gp, ref[0], tol[0], "grad_prev")
    close(d1[there], ref[1][there], tol[1][there], "dW1")
    assert bool((d1[~there] == start[0]).all())
    close(d2, ref[2], tol[2], "dW2")
    return gp, d1, d2


@pytest.mark.parametrize("rows", [1, 7, 8, 9, 16, 17, 32, 33])
@pytest.mark.parametrize("V,rank,gap", [
    (8, 64, 0), (128, 192, 8), (2424, 320, 0), (9736, 448, 24), (40000, 256, 0), (80008, 512, 0),
    (160008, 64, 0), (100000, 128, 0), (120008, 192, 0), (90008, 320, 0), (70000, 384, 0), (60008, 448, 0),
])
def test_markov_grad_few_rows(B, rows, V, rank, gap):
    """A block's rows: fewer elements than CTAs, pieces of them that end inside a stretch, ranks that leave threads over."""
    g, prev, W1, W2 = markov_case(40 + rows, rows, V, rank, gap)
    markov_holds(B, g, prev, W1, W2, start=(7.0, 9.0))
    markov_holds(B, g, prev, W1, W2, accumulate=True, start=(0.5, -2.0))


@pytest.mark.parametrize("rows", [4, 13, 29])
def test_markov_grad_few_rows_tokens(B, rows):
    """Rows of one token, rows without one, and rows whose token is none, with anything in them and behind them."""
    V, rank = 5000, 128
    g, prev, W1, W2 = markov_case(60, rows, V, rank)
    prev.fill_(V - 1)
    markov_holds(B, g, prev, W1, W2)
    prev.copy_(torch.arange(rows, device="cuda") % 3)
    markov_holds(B, g, prev, W1, W2, accumulate=True, start=(1.0, 2.0))
    prev[1], prev[3], prev[rows - 2] = -1, V, -2 ** 31
    seen = g.clone()
    seen[[1, 3, rows - 2]] = 0
    g[1, ::7], g[3], g[rows - 2, V - 1] = NAN, INF, -INF
    markov_holds(B, g, prev, W1, W2, status=DEVICE_INPUT, seen=seen)
    prev.fill_(-1)
    gp, d1, d2, status = markov(B, g, prev, W1, W2, start=(3.0, 4.0))
    assert status == 0 and (gp == 0).all() and (d1 == 3).all() and (d2 == 0).all()


def test_markov_grad_few_rows_infinities(B):
    """An infinity in the factors or in a row reaches what it takes part in, and nothing else."""
    rows, V, rank = 5, 3000, 64
    g, prev, W1, W2 = markov_case(61, rows, V, rank)
    g = torch.where(g == 0, torch.ones_like(g), g)
    prev.copy_(i32([4, -1, 9, 9, 2000]))
    W2[77, 3] = INF
    gp, d1, d2, status = markov(B, g, prev, W1, W2)
    assert status == 0 and (gp[1] == 0).all() and torch.isfinite(d2).all()
    odd = ~torch.isfinite(gp)
    assert odd[[0, 2, 3, 4], 3].all() and int(odd.sum()) == 4
    odd = ~torch.isfinite(d1)
    assert odd[[4, 9, 2000], 3].all() and int(odd.sum()) == 3
    W2[77, 3] = 0
    g[2, 1234] = NAN
    gp, d1, d2, status = markov(B, g, prev, W1, W2)
    odd = ~torch.isfinite(gp)
    assert status == 0 and odd[2].all() and int(odd.sum()) == rank
    odd = ~torch.isfinite(d1)
    assert odd[9].all() and int(odd.sum()) == rank
    odd = ~torch.isfinite(d2)
    assert odd[1234].all() and int(odd.sum()) == rank


@pytest.mark.parametrize("rows", [9, 20])
@pytest.mark.parametrize("want", [(False, False), (True, False), (False, True)])
def test_markov_grad_few_rows_in_part(B, want, rows):
    g, prev, W1, W2 = markov_case(62, rows, 2000, 128)
    all_of = markov(B, g, prev, W1, W2)
    some = markov(B, g, prev, W1, W2, want=want)
    for a, b in zip(all_of[:3], some[:3]):
        assert b is None or torch.equal(a, b)


def test_markov_grad_few_rows_replayed(B):
    """Calls of a few rows and of many on one workspace, captured and replayed on new rows: the bits of calls by themselves."""
    V, rank = 4104, 320
    sets = [markov_case(70 + k, rows, V, rank) for k, rows in enumerate((7, 200, 16, 1, 31, 7))]
    want = [markov(B, *s)[:3] for s in sets]
    ws = B.workspace(max(B.dspark_workspace_size(B.DSPARK_OP_MARKOV_GRAD, 0, 0, V, rank, s[0].shape[0]) for s in sets))
    at = [[torch.zeros_like(x) for x in s] for s in sets]
    got = [[torch.full_like(x, 9.0) for x in w] for w in want]
    for o in got:
        o[1].zero_()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        for (g, prev, W1, W2), (gp, d1, d2) in zip(at, got):
            B.dspark_markov_grad(g, prev, W1, W2, gp, dW1=d1, dW2=d2, ws=ws)
    for s, t in zip(sets, at):
        for x, y in zip(s, t):
            y.copy_(x)
    for _ in range(3):
        for o in got:
            o[1].zero_()
        graph.replay()
        torch.cuda.synchronize()
        for o, w in zip(got, want):
            assert all(torch.equal(a, b) for a, b in zip(o, w))


# ------------------------------------------------------------------------------------------- all of them
def chain(B, w, d, T=1.0, top=16):
    """A cycle's rows through the three of them: what the target says, what the drafter makes of it, what its head learns."""
    from speculative_decoding_dspark_gb300 import inputs
    R, gamma, V, rank = w["R"], w["gamma"], w["V"], w["rank"]
    g = H.gpu_draft(d, T, 0)
    target = H.dev(inputs.target_full(w, d["U"])[:, :gamma].reshape(R * gamma, V))
    rows = R * gamma
    ids, val = torch.empty(rows, top, dtype=I32, device="cuda"), torch.empty(rows, top, device="cuda")
    status = torch.zeros(1, dtype=I32, device="cuda")
    student = g["q_logits_dev"].reshape(rows, V)
    loss, grad = torch.empty(rows, device="cuda"), torch.empty(rows, V, dtype=BF16, device="cuda")
    prev = torch.cat([H.dev(d["anchor"])[:, None], g["y_dev"][:, :-1]], 1).reshape(-1).contiguous()
    W1, W2 = H.dev(d["W1"]), H.dev(d["W2"])
    gp, d1, d2 = torch.empty(rows, rank, device="cuda"), torch.zeros(V, rank, device="cuda"), torch.empty(V, rank, device="cuda")
    ws = B.workspace(B.dspark_workspace_size(B.DSPARK_OP_MARKOV_GRAD, 0, 0, V, rank, rows))

    def run(stream=None):
        B.dspark_token_logprobs(target, None, T, None, None, None, ids, val, dev_status=status, stream=stream)
        B.dspark_distill_loss(student, ids, val, 1.0, loss, grad=grad, rest=True, dev_status=status, stream=stream)
        B.dspark_markov_grad(grad, prev, W1, W2, gp, dW1=d1, dW2=d2, ws=ws, dev_status=status, stream=stream)
    outs = dict(ids=ids, val=val, loss=loss, grad=grad, gp=gp, d1=d1, d2=d2)
    return run, outs, status, dict(target=target, student=student, prev=prev, W1=W1, W2=W2)


def test_chain(B):
    w, d = H.cycle_inputs("batched_sampling", R=9, V=4096, gamma=5, rank=64, w_sigma=0.2)
    run, o, status, i = chain(B, w, d)
    run()
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    ref, tol = L.logprobs(i["target"], None, 1.0, 16)
    assert torch.equal(o["ids"].long(), ref[3])
    close(o["val"], ref[4], tol[3], "teacher")
    ref, tol = L.distill(i["student"], o["ids"], o["val"], 1.0, None, True, BF16)
    close(o["loss"], ref[0], tol[0], "loss")
    close(o["grad"], ref[1], tol[1], "grad")
    ref, tol = L.markov(o["grad"], i["prev"], i["W1"], i["W2"])
    for name, r, t in zip(("gp", "d1", "d2"), ref, tol):
        close(o[name], r, t, name)


def test_chain_in_a_graph_and_on_another_stream(B):
    """Captured once, replayed on changed inputs: the same bits as calls one by one, on a stream of their own."""
    w, d = H.cycle_inputs("batched_sampling", R=9, V=4096, gamma=5, rank=64, w_sigma=0.2)
    run, o, status, i = chain(B, w, d)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        run()
    torch.cuda.synchronize()
    first = {k: v.clone() for k, v in o.items()}
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    for v in o.values():
        v.zero_()
    graph.replay()
    torch.cuda.synchronize()
    for k in o:
        assert torch.equal(o[k], first[k]), k
    i["target"].copy_(i["target"].roll(1, 0))
    i["student"].mul_(0.5)
    for v in o.values():
        v.zero_()
    graph.replay()
    torch.cuda.synchronize()
    again = {k: v.clone() for k, v in o.items()}
    for v in o.values():
        v.zero_()
    run(side.cuda_stream)
    torch.cuda.synchronize()
    for k in o:
        assert torch.equal(o[k], again[k]), k
    assert int(status.item()) == 0


def test_markov_grad_calls_in_turn(B):
    """Calls one after the other without a wait, one workspace and one set of buffers whose contents change in between."""
    rows, V, rank = 300, 4104, 320
    sets = [markov_case(k, rows, V, rank) for k in (31, 32, 33)]
    want = [markov(B, *s)[:3] for s in sets]
    g, prev, W1, W2 = (t.clone() for t in sets[0])
    gp, d1, d2 = torch.empty(rows, rank, device="cuda"), torch.zeros(V, rank, device="cuda"), torch.empty(V, rank, device="cuda")
    ws = B.workspace(B.dspark_workspace_size(B.DSPARK_OP_MARKOV_GRAD, 0, 0, V, rank, rows))
    got = []
    for k in [0, 1, 2, 0, 0, 2, 1, 1, 0] * 3:
        for to, source in zip((g, prev, W1, W2), sets[k]):
            to.copy_(source)
        d1.zero_()
        B.dspark_markov_grad(g, prev, W1, W2, gp, dW1=d1, dW2=d2, ws=ws)
        got.append((k, gp.clone(), d1.clone(), d2.clone()))
    torch.cuda.synchronize()
    for k, *o in got:
        assert all(torch.equal(a, b) for a, b in zip(o, want[k]))


def test_two_streams_at_once(B):
    """The chain on two streams at the same time, each with buffers and a workspace of its own."""
    runs, outs = [], []
    for k in range(2):
        w, d = H.cycle_inputs("batched_sampling", seed_offset=k, R=40, V=8192, gamma=5, rank=128, w_sigma=0.2)
        run, o, status, _ = chain(B, w, d)
        run()
        torch.cuda.synchronize()
        runs.append(run)
        outs.append((o, {n: t.clone() for n, t in o.items()}, status))
    streams = [torch.cuda.Stream() for _ in runs]
    for o, _, _ in outs:
        for t in o.values():
            t.zero_()
    torch.cuda.synchronize()
    for _ in range(10):
        for run, stream in zip(runs, streams):
            run(stream.cuda_stream)
    torch.cuda.synchronize()
    for o, first, status in outs:
        assert int(status.item()) == 0 and all(torch.equal(o[n], first[n]) for n in o)


def test_offsets_past_32_bits(B):
    """More than 2^31 elements in the rows, and a stride that passes 2^31 bytes: the last rows are as good as the first."""
    rows, V, rank = 17001, 129280, 64
    x = torch.empty(rows, V, dtype=BF16, device="cuda")
    for a in range(0, rows, 1000):
        x[a:a + 1000].normal_(0.0, 3.0, generator=generator(a))
    assert x.numel() > 2 ** 31
    pick = torch.tensor([0, 1, 16611, 16612, rows - 2, rows - 1], device="cuda")  # row 16612 holds element 2^31
    tokens = torch.randint(0, V, (rows,), generator=generator(1), device="cuda", dtype=I32)
    lp, lse, ent, ids, val, status = logprobs(B, x, tokens, 1.0, 8)
    assert status == 0
    ref, tol = L.logprobs(x[pick], tokens[pick], 1.0, 8)
    for got, r, t in zip((lp, lse, ent, val), (ref[0], ref[1], ref[2], ref[4]), tol):
        close(got[pick], r, t, "logprobs")
    assert torch.equal(ids[pick].long(), ref[3])
    ref, tol = L.distill(x[pick], ids[pick], val[pick], 2.0, None, True, BF16)
    loss, g, status = distill(B, x, ids, val, 2.0, rest=True, in_place=True)
    assert status == 0
    close(loss[pick], ref[0], tol[0], "loss")
    close(g[pick], ref[1], tol[1], "grad")
    W1, W2 = (normal(k, (V, rank), 0.05).to(BF16) for k in (1, 2))
    prev = torch.arange(rows, device="cuda", dtype=I32)
    gp, d1, d2, status = markov(B, g, prev, W1, W2)
    assert status == 0
    ref, tol = L.markov(g[pick], prev[pick], W1, W2)
    close(gp[pick], ref[0], tol[0], "grad_prev")
    close(d1[pick], ref[0], tol[0], "dW1")
    part = g[:, -16:].double()
    E = W1[:rows].double()
    steps = (64 + rows / 1024 + 152) * 2.0 ** -22
    close(d2[-16:], part.T @ E, steps * (part.abs().T @ E.abs()), "dW2")
    # rows that lie far apart
    far = torch.empty(3 * 2 ** 30, dtype=BF16, device="cuda").as_strided((3, 1001), (2 ** 30 + 5, 1), 3)
    far.copy_(normal(2, (3, 1001), 3.0))
    check_logprobs(B, far, i32([0, 1000, 500]), 1.0, 5)
    ids, value = teacher_of(3, far, 5)
    check_distill(B, far, ids, value, 1.0, BF16, rest=True, in_place=True)


def test_same_results_every_time(B):
    x = normal(21, (40, 50001), 3.0).to(BF16)
    ids, value = teacher_of(22, x, 64)
    a = distill(B, x, ids, value, 1.0, BF16, rest=True)
    b = distill(B, x, ids, value, 1.0, BF16, rest=True)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    p, q = logprobs(B, x, None, 1.0, 128), logprobs(B, x, None, 1.0, 128)
    assert all(torch.equal(u, v) for u, v in zip(p[:5], q[:5]))
    g, prev, W1, W2 = markov_case(23, 500, 8200, 320)
    s, t = markov(B, g, prev, W1, W2), markov(B, g, prev, W1, W2)
    assert all(torch.equal(u, v) for u, v in zip(s[:3], t[:3]))


def test_binding_refuses(B):
    x = normal(24, (4, 64))
    lp, tok = torch.empty(4, device="cuda"), i32([0] * 4)
    top = torch.empty(4, 2, dtype=I32, device="cuda")
    with pytest.raises(ValueError):
        B.dspark_token_logprobs(x, tok[:3], 1.0, lp)
    with pytest.raises(ValueError):
        B.dspark_token_logprobs(x, tok, 1.0, lp, top_ids=top)
    with pytest.raises(ValueError):
        B.dspark_token_logprobs(x.t(), tok, 1.0, lp)
    with pytest.raises(ValueError):
        B.dspark_token_logprobs(x, tok, 1.0, lp, cu_seqlens=i32([0, 4]))
    with pytest.raises(TypeError):
        B.dspark_token_logprobs(x.half(), tok, 1.0, lp)
    with pytest.raises(TypeError):
        B.dspark_token_logprobs(x, tok.long(), 1.0, lp)
    with pytest.raises(B.DSparkError):
        B.dspark_token_logprobs(x, tok, 0.0, lp)
    with pytest.raises(ValueError):
        B.dspark_distill_loss(x, top, torch.empty(4, 3, device="cuda"), 1.0, lp)
    with pytest.raises(ValueError):
        B.dspark_distill_loss(x, top, torch.empty(4, 2, device="cuda"), 1.0, lp, grad=torch.empty(4, 65, device="cuda"))
    with pytest.raises(B.DSparkError):
        B.dspark_distill_loss(x[:1].expand(4, 64), top, torch.empty(4, 2, device="cuda"), 1.0, lp)
    W = torch.empty(64, 64, dtype=BF16, device="cuda")
    with pytest.raises(TypeError):
        B.dspark_markov_grad(x, tok, W, W, torch.empty(4, 64, device="cuda"), ws=B.workspace(1 << 20))
    with pytest.raises(B.DSparkError):
        B.dspark_markov_grad(x.to(BF16), tok, W, W, torch.empty(4, 64, device="cuda"), ws=B.workspace(256))


def test_two_host_threads(B):
    """Two host threads that call at once, with rows of different lengths: neither's call disturbs the other's."""
    import threading
    cases, errors = [], []
    for V, top in ((151936, 128), (700, 3)):
        x = normal(V, (5, V), 3.0)
        ids, value = teacher_of(V, x, top)
        want = logprobs(B, x, None, 1.0, top)[:5] + distill(B, x, ids, value, 1.0, F32, rest=True)[:2]
        cases.append((x, ids, value, top, want))

    def work(x, ids, value, top, want):
        try:
            stream = torch.cuda.Stream()
            lp, lse, ent = (torch.empty(5, device="cuda") for _ in range(3))
            oi, ov = torch.empty(5, top, dtype=I32, device="cuda"), torch.empty(5, top, device="cuda")
            loss, g = torch.empty(5, device="cuda"), torch.empty_like(x)
            stream.wait_stream(torch.cuda.default_stream())
            for _ in range(200):
                B.dspark_token_logprobs(x, None, 1.0, lp, lse, ent, oi, ov, stream=stream)
                B.dspark_distill_loss(x, ids, value, 1.0, loss, grad=g, rest=True, stream=stream)
            stream.synchronize()
            for a, b in zip((lp, lse, ent, oi, ov, loss, g), want):
                if not torch.equal(a, b):
                    errors.append("results differ")
        except Exception as e:  # noqa: BLE001 (shown by the test's own thread)
            errors.append(repr(e))
    torch.cuda.synchronize()
    threads = [threading.Thread(target=work, args=c) for c in cases]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors
