"""Where the operators on vocabulary rows and of the Markov factors' gradient could go wrong and test_gpu_learning.py does
not look: clusters that start beside other work, rests next to nothing, single terms of long sums, long chains, tokens
that repeat, buffers kept for the largest call, a verify's packed rows."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

import learning_reference as L  # noqa: E402
import parity_helpers as H  # noqa: E402
from test_gpu_learning import (BF16, F32, I32, B, close, distill, generator, i32, logprobs, markov,  # noqa: E402,F401
                               markov_case, normal, rows_of, teacher_of)


# ----------------------------------------------------------------------------------------- distillation
@pytest.mark.parametrize("V", [4001, 8003, 32003])
def test_distill_beside_other_work(B, V):
    """Rows shared by two, four and eight CTAs, whose clusters find room one CTA of theirs after the other while another
    stream fills the GPU: the bits of a call by itself."""
    rows, top = 5, 20
    x = normal(V, (rows, V), 3.0)
    ids, value = teacher_of(V, x, top)
    want = distill(B, x, ids, value, 1.0, F32, rest=True)
    assert want[2] == 0
    other, side = torch.cuda.Stream(), torch.cuda.Stream()
    a = normal(1, (1 << 24,))
    losses, grads = torch.empty(40, rows, device="cuda"), torch.empty(40, rows, V, device="cuda")
    status = torch.zeros(1, dtype=I32, device="cuda")
    torch.cuda.synchronize()
    for k in range(40):
        with torch.cuda.stream(other):
            a.mul_(1.0)
            a.view(-1, 64).sum(1)
        B.dspark_distill_loss(x, ids, value, 1.0, losses[k], grad=grads[k], rest=True, dev_status=status, stream=side)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    assert all(torch.equal(losses[k], want[0]) and torch.equal(grads[k], want[1]) for k in range(40))


@pytest.mark.parametrize("grad", [F32, None])
@pytest.mark.parametrize("others,left", [(5e-7, 5e-7), (1e-3, 1e-6), (0.4, 1e-5), (0.2, 1e-4), (0.3, 0.0), (0.0, 3e-8), (0.2, 1e-3)])
def test_distill_a_rest_next_to_nothing(B, others, left, grad):
    """A teacher that leaves next to nothing to the tokens that are not listed, and a drafter that leaves them twice as
    much: what their gradient is depends on every bit of the difference.

    The teacher's share of the rest is (1 - p of its surest token) - sum of the others, in 32 bits: the first off by a step
    of it (2u), the others by a step each and eight sums (10u), the difference by u: 13u (1 - p_top) in all, u = 2^-24,
    and the listed mass likewise by 13u where nothing is left; where less than 2^-10 of what the surest token leaves is
    left, it is taken in 64 bits (a sum of 64 exponentials: below 2^-46) and rounded.  The rest as in
    learning_reference.py: q (3u|a| + v + e_s + 12u), the share of the rest likewise with its own reference, the
    roundings of the type."""
    rows, V, top = 4, 3000, 64
    p = torch.rand(rows, top, generator=generator(31), device="cuda", dtype=torch.float64)
    p[:, 1:] *= others / p[:, 1:].sum(1, keepdim=True)
    p[:, 0] = 1 - others - left
    value = p.log().float()
    ids = torch.stack([torch.randperm(V, generator=generator(k), device="cuda")[:top] for k in range(rows)]).to(I32)
    exact_left = (1 - value.double().exp().sum(1)).clamp(min=0)
    free = torch.ones(rows, V, dtype=torch.bool, device="cuda").scatter_(1, ids.long(), False)
    x = normal(32, (rows, V), 0.5) + np.log(2 * max(left, 1e-7) / V)
    x.scatter_(1, ids.long(), value.clamp(min=-80.0))
    loss, g, status = distill(B, x, ids, value, 1.0, grad, rest=True)
    assert status == 0
    ref, tol = L.distill(x, ids, value, 1.0, None, True, grad)
    close(loss, ref[0], tol[0], "loss")
    if grad is None:
        return
    close(g, ref[1], tol[1], "grad")
    t, m, a, q, log_s, e_s, a1, a2, _, _ = L._sums(x, 1.0)
    free_a = torch.where(free, a, torch.full_like(a, L.NEG))
    share = torch.softmax(free_a, 1)
    extra = exact_left[:, None] * share
    own = 3 * L.U * (a - free_a.amax(1, keepdim=True)).abs()
    want = q - extra
    beside = -torch.expm1(value[:, :1].double())
    d_left = torch.where(exact_left[:, None] < beside * 2.0 ** -11, L.U * exact_left[:, None] + 2.0 ** -46, 13 * L.U * beside)
    tol = (q * (3 * L.U * a.abs() + L.V2 + e_s[:, None] + 25 * L.U) + extra * (own + 2 * L.V2 + 2 * e_s[:, None] + 8 * L.U) +
           share * d_left + 5 * L.U * want.abs() + 2.0 ** -120)
    close(g[free], want[free], tol[free], "the rest's gradient")


# ------------------------------------------------------------------------------ the Markov factors' gradient
def grad_prev_of(g, W2):
    """sum_v g W2 and sum_v |g W2| in 64 bits, a stretch of V at a time."""
    s, size = (torch.zeros(g.shape[0], W2.shape[1], dtype=torch.float64, device="cuda") for _ in range(2))
    for a in range(0, g.shape[1], 1 << 17):
        x, y = g[:, a:a + (1 << 17)].double(), W2[a:a + (1 << 17)].double()
        s += x @ y
        size += x.abs() @ y.abs()
    return s, size


@pytest.mark.parametrize("rows", [7, 16, 17, 32, 33])
@pytest.mark.parametrize("V,rank", [((1 << 21) + 8, 512), ((1 << 22), 64), (151936, 512)])
def test_markov_grad_long_sums(B, rows, V, rank):
    """Terms of one sign: what an accumulator cuts off goes the same way every time.

    A chain ends after 512 terms, 32 steps of which each may cut off 2^-22 of the sum so far; the chains' sums (at most 64
    to a warp or part here), those of eight groups, of two CTAs and of 152 parts are added in fp32, u each."""
    g = normal(rows, (rows, V)).abs_().to(BF16)
    W2 = torch.empty(V, rank, dtype=BF16, device="cuda").normal_(0.0, 0.05, generator=generator(2)).abs_()
    W1 = torch.zeros(V, rank, dtype=BF16, device="cuda")
    prev = torch.arange(rows, device="cuda", dtype=I32)
    gp, _, _, status = markov(B, g, prev, W1, W2, want=(False, False))
    assert status == 0
    ref, size = grad_prev_of(g, W2)
    close(gp, ref, (32 * 2.0 ** -22 + (64 + 8 + 2 + 152) * L.U) * size, "grad_prev")


@pytest.mark.parametrize("rows", [1, 7, 16, 17, 32, 33, 128, 129, 300])
@pytest.mark.parametrize("V,rank", [(8, 64), (640, 192), (40008, 256), (80008, 512), (151936, 64), (151936, 512)])
def test_markov_grad_every_term(B, rows, V, rank):
    """Whole numbers whose sums fp32 holds exactly, in any order: every term is there once, in all three gradients."""
    g = torch.randint(-2, 3, (rows, V), generator=generator(V + rows), device="cuda").to(BF16)
    W1, W2 = (torch.randint(-3, 4, (V, rank), generator=generator(V + k), device="cuda").to(BF16) for k in (1, 2))
    prev = torch.randint(-1, max(1, min(V, rows // 2 + 1)), (rows,), generator=generator(3), device="cuda", dtype=I32)
    assert V * 6 < 2 ** 24 and rows * V * 6 < 2 ** 53
    gp, d1, d2, status = markov(B, g, prev, W1, W2)
    assert status == 0
    there = prev >= 0
    want, _ = grad_prev_of(g, W2)
    want *= there[:, None]
    assert torch.equal(gp.double(), want)
    at = prev.clamp(min=0).long()
    sums = torch.zeros(V, rank, dtype=torch.float64, device="cuda").index_add_(0, at, want)
    assert float(sums.abs().max()) < 2 ** 24 and torch.equal(d1.double(), sums)
    E = W1.double()[at] * there[:, None]
    assert torch.equal(d2.double(), g.double().t() @ E)


@pytest.mark.parametrize("rows,rank", [(7, 256), (20, 512), (33, 64), (200, 512)])
def test_markov_grad_last_terms(B, rows, rank):
    """A gradient of one element, at the beginnings and ends of what CTAs, stages and parts may have."""
    V = 50008
    W1, W2 = (normal(k, (V, rank)).to(BF16) for k in (4, 5))
    prev = torch.arange(rows, device="cuda", dtype=I32) % 5
    places = [0, 15, 16, 63, 64, 127, 128, 255, 256, V // 2, V - 257, V - 65, V - 64, V - 17, V - 16, V - 9, V - 8, V - 1]
    for v in places:
        g = torch.zeros(rows, V, dtype=BF16, device="cuda")
        g[rows - 1, v] = 2.0
        gp, d1, d2, status = markov(B, g, prev, W1, W2)
        assert status == 0
        want = torch.zeros_like(gp)
        want[rows - 1] = 2 * W2[v].float()
        assert torch.equal(gp, want), v
        assert torch.equal(d1[int(prev[rows - 1])], want[rows - 1]) and int((d1 != 0).any(1).sum()) == 1, v
        assert torch.equal(d2[v], 2 * W1[int(prev[rows - 1])].float()) and int((d2 != 0).any(1).sum()) == 1, v


@pytest.mark.parametrize("rows,V,rank", [(2560, 136, 512), (20000, 64, 64), (4100, 72, 320), (33, 64, 64)])
@pytest.mark.parametrize("every", [1, 3])
def test_markov_grad_many_equal_tokens(B, rows, V, rank, every):
    """One token before all rows, or three in turn: dW1's error does not grow with their number.

    A compensated sum of n terms: 2u sum |x| and the second order, n u^2 sum |x|, a few times (here four); then the sum to
    the given value, one rounding."""
    g = normal(rows, (rows, V)).abs_().to(BF16)
    W1, W2 = (normal(k, (V, rank)).abs_().to(BF16) for k in (1, 2))
    prev = (torch.arange(rows, device="cuda") % every * 7).to(I32)
    for accumulate, start in ((False, 3.0), (True, 3.0)):
        gp, d1, _, status = markov(B, g, prev, W1, W2, accumulate, want=(True, False), start=(start, 0.0))
        assert status == 0
        for t in range(every):
            x = gp[prev == 7 * t].double()
            size = x.abs().sum(0) + start * accumulate
            want = x.sum(0) + start * accumulate
            close(d1[7 * t], want, (2 * L.U + 4 * rows * L.U ** 2) * size + L.U * want.abs(), "dW1")
        assert bool((d1[1:7] == start).all())


def test_markov_grad_equal_tokens_infinite(B):
    """An infinity among the rows of a token stays one in its sum, two of them of either sign are none."""
    rows, V, rank = 200, 136, 64
    g, prev, W1, W2 = markov_case(12, rows, V, rank)
    g = torch.where(g == 0, torch.ones_like(g), g).abs()
    prev.copy_(torch.arange(rows, device="cuda") % 2)
    W2.zero_()
    W2[0] = 1.0
    g[20, 0], g[21, 0], g[101, 0] = float("inf"), float("inf"), -float("inf")
    gp, d1, _, status = markov(B, g, prev, W1, W2, want=(True, False))
    assert status == 0 and bool((gp[20] == float("inf")).all()) and bool((gp[101] == -float("inf")).all())
    assert bool((d1[0] == float("inf")).all()) and bool(d1[1].isnan().all())


@pytest.mark.parametrize("V,rank,most", [(4104, 64, 700), (32000, 256, 896)])
def test_markov_grad_workspace_of_the_largest_call(B, V, rank, most):
    """One workspace, as large as the largest call's, holds calls of any fewer rows: the bits of calls with their own."""
    g, prev, W1, W2 = markov_case(17, most, V, rank)
    ws = B.workspace(B.dspark_workspace_size(B.DSPARK_OP_MARKOV_GRAD, 0, 0, V, rank, most))
    status = torch.zeros(1, dtype=I32, device="cuda")
    for rows in (1, 16, 17, 32, 33, 64, 128, 129, 256, 257, 400, 512, 513, 640, most):
        want = markov(B, g[:rows], prev[:rows], W1, W2)
        gp, d1, d2 = (torch.zeros_like(x) for x in want[:3])
        B.dspark_markov_grad(g[:rows], prev[:rows], W1, W2, gp, dW1=d1, dW2=d2, ws=ws, dev_status=status)
        assert all(torch.equal(a, b) for a, b in zip((gp, d1, d2), want[:3])), rows
    assert int(status.item()) == 0


# ------------------------------------------------------------------------------------------- all of them
def test_chain_on_a_verify_s_packed_rows(B):
    """From the rows a verify read to the factors' gradient.  The target's rows are packed (cu_seqlens[r] + j), the
    drafter's lie by blocks (r * gamma + j): the teacher's lists are laid beside the drafter's rows, and rows that no
    target row stands beside (behind a request's length) have no list: loss and gradient 0.  A request's last packed row is
    the bonus token's, beside which the drafter has nothing."""
    from speculative_decoding_dspark_gb300 import inputs
    R, gamma, V, rank, top, T = 17, 5, 8192, 64, 16, 0.7
    w, d = H.cycle_inputs("varlen_verify", R=R, V=V, gamma=gamma, rank=rank, w_sigma=0.2)
    g = H.gpu_draft(d, T, 2)
    l = inputs.verify_lengths(w)
    assert l.min() < gamma and l.max() > 0
    target = H.dev(inputs.pack_rows(inputs.target_full(w, d["U"]), l))
    cu = H.dev(inputs.cu_from_lengths(l))
    rows = target.shape[0]
    status = torch.zeros(1, dtype=I32, device="cuda")
    n_acc, out = torch.empty(R, dtype=I32, device="cuda"), torch.empty(R, gamma + 1, dtype=I32, device="cuda")
    ws = B.workspace(max(B.dspark_workspace_size(B.DSPARK_OP_VERIFY, R, gamma, V, 0, rows),
                         B.dspark_workspace_size(B.DSPARK_OP_MARKOV_GRAD, 0, 0, V, rank, R * gamma)))
    B.dspark_verify(target, cu, g["y_dev"], g["q_logits_dev"], g["q_lse_dev"], g["q_tok_dev"], H.dev(d["seeds"]), 2, T, rows,
                    n_acc, out, None, ws, dev_status=status)
    ids, val = torch.empty(rows, top, dtype=I32, device="cuda"), torch.empty(rows, top, device="cuda")
    B.dspark_token_logprobs(target, None, T, None, None, None, ids, val, dev_status=status)
    # each packed row's place among the drafter's
    row = torch.arange(rows, device="cuda")
    r = torch.searchsorted(cu.long(), row, right=True) - 1
    j = row - cu.long()[r]
    drafted = (j < H.dev(l).long()[r]).nonzero()[:, 0]
    at = (r * gamma + j)[drafted]
    teacher_ids = torch.full((R * gamma, top), -1, dtype=I32, device="cuda")
    teacher = torch.zeros(R * gamma, top, device="cuda")
    teacher_ids[at], teacher[at] = ids[drafted], val[drafted]
    # (q_logits are scaled already: temperature 1, and the gradient of U + W2 W1[prev] has 1 / T more)
    student = g["q_logits_dev"].reshape(R * gamma, V)
    weight = torch.full((R * gamma,), 1 / T, device="cuda")
    loss, grad = torch.empty(R * gamma, device="cuda"), torch.empty(R * gamma, V, dtype=BF16, device="cuda")
    B.dspark_distill_loss(student, teacher_ids, teacher, 1.0, loss, grad=grad, row_weight=weight, rest=True, dev_status=status)
    prev = torch.cat([H.dev(d["anchor"])[:, None], g["y_dev"][:, :-1]], 1).reshape(-1).contiguous()
    W1, W2 = H.dev(d["W1"]), H.dev(d["W2"])
    gp, d1, d2 = (torch.zeros(*s, device="cuda") for s in ((R * gamma, rank), (V, rank), (V, rank)))
    B.dspark_markov_grad(grad, prev, W1, W2, gp, dW1=d1, dW2=d2, ws=ws, dev_status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    # every step against its definition, row by row of a block: the target's row for position j stands at cu[r] + j
    behind = torch.ones(R * gamma, dtype=torch.bool, device="cuda")
    for q in range(R):
        n = int(l[q])
        behind[q * gamma:q * gamma + n] = False
        if n == 0:
            continue
        first = int(cu[q])
        ref, _ = L.logprobs(target[first:first + n], None, T, top)
        mine = slice(q * gamma, q * gamma + n)
        assert torch.equal(teacher_ids[mine].long(), ref[3])
        ref, tol = L.distill(student[mine], ids[first:first + n], val[first:first + n], 1.0, weight[mine], True, BF16)
        close(loss[mine], ref[0], tol[0], "loss")
        close(grad[mine], ref[1], tol[1], "grad")
    assert bool(behind.any()) and bool((loss[behind] == 0).all()) and bool((grad[behind] == 0).all())
    ref, tol = L.markov(grad, prev, W1, W2)
    for got, want, t, name in zip((gp, d1, d2), ref, tol, ("grad_prev", "dW1", "dW2")):
        close(got, want, t, name)
