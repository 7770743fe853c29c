"""64-bit definitions of the operators on vocabulary rows (token log probabilities, distillation, the Markov factors'
gradient), and how far an output may be from them.

Formulas as in include/dspark.h, in float64 on the device of the inputs.

Tolerances (u = 2^-24, half a step of fp32; v = 2^-21 covers the base-2 exponential's and the logarithm's own
error, 2^-22 each, with the roundings of their arguments' constants):

* a term e_v = exp(t_v - m): its exponent a is off by 3u|a| (difference, product, scale), so e_v by 3u|a| + v.
* their sum s: the terms' errors, weighted by p: e_s = 3u A1 + v + depth u, A1 = sum p |t - m|.  A thread adds
  V / 256 terms (in two chains; a row shared by several blocks: fewer) and rescales once a batch of at least 16,
  each time by a factor off by v; ten joins follow: depth = V / 256 + 40, rescalings V / 4096 + 30, v each.
* log s is then off by e_s + v + u|log s|; lse by that and 3u|m| + u|lse|; logprob by that and 3u|t - m| + u|logprob|.
* entropy = log s - sum p |a|: the sum is off by (3u A2 + (v + e_s) A1 + depth u A1) + e_s A1, A2 = sum p a^2, and
  rescaled as s is.
* the teacher's p_k are off by e_p = 2v + 3u|value| + 32u each (sum of up to 128 by a tree), p_rest by 2 (e_p mass + 2u).
* a loss: sum of p (err(log p) + err(log q)) + e_p p |log p - log q|, and for the rest its p_rest's error times
  (|log p_rest| + |log q_rest| + 1); 128 terms by a tree: 16u of the sum of magnitudes.
* a gradient: q M (3u|a| + v + e_s + 8u) + p e_p + the rest's share likewise and with p_rest's error; then the
  rounding of the type, u or 2^-9.
* a product's sum (the Markov factors): the tensor cores add 16 products at a time to an accumulator and may cut off
  what lies below it: 2^-22 of the sum of magnitudes for each of the 32 steps of a chain, and likewise for the chains
  of a part and the parts, at most 152, added in fp32: (64 + K / 1024 + 152) 2^-22 of sum |a b| is never passed (K / 512
  chains in all, of which a part has K / 512 over the number of parts; up to K = 180000 in one part).
"""
from __future__ import annotations

import torch

U = 2.0 ** -24
UBF = 2.0 ** -8
V2 = 2.0 ** -21
NEG = float("-inf")


def _sums(x, invT):
    """t - max t, p, log s, e_s and the moments A1, A2 of |t - max t| of the rows of x."""
    V = x.shape[1]
    t = x.double() * invT
    m = t.amax(1, keepdim=True)
    a = t - m
    e = a.exp()
    s = e.sum(1, keepdim=True)
    p = e / s
    near = torch.where(p > 0, a.abs(), torch.zeros_like(a))
    a1, a2 = (p * near).sum(1), (p * near * near).sum(1)
    depth, rescale = V / 256 + 40, V / 4096 + 30
    e_s = 3 * U * a1 + V2 + depth * U + rescale * V2
    return t, m[:, 0], a, p, s.log()[:, 0], e_s, a1, a2, depth, rescale


def invT32(T):
    return float(torch.tensor(1.0, dtype=torch.float32) / torch.tensor(T, dtype=torch.float32))


def logprobs(x, token, T, top_k):
    """(logprob, lse, entropy, ids, values) of rows x [n, V] with tokens [n] (or None), and the tolerances of the floats."""
    invT = invT32(T)
    t, m, a, p, log_s, e_s, a1, a2, depth, rescale = _sums(x, invT)
    lse = m + log_s
    e_log = e_s + V2 + U * log_s.abs()
    lse_tol = e_log + 3 * U * m.abs() + U * lse.abs()
    entropy = log_s + (p * torch.where(p > 0, -a, torch.zeros_like(a))).sum(1)
    entropy_tol = e_log + 3 * U * a2 + (V2 * (2 + rescale) + 2 * e_s + (depth + 4) * U) * a1 + U * entropy.abs()

    def value(ids):
        at = a.gather(1, ids)
        y = at - log_s[:, None]
        return y, e_log[:, None] + 3 * U * at.abs() + U * y.abs()
    if token is None:
        lp = lp_tol = torch.zeros_like(lse)
    else:
        lp, lp_tol = (z[:, 0] for z in value(token.long()[:, None]))
    n, V = x.shape
    k = min(top_k, V)
    order = torch.sort(x.double() + 0.0, dim=1, descending=True, stable=True)
    ids = torch.full((n, top_k), -1, dtype=torch.int64, device=x.device)
    values = torch.full((n, top_k), NEG, dtype=torch.float64, device=x.device)
    values_tol = torch.zeros_like(values)
    if k:
        listed = order.values[:, :k] > NEG
        y, tol = value(order.indices[:, :k])
        ids[:, :k] = torch.where(listed, order.indices[:, :k], torch.full_like(order.indices[:, :k], -1))
        values[:, :k] = torch.where(listed, y, torch.full_like(y, NEG))
        values_tol[:, :k] = torch.where(listed, tol, torch.zeros_like(tol))
    return (lp, lse, entropy, ids, values), (lp_tol, lse_tol, entropy_tol, values_tol)


def distill(x, ids, value, T, weight=None, rest=False, out_dtype=None):
    """(loss, grad) of rows x [n, V], and their tolerances.  Good rows only: no NaN, no id twice."""
    n, V = x.shape
    invT = invT32(T)
    t, m, a, p_q, log_s, e_s, a1, a2, _, _ = _sums(x, invT)
    w = torch.ones(n, dtype=torch.float64, device=x.device) if weight is None else weight.double()
    ids, value = ids.long(), value.double()
    there = (ids >= 0) & (value > NEG)
    at = ids.clamp(min=0)
    val = torch.where(there, value, torch.zeros_like(value))
    raw = torch.where(there, (value if rest else value - torch.where(there, value, torch.full_like(value, -1e300)).amax(
        1, keepdim=True)).exp(), torch.zeros_like(value))
    mass = raw.sum(1, keepdim=True)
    e_p = 2 * V2 + 3 * U * val.abs() + 32 * U
    listed = torch.zeros(n, V + 1, dtype=torch.bool, device=x.device)
    listed.scatter_(1, torch.where(ids >= 0, ids, torch.full_like(ids, V)), True)
    free = ~listed[:, :V]
    if rest:
        p, log_p = raw, val
        # (from differences: beside a maximum of -3e38 the sum's logarithm would be lost in 64 bits too)
        free_a = torch.where(free, a, torch.full_like(a, NEG))
        log_rest = torch.logsumexp(free_a, 1) - log_s
        some = free_a.amax(1) > NEG
        p_rest = torch.where(some, (1.0 - mass[:, 0]).clamp(min=0), torch.zeros_like(m))
        d_rest = torch.where(some, 2 * ((e_p * raw).sum(1) + 2 * U), torch.zeros_like(m))
        M = mass[:, 0] + p_rest
    else:
        p = torch.where(mass > 0, raw / mass.clamp(min=1e-300), raw)
        log_p = torch.where(p > 0, p.clamp(min=1e-300).log(), torch.zeros_like(p))
        p_rest = d_rest = torch.zeros_like(m)
        log_rest = torch.zeros_like(m)
        M = (mass[:, 0] > 0).double()
    e_log = e_s + V2 + U * log_s.abs()
    at_a = a.gather(1, at)
    log_q = at_a - log_s[:, None]
    on = p > 0
    zero = torch.zeros_like(p)
    diff = torch.where(on, log_p - log_q, zero)
    loss = torch.where(on, p * diff, zero).sum(1)
    magnitude = torch.where(on, p * (log_p.abs() + log_q.abs()), zero).sum(1)
    err = torch.where(on, p * ((e_p + 4 * U) * diff.abs() + 2 * V2 + 4 * U * (val.abs() + log_p.abs()) + e_p + e_log[:, None] +
                               3 * U * at_a.abs() + 2 * U * log_q.abs()), zero).sum(1)
    if rest:
        safe = p_rest.clamp(min=1e-300)
        far = torch.where(log_rest > NEG, log_rest, torch.zeros_like(log_rest))
        loss = loss + torch.where(p_rest > 0, p_rest * (safe.log() - log_rest), torch.zeros_like(loss))
        # (p log p changes by at most d (|log d| + 1) when p does by d)
        small = torch.maximum(p_rest, d_rest).clamp(min=1e-300)
        magnitude = magnitude + p_rest * (safe.log().abs() + far.abs())
        span = torch.logsumexp(free_a, 1).clamp(min=-1e300)
        err = err + d_rest * (torch.minimum(small, d_rest.clamp(min=1e-300)).log().abs() + far.abs() + 1) + p_rest * (
            2 * e_log + V2 + 3 * U * torch.where(some, span.abs(), torch.zeros_like(m)) + 4 * U * far.abs())
    err = err + 16 * U * magnitude
    loss_tol = (w.abs() * err + 2 * U * (w * loss).abs())
    loss_tol = torch.where(loss.isfinite(), loss_tol, torch.zeros_like(loss_tol))
    loss = torch.where(w != 0, w * loss, torch.zeros_like(loss))
    # the gradient
    e_q = 3 * U * a.abs().clamp(max=200) + V2 + e_s[:, None] + 8 * U
    grad = p_q * M[:, None]
    tol = grad * (e_q + 4 * U) + p_q * d_rest[:, None]
    if rest:
        share = torch.where(free & (p_rest > 0)[:, None], torch.softmax(free_a, 1), torch.zeros_like(t))
        own = 3 * U * (a - free_a.amax(1, keepdim=True).clamp(min=-1e300)).abs().clamp(max=200)
        extra = p_rest[:, None] * share
        grad = grad - extra
        tol = tol + extra * (own + 2 * V2 + e_s[:, None] * 2 + 8 * U) + share * d_rest[:, None]
    grad = grad.scatter_add(1, at, torch.where(there, -p, zero))
    tol = tol.scatter_add(1, at, torch.where(there, p * (2 * e_p + 4 * U), zero))
    scale = (w * invT)[:, None]
    grad, tol = grad * scale, tol * scale.abs() + 4 * U * (grad * scale).abs() + 2.0 ** -120
    u = UBF if out_dtype == torch.bfloat16 else U
    tol = tol * (1 + u) + u * grad.abs()
    return (loss, torch.where((w != 0)[:, None], grad, torch.zeros_like(grad))), (loss_tol, tol)


def markov(g, prev, W1, W2, dW1=None, dW2=None):
    """(grad_prev, dW1, dW2) with the sums added to the given ones, and their tolerances."""
    rows, V = g.shape
    rank = W1.shape[1]
    g, W1, W2, prev = g.double(), W1.double(), W2.double(), prev.long()
    there = (prev >= 0) & (prev < V)
    at = torch.where(there, prev, torch.zeros_like(prev))
    E = W1[at] * there[:, None]

    def steps(K):
        return (64 + K / 1024 + 152) * 2.0 ** -22
    gp = (g @ W2) * there[:, None]
    gp_tol = steps(V) * (g.abs() @ W2.abs()) * there[:, None] + 1e-37
    base1 = torch.zeros(V, rank, dtype=torch.float64, device=g.device) if dW1 is None else dW1.double()
    base2 = torch.zeros(V, rank, dtype=torch.float64, device=g.device) if dW2 is None else dW2.double()
    sums = torch.zeros_like(base1).index_add_(0, at, gp)
    size = torch.zeros_like(base1).index_add_(0, at, gp.abs())
    tol1 = torch.zeros_like(base1).index_add_(0, at, gp_tol) + (rows + 1) * U * (size + base1.abs())
    d2 = g.T @ E
    tol2 = steps(rows) * (g.abs().T @ E.abs()) + 2 * U * (base2.abs() + d2.abs()) + 1e-37
    gp = torch.where((prev >= V)[:, None], torch.full_like(gp, float("nan")), gp)
    return (gp, base1 + sums, base2 + d2), (gp_tol, tol1, tol2)
