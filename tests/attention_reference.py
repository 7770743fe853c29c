"""Plain 64-bit definitions of the attention step's operators, and how far an output may be from them.

Formulas as in include/dspark.h; everything on the CPU in float64, one request and row at a time.

Tolerances (u = 2^-24 for fp32, ub = 2^-8 for a bf16 rounding, each the largest relative error of
one rounding):

* a normed and rotated element: the sum of squares, the mean, the root, two products and the
  rotation are under 32 fp32 roundings of the pair's magnitude (the lane sums are 8 long, then a
  tree), the angle's sine and cosine within 2^-22 of theirs; then one rounding to the output type.
* an attention output: weights p_j rounded to bf16 (ub), scores off by
  delta = scale * (d + 8) * 2u * max_j sum_i |q_i k_ji| + 2^-21 (|s| + 1) for the base-2 exponential's argument and
  value, both relative errors of p_j against A = sum_j p_j |v_j|; the sum over the keys adds
  2u per key (accumulators may truncate); then one rounding of the output.
* lse: delta, 2u per key, and four roundings of its own size.
"""
from __future__ import annotations

import math

import numpy as np
import torch

U32 = 2.0 ** -24
UB = 2.0 ** -8


def heads(x, w, eps, positions, inv_freq, pairs):
    """(y, size): the normed, rotated heads of x [rows, h, d] in float64, and each element's pair magnitude."""
    x = x.double().cpu()
    y = x if w is None else x * w.double().cpu() / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
    out, size = y.clone(), y.abs().clone()
    if inv_freq is not None:
        f = inv_freq.double().cpu()
        half = f.numel()
        for t, pos in enumerate(positions.tolist()):
            for j in range(half):
                a, b = (2 * j, 2 * j + 1) if pairs else (j, j + half)
                c, s = math.cos(pos * float(f[j])), math.sin(pos * float(f[j]))
                out[t, :, a] = y[t, :, a] * c - y[t, :, b] * s
                out[t, :, b] = y[t, :, b] * c + y[t, :, a] * s
                size[t, :, a] = size[t, :, b] = y[t, :, a].abs() + y[t, :, b].abs()
    return out, size


def heads_tol(ref, size, dtype):
    u = UB if dtype == torch.bfloat16 else U32
    inner = size * (32 * U32 + 2.0 ** -22)
    return u * (ref.abs() + inner) + inner


def attention(q, k_cache, v_cache, table, kv_len, cu, scale, full):
    """out, lse and their tolerances, in float64; rows past cu[-1] are NaN in out."""
    rows, hq, d = q.shape
    _, hkv, page, _ = k_cache.shape
    g = hq // hkv
    q = q.double().cpu()
    table, kv_len, cu = (np.asarray(x.cpu()) if torch.is_tensor(x) else np.asarray(x) for x in (table, kv_len, cu))
    out = torch.full((rows, hq, d), float("nan"), dtype=torch.float64)
    lse = torch.full((rows, hq), float("nan"), dtype=torch.float64)
    out_tol, lse_tol = torch.zeros_like(out), torch.zeros_like(lse)
    for r in range(len(kv_len)):
        n = int(cu[r + 1] - cu[r])
        total = int(kv_len[r]) + n
        if n == 0:
            continue
        ids = torch.as_tensor(table[r, :-(-total // page)].astype(np.int64))
        k, v = (c[ids.to(c.device)].double().cpu().permute(1, 0, 2, 3).reshape(hkv, -1, d)[:, :total]
                for c in (k_cache, v_cache))
        for i in range(n):
            row = int(cu[r]) + i
            seen = total if full else int(kv_len[r]) + i + 1
            for h in range(hkv):
                kk, vv, qq = k[h, :seen], v[h, :seen], q[row, h * g:(h + 1) * g]
                s = scale * qq @ kk.T
                z = torch.logsumexp(s, -1)
                p = torch.exp(s - z[:, None])
                o = p @ vv
                delta = (abs(scale) * (d + 8) * 2 * U32 * (qq.abs() @ kk.abs().T).amax(-1) +
                         2.0 ** -21 * (s.abs().amax(-1) + 1))
                out[row, h * g:(h + 1) * g], lse[row, h * g:(h + 1) * g] = o, z
                out_tol[row, h * g:(h + 1) * g] = (UB * o.abs() + (p @ vv.abs()) * (1 + UB) *
                                                   (UB + 2 * delta + seen * 2 * U32)[:, None])
                lse_tol[row, h * g:(h + 1) * g] = delta + seen * 2 * U32 + 4 * U32 * z.abs()
    return out, lse, out_tol, lse_tol


def pages_for(rng, kv_len, cu, page, shared=0, spare=3):
    """A block table over a shuffled pool: (table [R, blocks] int32, pages of the pool).  The first `shared` positions
    lie in the same pages for every request."""
    R = len(kv_len)
    total = [int(kv_len[r]) + int(cu[r + 1] - cu[r]) for r in range(R)]
    blocks = max(1, max(-(-t // page) for t in total)) + 1
    head = shared // page
    need = [max(0, -(-t // page) - head) for t in total]
    pool = head + sum(need) + spare
    ids = rng.permutation(pool).astype(np.int32)
    table = np.full((R, blocks), -1, np.int32)
    at = head
    for r in range(R):
        table[r, :head] = ids[:head]
        table[r, head:head + need[r]] = ids[at:at + need[r]]
        at += need[r]
    return table, pool
