"""One attention layer of a target model over several verify cycles, its keys and values in the paged cache.

R requests share a system prompt.  The prompt's rows are appended to the cache and attended once
(dspark_kv_append, dspark_verify_attention); then each cycle
  drafts      gamma rows a request, whose positions see each other (dspark_qk_norm_rope on the block's own
              queries and keys),
  reserves    pages for the l + 1 rows of each request (dspark_kv_reserve),
  appends     them: norm, rotation, cache (dspark_kv_append),
  attends     the shared prompt once for all requests, then their own keys (dspark_prefix_attention),
  commits     what was accepted and gives back the other rows' pages (dspark_kv_commit).
Weights and hidden states are random, and so is what is accepted.  At the end the last cycle's outputs are compared
with a plain computation in float64 from the projected rows.

    python examples/attention_layer.py [--requests 32] [--cycles 4]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from speculative_decoding_dspark_gb300 import binding as B  # noqa: E402

EPS = 1e-6


class Layer:
    def __init__(self, hidden, hq, hkv, d, gen):
        def normal(*shape, scale=1.0):
            return (torch.randn(*shape, device="cuda", generator=gen) * scale).bfloat16()
        self.hq, self.hkv, self.d = hq, hkv, d
        self.w_qkv = normal(hidden, (hq + 2 * hkv) * d, scale=hidden ** -0.5)
        self.w_out = normal(hq * d, hidden, scale=(hq * d) ** -0.5)
        self.q_norm, self.k_norm = 1 + normal(d, scale=0.1), 1 + normal(d, scale=0.1)
        self.inv_freq = 10000.0 ** (-torch.arange(0, d, 2, device="cuda").float() / d)

    def project(self, x):
        qkv = (x @ self.w_qkv).view(-1, self.hq + 2 * self.hkv, self.d)
        return qkv, qkv[:, :self.hq], qkv[:, self.hq:self.hq + self.hkv], qkv[:, self.hq + self.hkv:]


class Cache:
    """The paged cache of R requests whose first `shared` positions lie in the same pages."""

    def __init__(self, layer, R, shared, page, max_len):
        head, blocks = shared // page, -(-max_len // page)
        pool = head + R * (blocks - head)
        shape = (pool, layer.hkv, page, layer.d)
        self.k = torch.zeros(shape, dtype=torch.bfloat16, device="cuda")
        self.v = torch.zeros_like(self.k)
        self.page, self.shared = page, shared
        self.kv_len = torch.full((R,), shared, dtype=torch.int32, device="cuda")
        self.table = torch.full((R, blocks), -1, dtype=torch.int32, device="cuda")
        self.table[:, :head] = torch.arange(head, dtype=torch.int32, device="cuda")
        self.free_pages = torch.full((pool,), -1, dtype=torch.int32, device="cuda")
        self.free_pages[:pool - head] = torch.arange(head, pool, dtype=torch.int32, device="cuda")
        self.free_top = torch.tensor([pool - head], dtype=torch.int32, device="cuda")


def i32(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def prompt(layer, cache, x, status):
    """The shared prompt's rows into the cache, and their attention."""
    rows = x.shape[0]
    qkv, q, k, v = layer.project(x)
    q_out = torch.empty(rows, layer.hq, layer.d, dtype=torch.bfloat16, device="cuda")
    out = torch.empty_like(q_out)
    at = (i32([0, rows]), i32([0]), cache.table[:1])  # cu_seqlens, kv_len, block_table
    B.dspark_kv_append(q, k, v, layer.q_norm, layer.k_norm, EPS, layer.inv_freq, *at, cache.k, cache.v, q_out,
                       dev_status=status)
    ws = B.workspace(B.dspark_attention_workspace_size(1, 0, rows, layer.hq, layer.hkv, layer.d))
    B.dspark_verify_attention(q_out, cache.k, cache.v, at[2], at[1], at[0], layer.d ** -0.5, out, ws=ws, dev_status=status)
    return qkv, out.view(rows, -1) @ layer.w_out


def draft(layer, x, first, status):
    """A block of positions from `first` [R] on that see each other: x [R, block, hidden] mixed by attention."""
    R, block, hidden = x.shape
    qkv, q, k, v = layer.project(x.reshape(R * block, hidden))
    at = (first[:, None] + torch.arange(block, dtype=torch.int32, device="cuda")).reshape(-1)
    B.dspark_qk_norm_rope(q, k, layer.q_norm, layer.k_norm, EPS, at, layer.inv_freq, q, k, dev_status=status)
    heads = [t.reshape(R, block, -1, layer.d).transpose(1, 2) for t in (q, k, v)]
    mixed = torch.nn.functional.scaled_dot_product_attention(*heads, enable_gqa=True)
    return x + (mixed.transpose(1, 2).reshape(R * block, -1) @ layer.w_out).view_as(x)


def verify(layer, cache, x, l, cu, ws, status):
    """The rows of all requests appended and attended; (their projections, the layer's output, the heads' output)."""
    R, rows = l.numel(), x.shape[0]
    B.dspark_kv_reserve(cache.kv_len, l, cache.page, cache.table, cache.free_pages, cache.free_top, dev_status=status)
    qkv, q, k, v = layer.project(x)
    q_out = torch.empty(rows, layer.hq, layer.d, dtype=torch.bfloat16, device="cuda")
    out = torch.empty_like(q_out)
    B.dspark_kv_append(q, k, v, layer.q_norm, layer.k_norm, EPS, layer.inv_freq, cu, cache.kv_len, cache.table,
                       cache.k, cache.v, q_out, dev_status=status)
    B.dspark_prefix_attention(q_out, cache.k, cache.v, cache.table, cache.kv_len, cu, i32([0, R]), i32([cache.shared]),
                              layer.d ** -0.5, out, ws=ws, dev_status=status)
    return qkv, out.view(rows, -1) @ layer.w_out, out


def plain(layer, qkv, rows):
    """The attention of the last `rows` of one request, in float64 from all its projected rows."""
    x = qkv.double().cpu()
    n, (hq, hkv, d) = x.shape[0], (layer.hq, layer.hkv, layer.d)
    angle = torch.arange(n).double()[:, None, None] * layer.inv_freq.double().cpu()

    def turned(x, w):  # as the cache and the attention hold them: rounded to bf16
        x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS) * w.double().cpu()
        a, b = x[..., :d // 2], x[..., d // 2:]
        x = torch.cat([a * angle.cos() - b * angle.sin(), b * angle.cos() + a * angle.sin()], -1)
        return x.bfloat16().double()

    q, k, v = turned(x[:, :hq], layer.q_norm), turned(x[:, hq:hq + hkv], layer.k_norm), x[:, hq + hkv:]
    k, v = k.repeat_interleave(hq // hkv, 1), v.repeat_interleave(hq // hkv, 1)
    s = torch.einsum("ihd,jhd->hij", q[n - rows:], k) * d ** -0.5
    s.masked_fill_(torch.arange(n) > torch.arange(n - rows, n)[:, None], float("-inf"))
    return torch.einsum("hij,jhd->ihd", s.softmax(-1), v)


def run(requests=32, cycles=4, gamma=7, hidden=1024, hq=32, hkv=8, d=128, shared=512, page=16, seed=0):
    """The largest error of the last cycle's outputs over the largest output, and the pages in use at the end."""
    gen = torch.Generator("cuda").manual_seed(seed)
    layer = Layer(hidden, hq, hkv, d, gen)
    cache = Cache(layer, requests, shared, page, shared + cycles * (gamma + 1))
    status = i32([0])

    def normal(*shape):
        return torch.randn(*shape, device="cuda", generator=gen).bfloat16()

    prompt_rows, _ = prompt(layer, cache, normal(shared, hidden), status)
    history = [[prompt_rows] for _ in range(requests)]
    ws = B.workspace(B.dspark_attention_workspace_size(requests, 1, requests * (gamma + 1), hq, hkv, d))
    host = torch.Generator().manual_seed(seed)
    for cycle in range(cycles):
        l = torch.randint(0, gamma + 1, (requests,), generator=host)  # verified drafts of each request
        x = draft(layer, normal(requests, gamma + 1, hidden), cache.kv_len, status)
        x = torch.cat([x[r, :int(l[r]) + 1] for r in range(requests)])
        cu = torch.cat([torch.zeros(1, dtype=torch.int64), (l + 1).cumsum(0)])
        l_dev = l.to(torch.int32).cuda()
        qkv, _, heads = verify(layer, cache, x, l_dev, cu.to(torch.int32).cuda(), ws, status)
        last = cycle == cycles - 1
        n_accepted = l if last else (torch.rand(requests, generator=host) * (l + 1)).long()
        B.dspark_kv_commit(cache.kv_len, l_dev, n_accepted.to(torch.int32).cuda(), page, cache.table,
                           cache.free_pages, cache.free_top, dev_status=status)
        for r in range(requests):
            history[r].append(qkv[int(cu[r]):int(cu[r]) + int(n_accepted[r]) + 1])
    if int(status.item()) != 0:
        raise RuntimeError(B.dspark_status_string(int(status.item())))
    worst = size = 0.0
    for r in range(requests):
        want = plain(layer, torch.cat(history[r]), int(l[r]) + 1)
        got = heads[int(cu[r]):int(cu[r + 1])].double().cpu()
        worst, size = max(worst, float((got - want).abs().max())), max(size, float(want.abs().max()))
    return worst / size, cache.k.shape[0] - int(cache.free_top.item()), cache.kv_len.cpu()


if __name__ == "__main__":
    args = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    args.add_argument("--requests", type=int, default=32)
    args.add_argument("--cycles", type=int, default=4)
    args = args.parse_args()
    error, pages, kv_len = run(args.requests, args.cycles)
    print(f"{args.requests} requests, {args.cycles} cycles: {pages} pages in use, lengths {int(kv_len.min())} to "
          f"{int(kv_len.max())}, outputs within {error:.1e} of the largest in float64")
