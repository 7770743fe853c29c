"""The target model's attention step around one verify: what is measured, and its plain form.

Four operators of the library, each with the cases it meets in a decode cycle:

* ``norm_rope``  ``dspark_qk_norm_rope``: RMS norm of every query and key head and the position
  rotation, in one pass.
* ``append``     ``dspark_kv_append``: the same on the rows of a packed batch, the keys and
  values going to their places in the paged cache.
* ``attend``     ``dspark_verify_attention``: the l + 1 verify rows of each request (one row for
  plain decoding) over the request's pages.
* ``prefix``     ``dspark_prefix_attention``: the same where groups of requests share their
  leading pages, the shared part computed once for the group.

The plain form is elementary torch in 32 bits (the angles of the rotation in 64), rounded once at
the end.
"""
import math
import random

import torch

own = False

#: requests, rows and lengths of a case are spread by this generator, so that work() knows them
SPREAD = 20011

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


# ---------------------------------------------------------------------------------------- cases
def listed():
    return [
        # one decoded token's heads, where only latency counts
        dict(name="norm_rope_token", op="norm_rope", rows=1, hq=32, hkv=8, d=128, rot=128, style="half",
             dtype="bf16", out="bf16", first=4095),
        # the drafter's block positions of a batch, 32-bit activations, part of each head rotated in pairs
        dict(name="norm_rope_block", op="norm_rope", rows=896, hq=16, hkv=4, d=64, rot=48, style="pairs",
             dtype="f32", out="bf16", first=100000),
        # a prompt chunk far into a long context
        dict(name="norm_rope_prompt", op="norm_rope", rows=16384, hq=32, hkv=8, d=128, rot=128, style="half",
             dtype="bf16", out="bf16", first=500000),
        # one request decoding one token
        dict(name="append_token", op="append", requests=1, n_low=1, n_high=1, len_low=777, len_high=777, page=16,
             hq=32, hkv=8, d=128, rot=128, style="half", dtype="bf16"),
        # the packed verify rows of a batch of 128 requests, ragged lengths
        dict(name="append_verify", op="append", requests=128, n_low=1, n_high=8, len_low=0, len_high=900, page=16,
             hq=32, hkv=8, d=128, rot=128, style="half", dtype="bf16"),
        # prompts of several requests, 32-bit activations, pages of an odd size
        dict(name="append_prompt", op="append", requests=7, n_low=300, n_high=4001, len_low=0, len_high=50, page=12,
             hq=24, hkv=8, d=64, rot=64, style="pairs", dtype="f32"),
        # one request decoding one token of a short context
        dict(name="attend_token", op="attend", requests=1, n_low=1, n_high=1, len_low=777, len_high=777, page=16,
             hq=32, hkv=8, d=128, full=False),
        # two very long contexts under verification: the work of few rows split over the keys
        dict(name="attend_long", op="attend", requests=2, n_low=5, n_high=8, len_low=100001, len_high=131000, page=64,
             hq=32, hkv=8, d=128, full=False),
        # the serving batch: 128 requests, 1 to 8 rows each, ragged contexts
        dict(name="attend_verify", op="attend", requests=128, n_low=1, n_high=8, len_low=17, len_high=5000, page=16,
             hq=32, hkv=8, d=128, full=False),
        # a drafter's block over its context, every row seeing the whole block; 17 x 8 rows a head, odd pages
        dict(name="attend_block", op="attend", requests=48, n_low=17, n_high=17, len_low=0, len_high=2000, page=10,
             hq=64, hkv=8, d=64, full=True),
        # 128 requests behind one long system prompt
        dict(name="prefix_batch", op="prefix", requests=128, n_low=1, n_high=8, len_low=0, len_high=500, page=16,
             hq=32, hkv=8, d=128, full=False, shared="8192"),
        # several groups behind prompts of their own, one of them sharing nothing
        dict(name="prefix_groups", op="prefix", requests=45, n_low=1, n_high=6, len_low=0, len_high=1000, page=32,
             hq=16, hkv=2, d=64, full=False, shared="2048,0,6400,96"),
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["norm_rope", "append", "attend", "attend", "prefix", "prefix"])
    hkv = rng.choice([1, 2, 4, 8])
    hq = hkv * rng.choice([1, 2, 3, 4, 5, 8])
    d = rng.choice([64, 128])
    style = rng.choice(["half", "pairs"])
    rot = rng.choice([d, d, d // 2, d - 16])
    if op == "norm_rope":
        return dict(op=op, rows=_log(rng, 1, 16384), hq=min(hq, 32), hkv=hkv, d=d, rot=rot, style=style,
                    dtype=rng.choice(["bf16", "f32"]), out=rng.choice(["bf16", "bf16", "f32"]),
                    first=_log(rng, 1, 500000))
    page = rng.choice([1, 7, 10, 16, 16, 32, 64, 100, 128, 256])
    if op == "append":
        requests = _log(rng, 1, 256)
        n_high = _log(rng, 1, max(2, 8192 // requests))
        return dict(op=op, requests=requests, n_low=rng.randint(0, n_high), n_high=n_high, len_low=0,
                    len_high=_log(rng, 1, max(2, 60000 // requests)), page=page, hq=min(hq, 32), hkv=hkv, d=d, rot=rot,
                    style=style, dtype=rng.choice(["bf16", "f32"]))
    requests = _log(rng, 1, 200)
    n_high = _log(rng, 1, 17)
    common = dict(op=op, requests=requests, n_low=rng.randint(0, n_high), n_high=n_high, page=page, hq=hq,
                  hkv=hkv, d=d, full=rng.random() < 0.25)
    if op == "attend":
        high = _log(rng, 1, max(2, min(131072, 300000 // requests)))
        return dict(common, len_low=rng.randint(0, high), len_high=high)
    groups = rng.randint(1, min(4, requests))
    shared = [0 if rng.random() < 0.15 else page * max(1, _log(rng, 16, 8192) // page) for _ in range(groups)]
    return dict(common, requests=min(requests, 128), len_low=0, len_high=_log(rng, 1, 600),
                n_low=1, n_high=min(n_high, 8), hq=min(hq, 32), shared=",".join(map(str, shared)))


class Shape:
    """Rows and lengths of a case's requests, and where each request's pages are."""

    def __init__(self, case):
        r = random.Random(SPREAD)
        self.n = [r.randint(case["n_low"], case["n_high"]) for _ in range(case["requests"])]
        own_len = [r.randint(case["len_low"], case["len_high"]) for _ in range(case["requests"])]
        if case["requests"] == 1:
            self.n, own_len = [case["n_high"]], [case["len_high"]]
        self.n[0] = max(1, self.n[0])
        self.shared = [int(x) for x in case["shared"].split(",")] if "shared" in case else []
        # the requests of group g are start[g] .. start[g + 1] - 1
        g = max(1, len(self.shared))
        self.start = [case["requests"] * i // g for i in range(g + 1)]
        self.of = [max(i for i in range(g) if self.start[i] <= k) for k in range(case["requests"])]
        self.front = [self.shared[self.of[k]] if self.shared else 0 for k in range(case["requests"])]
        self.kv = [f + x for f, x in zip(self.front, own_len)]
        self.total = [a + b for a, b in zip(self.kv, self.n)]
        self.cu = [0]
        for x in self.n:
            self.cu.append(self.cu[-1] + x)
        p = case["page"]
        self.blocks = max(1, max(-(-t // p) for t in self.total))
        # pages: each group's shared ones, then each request's own
        self.table, at = [], 0
        first = []
        for s in self.shared or [0]:
            first.append(list(range(at, at + s // p)))
            at += s // p
        for k in range(case["requests"]):
            own_pages = -(-self.total[k] // p) - self.front[k] // p
            row = first[self.of[k]] + list(range(at, at + own_pages))
            at += own_pages
            self.table.append(row + [-1] * (self.blocks - len(row)))
        self.pages = max(1, at)


# -------------------------------------------------------------------------------------- inputs
def _normal(gen, shape, dtype, scale=1.0):
    return (torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32) * scale).to(dtype)


def _inv_freq(rot):
    return torch.tensor([10000.0 ** (-2.0 * i / rot) for i in range(rot // 2)], dtype=torch.float64).float().cuda()


def prepare(case, seed):
    gen = torch.Generator("cuda")
    gen.manual_seed(seed)
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    i32 = dict(dtype=torch.int32, device="cuda")
    s = dict(case)
    s["status"] = torch.zeros(1, **i32)
    if case["op"] in ("norm_rope", "append"):
        t = DTYPES[case["dtype"]]
        s["inv_freq"] = _inv_freq(case["rot"])
        s["wq"] = (1.0 + 0.2 * torch.randn(d, generator=gen, device="cuda")).to(t)
        s["wk"] = (1.0 + 0.2 * torch.randn(d, generator=gen, device="cuda")).to(t)
    if case["op"] == "norm_rope":
        rows = case["rows"]
        # the q and k parts of one projection's output, where they stand
        qkv = _normal(gen, (rows, hq + 2 * hkv, d), t, 3.0)
        s["q"], s["k"] = qkv[:, :hq], qkv[:, hq:hq + hkv]
        s["positions"] = torch.arange(case["first"], case["first"] + rows, **i32)
        s["q_out"] = torch.empty(rows, hq, d, dtype=DTYPES[case["out"]], device="cuda")
        s["k_out"] = torch.empty(rows, hkv, d, dtype=DTYPES[case["out"]], device="cuda")
        return s
    shape = Shape(case)
    rows = shape.cu[-1]
    shuffled = torch.randperm(shape.pages, generator=gen, device="cuda").to(torch.int32)
    table = torch.tensor(shape.table, dtype=torch.int64).cuda()
    s["table"] = torch.where(table >= 0, shuffled[table.clamp(min=0)], torch.full_like(table, -1, dtype=torch.int32))
    s["kv_len"] = torch.tensor(shape.kv, **i32)
    s["cu"] = torch.tensor(shape.cu, **i32)
    place = (shape.pages, hkv, case["page"], d)
    # trained value heads have a mean of their own in each channel; keys of a trained model are spread likewise
    s["k_cache"] = _normal(gen, place, torch.bfloat16)
    s["v_cache"] = (torch.randn(place, generator=gen, device="cuda") +
                    0.5 * torch.randn((1, hkv, 1, d), generator=gen, device="cuda")).to(torch.bfloat16)
    if case["op"] == "append":
        qkv = _normal(gen, (rows, hq + 2 * hkv, d), t, 3.0)
        s["q"], s["k"], s["v"] = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
        s["q_out"] = torch.empty(rows, hq, d, dtype=torch.bfloat16, device="cuda")
        return s
    s["q"] = _normal(gen, (rows, hq, d), torch.bfloat16, 2.0)
    s["scale"] = d ** -0.5
    s["out"] = torch.empty_like(s["q"])
    s["lse"] = torch.empty(rows, hq, dtype=torch.float32, device="cuda")
    if case["op"] == "prefix":
        s["group_start"] = torch.tensor(shape.start, **i32)
        s["shared_len"] = torch.tensor(shape.shared, **i32)
    if own:
        from speculative_decoding_dspark_gb300 import binding as B
        s["ws"] = B.workspace(B.dspark_attention_workspace_size(case["requests"], len(shape.shared), rows, hq, hkv, d))
    return s


# -------------------------------------------------------------------------------------- one pass
def run(s):
    if own:
        return _own(s)
    if s["op"] == "norm_rope":
        q = _norm_rotate(s["q"].float(), s["wq"].float(), s["positions"], s["inv_freq"], s["style"])
        k = _norm_rotate(s["k"].float(), s["wk"].float(), s["positions"], s["inv_freq"], s["style"])
        t = s["q_out"].dtype
        return [q.to(t), k.to(t)]
    if s["op"] == "append":
        rows = torch.arange(s["q"].shape[0], device="cuda")
        request = torch.searchsorted(s["cu"], rows, right=True) - 1
        position = s["kv_len"][request] + rows - s["cu"][request]
        q = _norm_rotate(s["q"].float(), s["wq"].float(), position, s["inv_freq"], s["style"])
        k = _norm_rotate(s["k"].float(), s["wk"].float(), position, s["inv_freq"], s["style"])
        page = s["table"][request, position // s["page"]].long()
        slot = position % s["page"]
        s["k_cache"][page, :, slot] = k.to(torch.bfloat16)
        s["v_cache"][page, :, slot] = s["v"].to(torch.bfloat16)
        return [q.to(torch.bfloat16), s["k_cache"], s["v_cache"]]
    return _attend(s)


EPS = 1e-6


def _norm_rotate(x, w, position, inv_freq, style):
    x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * w
    rot = 2 * inv_freq.numel()
    angle = position.double()[:, None, None] * inv_freq.double()
    cos, sin = angle.cos().float(), angle.sin().float()
    if style == "half":
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    else:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    return torch.cat([turned, x[..., rot:]], -1)


def _attend(s):
    """All requests at once, padded to the longest."""
    cu, kv_len, table, page = s["cu"].long(), s["kv_len"].long(), s["table"].long(), s["page"]
    rows, hq, d = s["q"].shape
    hkv = s["k_cache"].shape[1]
    n = cu[1:] - cu[:-1]
    longest, most = table.shape[1] * page, min(s["n_high"], rows)
    requests = n.numel()
    at = torch.arange(most, device="cuda")
    there = at < n[:, None]
    row = (cu[:-1, None] + at).clamp(max=rows - 1)
    q = s["q"][row].float().view(requests, most, hkv, hq // hkv, d).transpose(1, 2)  # [R, hkv, n, g, d]
    key = torch.arange(longest, device="cuda")
    total = kv_len + n
    within = (key < total[:, None])[:, :, None, None]
    pages = table.clamp(min=0)

    def gathered(cache):
        x = cache[pages].transpose(2, 3).reshape(requests, longest, hkv, d)
        return torch.where(within, x, 0).float().transpose(1, 2)  # [R, hkv, L, d]

    scores = torch.matmul(q.reshape(requests, hkv, -1, d), gathered(s["k_cache"]).transpose(2, 3)) * s["scale"]
    last = (total[:, None] - 1).expand(-1, most) if s["full"] else kv_len[:, None] + at
    seen = key <= last[:, :, None]  # [R, n, L]
    scores = scores.view(requests, hkv, most, hq // hkv, longest)
    scores = scores.masked_fill(~seen[:, None, :, None], float("-inf"))
    top = scores.amax(-1, keepdim=True)
    p = (scores - top).exp_()
    total_p = p.sum(-1, keepdim=True)
    out = torch.matmul(p.view(requests, hkv, -1, longest), gathered(s["v_cache"]))
    out = out.view(requests, hkv, most, hq // hkv, d) / total_p
    lse = (top + total_p.log()).squeeze(-1)
    out = out.transpose(1, 2).reshape(requests, most, hq, d)[there]
    lse = lse.transpose(1, 2).reshape(requests, most, hq)[there]
    return [out.to(torch.bfloat16), lse]


def _own(s):
    from speculative_decoding_dspark_gb300 import binding as B
    pairs = s.get("style") == "pairs"
    if s["op"] == "norm_rope":
        B.dspark_qk_norm_rope(s["q"], s["k"], s["wq"], s["wk"], EPS, s["positions"], s["inv_freq"], s["q_out"],
                              s["k_out"], interleaved=pairs, dev_status=s["status"])
        return [s["q_out"], s["k_out"]]
    if s["op"] == "append":
        B.dspark_kv_append(s["q"], s["k"], s["v"], s["wq"], s["wk"], EPS, s["inv_freq"], s["cu"], s["kv_len"],
                           s["table"], s["k_cache"], s["v_cache"], s["q_out"], interleaved=pairs,
                           dev_status=s["status"])
        return [s["q_out"], s["k_cache"], s["v_cache"]]
    args = [s["q"], s["k_cache"], s["v_cache"], s["table"], s["kv_len"], s["cu"]]
    more = dict(lse=s["lse"], full_block=s["full"], ws=s["ws"], dev_status=s["status"])
    if s["op"] == "prefix":
        B.dspark_prefix_attention(*args, s["group_start"], s["shared_len"], s["scale"], s["out"], **more)
    else:
        B.dspark_verify_attention(*args, s["scale"], s["out"], **more)
    return [s["out"], s["lse"]]


# ---------------------------------------------------------------------------- the floor of a pass
def work(case):
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    if case["op"] == "norm_rope":
        rows = case["rows"]
        size = {"f32": 4, "bf16": 2}
        return {"bytes": rows * (hq + hkv) * d * (size[case["dtype"]] + size[case["out"]]) + 4 * rows,
                "flops": 9 * rows * (hq + hkv) * d}
    shape = Shape(case)
    rows = shape.cu[-1]
    if case["op"] == "append":
        size = {"f32": 4, "bf16": 2}[case["dtype"]]
        return {"bytes": rows * (hq + 2 * hkv) * d * (size + 2) + 12 * case["requests"] + 4,
                "flops": 9 * rows * (hq + hkv) * d}
    keys = sum(shape.shared) + sum(t - f for t, f in zip(shape.total, shape.front))
    seen = sum(n * t if case["full"] else sum(kv + j + 1 for j in range(n))
               for n, kv, t in zip(shape.n, shape.kv, shape.total))
    return {"bytes": keys * hkv * d * 4 + rows * hq * (4 * d + 4), "flops": 4 * seen * hq * d}


# --------------------------------------------------------------------------- the answer in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm_rope":
        return [_exact_heads(s[x], s["w" + x], s["positions"], s["inv_freq"], case) for x in ("q", "k")]
    if case["op"] == "append":
        position, place = [], []
        cu, kv_len, table = s["cu"].tolist(), s["kv_len"].tolist(), s["table"].tolist()
        for r in range(case["requests"]):
            for i in range(cu[r + 1] - cu[r]):
                b, slot = divmod(kv_len[r] + i, case["page"])
                position.append(kv_len[r] + i)
                place.append((table[r][b], slot))
        position = torch.tensor(position, device="cuda")
        place = torch.tensor(place, device="cuda")
        k_cache, v_cache = s["k_cache"].double(), s["v_cache"].double()
        k_cache[place[:, 0], :, place[:, 1]] = _exact_heads(s["k"], s["wk"], position, s["inv_freq"], case)
        v_cache[place[:, 0], :, place[:, 1]] = s["v"].double()
        return [_exact_heads(s["q"], s["wq"], position, s["inv_freq"], case), k_cache, v_cache]
    out, lse = [], []
    g = case["hq"] // case["hkv"]
    cu, kv_len = s["cu"].tolist(), s["kv_len"].tolist()
    for r in range(case["requests"]):
        n = cu[r + 1] - cu[r]
        if n == 0:
            continue
        total = kv_len[r] + n
        ids = s["table"][r, :-(-total // case["page"])].long()
        k, v = (s[c][ids].double().permute(1, 0, 2, 3).flatten(1, 2)[:, :total] for c in ("k_cache", "v_cache"))
        q = s["q"][cu[r]:cu[r + 1]].double().unflatten(1, (case["hkv"], g))
        x = torch.einsum("nhgd,hkd->nhgk", q, k) * s["scale"]
        if not case["full"]:
            later = torch.arange(total, device="cuda") > kv_len[r] + torch.arange(n, device="cuda")[:, None]
            x = x.masked_fill(later[:, None, None], float("-inf"))
        norm = torch.logsumexp(x, -1)
        out.append(torch.einsum("nhgk,hkd->nhgd", torch.exp(x - norm[..., None]), v).flatten(1, 2))
        lse.append(norm.flatten(1, 2))
    return [torch.cat(out), torch.cat(lse)]


def _exact_heads(x, w, position, inv_freq, case):
    x = x.double()
    y = x / (x.square().mean(-1, keepdim=True) + EPS).sqrt() * w.double()
    z = y.clone()
    turn = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"),
                       position.double()[:, None, None] * inv_freq.double())
    rot = case["rot"]
    first, second = ((slice(0, rot // 2), slice(rot // 2, rot)) if case["style"] == "half" else
                     (slice(0, rot, 2), slice(1, rot, 2)))
    turned = torch.complex(y[..., first], y[..., second]) * turn
    z[..., first], z[..., second] = turned.real, turned.imag
    return z
