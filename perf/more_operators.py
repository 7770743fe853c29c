"""What the target says about its rows, and what a drafter learns from it: what is measured, and its plain form.

Three operators of the library around one verify, from the target's logits to the gradients of the drafter's head:

* ``logprobs``  ``dspark_token_logprobs``: the log probability of a given token of every row, the row's entropy and
  its top alternatives, over packed verify rows, prompts, or all rows of a teacher.
* ``distill``   ``dspark_distill_loss``: a drafter's rows held to the teacher's top tokens (their divergence, with the
  rest of the vocabulary as a class of its own or left out), and the gradient of its logits.
* ``markov``    ``dspark_markov_grad``: what that gradient says to the Markov factors W1 and W2.

The plain form is elementary torch in 32 bits, rounded once at the end.
"""
import math
import random

import torch

own = False

#: which rows of a case are asked for is spread by this generator, so that work() knows them
SPREAD = 20021

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "bf16": 2}


# ---------------------------------------------------------------------------------------- cases
def listed():
    return [
        # one decoded token with its alternatives, where only latency counts
        dict(name="logprobs_token", op="logprobs", rows=1, V=151936, dtype="f32", top=5, tokens="rows", T=1.0, masked=0.0),
        # what 128 requests get back from a verify: the emitted tokens of up to 8 rows each, the rest of the rows not asked for
        dict(name="logprobs_verify", op="logprobs", rows=0, requests=128, width=8, V=151936, dtype="f32", top=20,
             tokens="packed", T=0.7, masked=0.0),
        # a prompt's tokens scored, no alternatives
        dict(name="logprobs_prompt", op="logprobs", rows=4096, V=129280, dtype="bf16", top=0, tokens="rows", T=1.0, masked=0.0),
        # a teacher's top tokens of a batch of blocks, to be learned from
        dict(name="logprobs_teacher", op="logprobs", rows=2560, V=129280, dtype="bf16", top=64, tokens="none", T=1.0, masked=0.0),
        # rows of an odd length under a grammar that leaves a tenth of the vocabulary
        dict(name="logprobs_masked", op="logprobs", rows=333, V=50001, dtype="bf16", top=20, tokens="rows", T=0.8, masked=0.9),
        # one request's block, learned from as it is served
        dict(name="distill_block", op="distill", rows=7, V=32000, dtype="f32", grad="f32", top=8, rest=True, T=1.0, weights=False),
        # a held-out batch: the loss alone
        dict(name="distill_eval", op="distill", rows=896, V=151936, dtype="f32", grad="none", top=20, rest=True, T=1.0,
             weights=False),
        # the drafter's own 32-bit logits of a batch, their gradient in 16 bits for the product with the factors
        dict(name="distill_batch", op="distill", rows=896, V=151936, dtype="f32", grad="bf16", top=64, rest=True, T=1.0,
             weights=True),
        # a training step's rows in 16 bits, the listed tokens alone
        dict(name="distill_step", op="distill", rows=4096, V=129280, dtype="bf16", grad="bf16", top=128, rest=False, T=2.0,
             weights=True),
        # one request's block
        dict(name="markov_block", op="markov", rows=7, V=32000, rank=256),
        # the blocks of 128 requests
        dict(name="markov_batch", op="markov", rows=896, V=151936, rank=512),
        # the blocks of 512 requests
        dict(name="markov_step", op="markov", rows=2560, V=129280, rank=512),
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["logprobs", "logprobs", "distill", "distill", "markov"])
    V = _log(rng, 64, 160000)
    if op == "markov":
        V = max(64, V // 8 * 8)
        return dict(op=op, rows=_log(rng, 1, max(2, min(2560, 330000000 // V))), V=V, rank=64 * rng.randint(1, 8))
    rows = _log(rng, 1, max(2, min(4096, 250000000 // V)))
    dtype = rng.choice(["f32", "bf16"])
    T = rng.choice([1.0, 1.0, 0.7, 1.3, 2.0])
    if op == "logprobs":
        case = dict(op=op, rows=rows, V=V, dtype=dtype, top=rng.choice([0, 1, 5, 20, 50, 64, 128]),
                    tokens=rng.choice(["rows", "packed", "none"]), T=T, masked=rng.choice([0.0, 0.0, 0.3, 0.95]))
        if case["tokens"] == "packed":
            case.update(rows=0, width=rng.randint(1, 9))
            case["requests"] = max(1, rows // case["width"])
        return case
    return dict(op=op, rows=rows, V=V, dtype=dtype, grad=rng.choice(["none", "f32", "bf16"]),
                top=min(V, _log(rng, 1, 128)), rest=rng.random() < 0.5, T=T, weights=rng.random() < 0.5)


class Packed:
    """Lengths of a packed batch's requests, and how many of each request's rows have a token."""

    def __init__(self, case):
        r = random.Random(SPREAD)
        self.n = [r.randint(1, case["width"]) for _ in range(case["requests"])]
        self.asked = [r.randint(1, n) for n in self.n]
        self.cu = [0]
        for n in self.n:
            self.cu.append(self.cu[-1] + n)


def _weights(case):
    r = random.Random(SPREAD)
    return [0.0 if r.random() < 0.1 else r.uniform(0.2, 1.0) for _ in range(case["rows"])]


# -------------------------------------------------------------------------------------- inputs
def _normal(gen, shape, scale=1.0):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32).mul_(scale)


def prepare(case, seed):
    gen = torch.Generator("cuda")
    gen.manual_seed(seed)
    i32 = dict(dtype=torch.int32, device="cuda")
    f32 = dict(dtype=torch.float32, device="cuda")
    s = dict(case)
    s["status"] = torch.zeros(1, **i32)
    V = case["V"]
    if case["op"] == "logprobs":
        rows = case["rows"]
        if case["tokens"] == "packed":
            p = Packed(case)
            rows = p.cu[-1]
            s["cu"] = torch.tensor(p.cu, **i32)
            there = torch.arange(case["width"], device="cuda") < torch.tensor(p.asked, **i32)[:, None]
            any_token = torch.randint(0, V, there.shape, generator=gen, device="cuda", dtype=torch.int32)
            s["tokens"] = torch.where(there, any_token, -1).to(torch.int32)
        elif case["tokens"] == "rows":
            s["tokens"] = torch.randint(0, V, (rows,), generator=gen, device="cuda", dtype=torch.int32)
        else:
            s["tokens"] = None
        x = _normal(gen, (rows, V), 3.0)
        if case["masked"]:
            off = torch.rand((rows, V), generator=gen, device="cuda") < case["masked"]
            off[:, 0] = False  # a grammar always leaves a token
            x.masked_fill_(off, float("-inf"))
        s["logits"] = x.to(DTYPES[case["dtype"]])
        s["out"] = [torch.empty(rows, **f32) for _ in range(3)]
        s["top_ids"] = torch.empty(rows, case["top"], **i32) if case["top"] else None
        s["top_logprobs"] = torch.empty(rows, case["top"], **f32) if case["top"] else None
        return s
    rows = case["rows"]
    student = _normal(gen, (rows, V), 3.0)
    if case["op"] == "distill":
        # a teacher that the drafter has learned something of
        teacher = _normal(gen, (rows, V), 2.4).add_(student, alpha=0.6)
        best, ids = teacher.topk(case["top"], dim=1)
        norm = teacher.logsumexp(1, keepdim=True)
        s["student"] = student.to(DTYPES[case["dtype"]])
        s["ids"], s["teacher"] = ids.to(torch.int32), best - norm
        s["weight"] = torch.tensor(_weights(case), **f32) if case["weights"] else None
        s["loss"] = torch.empty(rows, **f32)
        s["out"] = None if case["grad"] == "none" else torch.empty(rows, V, dtype=DTYPES[case["grad"]], device="cuda")
        return s
    # a distilled block's gradient: what the drafter gives its tokens, less the teacher's few
    d = torch.softmax(student, 1)
    ids = torch.randint(0, V, (rows, 8), generator=gen, device="cuda")
    d.scatter_add_(1, ids, torch.full(ids.shape, -0.125, **f32))
    s["grad"] = (d / rows).to(torch.bfloat16)
    s["prev"] = torch.randint(-1, max(1, min(V, rows)), (rows,), generator=gen, device="cuda", dtype=torch.int32)
    s["W1"] = _normal(gen, (V, case["rank"]), 0.02).to(torch.bfloat16)
    s["W2"] = _normal(gen, (V, case["rank"]), 0.02).to(torch.bfloat16)
    s["grad_prev"] = torch.empty(rows, case["rank"], **f32)
    s["dW1"] = torch.zeros(V, case["rank"], **f32)
    s["dW2"] = torch.empty(V, case["rank"], **f32)
    if own:
        from speculative_decoding_dspark_gb300 import binding as B
        s["ws"] = B.workspace(B.dspark_workspace_size(B.DSPARK_OP_MARKOV_GRAD, 0, 0, V, case["rank"], rows, B.DSPARK_BF16))
    return s


# -------------------------------------------------------------------------------------- one pass
def run(s):
    if own:
        return _own(s)
    return {"logprobs": _logprobs, "distill": _distill, "markov": _markov}[s["op"]](s)


def _row_tokens(s):
    """The token of every row, -1 where there is none."""
    if s["tokens"] is None or s["tokens"].dim() == 1:
        return s["tokens"]
    cu = s["cu"].long()
    row = torch.arange(s["logits"].shape[0], device="cuda")
    request = torch.searchsorted(cu, row, right=True) - 1
    return s["tokens"][request, row - cu[request]]


def _logprobs(s):
    x = s["logits"].float()
    token = _row_tokens(s)
    asked = torch.ones(x.shape[0], dtype=torch.bool, device="cuda") if token is None else token >= 0
    t = x * (1.0 / s["T"])
    top = t.amax(1, keepdim=True)
    e = (t - top).exp_()
    total = e.sum(1)
    lse = top[:, 0] + total.log()
    entropy = total.log() - torch.where(e > 0, e * (t - top), 0.0).sum(1) / total
    logprob = torch.zeros_like(lse) if token is None else t.gather(1, token.clamp(min=0).long()[:, None])[:, 0] - lse
    out = [torch.where(asked, v, 0.0) for v in (logprob, lse, entropy)]
    if not s["top"]:
        return out
    # one whole number for the value (in the order of the numbers) and the place, the lowest first among equals
    bits = (x + 0.0).view(torch.int32)
    order = torch.where(bits < 0, bits ^ 0x7FFFFFFF, bits).long()
    place = torch.arange(x.shape[1] - 1, -1, -1, device="cuda")
    k = min(s["top"], x.shape[1])
    ids = x.shape[1] - 1 - (order * 2**32 + place).topk(k, dim=1).values % 2**32
    values = t.gather(1, ids) - lse[:, None]
    there = asked[:, None] & (values > float("-inf"))
    pad = (0, s["top"] - k)
    ids = torch.nn.functional.pad(torch.where(there, ids, -1), pad, value=-1)
    values = torch.nn.functional.pad(torch.where(there, values, float("-inf")), pad, value=float("-inf"))
    return out + [ids.to(torch.int32), values]


def _distill(s):
    t = s["student"].float() * (1.0 / s["T"])
    ids, w = s["ids"].long(), s["weight"]
    listed = t.gather(1, ids)
    p = s["teacher"].exp()
    rest = t.scatter(1, ids, float("-inf"))
    top = t.amax(1, keepdim=True)
    total = (t - top).exp().sum(1, keepdim=True)
    log_q = listed - top - total.log()
    if s["rest"]:
        p_rest = (1.0 - p.double().sum(1, keepdim=True)).clamp(min=0).float()
        rest_top = rest.amax(1, keepdim=True)
        p_rest = torch.where(rest_top > float("-inf"), p_rest, 0.0)
        rest_top = rest_top.clamp(min=-3e38)
        rest_total = (rest - rest_top).exp().sum(1, keepdim=True)
        log_rest = rest_top - top + rest_total.log() - total.log()
        loss = (p * (s["teacher"] - log_q)).sum(1) + torch.where(p_rest > 0, p_rest * (p_rest.log() - log_rest), 0.0)[:, 0]
        mass = p.sum(1, keepdim=True) + p_rest
    else:
        log_p = s["teacher"] - p.sum(1, keepdim=True).log()
        p = log_p.exp()
        loss = (p * (log_p - log_q)).sum(1)
        mass = 1.0
    weight = torch.ones_like(loss) if w is None else w
    loss = torch.where(weight != 0, loss * weight, 0.0)
    if s["out"] is None:
        return [loss]
    grad = mass * ((t - top).exp() / total)
    if s["rest"]:
        grad = grad - torch.where(p_rest > 0, p_rest * (rest - rest_top).exp() / rest_total, 0.0)
    grad = grad.scatter_add(1, ids, -p)
    grad = torch.where(weight[:, None] != 0, grad * (weight[:, None] / s["T"]), 0.0)
    return [loss, grad.to(s["out"].dtype)]


def _markov(s):
    d, prev = s["grad"].float(), s["prev"].long()
    there = prev >= 0
    at = prev.clamp(min=0)
    grad_prev = torch.matmul(d, s["W2"].float()) * there[:, None]
    before = s["W1"][at].float() * there[:, None]
    dW2 = torch.matmul(d.t(), before)
    sums = torch.zeros_like(s["dW1"]).index_add_(0, at, grad_prev)
    seen = torch.zeros(d.shape[1], dtype=torch.bool, device="cuda").index_fill_(0, at[there], True)
    return [grad_prev, torch.where(seen[:, None], sums, s["dW1"]), dW2]


def _own(s):
    from speculative_decoding_dspark_gb300 import binding as B
    if s["op"] == "logprobs":
        B.dspark_token_logprobs(s["logits"], s["tokens"], s["T"], *s["out"], s["top_ids"], s["top_logprobs"],
                                cu_seqlens=s.get("cu"), dev_status=s["status"])
        return s["out"] + ([s["top_ids"], s["top_logprobs"]] if s["top"] else [])
    if s["op"] == "distill":
        B.dspark_distill_loss(s["student"], s["ids"], s["teacher"], s["T"], s["loss"], grad=s["out"],
                              row_weight=s["weight"], rest=s["rest"], dev_status=s["status"])
        return [s["loss"]] + ([] if s["out"] is None else [s["out"]])
    B.dspark_markov_grad(s["grad"], s["prev"], s["W1"], s["W2"], s["grad_prev"], dW1=s["dW1"], dW2=s["dW2"], ws=s["ws"],
                         dev_status=s["status"])
    return [s["grad_prev"], s["dW1"], s["dW2"]]


# ---------------------------------------------------------------------------- the floor of a pass
def work(case):
    V = case["V"]
    if case["op"] == "logprobs":
        rows = asked = case["rows"]
        if case["tokens"] == "packed":
            p = Packed(case)
            rows, asked = p.cu[-1], sum(p.asked)
        return {"bytes": asked * V * SIZE[case["dtype"]] + rows * (16 + 8 * case["top"]), "flops": 6 * asked * V}
    rows = case["rows"]
    if case["op"] == "distill":
        asked = sum(w != 0 for w in _weights(case)) if case["weights"] else rows
        read = asked * (V * SIZE[case["dtype"]] + 8 * case["top"])
        written = 0 if case["grad"] == "none" else rows * V * SIZE[case["grad"]]
        return {"bytes": read + written + 8 * rows, "flops": (4 if case["grad"] == "none" else 8) * asked * V}
    rank = case["rank"]
    # the gradient and W2 read, dW2 written; of W1 and its gradient the rows that occur (at most one to a row)
    return {"bytes": rows * V * 2 + V * rank * (2 + 4) + rows * rank * (2 + 4 + 4), "flops": 4 * rows * V * rank}


# --------------------------------------------------------------------------- the answer in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    parts = {"logprobs": _exact_logprobs, "distill": _exact_distill, "markov": _exact_markov}[case["op"]](s, case)
    return parts


def _in_parts(s, case, rows, one):
    """`one` over a few hundred million values at a time, the results joined."""
    step = max(1, 200000000 // case["V"])
    got = [one(slice(a, min(rows, a + step))) for a in range(0, rows, step)]
    return [torch.cat(x) for x in zip(*got)]


def _exact_logprobs(s, case):
    rows, V, k = s["logits"].shape[0], case["V"], case["top"]
    token = torch.full((rows,), 0, dtype=torch.int64, device="cuda")
    if case["tokens"] == "rows":
        token = s["tokens"].long()
    if case["tokens"] == "packed":
        p = Packed(case)
        given = s["tokens"].tolist()
        token = torch.tensor([given[r][j] for r, n in enumerate(p.n) for j in range(n)], device="cuda")

    def one(at):
        x = s["logits"][at].double()
        log_p = torch.log_softmax(x / case["T"], 1)
        lse = torch.logsumexp(x / case["T"], 1)
        p = log_p.exp()
        entropy = -torch.where(p > 0, p * log_p, torch.zeros_like(p)).sum(1)
        skip = token[at] < 0
        logprob = log_p.gather(1, token[at].clamp(min=0)[:, None])[:, 0]
        if case["tokens"] == "none":
            logprob = torch.zeros_like(logprob)
        out = [v.masked_fill(skip, 0.0) for v in (logprob, lse, entropy)]
        if k:
            # equal values are in order of their places: a stable sort
            n = min(k, V)
            best, ids = torch.sort(x, dim=1, descending=True, stable=True)
            best, ids = best[:, :n], ids[:, :n].clone()
            value = log_p.gather(1, ids)
            gone = skip[:, None] | (best == float("-inf"))
            wide = torch.full((x.shape[0], k), float("-inf"), dtype=torch.float64, device="cuda")
            wide[:, :n] = value.masked_fill(gone, float("-inf"))
            places = torch.full((x.shape[0], k), -1, dtype=torch.int32, device="cuda")
            places[:, :n] = ids.masked_fill(gone, -1).to(torch.int32)
            out += [places, wide]
        return out
    return _in_parts(s, case, rows, one)


def _exact_distill(s, case):
    def one(at):
        x = s["student"][at].double() / case["T"]
        n = x.shape[0]
        ids = s["ids"][at].long()
        log_q = torch.log_softmax(x, 1)
        teacher = s["teacher"][at].double()
        p = torch.zeros_like(x)
        if case["rest"]:
            p.scatter_(1, ids, teacher.exp())
            free = torch.ones_like(x, dtype=torch.bool).scatter_(1, ids, False)
            left = (1.0 - p.sum(1)).clamp(min=0) * free.any(1)
            log_rest = torch.logsumexp(log_q.masked_fill(~free, float("-inf")), 1)
            loss = (teacher.exp() * (teacher - log_q.gather(1, ids))).sum(1)
            loss = loss + torch.where(left > 0, left * (left.clamp(min=1e-300).log() - log_rest), torch.zeros_like(left))
            # within the rest the teacher says nothing: its mass lies as the student's does
            share = torch.where(left > 0, left, torch.zeros_like(left))[:, None]
            inside = (log_q - log_rest.clamp(min=-1e300)[:, None]).exp() * free
            grad = log_q.exp() * (p.sum(1) + left)[:, None] - p - share * inside
        else:
            log_p = torch.log_softmax(teacher, 1)
            p.scatter_(1, ids, log_p.exp())
            loss = (log_p.exp() * (log_p - log_q.gather(1, ids))).sum(1)
            grad = log_q.exp() - p
        w = torch.ones(n, dtype=torch.float64, device="cuda") if s["weight"] is None else s["weight"][at].double()
        return [loss * w] + ([] if s["out"] is None else [grad * (w / case["T"])[:, None]])
    return _in_parts(s, case, case["rows"], one)


def _exact_markov(s, case):
    d, W2 = s["grad"].double(), s["W2"].double()
    prev = s["prev"].tolist()
    grad_prev = d @ W2
    before = torch.zeros(case["rows"], case["rank"], dtype=torch.float64, device="cuda")
    dW1 = s["dW1"].double()
    have = [n for n, v in enumerate(prev) if v >= 0]
    if have:
        at = torch.tensor([prev[n] for n in have], device="cuda")
        before[have] = s["W1"][at].double()
        dW1.index_put_((at,), grad_prev[have], accumulate=True)  # (the buffer was zero)
    none = [n for n, v in enumerate(prev) if v < 0]
    if none:
        grad_prev[none] = 0.0
    return [grad_prev, dW1, d.t() @ before]
