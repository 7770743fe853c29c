"""Host-side checks of dspark_token_logprobs, dspark_distill_loss and dspark_markov_grad, and pins of the 64-bit
reference the GPU tests compare with."""
import ctypes
import math

import pytest

torch = pytest.importorskip("torch")

import learning_reference as L  # noqa: E402

INVALID, UNSUPPORTED, WORKSPACE = -1, -2, -7
vp, i32, i64, f32, u32, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_float, ctypes.c_uint, ctypes.c_size_t
F = vp(4096)  # never dereferenced: every call here is refused, or has nothing to do


@pytest.fixture(scope="module")
def lib():
    from speculative_decoding_dspark_gb300 import build
    try:
        build.nvcc()
    except RuntimeError:
        pytest.skip("nvcc not available")
    return ctypes.CDLL(build.build())


LOGPROBS = dict(logits=F, stride=1000, dtype=0, tokens=F, cu=None, R=0, width=0, T=1.0, rows=5, V=1000, top=4, logprob=F,
                lse=F, entropy=F, ids=F, values=F, status=None, stream=None)
LOGPROBS_T = [vp, i64, i32, vp, vp, i32, i32, f32, i32, i32, i32] + [vp] * 7
DISTILL = dict(x=F, stride=1000, dtype=0, ids=F, values=F, top=4, weight=None, T=1.0, rows=5, V=1000, loss=F, grad=vp(8192),
               grad_stride=1000, grad_dtype=1, flags=0, status=None, stream=None)
DISTILL_T = [vp, i64, i32, vp, vp, i32, vp, f32, i32, i32, vp, vp, i64, i32, u32, vp, vp]
MARKOV = dict(g=F, stride=1000, prev=F, W1=F, W2=F, rows=5, V=1000, rank=64, gp=F, dW1=F, dW2=F, flags=0, ws=vp(256 * 64),
              ws_bytes=1 << 40, status=None, stream=None)
MARKOV_T = [vp, i64, vp, vp, vp, i32, i32, i32, vp, vp, vp, u32, vp, sz, vp, vp]


def call(lib, name, types, base, **change):
    f = getattr(lib, name)
    f.restype, f.argtypes = i32, types
    assert set(change) <= set(base)
    return f(*{**base, **change}.values())


@pytest.mark.parametrize("change,status", [
    (dict(rows=-1), INVALID), (dict(V=0), INVALID), (dict(top=-1), INVALID), (dict(dtype=2), INVALID),
    (dict(stride=999), INVALID), (dict(logits=vp(4098)), INVALID), (dict(dtype=1, logits=vp(4097)), INVALID),
    (dict(logits=None), INVALID), (dict(logprob=None), INVALID), (dict(ids=None), INVALID), (dict(values=None), INVALID),
    (dict(T=0.0), INVALID), (dict(T=-1.0), INVALID), (dict(T=math.inf), INVALID), (dict(T=math.nan), INVALID),
    (dict(T=1e-39), INVALID), (dict(cu=F, R=0, width=4), INVALID), (dict(cu=F, R=3, width=0), INVALID),
    (dict(cu=F, R=3, width=4, tokens=None), INVALID), (dict(top=129), UNSUPPORTED), (dict(V=(1 << 22) + 1, stride=1 << 23), UNSUPPORTED),
    (dict(rows=1 << 27), UNSUPPORTED), (dict(cu=F, R=1 << 20, width=1 << 8), UNSUPPORTED),
])
def test_logprobs_refusals(lib, change, status):
    assert call(lib, "dspark_token_logprobs", LOGPROBS_T, LOGPROBS, **change) == status


@pytest.mark.parametrize("change,status", [
    (dict(rows=-1), INVALID), (dict(V=0), INVALID), (dict(top=0), INVALID), (dict(dtype=-1), INVALID),
    (dict(stride=999), INVALID), (dict(grad_stride=999), INVALID), (dict(grad_dtype=7), INVALID), (dict(x=vp(4097)), INVALID),
    (dict(grad=vp(8193)), INVALID), (dict(x=None), INVALID), (dict(ids=None), INVALID), (dict(values=None), INVALID),
    (dict(loss=None), INVALID), (dict(flags=2), INVALID), (dict(T=0.0), INVALID), (dict(T=math.nan), INVALID),
    (dict(grad=F), INVALID), (dict(grad=F, grad_dtype=0, grad_stride=1001), INVALID),  # in place, but not alike
    (dict(top=129), UNSUPPORTED), (dict(V=(1 << 22) + 1, stride=1 << 23, grad_stride=1 << 23), UNSUPPORTED),
    (dict(rows=1 << 27), UNSUPPORTED),
])
def test_distill_refusals(lib, change, status):
    assert call(lib, "dspark_distill_loss", DISTILL_T, DISTILL, **change) == status


@pytest.mark.parametrize("change,status", [
    (dict(rows=-1), INVALID), (dict(V=0), INVALID), (dict(rank=0), INVALID), (dict(g=None), INVALID), (dict(prev=None), INVALID),
    (dict(W1=None), INVALID), (dict(W2=None), INVALID), (dict(gp=None), INVALID), (dict(stride=992), INVALID),
    (dict(flags=2), INVALID), (dict(rank=96), UNSUPPORTED), (dict(rank=576), UNSUPPORTED), (dict(V=996), UNSUPPORTED),
    (dict(stride=1004), UNSUPPORTED), (dict(rows=(1 << 19) + 1), UNSUPPORTED), (dict(V=(1 << 22) + 8, stride=1 << 23), UNSUPPORTED), (dict(g=vp(4104)), UNSUPPORTED),
    (dict(W2=vp(4104)), UNSUPPORTED), (dict(dW2=vp(4104)), UNSUPPORTED), (dict(ws=None), WORKSPACE),
    (dict(ws=vp(4096 + 16)), WORKSPACE), (dict(ws_bytes=100), WORKSPACE),
])
def test_markov_refusals(lib, change, status):
    assert call(lib, "dspark_markov_grad", MARKOV_T, MARKOV, **change) == status


def test_nothing_to_do(lib):
    assert call(lib, "dspark_token_logprobs", LOGPROBS_T, LOGPROBS, rows=0, logits=None, logprob=None) == 0
    assert call(lib, "dspark_distill_loss", DISTILL_T, DISTILL, rows=0, loss=None) == 0
    assert call(lib, "dspark_markov_grad", MARKOV_T, MARKOV, rows=0, dW2=None) == 0


def test_workspace(lib):
    f = lib.dspark_workspace_size
    f.restype, f.argtypes = sz, [i32] * 7 + [u32]
    assert f(6, 0, 0, 1000, 64, 5, 1, 0) > 0
    for V, rank, rows in [(1000, 96, 5), (1004, 64, 5), (1000, 64, -1), (1000, 576, 5), (0, 64, 5), (2 ** 31 - 8, 64, 5)]:
        assert f(6, 0, 0, V, rank, rows, 1, 0) == 0


# ------------------------------------------------------------------------------ pins of the reference
def test_reference_logprobs_by_hand():
    x = torch.tensor([[0.0, math.log(3.0), -math.inf, -0.0]])
    (lp, lse, ent, ids, val), _ = L.logprobs(x, torch.tensor([1]), 1.0, 5)
    x2 = float(x[0, 1])
    s = 2 + math.exp(x2)
    assert lp.item() == pytest.approx(x2 - math.log(s)) and lse.item() == pytest.approx(math.log(s))
    assert ent.item() == pytest.approx(-(0.6 * math.log(0.6) + 0.4 * math.log(0.2)))
    assert ids.tolist() == [[1, 0, 3, -1, -1]]  # 0 and -0 are equal: by place
    assert val[0, 3:].tolist() == [-math.inf, -math.inf]


@pytest.mark.parametrize("rest", [False, True])
def test_reference_gradient_is_the_losses_slope(rest):
    g = torch.Generator().manual_seed(3)
    x = torch.randn(3, 11, generator=g, dtype=torch.float64)
    ids = torch.tensor([[4, 0, 9], [1, -1, 2], [10, 3, 5]], dtype=torch.int32)
    value = torch.log_softmax(torch.randn(3, 11, generator=g, dtype=torch.float64), 1)[:, :3]
    weight = torch.tensor([1.0, -0.5, 2.0])
    T = 0.5
    _, grad = L.distill(x, ids, value, T, weight, rest)[0]
    h = 1e-5
    for v in range(11):
        up, down = x.clone(), x.clone()
        up[:, v] += h
        down[:, v] -= h
        slope = (L.distill(up, ids, value, T, weight, rest)[0][0] - L.distill(down, ids, value, T, weight, rest)[0][0]) / (2 * h)
        # a central difference: h^2 / 6 of the third derivative (below 8 |w| / T^3) and 1e-16 / h of rounding
        assert torch.allclose(slope, grad[:, v], rtol=0, atol=h * h * 8 * 2 / T ** 3 + 1e-9)


def test_reference_rest_is_the_divergence_of_classes():
    g = torch.Generator().manual_seed(4)
    x, z = (torch.randn(2, 9, generator=g, dtype=torch.float64) for _ in range(2))
    ids = torch.tensor([[0, 5], [8, 2]], dtype=torch.int32)
    p, q = z.softmax(1), x.softmax(1)
    (loss, _), _ = L.distill(x, ids, z.log_softmax(1).gather(1, ids.long()), 1.0, None, True)
    for n in range(2):
        a = [p[n, i].item() for i in ids[n].tolist()]
        b = [q[n, i].item() for i in ids[n].tolist()]
        a, b = a + [1 - sum(a)], b + [1 - sum(b)]
        assert loss[n].item() == pytest.approx(sum(s * math.log(s / t) for s, t in zip(a, b)))


def test_reference_markov_is_the_forward_passes_gradient():
    g = torch.Generator().manual_seed(5)
    rows, V, rank = 6, 8, 4
    W1, W2 = (torch.randn(V, rank, generator=g, dtype=torch.float64, requires_grad=True) for _ in range(2))
    d = torch.randn(rows, V, generator=g, dtype=torch.float64)
    prev = torch.tensor([3, -1, 3, 0, 7, 3])
    E = W1[prev.clamp(min=0)] * (prev >= 0)[:, None]
    ((E @ W2.T) * d).sum().backward()
    (_, d1, d2), _ = L.markov(d, prev, W1.detach(), W2.detach())
    assert torch.allclose(d1, W1.grad, rtol=1e-12, atol=1e-12) and torch.allclose(d2, W2.grad, rtol=1e-12, atol=1e-12)
