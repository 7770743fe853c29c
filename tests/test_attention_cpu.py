"""Host-side checks of the attention step's entry points, and pins of the 64-bit reference the GPU tests compare with."""
import ctypes
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import attention_reference as A  # noqa: E402

INVALID, UNSUPPORTED, WORKSPACE = -1, -2, -7
vp, i32, i64, f32, u32 = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_float, ctypes.c_uint
F = vp(4096)  # never dereferenced: every call here is refused on the host


@pytest.fixture(scope="module")
def lib():
    from speculative_decoding_dspark_gb300 import build
    try:
        build.nvcc()
    except RuntimeError:
        pytest.skip("nvcc not available")
    return ctypes.CDLL(build.build())


ROPE = dict(q=F, q_stride=8 * 128, k=F, k_stride=2 * 128, in_dtype=1, wq=F, wk=F, eps=1e-6, positions=F, inv_freq=F,
            rot=128, rows=5, hq=8, hkv=2, d=128, q_out=F, qo_stride=8 * 128, k_out=F, ko_stride=2 * 128, out_dtype=1,
            flags=0, status=None, stream=None)
ROPE_T = [vp, i64, vp, i64, i32, vp, vp, f32, vp, vp, i32, i32, i32, i32, i32, vp, i64, vp, i64, i32, u32, vp, vp]
APPEND = dict(q=F, q_stride=8 * 128, k=F, k_stride=2 * 128, v=F, v_stride=2 * 128, in_dtype=1, wq=F, wk=F, eps=1e-6,
              inv_freq=F, rot=128, cu=F, kv_len=F, table=F, R=4, rows=9, hq=8, hkv=2, d=128, page=16, blocks=8, pool=32,
              k_cache=F, v_cache=F, q_out=F, out_dtype=1, flags=0, status=None, stream=None)
APPEND_T = [vp, i64, vp, i64, vp, i64, i32, vp, vp, f32, vp, i32, vp, vp, vp] + [i32] * 8 + [vp, vp, vp, i32, u32, vp, vp]
ATT = dict(q=F, k=F, v=F, table=F, kv_len=F, cu=F, scale=0.1, R=4, rows=9, hq=8, hkv=2, d=128, page=16, blocks=8,
           pool=32, out=F, lse=F, flags=0, ws=vp(256 * 64), ws_bytes=1 << 40, status=None, stream=None)
ATT_T = [vp] * 6 + [f32] + [i32] * 8 + [vp, vp, u32, vp, ctypes.c_size_t, vp, vp]
PRE = dict(q=F, k=F, v=F, table=F, kv_len=F, cu=F, group_start=F, shared=F, n_groups=2, scale=0.1, R=4, rows=9, hq=8,
           hkv=2, d=128, page=16, blocks=8, pool=32, out=F, lse=F, flags=0, ws=vp(256 * 64), ws_bytes=1 << 40,
           status=None, stream=None)
PRE_T = [vp] * 8 + [i32, f32] + [i32] * 8 + [vp, vp, u32, vp, ctypes.c_size_t, vp, vp]


def call(lib, name, types, base, **change):
    f = getattr(lib, name)
    f.restype, f.argtypes = i32, types
    assert set(change) <= set(base)
    return f(*{**base, **change}.values())


BAD_HEADS = [
    (dict(k=None), INVALID), (dict(in_dtype=2), INVALID), (dict(out_dtype=-1), INVALID), (dict(hkv=0), INVALID),
    (dict(d=0), INVALID), (dict(rot=7), INVALID), (dict(rot=144), INVALID), (dict(rot=-16), INVALID),
    (dict(eps=-1.0), INVALID), (dict(eps=float("nan")), INVALID), (dict(inv_freq=None), INVALID),
    (dict(q_stride=8 * 128 - 1), INVALID), (dict(k_stride=8), INVALID), (dict(flags=2), INVALID), (dict(rows=-1), INVALID),
    (dict(d=60, rot=48), UNSUPPORTED), (dict(rot=24), UNSUPPORTED), (dict(q=vp(4104)), UNSUPPORTED),
    (dict(wk=vp(4100)), UNSUPPORTED), (dict(q_stride=8 * 128 + 4), UNSUPPORTED), (dict(q_out=vp(4104)), UNSUPPORTED),
    (dict(d=264, q_stride=1 << 20, k_stride=1 << 20), UNSUPPORTED),
]


@pytest.mark.parametrize("change,status", BAD_HEADS)
def test_heads_refusals(lib, change, status):
    rope = dict(change)
    if "d" in change:
        rope.update(qo_stride=1 << 20, ko_stride=1 << 20)
    if change.get("d") == 264 or "rows" in change:
        assert call(lib, "dspark_kv_append", APPEND_T, {**APPEND, "v_stride": 1 << 20}, **change) == status
    else:
        assert call(lib, "dspark_kv_append", APPEND_T, APPEND, **change) == status
    assert call(lib, "dspark_qk_norm_rope", ROPE_T, ROPE, **rope) == status


def test_heads_refusals_of_one_call(lib):
    assert call(lib, "dspark_qk_norm_rope", ROPE_T, ROPE, positions=None) == INVALID
    assert call(lib, "dspark_qk_norm_rope", ROPE_T, ROPE, ko_stride=2) == INVALID
    assert call(lib, "dspark_qk_norm_rope", ROPE_T, ROPE, hq=0) == INVALID
    assert call(lib, "dspark_qk_norm_rope", ROPE_T, ROPE, k_out=None) == INVALID
    assert call(lib, "dspark_qk_norm_rope", ROPE_T, ROPE, in_dtype=0, q_stride=8 * 128 + 2) == UNSUPPORTED
    assert call(lib, "dspark_kv_append", APPEND_T, APPEND, q=None) == INVALID          # n_q_heads without q
    assert call(lib, "dspark_kv_append", APPEND_T, APPEND, hq=0) == INVALID            # q without heads
    assert call(lib, "dspark_kv_append", APPEND_T, APPEND, R=0) == INVALID
    assert call(lib, "dspark_kv_append", APPEND_T, APPEND, page=0) == INVALID
    assert call(lib, "dspark_kv_append", APPEND_T, APPEND, v_stride=100) == INVALID
    assert call(lib, "dspark_kv_append", APPEND_T, APPEND, k_cache=vp(4104)) == UNSUPPORTED
    # no rows: nothing to do
    assert call(lib, "dspark_qk_norm_rope", ROPE_T, ROPE, rows=0) == 0
    assert call(lib, "dspark_kv_append", APPEND_T, APPEND, rows=0) == 0


@pytest.mark.parametrize("change,status", [
    (dict(q=None), INVALID), (dict(table=None), INVALID), (dict(out=None), INVALID), (dict(R=0), INVALID),
    (dict(rows=-1), INVALID), (dict(hq=9), INVALID), (dict(page=0), INVALID), (dict(blocks=0), INVALID),
    (dict(scale=float("nan")), INVALID), (dict(scale=float("inf")), INVALID), (dict(scale=-0.1), INVALID), (dict(flags=2), INVALID),
    (dict(pool=-1), INVALID), (dict(d=96), UNSUPPORTED), (dict(hq=258), UNSUPPORTED), (dict(pool=1 << 30), UNSUPPORTED), (dict(rows=1 << 29), UNSUPPORTED), (dict(q=vp(4104)), UNSUPPORTED),
    (dict(v=vp(4098)), UNSUPPORTED), (dict(ws=None), WORKSPACE), (dict(ws=vp(4100)), WORKSPACE),
    (dict(ws_bytes=16), WORKSPACE), (dict(rows=0), 0),
])
def test_attention_refusals(lib, change, status):
    assert call(lib, "dspark_verify_attention", ATT_T, ATT, **change) == status
    assert call(lib, "dspark_prefix_attention", PRE_T, PRE, **change) == status


def test_prefix_refusals_and_workspace(lib):
    assert call(lib, "dspark_prefix_attention", PRE_T, PRE, group_start=None) == INVALID
    assert call(lib, "dspark_prefix_attention", PRE_T, PRE, shared=None) == INVALID
    assert call(lib, "dspark_prefix_attention", PRE_T, PRE, n_groups=0) == INVALID
    assert call(lib, "dspark_prefix_attention", PRE_T, PRE, R=1 << 30, n_groups=1 << 30) == UNSUPPORTED
    size = lib.dspark_attention_workspace_size
    size.restype, size.argtypes = ctypes.c_size_t, [i32] * 6
    assert size(4, 0, 9, 8, 2, 128) > 0 and size(4, 2, 9, 8, 2, 128) >= size(4, 0, 9, 8, 2, 128)
    for bad in ((0, 0, 9, 8, 2, 128), (4, -1, 9, 8, 2, 128), (4, 0, -1, 8, 2, 128), (4, 0, 9, 8, 3, 128),
                (4, 0, 9, 8, 2, 96), (4, 0, 9, 0, 2, 128)):
        assert size(*bad) == 0


# ------------------------------------------------------------------ pins of the reference
def test_reference_heads_worked_example():
    """d = 2, one pair, a quarter turn: (3, 4) normed by its root mean square sqrt(12.5) is turned to (-4, 3)."""
    x = torch.tensor([[[3.0, 4.0]]])
    for pairs in (False, True):
        y, _ = A.heads(x, torch.ones(2), 0.0, torch.tensor([1]), torch.tensor([math.pi / 2], dtype=torch.float64), pairs)
        np.testing.assert_allclose(y[0, 0].numpy(), np.array([-4.0, 3.0]) / math.sqrt(12.5), atol=1e-12)
    y, _ = A.heads(x, None, 0.0, torch.tensor([0]), torch.tensor([1.0]), False)
    np.testing.assert_array_equal(y.numpy(), x.double().numpy())


def test_reference_rotation_keeps_relative_positions():
    """q(m) . k(n) depends on m - n alone."""
    rng = np.random.default_rng(1)
    q, k = (torch.tensor(rng.normal(size=(1, 1, 8))) for _ in range(2))
    f = torch.tensor([1.0, 0.3, 0.02, 0.001])
    dot = []
    for m, n in ((7, 3), (1007, 1003)):
        a, _ = A.heads(q, None, 0.0, torch.tensor([m]), f, True)
        b, _ = A.heads(k, None, 0.0, torch.tensor([n]), f, True)
        dot.append(float((a * b).sum()))
    assert abs(dot[0] - dot[1]) < 1e-9


def test_reference_attention_worked_example():
    """Two keys with scores 0 and log 3: weights 1/4 and 3/4; the first of two causal rows sees one key less."""
    page, d = 2, 64
    k, v = torch.zeros(2, 1, page, d), torch.zeros(2, 1, page, d)
    k[1, 0, 1, 0] = math.log(3.0)          # position 1: page 1 of the pool, slot 1
    v[1, 0, 0, :], v[1, 0, 1, :] = 4.0, 8.0
    q = torch.zeros(2, 1, d)
    q[:, 0, 0] = 1.0
    table = np.array([[1, -1]], np.int32)
    out, lse, tol, _ = A.attention(q, k, v, table, [0], [0, 2], 1.0, False)
    np.testing.assert_allclose(out[0].numpy(), 4.0)
    np.testing.assert_allclose(out[1].numpy(), 7.0)
    np.testing.assert_allclose(lse.numpy().ravel(), [0.0, math.log(4.0)], atol=1e-12)
    full, _, _, _ = A.attention(q, k, v, table, [0], [0, 2], 1.0, True)
    np.testing.assert_allclose(full.numpy(), 7.0)
    assert float(tol.max()) < 0.1
