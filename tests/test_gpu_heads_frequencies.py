"""Frequencies that are not finite, in the rotation of dspark_qk_norm_rope (tolerances: attention_reference.py)."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

import attention_reference as A  # noqa: E402


@pytest.mark.parametrize("pairs", [False, True])
def test_frequencies_that_are_not_finite(pairs):
    """An angle without a value leaves its pair without one, and only that pair; position 0 is no exception (0 times
    infinity)."""
    from speculative_decoding_dspark_gb300 import build
    build.build()
    from speculative_decoding_dspark_gb300 import binding as B
    rows, hq, hkv, d, rot = 4, 3, 1, 64, 48
    g = torch.Generator("cuda")
    g.manual_seed(1)
    q = torch.randn((rows, hq, d), generator=g, device="cuda")
    k = torch.randn((rows, hkv, d), generator=g, device="cuda")
    f = torch.tensor([10000.0 ** (-2.0 * i / rot) for i in range(rot // 2)], device="cuda")
    odd = {3: float("inf"), 8: float("nan"), 23: float("-inf")}
    finite = f.clone()
    for i, x in odd.items():
        f[i], finite[i] = x, 0.0
    pos = torch.tensor([0, 1, 77, 100000], dtype=torch.int32, device="cuda")
    qo, ko = torch.empty_like(q), torch.empty_like(k)
    B.dspark_qk_norm_rope(q, k, None, None, 1e-6, pos, f, qo, ko, interleaved=pairs)
    torch.cuda.synchronize()
    lost = torch.zeros(d, dtype=torch.bool)
    for i in odd:
        lost[[2 * i, 2 * i + 1] if pairs else [i, i + rot // 2]] = True
    for x, y in ((q, qo), (k, ko)):
        y = y.double().cpu()
        ref, size = A.heads(x, None, 1e-6, pos, finite, pairs)
        assert bool(torch.isnan(y[..., lost]).all())
        assert bool(((y - ref).abs() <= A.heads_tol(ref, size, torch.float32))[..., ~lost].all())
