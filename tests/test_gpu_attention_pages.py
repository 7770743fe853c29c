"""A request whose pages are not all there gets NaN rows, all of them, however its rows are cut into items."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

import attention_reference as A  # noqa: E402
from test_gpu_attention import B, DEVICE_INPUT, attend, attention_case, close  # noqa: E402,F401


@pytest.mark.parametrize("missing", ["last", "middle", "first"])
@pytest.mark.parametrize("full", [False, True])
@pytest.mark.parametrize("n,kv_len,page,hq,hkv,d", [
    ([2, 300, 5], [40, 20, 300], 16, 8, 2, 128),   # 1200 rows a key head: five items
    ([200, 3, 600], [0, 77, 0], 12, 4, 1, 64),     # several of them in one batch, pages that end anywhere
    ([300, 300], [500, 500], 1, 4, 2, 64),
])
def test_a_missing_page_spoils_its_request(B, n, kv_len, page, hq, hkv, d, full, missing):
    case = attention_case(23, n, kv_len, page, hq, hkv, d)
    q, kc, vc, table, cu = case
    ref, lse, tol, ztol = A.attention(q, kc, vc, table, kv_len, cu, float(np.float32(d ** -0.5)), full)
    bad = int(np.argmax(n))
    last = (kv_len[bad] + n[bad] - 1) // page
    for groups in (None, ([0, len(n)], [0])):
        for value in (-1, kc.shape[0]):
            t = table.copy()
            t[bad, {"last": last, "middle": last // 2 + 1, "first": 0}[missing]] = value
            out, z, status = attend(B, q, kc, vc, t, kv_len, cu, full, groups)
            assert status == DEVICE_INPUT
            rows = torch.zeros(int(cu[-1]), dtype=torch.bool)
            rows[int(cu[bad]):int(cu[bad + 1])] = True
            assert bool(torch.isnan(out.cpu()[rows]).all()) and bool(torch.isnan(z.cpu()[rows]).all())
            close(out.cpu()[~rows], ref[~rows], tol[~rows], "out")
            close(z.cpu()[~rows], lse[~rows], ztol[~rows], "lse")
