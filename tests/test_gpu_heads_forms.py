"""Forms of dspark_qk_norm_rope and dspark_kv_append whose CTAs need about 48 KB of shared memory, each in a process of its
own (what a kernel may use is raised once for the process, so an earlier call could hide a later one's refusal).
Definitions and tolerances: attention_reference.py."""
import json
import os
import subprocess
import sys
import textwrap

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

TESTS = os.path.dirname(os.path.abspath(__file__))

CHILD = textwrap.dedent(r"""
    import json, sys
    import torch
    TESTS, name, rows, hq, hkv, d, rot, pairs = json.loads(sys.argv[1])
    sys.path[:0] = [TESTS, TESTS + "/.."]
    import attention_reference as A
    from speculative_decoding_dspark_gb300 import binding as B
    g = torch.Generator("cuda")
    g.manual_seed(rows)
    qkv = torch.randn((rows, hq + 2 * hkv, d), generator=g, device="cuda")
    w = torch.randn((d,), generator=g, device="cuda")
    q, k, v = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
    f = torch.tensor([10000.0 ** (-2.0 * i / rot) for i in range(rot // 2)], device="cuda") if rot else None
    at = torch.arange(rows, dtype=torch.int32, device="cuda") + 1000
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    qo = torch.empty(rows, hq, d, dtype=torch.bfloat16, device="cuda")
    if name == "norm_rope":
        ko = torch.empty(rows, hkv, d, dtype=torch.bfloat16, device="cuda")
        B.dspark_qk_norm_rope(q, k, w, w, 1e-6, at if rot else None, f, qo, ko, interleaved=pairs, dev_status=status)
        sides = [(q, qo), (k, ko)]
    else:
        page, R = 16, 3
        n = [rows // 2, 0, rows - rows // 2]
        blocks = -(-(1000 + rows) // page)
        kc = torch.zeros(2 * blocks, hkv, page, d, dtype=torch.bfloat16, device="cuda")
        vc = torch.zeros_like(kc)
        table = torch.arange(2 * blocks, dtype=torch.int32, device="cuda").view(2, blocks)[[0, 0, 1]].contiguous()
        cu = torch.tensor([0, n[0], n[0], rows], dtype=torch.int32, device="cuda")
        kv_len = torch.tensor([1000, 5, 1000 + n[0]], dtype=torch.int32, device="cuda")  # so that row t stands at 1000 + t
        B.dspark_kv_append(q, k, v, w, w, 1e-6, f, cu, kv_len, table, kc, vc, qo, interleaved=pairs, dev_status=status)
        side = (torch.arange(rows, device="cuda") >= n[0]).long()
        place = table[2 * side, (at // page).long()].long()
        assert torch.equal(vc[place, :, (at % page).long()], v.bfloat16())
        sides = [(q, qo), (k, kc[place, :, (at % page).long()])]
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    few = torch.tensor(sorted({0, 1, 2, rows // 2 - 1, rows // 2, rows // 2 + 1, rows - 9, rows - 2, rows - 1}))
    worst = 0.0
    for x, y in sides:
        ref, size = A.heads(x[few], w, float(torch.tensor(1e-6)), at[few], f, pairs)
        err = (y[few].double().cpu() - ref).abs() / A.heads_tol(ref, size, torch.bfloat16)
        worst = max(worst, float(err.nan_to_num(1e9).max()))
    print("RESULT " + json.dumps(worst))
""")


@pytest.mark.parametrize("name,rows,hq,hkv,d,rot,pairs", [
    ("norm_rope", 153, 24, 8, 128, 0, False), ("norm_rope", 700, 24, 8, 128, 0, True),
    ("append", 153, 16, 8, 128, 0, False), ("append", 400, 48, 8, 64, 0, False),
    ("norm_rope", 4900, 32, 8, 192, 160, False), ("norm_rope", 4900, 32, 8, 192, 176, True),
    ("norm_rope", 4900, 32, 8, 192, 192, False), ("append", 4900, 16, 8, 128, 128, False),
])
def test_fp32_heads_that_fill_a_cta(name, rows, hq, hkv, d, rot, pairs):
    from speculative_decoding_dspark_gb300 import build
    build.build()
    arg = json.dumps([TESTS, name, rows, hq, hkv, d, rot, pairs])
    r = subprocess.run([sys.executable, "-c", CHILD, arg], capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stderr[-2000:]
    line = [x for x in r.stdout.splitlines() if x.startswith("RESULT ")][-1]
    assert json.loads(line[len("RESULT "):]) <= 1.0
