"""The DSPARK_DEBUG build of the attention step's kernels (checks of the rows, pages and workspace slots that they compute):
on valid inputs and on bad pages the same bits and the same status as the normal build, which each runs in a process of its
own (DSPARK_LIBRARY names it)."""
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
    import hashlib, json, sys
    import numpy as np
    import torch
    sys.path[:0] = [TESTS, TESTS + "/.."]
    from speculative_decoding_dspark_gb300 import binding as B
    from test_gpu_attention import append_case, attend, attention_case, freqs, i32, normal
    out = {"lib": B.LIB_PATH}

    def bits(*tensors):
        torch.cuda.synchronize()
        return [hashlib.sha256(t.contiguous().view(torch.uint8).cpu().numpy().tobytes()).hexdigest() for t in tensors]

    for seed, n, kv_len, page, hq, hkv, d, full, shared in [
            (1, [8] * 40, list(range(0, 800, 20)), 16, 8, 2, 128, False, 0), (2, [1, 0, 17], [90, 3, 2000], 7, 16, 2, 64, False, 0),
            (3, [40, 3, 300], [500, 30000, 0], 16, 8, 1, 128, False, 0), (4, [20] * 9, [300] * 9, 10, 16, 2, 64, True, 0),
            (5, [5] * 30, [1040 + r for r in range(30)], 16, 8, 2, 128, False, 1024)]:
        q, kc, vc, table, cu = attention_case(seed, n, kv_len, page, hq, hkv, d)
        groups = None
        if shared:
            table[:, :shared // page] = table[0, :shared // page]
            groups = ([0, len(n)], [shared])
        vc[int(table[0, (kv_len[0] + n[0] - 1) // page]), 0, (kv_len[0] + n[0] - 1) % page, 3] = float("inf")
        o, z, status = attend(B, q, kc, vc, table, kv_len, cu, full, groups)
        out[f"attend {seed}"] = [status, bits(o, z)]
        t = table.copy()
        t[-1, (kv_len[-1] + n[-1] - 1) // page] = kc.shape[0] + 3
        o, z, status = attend(B, q, kc, vc, t, kv_len, cu, full, groups)
        out[f"bad page {seed}"] = [status, bits(o, z)]
    for seed, n, kv_len, page, hq, hkv, d, rot, pairs, dt in [
            (1, [3, 0, 8, 1], [15, 4, 0, 300], 16, 32, 8, 128, 128, False, torch.bfloat16),
            (2, [900, 5], [0, 70], 7, 6, 2, 64, 48, True, torch.float32)]:
        cu, table, kc, vc = append_case(seed, n, kv_len, page, hkv, d, torch.bfloat16)
        rows = int(cu[-1]) + 3
        qkv, w, f = normal(9, (rows, hq + 2 * hkv, d), dt, 2.0), normal(5, (d,), dt), freqs(rot)
        for bad in (False, True):
            if bad:
                table[0, 0] = -1
            k, v, qo, status = kc.clone(), vc.clone(), torch.zeros(rows, hq, d, dtype=torch.bfloat16, device="cuda"), i32([0])
            B.dspark_kv_append(qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:], w, w, 1e-6, f, i32(cu), i32(kv_len), i32(table),
                               k, v, qo, interleaved=pairs, dev_status=status)
            out[f"append {seed} {bad}"] = [int(status.item()), bits(k, v, qo)]
        pos, qo, ko = i32(np.arange(rows)), torch.empty(rows, hq, d, device="cuda"), torch.empty(rows, hkv, d, device="cuda")
        status = i32([0])
        B.dspark_qk_norm_rope(qkv[:, :hq], qkv[:, hq:hq + hkv], w, w, 1e-6, pos, f, qo, ko, interleaved=pairs, dev_status=status)
        out[f"norm_rope {seed}"] = [int(status.item()), bits(qo, ko)]
    print("RESULT " + json.dumps(out))
""")


def run(lib):
    env = dict(os.environ)
    env.pop("DSPARK_LIBRARY", None)
    if lib:
        env["DSPARK_LIBRARY"] = lib
    r = subprocess.run([sys.executable, "-c", f"TESTS = {TESTS!r}\n" + CHILD], capture_output=True, text=True, env=env, timeout=600)
    assert r.returncode == 0, r.stderr[-3000:]
    return json.loads([x for x in r.stdout.splitlines() if x.startswith("RESULT ")][-1][len("RESULT "):])


def test_debug_build_of_the_attention_step():
    from speculative_decoding_dspark_gb300 import build
    build.build()
    normal, debug = run(None), run(build.build(debug=True))
    assert debug.pop("lib").endswith("libdspark_debug.so") and normal.pop("lib").endswith("libdspark.so")
    assert normal == debug
    for name, (status, _) in normal.items():
        assert status == (-6 if "bad" in name or name.endswith("True") else 0), name
