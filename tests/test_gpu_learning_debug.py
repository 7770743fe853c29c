"""The DSPARK_DEBUG build of the kernels on vocabulary rows and of the Markov factors' gradient: on valid inputs and on bad
tokens, lengths and lists the same bits and the same status as the normal build, each in a process of its own
(DSPARK_LIBRARY names it)."""
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
    from test_gpu_learning import BF16, F32, INF, distill, i32, logprobs, markov, markov_case, normal, rows_of, teacher_of
    out = {"lib": B.LIB_PATH}

    def bits(*tensors):
        torch.cuda.synchronize()
        return [hashlib.sha256(t.contiguous().view(torch.uint8).cpu().numpy().tobytes()).hexdigest() for t in tensors if t is not None]

    for dtype in (F32, BF16):
        for rows, V, top in ((1, 50001, 20), (40, 1001, 128), (300, 20000, 5), (2, 300000, 128)):
            x = rows_of(normal(V, (rows, V), 3.0), dtype, 3, 1)
            x[0, :V // 2] = -INF
            *o, status = logprobs(B, x, i32(np.arange(rows) * 7 % V), 0.7, top)
            out[f"logprobs {dtype} {V}"] = [status, bits(*o)]
            ids, value = teacher_of(3, x, top)
            for grad in (None, F32, BF16):
                loss, g, status = distill(B, x, ids, value, 1.0, grad, rest=V % 2 == 0)
                out[f"distill {dtype} {V} {grad}"] = [status, bits(loss, g)]
            ids[rows - 1, 0] = V + 5
            if top > 1:
                ids[0, 1] = ids[0, 0]
            loss, g, status = distill(B, x, ids, value, 1.0, dtype, rest=True)
            out[f"bad list {dtype} {V}"] = [status, bits(torch.isnan(loss))]
        x = torch.full((3, 9000), 1.5, device="cuda").to(dtype)
        *o, status = logprobs(B, x, i32([1, 9000, -1]), 1.0, 64)
        out[f"equal {dtype}"] = [status, bits(*o)]
        *o, status = logprobs(B, x, i32(np.zeros((2, 2))), 1.0, 4, cu=i32([0, 2, 9]))
        out[f"lengths {dtype}"] = [status, bits(*o)]
    for rows, V, rank in ((7, 640, 64), (300, 4104, 320)):
        g, prev, W1, W2 = markov_case(rows, rows, V, rank)
        for bad in (False, True):
            if bad:
                prev[2], prev[rows - 1] = V, -4
                g[rows - 1] = INF
            *o, status = markov(B, g, prev, W1, W2)
            out[f"markov {rows} {bad}"] = [status, bits(*o)]
    print("RESULT " + json.dumps(out))
""")


def run(lib=None):
    env = dict(os.environ)
    env.pop("DSPARK_LIBRARY", None)
    if lib:
        env["DSPARK_LIBRARY"] = lib
    r = subprocess.run([sys.executable, "-c", f"TESTS = {TESTS!r}\n" + CHILD], capture_output=True, text=True, env=env, timeout=300)
    assert r.returncode == 0, r.stderr[-3000:]
    return json.loads([line for line in r.stdout.splitlines() if line.startswith("RESULT ")][-1][7:])


def test_debug_build_gives_the_same_bits():
    from speculative_decoding_dspark_gb300 import build
    normal, debug = run(build.build()), run(build.build(debug=True))
    assert normal.pop("lib") != debug.pop("lib")
    assert normal.keys() == debug.keys()
    for k in normal:
        assert normal[k] == debug[k], k
        assert normal[k][0] in (0, -6), k
