"""The attention example: prompt, drafts, reserve, append, attention and commit together."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)


@pytest.mark.parametrize("sizes", [dict(), dict(requests=5, hidden=256, hq=8, hkv=2, d=64, shared=96, page=12, cycles=3)])
def test_attention_layer(sizes):
    from speculative_decoding_dspark_gb300 import build
    build.build()
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "attention_layer.py")
    spec = importlib.util.spec_from_file_location("attention_layer", path)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    error, pages, kv_len = example.run(**sizes)
    # Of the largest output: the weights' rounding and the output's (2^-8 each at most), and a query or key that fp32
    # rounds to the other neighbour (a step of 2^-7 on some elements moves a score by some 2^-8).
    assert error < 4 * 2.0 ** -8
    page, shared = sizes.get("page", 16), sizes.get("shared", 512)
    assert pages == shared // page + sum(-(-int(n) // page) - shared // page for n in kv_len)  # none lost
