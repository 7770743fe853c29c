"""Where the operators on vocabulary rows and of the Markov factors' gradient could go wrong and test_gpu_learning.py does
not look: clusters that start beside other work, rests next to nothing, single terms of long sums, long chains, tokens
that repeat, buffers kept for the largest call, a verify's packed rows."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

import learning_reference as L  # noqa: E402
import parity_helpers as H  # noqa: E402
from test_gpu_learning import (BF16, F32, I32, B, close, distill, generator, i32, logprobs, markov,  # noqa: E402,F401
                               markov_case, normal, rows_of, teacher_of)


# ----------------------------------------------------------------------------------------- distillation
@pytest.mark.parametrize("V", [4001, 8003, 32003])
def test_distill_beside_other_work(B, V):
    """Rows shared by two, four and eight CTAs, whose clusters find room one CTA of theirs after the other while another
    stream fills the GPU: the bits of a call by itself."""
    rows, top = 5, 20
    x = normal(V, (rows, V), 3.0)
    ids, value = teacher_of(V, x, top)
    want = distill(B, x, ids, value, 1.0, F32, rest=True)
    assert want[2] == 0
    other, side = torch.cuda.Stream(), torch.cuda.Stream()
    a = normal(1, (1 << 24,))
    losses, grads = torch.empty(40, rows, device="cuda"), torch.empty(40, rows, V, device="cuda")
    status = torch.zeros(1, dtype=I32, device="cuda")
    torch.cuda.synchronize()
    for k in range(40):
        with torch.cuda.stream(other):
            a.mul_(1.0)
            a.view(-1, 64).sum(1)
        B.dspark_distill_loss(x, ids, value, 1.0, losses[k], grad=grads[k], rest=True, dev_status=status, stream=side)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    assert all(torch.equal(losses[k], want[0]) and torch.equal(grads[k], want[1]) for k in range(40))
