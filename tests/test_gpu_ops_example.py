"""The example that runs the training operators and the optimizer step
together (examples/distill_student.py)."""
import importlib.util
import os

import pytest

from gpu_util import gpu_or_skip

pytestmark = pytest.mark.gpu


def _example():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                        "distill_student.py")
    spec = importlib.util.spec_from_file_location("distill_student", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_student_learns_and_repeats_bitwise():
    gpu_or_skip()
    m = _example()
    quiet = dict(steps=20, log=lambda *_: None)
    a = m.train(**quiet)
    assert all(x == x and x >= 0 for x in a)
    assert a[-1] < a[0]
    # every sum in the operators and in the step has a fixed order
    assert m.train(**quiet) == a


def test_student_of_one_token_rows():
    """The smallest rows: one visible token each, padding behind it."""
    torch = gpu_or_skip()
    m = _example()
    s = m.Student(3, 9)
    flat = s.initial(2).to(torch.bfloat16)
    b = m.batch(s, 4)
    b["doc"].fill_(-1)
    b["doc"][:, 0] = 0
    b["weight"].zero_()
    b["weight"].view(3, 9)[:, 0] = 1 / 3
    grad = torch.full((s.n,), float("nan"), dtype=torch.bfloat16, device="cuda")
    loss = s.run(flat, grad, **b)
    g = s.views(grad)
    assert bool(torch.isfinite(loss))
    assert all(bool(torch.isfinite(x).all()) for x in g.values())
    # a query that sees one key has the softmax 1 whatever its score: no gradient
    # reaches the norms' weights or the bias but the roundings of do . o, a bf16 o and
    # products summed in binary32 (|do|, |o| < 4 here, D = 64: below 64 * 16 * 2^-8)
    for name in ("wq", "wk", "bias"):
        assert float(g[name].float().abs().max()) < 64 * 16 * 2.0 ** -8
