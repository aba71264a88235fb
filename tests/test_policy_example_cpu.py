"""That the comparison of test_gpu_policy_example_more tells a wrong gradient of the example from a
rounded one, without a GPU: in its 64-bit student every path's gradient in turn is taken 10 % too
small, and the parameters behind the path have to leave their tolerances."""
import math
import types

import pytest

torch = pytest.importorskip("torch")

import test_gpu_policy_example_more as M  # noqa: E402
import zero_sharded_mixed_step_amd as zs  # noqa: E402


def _student(B, T, V=67, C=128, Hq=4, Hk=2, D=32, L=2):
    s = types.SimpleNamespace(B=B, T=T, V=V, C=C, L=L, Hq=Hq, Hk=Hk, D=D, scale=C ** 0.5,
                              inv_freq=zs.rope_inv_freq(D))
    g = torch.Generator()
    g.manual_seed(3)
    r = lambda *sh: torch.randn(*sh, generator=g)
    p = dict(emb=r(V, C) / s.scale, pre0=torch.ones(C))
    for b in range(L):
        p.update({f"proj{b}": r(C, (Hq + 2 * Hk) * D) * C ** -0.5, f"wq{b}": torch.ones(D),
                  f"wk{b}": torch.ones(D), f"out{b}": r(Hq * D, C) * (Hq * D) ** -0.5,
                  f"post{b}": torch.ones(C), f"gate{b}": torch.full((C,), 0.3),
                  f"pre{b + 1}": torch.ones(C)})
    return s, {n: v.to(torch.bfloat16) for n, v in p.items()}, g


class Wrong(M.Stored):
    cut = None

    def __call__(self, name, x, back=True):
        y = super().__call__(name, x, back)
        return y.detach() + 0.9 * (y - y.detach()) if name == self.cut else y


# a path, and parameters behind it
PATHS = {"x": ["emb"], "z0": ["pre0"], "qkv0": ["proj0", "pre0"], "yq0": ["wq0"], "yk0": ["wk0"],
         "yq1": ["wq1"], "yk1": ["wk1"], "y0": ["out0", "proj0"], "y1": ["out1"], "h0": ["gate0", "post0"],
         "h1": ["gate1", "post1", "out0"], "z1": ["pre1"], "z2": ["pre2", "gate1"], "qkv1": ["proj1", "pre1"],
         "logits": ["emb", "pre2"]}


@pytest.mark.parametrize("B,T", [(2, 9), (3, 70)])
def test_tolerances_notice_wrong_gradients(B, T):
    s, param, g = _student(B, T)
    N = B * T
    tokens = torch.randint(s.V, (B, T), generator=g, dtype=torch.int32)
    r = dict(action=torch.randint(s.V, (N,), generator=g, dtype=torch.int32),
             advantage=torch.randn(N, generator=g).double(), weight=torch.full((N,), 1.0 / N).double(),
             old=torch.zeros(N).double(), ref=torch.zeros(N).double())
    stored = {}
    M.student_loss(torch, s, {n: v.double() for n, v in param.items()}, tokens, r, 0.1, M.Stored(torch, stored))
    lp = torch.log_softmax(stored["logits"].double().view(N, -1), 1).gather(1, r["action"].long()[:, None])[:, 0]
    r["old"] = lp - (torch.arange(N) % 2) * math.log(1.6)
    r["ref"] = lp + 0.5 * torch.randn(N, generator=g)
    want = M.gradients(torch, s, param, tokens, r, 0.1, stored)
    tol = M.tolerances(torch, s, param, tokens, r, 0.1, stored, want)
    for n, w in want.items():
        assert tol[n] < 0.05 * float(w.norm()), n
    for cut, behind in PATHS.items():
        p = {n: v.double().requires_grad_() for n, v in param.items()}
        at = Wrong(torch, stored)
        at.cut = cut
        M.student_loss(torch, s, p, tokens, r, 0.1, at).backward()
        for n in behind:
            assert float((p[n].grad - want[n]).norm()) > tol[n], (cut, n)
