"""The example that runs the operators around a student's blocks and the optimizer
step together (examples/policy_student.py): it runs, repeats bit for bit, and its
gradients are those of the same student in 64 bits."""
import importlib.util
import math
import os

import pytest

from gpu_util import gpu_or_skip

pytestmark = pytest.mark.gpu


def _example():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                        "policy_student.py")
    spec = importlib.util.spec_from_file_location("policy_student", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_student_runs_and_repeats_bitwise():
    gpu_or_skip()
    m = _example()
    quiet = dict(steps=3, log=lambda *_: None)
    a = m.train(**quiet)
    assert all(0 <= x <= 1 for x in a)
    # every sum in the operators and in the step has a fixed order
    assert m.train(**quiet) == a


def _loss64(torch, s, p, tokens, r, kl):
    """The same student and loss, elementary operations in 64 bits on the host."""
    B, T, Hq, Hk, D = s.B, s.T, s.Hq, s.Hk, s.D
    rms = lambda v, w: v / torch.sqrt((v * v).mean(-1, keepdim=True) + 1e-6) * w
    pos = torch.arange(T, dtype=torch.float64)
    ang = pos[:, None] * s.inv_freq.cpu()[None]
    cos, sin = torch.cos(ang)[None, :, None], torch.sin(ang)[None, :, None]

    def turn(v):
        a, b = v[..., :D // 2], v[..., D // 2:]
        return torch.cat([a * cos - b * sin, b * cos + a * sin], -1)

    x = p["emb"][tokens.long()] * s.scale                       # (B, T, C)
    z = rms(x, p["pre0"])
    mask = torch.ones(T, T).tril().bool()
    for b in range(s.L):
        qkv = (z @ p[f"proj{b}"]).view(B, T, Hq + 2 * Hk, D)
        q = turn(rms(qkv[:, :, :Hq], p[f"wq{b}"])).permute(0, 2, 1, 3)
        k = turn(rms(qkv[:, :, Hq:Hq + Hk], p[f"wk{b}"])).permute(0, 2, 1, 3)
        v = qkv[:, :, Hq + Hk:].permute(0, 2, 1, 3)
        k, v = (t.repeat_interleave(Hq // Hk, 1) for t in (k, v))
        a = (q @ k.transpose(2, 3) * D ** -0.5).masked_fill(~mask, -math.inf).softmax(-1) @ v
        y = a.permute(0, 2, 1, 3).reshape(B, T, Hq * D) @ p[f"out{b}"]
        x = x + p[f"gate{b}"] * rms(y, p[f"post{b}"])
        z = rms(x, p[f"pre{b + 1}"])
    logp = torch.log_softmax((z @ p["emb"].t()).view(B * T, s.V), 1)
    lp = logp.gather(1, r["action"].long()[:, None])[:, 0]
    ratio = torch.exp(lp - r["old"])
    gain = torch.minimum(ratio * r["advantage"], ratio.clamp(0.8, 1.2) * r["advantage"])
    e = r["ref"] - lp
    return (r["weight"] * (kl * (torch.exp(e) - e - 1) - gain)).sum()


@pytest.mark.parametrize("B,T", [(1, 1), (2, 9), (3, 70)])
def test_gradients_against_64_bits(B, T):
    torch = gpu_or_skip()
    m = _example()
    s = m.Student(B, T, vocab=67)
    param = s.initial(3).to(torch.bfloat16)
    g = torch.Generator()
    g.manual_seed(4)
    N = B * T
    tokens = torch.randint(s.V, (B, T), generator=g, dtype=torch.int32)
    rollout = dict(action=torch.randint(s.V, (N,), generator=g, dtype=torch.int32),
                   advantage=torch.randn(N, generator=g), weight=torch.full((N,), 1.0 / N))
    logits, _ = s.forward(param, tokens.cuda())
    lp = torch.log_softmax(logits.float(), 1).cpu().gather(1, rollout["action"].long()[:, None])[:, 0]
    # ratios of 1 and of 1.6, clear of the borders by far more than the logits' roundings
    rollout["old"] = lp - (torch.arange(N) % 2) * math.log(1.6)
    rollout["ref"] = lp + 0.5 * torch.randn(N, generator=g)
    grad = torch.full((s.n,), float("nan"), dtype=torch.bfloat16, device="cuda")
    loss = s.update(param, grad, tokens.cuda(), {k: v.cuda() for k, v in rollout.items()}, 0.1)
    p = {n: v.cpu().double().requires_grad_() for n, v in s.views(param).items()}
    want = _loss64(torch, s, p, tokens, {k: v.double() if v.is_floating_point() else v
                                         for k, v in rollout.items()}, 0.1)
    want.backward()
    want = want.detach()
    # Roundings to bf16 that a gradient goes through: in every block z, the projection, q and
    # k, p, o and y forward, and seven backward; the embedding, the logits and their gradients: 2 (7 + 7)
    # + 6 = 34 of 2^-8 at most each, of a size that the norms keep.
    bound = 34 * 2.0 ** -8
    assert abs(float(loss) - float(want)) < bound * (abs(float(want)) + 1)
    for n, got in s.views(grad).items():
        w = p[n].grad
        off = float((got.cpu().double() - w).norm())
        # (one visible token: the softmax's gradient is 0 but for roundings of its parts)
        floor = 2.0 ** -8 * float(p["emb"].grad.norm())
        assert off <= bound * float(w.norm()) + floor, (n, off, float(w.norm()))
