"""examples/policy_student.py: a run's whole state repeats bit for bit; from what its forward pass has
stored, every parameter's gradient is as near to the formulas' in 64 bits as their own roundings
allow."""
import math

import pytest

from gpu_util import gpu_or_skip
from test_gpu_policy_example import _example

pytestmark = pytest.mark.gpu


def test_state_repeats_bitwise_and_moves():
    torch = gpu_or_skip()
    m = _example()
    runs = []
    for _ in range(2):
        state = {}
        m.train(steps=3, log=lambda *_: None, state=state)
        step = state["step"]
        runs.append([t.clone().view(-1).view(torch.uint8)
                     for t in (step.master, step.m, step.v, step.param, state["norm"])])
        # every parameter has moved, and no gradient was lost on its way to its moments
        s = state["student"]
        first, now, moved = (s.views(t) for t in (s.initial(1), step.master, step.m))
        for n in s.shapes:
            assert bool((first[n] != now[n]).any()), n
            assert bool((moved[n] != 0).float().mean() > 0.5), n
            assert bool(torch.isfinite(now[n]).all()), n
        assert 0.0 < float(state["norm"]) < math.inf
    for a, b in zip(*runs):
        assert torch.equal(a, b)


class Stored:
    """64-bit arithmetic that goes on from what the GPU has stored, so that a tensor's forward roundings
    are the GPU's own, and rounds gradients to bf16 where the example does.  With `noise` what is
    rounded first moves by 2^-19 of the tensor's size, more than sums in binary32 are off by, so that
    values next to a border of the rounding cross it as they may in another order, and what only
    the attention's backward rounds moves by up to a half step."""

    def __init__(self, torch, tensors, noise=None):
        self.torch, self.tensors, self.g = torch, tensors, None
        if noise is not None:
            self.g = torch.Generator()
            self.g.manual_seed(noise)

    def u(self, x):
        return 2 * self.torch.rand(x.shape, generator=self.g, dtype=x.dtype) - 1

    def bf16(self, x):
        if self.g is not None:
            x = x + 2.0 ** -19 * x.square().mean().sqrt() * self.u(x)
        return x.to(self.torch.bfloat16).double()

    def inside(self, x):
        return x if self.g is None else x * (1 + 2.0 ** -8 * self.u(x))

    def __call__(self, name, x, back=True):
        """What the GPU has stored as `name`, which has to be x but for its rounding and those of
        the operator inside; its gradient is rounded (where `back`)."""
        me, kept = self, self.tensors.get(name)
        if kept is None:                       # (the test of the test has no GPU: store x)
            kept = self.tensors[name] = x.detach().to(self.torch.bfloat16 if back or name == "x"
                                                      else self.torch.float32)
        kept = kept.double().view(x.shape)
        assert float((kept - x.detach()).norm()) <= 2.0 ** -7 * float(x.detach().norm()), name

        class Replace(self.torch.autograd.Function):
            @staticmethod
            def forward(ctx, x):
                return kept.clone()

            @staticmethod
            def backward(ctx, g):
                return me.bf16(g) if back else g

        return Replace.apply(x)

    def attention(self, name, q, k, v, mask, scale):
        """Softmax attention over (B, H, T, D) whose backward takes the row sums of do * o from the
        stored output; the weights and their gradients are rounded inside."""
        me, torch = self, self.torch

        class Attention(torch.autograd.Function):
            @staticmethod
            def forward(ctx, q, k, v):
                p = (q @ k.transpose(2, 3) * scale).masked_fill(~mask, -math.inf).softmax(-1)
                o = p @ v
                kept = me.tensors.get(name)
                if kept is not None:
                    kept = kept.double().view(o.transpose(1, 2).shape).transpose(1, 2)
                    assert float((kept - o).norm()) <= 2.0 ** -7 * float(o.norm()), name
                    o = kept
                else:
                    o = o.to(torch.bfloat16).double()
                    me.tensors[name] = o.transpose(1, 2).contiguous()
                ctx.save_for_backward(q, k, v, p, o)
                return o.clone()

            @staticmethod
            def backward(ctx, do):
                q, k, v, p, o = ctx.saved_tensors
                do = me.bf16(do)
                dp = do @ v.transpose(2, 3)
                if me.g is not None:
                    dp = dp + 2.0 ** -19 * (do.abs() @ v.abs().transpose(2, 3)) * me.u(dp)
                ds = me.inside(p * (dp - (do * o).sum(-1, keepdim=True))) * scale
                return ds @ k, ds.transpose(2, 3) @ q, me.inside(p).transpose(2, 3) @ do

        return Attention.apply(q, k, v)


def student_loss(torch, s, p, tokens, r, kl, at):
    """The example's student and loss, elementary operations in 64 bits."""
    B, T, Hq, Hk, D = s.B, s.T, s.Hq, s.Hk, s.D
    rms = lambda v, w: v / torch.sqrt((v * v).mean(-1, keepdim=True) + 1e-6) * w
    ang = torch.arange(T, dtype=torch.float64)[:, None] * s.inv_freq.cpu()[None]
    cos, sin = torch.cos(ang)[None, :, None], torch.sin(ang)[None, :, None]

    def turn(v):
        a, b = v[..., :D // 2], v[..., D // 2:]
        return torch.cat([a * cos - b * sin, b * cos + a * sin], -1)

    x = at("x", p["emb"][tokens.long()] * s.scale, back=False)
    z = at("z0", rms(x, p["pre0"]))
    mask = torch.ones(T, T).tril().bool()
    for b in range(s.L):
        qkv = at(f"qkv{b}", z @ p[f"proj{b}"]).view(B, T, Hq + 2 * Hk, D)
        q = at(f"yq{b}", turn(rms(qkv[:, :, :Hq], p[f"wq{b}"]))).permute(0, 2, 1, 3)
        k = at(f"yk{b}", turn(rms(qkv[:, :, Hq:Hq + Hk], p[f"wk{b}"]))).permute(0, 2, 1, 3)
        v = qkv[:, :, Hq + Hk:].permute(0, 2, 1, 3)
        k, v = (t.repeat_interleave(Hq // Hk, 1) for t in (k, v))
        a = at.attention(f"o{b}", q, k, v, mask, D ** -0.5)
        y = at(f"y{b}", a.permute(0, 2, 1, 3).reshape(B, T, Hq * D) @ p[f"out{b}"])
        x = at(f"h{b}", x + p[f"gate{b}"] * rms(y, p[f"post{b}"]), back=False)
        z = at(f"z{b + 1}", rms(x, p[f"pre{b + 1}"]))
    logp = torch.log_softmax(at("logits", z @ p["emb"].t()).view(B * T, s.V), 1)
    lp = logp.gather(1, r["action"].long()[:, None])[:, 0]
    ratio = torch.exp(lp - r["old"])
    gain = torch.minimum(ratio * r["advantage"], ratio.clamp(0.8, 1.2) * r["advantage"])
    e = r["ref"] - lp
    return (r["weight"] * (kl * (torch.exp(e) - e - 1) - gain)).sum()


def gradients(torch, s, param, tokens, r, kl, stored, noise=None):
    """{name: gradient} and "loss"."""
    p = {n: v.double().requires_grad_() for n, v in param.items()}
    loss = student_loss(torch, s, p, tokens, r, kl, Stored(torch, stored, noise))
    loss.backward()
    return dict({n: v.grad for n, v in p.items()}, loss=loss.detach())


def tolerances(torch, s, param, tokens, r, kl, stored, want, runs=8):
    """What each may be off by: three times the furthest of some runs whose roundings move, and of
    its own size three half steps (one rounding of the result, and single values on the other side of a
    border that no run may have met)."""
    off = {n: 0.0 for n in want}
    for noise in range(runs):
        other = gradients(torch, s, param, tokens, r, kl, stored, noise)
        for n in want:
            off[n] = max(off[n], float((other[n] - want[n]).norm()))
    return {n: 3 * off[n] + 3 * 2.0 ** -8 * float(want[n].norm()) + 1e-12 for n in want}


@pytest.mark.parametrize("B,T", [(1, 1), (2, 9), (3, 70)])
def test_each_gradient_from_what_is_stored(B, T):
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
    logits, (saved, z) = s.forward(param, tokens.cuda())
    stored = {"logits": logits, f"z{s.L}": z}
    for b, kept in enumerate(saved):
        stored.update({n + str(b): t for n, t in zip(("z", "qkv", "yq", "yk", "o", "lse", "y", "h"), kept)})
    stored = {n: t.cpu() for n, t in stored.items()}
    lp = torch.log_softmax(stored["logits"].double(), 1).gather(1, rollout["action"].long()[:, None])[:, 0]
    # ratios of 1 and of 1.6, clear of the borders
    rollout["old"] = (lp - (torch.arange(N) % 2) * math.log(1.6)).float()
    rollout["ref"] = (lp + 0.5 * torch.randn(N, generator=g)).float()
    grad = torch.full((s.n,), float("nan"), dtype=torch.bfloat16, device="cuda")
    loss = s.update(param, grad, tokens.cuda(), {k: v.cuda() for k, v in rollout.items()}, 0.1)
    got = {n: v.cpu().double() for n, v in s.views(grad).items()}
    got["loss"] = loss.cpu().double()
    host = {n: v.cpu() for n, v in s.views(param).items()}
    r = {k: v.double() if v.is_floating_point() else v for k, v in rollout.items()}
    want = gradients(torch, s, host, tokens, r, 0.1, stored)
    tol = tolerances(torch, s, host, tokens, r, 0.1, stored, want)
    for n, w in want.items():
        # (a wrong factor or a missing term shows; of one visible token the softmax has no gradient)
        assert T == 1 or tol[n] < 0.05 * float(w.norm()), (n, tol[n], float(w.norm()))
        off = float((got[n] - w).norm())
        assert off <= tol[n], (n, off, tol[n], float(w.norm()))
