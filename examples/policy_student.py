"""A small student improved on its own samples: the operators around its blocks and
the optimizer step together, as a training program uses them.

The student is two attention blocks between norms, with an fp32 residual stream
and a tied embedding:

  zero_embed -> zero_block_norm (the first norm), then in every block
  projection -> zero_qk_norm_rope -> zero_attn -> projection -> zero_block_norm (the
  output's norm, its gate, the residual sum, the next block's norm), then
  logits -> zero_policy

At every position it samples a token and is rewarded where its rest by 4 is one more than
that of the token before it; each rollout serves a few updates with the clipped policy
loss and a KL term to the initial student.  The gradients of all parameters are
views of one vector; their global norm and clipping (zero_grads_norm, zero_grads_clip)
write the bf16 replica that `ShardStep` reduces.  Plain matrix products are torch's.

One rank trains here, whose gradient is the whole one.  With several, every rank's gradient goes to
the step unclipped: the norm to clip by is that of the reduced gradient, whose shards' accumulators
add up (zero_grad_norm of each rank's shard, or zero_grads_norm of its pieces), and the
step clips by it itself.

  python examples/policy_student.py [--steps 40]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import zero_sharded_mixed_step_amd as zs  # noqa: E402

BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32


class Student:
    """Parameters, buffers and both passes of one batch of (B, T) tokens."""

    def __init__(self, B, T, vocab=256, width=128, Hq=4, Hk=2, D=32, blocks=2):
        self.B, self.T, self.V, self.C, self.L = B, T, vocab, width, blocks
        self.Hq, self.Hk, self.D = Hq, Hk, D
        H, N = Hq + 2 * Hk, B * T
        self.shapes = dict(emb=(vocab, width), pre0=(width,))
        for b in range(blocks):
            self.shapes.update({f"proj{b}": (width, H * D), f"wq{b}": (D,), f"wk{b}": (D,),
                                f"out{b}": (Hq * D, width), f"post{b}": (width,),
                                f"gate{b}": (width,), f"pre{b + 1}": (width,)})
        self.n = -(-sum(torch.Size(s).numel() for s in self.shapes.values()) // 32) * 32
        dev = "cuda"

        def new(*shape, dtype=BF):
            return torch.empty(*shape, dtype=dtype, device=dev)

        self.inv_freq = zs.rope_inv_freq(D).to(dev)
        self.pos = torch.arange(T, dtype=I32, device=dev).repeat(B)
        self.scale = width ** 0.5
        self.loss, self.stats = new(N, dtype=F32), new(N, 4, dtype=F32)
        # one workspace for all calls of the stream: they follow one another
        self.ws = torch.empty(max(
            zs.zero_attn_workspace_bytes(B, T, T, Hq, Hk, D),
            zs.zero_attn_workspace_bytes(B, T, T, Hq, Hk, D, backward=True),
            zs.zero_qk_norm_rope_workspace_bytes(N, D), zs.zero_block_norm_workspace_bytes(N, width),
            zs.zero_embed_workspace_bytes(N, width), zs.zero_grads_workspace_bytes()),
            dtype=torch.uint8, device=dev)

    def views(self, flat):
        """The parameters' views of a flat vector."""
        out, at = {}, 0
        for name, shape in self.shapes.items():
            n = torch.Size(shape).numel()
            out[name] = flat[at:at + n].view(shape)
            at += n
        return out

    def initial(self, seed):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        flat = torch.zeros(self.n, dtype=F32, device="cuda")
        for name, p in self.views(flat).items():
            if name == "emb":
                p.copy_(torch.randn(p.shape, generator=g, device="cuda") / self.scale)
            elif p.dim() == 2:
                p.copy_(torch.randn(p.shape, generator=g, device="cuda") * p.shape[0] ** -0.5)
            else:
                p.fill_(0.3 if name.startswith("gate") else 1.0)
        return flat

    def _heads(self, qkv):
        heads = qkv.view(self.B * self.T, self.Hq + 2 * self.Hk, self.D)
        return (heads[:, :self.Hq], heads[:, self.Hq:self.Hq + self.Hk],
                heads[:, self.Hq + self.Hk:].view(self.B, self.T, self.Hk, self.D))

    def forward(self, param, tokens):
        """The logits (B T, V), and what the backward pass needs."""
        B, T, Hq, Hk, D, N = self.B, self.T, self.Hq, self.Hk, self.D, self.B * self.T
        p, ids = self.views(param), tokens.view(-1)
        x = torch.empty(N, self.C, dtype=BF, device="cuda")
        zs.zero_embed_fwd(p["emb"], ids, x, scale=self.scale)
        x = x.float()
        z = torch.empty(N, self.C, dtype=BF, device="cuda")
        zs.zero_block_norm_fwd(x, None, None, z, pre_weight=p["pre0"])
        saved = []
        for b in range(self.L):
            qkv = z @ p[f"proj{b}"]
            q, k, v = self._heads(qkv)
            yq, yk = q.new_empty(q.shape), k.new_empty(k.shape)
            zs.zero_qk_norm_rope_fwd(q, k, yq, yk, wq=p[f"wq{b}"], wk=p[f"wk{b}"], pos=self.pos,
                                     inv_freq=self.inv_freq)
            o = x.new_empty((B, T, Hq, D), dtype=BF)
            lse = x.new_empty((B, Hq, T))
            zs.zero_attn_fwd(yq.view(B, T, Hq, D), yk.view(B, T, Hk, D), v, o, lse, causal=True,
                             workspace=self.ws)
            y = o.view(N, Hq * D) @ p[f"out{b}"]
            h, znext = torch.empty_like(x), torch.empty_like(z)
            zs.zero_block_norm_fwd(x, y, h, znext, **self._norms(p, b))
            saved.append((z, qkv, yq, yk, o, lse, y, h))
            x, z = h, znext
        return z @ p["emb"].t(), (saved, z)

    def _norms(self, p, b):
        return dict(post_norm=True, post_weight=p[f"post{b}"], gate=p[f"gate{b}"],
                    pre_weight=p[f"pre{b + 1}"])

    def backward(self, param, grad, tokens, saved, dlogits):
        """The gradients of all parameters into the flat vector `grad`, from the logits'."""
        B, T, Hq, Hk, D, N = self.B, self.T, self.Hq, self.Hk, self.D, self.B * self.T
        p, g = self.views(param), self.views(grad)
        saved, z = saved
        dz = dlogits @ p["emb"]
        demb = dlogits.t().float() @ z.float()
        dx = None
        for b in reversed(range(self.L)):
            zin, qkv, yq, yk, o, lse, y, h = saved[b]
            dh, dy = torch.empty_like(h), torch.empty_like(y)
            zs.zero_block_norm_bwd(y, h, dx, dz, dh, dy, dpost_weight=g[f"post{b}"],
                                   dgate=g[f"gate{b}"], dpre_weight=g[f"pre{b + 1}"],
                                   workspace=self.ws, **self._norms(p, b))
            att = o.view(N, Hq * D)
            g[f"out{b}"].copy_(att.t() @ dy)
            datt = (dy @ p[f"out{b}"].t()).view(B, T, Hq, D)
            q, k, v = self._heads(qkv)
            dqkv = torch.empty_like(qkv)
            dq, dk, dv = self._heads(dqkv)
            dyq, dyk = torch.empty_like(yq), torch.empty_like(yk)
            zs.zero_attn_bwd(yq.view(B, T, Hq, D), yk.view(B, T, Hk, D), v, o, lse, datt,
                             dyq.view(B, T, Hq, D), dyk.view(B, T, Hk, D), dv, causal=True,
                             workspace=self.ws)
            zs.zero_qk_norm_rope_bwd(q, k, dyq, dyk, dq, dk, wq=p[f"wq{b}"], wk=p[f"wk{b}"],
                                     dwq=g[f"wq{b}"], dwk=g[f"wk{b}"], pos=self.pos,
                                     inv_freq=self.inv_freq, workspace=self.ws)
            g[f"proj{b}"].copy_(zin.t() @ dqkv)
            dz, dx = dqkv @ p[f"proj{b}"].t(), dh
        # the first norm: its input is the embedding itself
        first = torch.empty(N, self.C, dtype=BF, device="cuda")
        zs.zero_embed_fwd(p["emb"], tokens.view(-1), first, scale=self.scale)
        zs.zero_block_norm_bwd(None, first.float(), dx, dz, dx, None, pre_weight=p["pre0"],
                               dpre_weight=g["pre0"], workspace=self.ws)
        # the tied table: the logits' part and the tokens' sums, rounded once
        zs.zero_embed_bwd(tokens.view(-1), dx, g["emb"], scale=self.scale, base=demb,
                          workspace=self.ws)

    def update(self, param, grad, tokens, rollout, kl_coef):
        """The mean loss of a batch, and its gradients into `grad`."""
        logits, saved = self.forward(param, tokens)
        # the loss, and its gradient in place of the logits
        zs.zero_policy_fwd(logits, rollout["action"], rollout["advantage"], self.loss, self.stats,
                           dlogits=logits, old_logp=rollout["old"], ref_logp=rollout["ref"],
                           row_weight=rollout["weight"], kl_coef=kl_coef)
        self.backward(param, grad, tokens, saved, logits)
        return self.loss.sum()


def sample(student, param, ref, tokens, generator):
    """A token at every position, its log probability under the student and under `ref`, and
    its advantage, the reward less its mean."""
    logits, _ = student.forward(param, tokens)
    logp = torch.log_softmax(logits.float(), 1)
    action = torch.multinomial(logp.exp(), 1, generator=generator)
    ref_logp = torch.log_softmax(student.forward(ref, tokens)[0].float(), 1)
    reward = (action[:, 0] % 4 == (tokens.view(-1) + 1) % 4).float()
    n = reward.numel()
    return dict(action=action[:, 0].to(I32), old=logp.gather(1, action)[:, 0],
                ref=ref_logp.gather(1, action)[:, 0],
                advantage=(reward - reward.mean()) / (reward.std() + 1e-3),
                weight=torch.full((n,), 1.0 / n, device="cuda")), float(reward.mean())


def train(steps=40, updates=4, B=8, T=64, log=print, state=None):
    """Rollouts of `updates` updates each; the mean rewards.  `state`, a dict, gets the student, its
    step and the norm of the last gradient."""
    student = Student(B, T)
    step = zs.ShardStep(student.n, 1, BF, lr=2e-2, beta2=0.95)
    step.master.copy_(student.initial(1))
    step.param.copy_(step.master.to(BF).view(torch.int16))
    param = step.param.view(BF)
    ref = param.clone()
    grad = torch.zeros(student.n, dtype=BF, device="cuda")
    replica = torch.zeros(student.n, dtype=BF, device="cuda")
    table = zs.GradTable(student.views(grad).values(), student.views(replica).values())
    acc, norm = zs.new_norm_acc(1), torch.zeros(1, device="cuda")
    g = torch.Generator(device="cuda")
    g.manual_seed(5)
    rewards = []
    for s in range(steps):
        tokens = torch.randint(student.V, (B, T), generator=g, device="cuda").to(I32)
        rollout, reward = sample(student, param, ref, tokens, g)
        for _ in range(updates):
            student.update(param, grad, tokens, rollout, kl_coef=0.01)
            zs.zero_grads_norm(table, acc, workspace=student.ws)
            zs.zero_grads_clip(table, acc, max_norm=1.0, norm_out=norm)
            step.step([replica])
        rewards.append(reward)
        if s % 10 == 0 or s == steps - 1:
            log("step %3d  reward %.4f  gradient norm %.4f" % (s, reward, float(norm)))
    if state is not None:
        state.update(student=student, step=step, norm=norm)
    return rewards


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--steps", type=int, default=40)
    train(ap.parse_args().steps)
