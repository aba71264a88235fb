"""A small student trained on a teacher's top entries: the operators and the
optimizer step together, as a training program uses them.

The student is one attention block over a tied embedding.  Its parameters are
one flat bf16 vector (the step's `param`) and its gradients one flat bf16
replica a micro-batch, with the matrices as views of both; every gradient is
written where the step reads it.  Rows hold packed documents and padding; the
forward of a micro-batch is

  embedding -> projection -> zero_qk_norm_rope -> zero_attn (documents' ranges,
  distance bias) -> projection + residual -> logits -> zero_distill

with the loss's gradient from the same pass over the logits, and the backward runs
the operators' backward calls in reverse.  Plain matrix products are torch's.

  python examples/distill_student.py [--steps 40]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import zero_sharded_mixed_step_amd as zs  # noqa: E402

BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32


class Student:
    """Parameters, buffers and both passes of one micro-batch of (B, T) tokens."""

    def __init__(self, B, T, vocab=512, width=128, Hq=4, Hk=2, D=64, K=8, buckets=16, reach=64):
        self.B, self.T, self.V, self.C = B, T, vocab, width
        self.Hq, self.Hk, self.D, self.K = Hq, Hk, D, K
        H = Hq + 2 * Hk
        self.shapes = dict(emb=(vocab, width), proj=(width, H * D), wq=(D,), wk=(D,),
                           bias=(buckets, Hq), out=(Hq * D, width))
        self.n = -(-sum(torch.Size(s).numel() for s in self.shapes.values()) // 32) * 32
        dev, N = "cuda", B * T

        def new(*shape, dtype=BF):
            return torch.empty(*shape, dtype=dtype, device=dev)

        self.inv_freq = zs.rope_inv_freq(D).to(dev)
        self.buckets = zs.relpos_buckets(buckets, reach, device=dev)
        self.yq, self.yk = new(N, Hq, D), new(N, Hk, D)
        self.o, self.lse = new(B, T, Hq, D), new(B, Hq, T, dtype=F32)
        self.ranges = new(B, T, 2, dtype=I32)
        self.loss, self.stats = new(N, dtype=F32), new(N, 2, dtype=F32)
        self.dqkv, self.dyq, self.dyk = new(N, H * D), new(N, Hq, D), new(N, Hk, D)
        # one workspace for all calls of the stream: they follow one another
        self.ws = torch.empty(max(
            zs.zero_attn_workspace_bytes(B, T, T, Hq, Hk, D, buckets),
            zs.zero_attn_workspace_bytes(B, T, T, Hq, Hk, D, buckets, backward=True),
            zs.zero_qk_norm_rope_workspace_bytes(N, D)), dtype=torch.uint8, device=dev)

    def views(self, flat):
        """The parameters' views of a flat bf16 vector."""
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
        v = self.views(flat)
        for name, scale in (("emb", 0.5), ("proj", self.C ** -0.5),
                            ("out", (self.Hq * self.D) ** -0.5)):
            v[name].copy_(torch.randn(v[name].shape, generator=g, device="cuda") * scale)
        v["wq"].fill_(1.0)
        v["wk"].fill_(1.0)
        return flat

    def run(self, param, grad, tokens, doc, pos, teacher_idx, teacher_val, teacher_lse, weight):
        """One micro-batch: the mean loss, and the gradients into the flat
        vector `grad`.  tokens, doc (negative: padding) and pos are (B, T) int32, the
        teacher's entries (B T, K), its logsumexp and the rows' weights (B T)."""
        B, T, Hq, Hk, D = self.B, self.T, self.Hq, self.Hk, self.D
        p, g = self.views(param), self.views(grad)
        ids, N = tokens.view(-1).long(), B * T
        pos = pos.view(-1)

        # forward
        x = p["emb"][ids]
        qkv = x @ p["proj"]
        heads = qkv.view(N, Hq + 2 * Hk, D)
        q, k = heads[:, :Hq], heads[:, Hq:Hq + Hk]
        v = heads[:, Hq + Hk:].view(B, T, Hk, D)
        turn = dict(wq=p["wq"], wk=p["wk"], pos=pos, inv_freq=self.inv_freq)
        zs.zero_qk_norm_rope_fwd(q, k, self.yq, self.yk, **turn)
        zs.zero_attn_ranges(doc, self.ranges)
        yq, yk = self.yq.view(B, T, Hq, D), self.yk.view(B, T, Hk, D)
        mask = dict(ranges=self.ranges, bias_table=p["bias"], bias_buckets=self.buckets,
                    workspace=self.ws)
        zs.zero_attn_fwd(yq, yk, v, self.o, self.lse, **mask)
        att = self.o.view(N, Hq * D)
        h = x + att @ p["out"]
        logits = h @ p["emb"].t()
        # the loss, and its gradient in place of the logits
        zs.zero_distill_fwd(logits, teacher_idx, teacher_val, self.loss, self.stats,
                            dlogits=logits, temperature=2.0, teacher_lse=teacher_lse,
                            row_weight=weight)
        # backward
        dh = logits @ p["emb"]
        torch.mm(att.t(), dh, out=g["out"])
        datt = (dh @ p["out"].t()).view(B, T, Hq, D)
        dheads = self.dqkv.view(N, Hq + 2 * Hk, D)
        dv = dheads[:, Hq + Hk:].view(B, T, Hk, D)
        dyq, dyk = self.dyq.view(B, T, Hq, D), self.dyk.view(B, T, Hk, D)
        zs.zero_attn_bwd(yq, yk, v, self.o, self.lse, datt, dyq, dyk, dv, dbias_table=g["bias"],
                         **mask)
        zs.zero_qk_norm_rope_bwd(q, k, self.dyq, self.dyk, dheads[:, :Hq], dheads[:, Hq:Hq + Hk],
                                 dwq=g["wq"], dwk=g["wk"], workspace=self.ws, **turn)
        torch.mm(x.t(), self.dqkv, out=g["proj"])
        dx = (dh + self.dqkv @ p["proj"].t()).float()
        demb = logits.t().float() @ h.float()
        # (the rows of one token in a fixed order: sorted, and summed by a matrix product)
        one_hot = torch.nn.functional.one_hot(ids, self.V).to(F32)
        g["emb"].copy_(demb + one_hot.t() @ dx)
        return self.loss.sum()


def batch(student, seed):
    """Tokens in packed documents with padding at the end, and the teacher: the
    K likeliest next tokens by a fixed random table, of all of the vocabulary's."""
    B, T, V, K = student.B, student.T, student.V, student.K
    g = torch.Generator()
    g.manual_seed(seed)
    tokens = torch.randint(V, (B, T), generator=g)
    doc, pos = torch.full((B, T), -1, dtype=I32), torch.zeros(B, T, dtype=I32)
    for b in range(B):
        room = T - 3 - b                               # (the rest is padding)
        cut = int(torch.randint(1, room, (1,), generator=g))
        doc[b, :cut], doc[b, cut:room] = 0, 1
        pos[b, :cut] = torch.arange(cut, dtype=I32)
        pos[b, cut:room] = torch.arange(room - cut, dtype=I32)
    table = torch.Generator()
    table.manual_seed(7)
    teacher = (torch.randn(V, V, generator=table) * 4).to(BF).float()[tokens.view(-1)]
    val, idx = teacher.topk(K, dim=1)
    lse = torch.logsumexp(teacher / 2.0, dim=1)        # at the loss's temperature
    real = (doc >= 0).view(-1).float()
    return dict(tokens=tokens.to(I32).cuda(), doc=doc.cuda(), pos=pos.cuda(),
                teacher_idx=idx.to(I32).cuda(), teacher_val=val.to(BF).cuda(),
                teacher_lse=lse.cuda(), weight=(real / real.sum()).cuda())


def train(steps=40, B=2, T=96, log=print):
    """Two micro-batches a step, reduced as two replicas; the mean losses."""
    student = Student(B, T)
    step = zs.ShardStep(student.n, 2, BF, lr=1e-2, max_norm=1.0, check_overflow=True)
    step.master.copy_(student.initial(1))
    step.param.copy_(step.master.to(BF).view(torch.int16))
    param = step.param.view(BF)
    replicas = [torch.zeros(student.n, dtype=BF, device="cuda") for _ in range(2)]
    batches = [batch(student, 10 + r) for r in range(2)]
    losses = []
    for s in range(steps):
        loss = sum(student.run(param, replicas[r], **batches[r]) for r in range(2)) / 2
        step.step(replicas)
        losses.append(float(loss))
        if s % 10 == 0 or s == steps - 1:
            log("step %3d  loss %.4f" % (s, losses[-1]))
    return losses


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--steps", type=int, default=40)
    train(ap.parse_args().steps)
