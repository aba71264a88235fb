"""Workloads of the student-training operators: the attention with a tanh cap,
a learned distance bias and document/prefix masks, the per-head norm of
queries and keys with the position rotation, and the distillation loss from a
teacher's top logits.

Each case is one call a training program makes.  `run` computes it either with
elementary torch operations (`own` false) or through this package's entry
points (`own` true); `exact` computes it from the definition in 64 bits.
"""
import math
import random

import numpy as np
import torch

own = False

# Bucket count and reach of the learned distance bias: 32 buckets that
# saturate at distance 128 are the usual setting of such a table.
BUCKETS, REACH = 32, 128


# --------------------------------------------------------------- the cases ---

def listed():
    return [
        # One new token per sequence against the keys so far: what sampling
        # from the student between updates costs.  Latency counts.
        dict(name="attn-fwd-one-token", op="attn", pass_="fwd", B=4, Tq=1, Tk=5003, Hq=12, Hk=12,
             D=64, cap=0.0, bias=True, mode="causal", docs=0, pad=0),
        # A micro-batch of a GPT-2-small-sized student (12 heads of 64, 1024
        # tokens), several packed documents a row, distance bias.
        dict(name="attn-fwd-1k-bias", op="attn", pass_="fwd", B=8, Tq=1024, Tk=1024, Hq=12, Hk=12,
             D=64, cap=0.0, bias=True, mode="docs", docs=3, pad=9),
        dict(name="attn-bwd-1k-bias", op="attn", pass_="bwd", B=8, Tq=1024, Tk=1024, Hq=12, Hk=12,
             D=64, cap=0.0, bias=True, mode="docs", docs=3, pad=9),
        # A long row of a larger student: 32 query heads on 8 key heads of
        # 128, capped scores, documents that each open with a prefix.
        dict(name="attn-fwd-4k-cap", op="attn", pass_="fwd", B=1, Tq=4096, Tk=4096, Hq=32, Hk=8,
             D=128, cap=30.0, bias=False, mode="prefix", docs=2, pad=0),
        # The same in training, at a length that ends inside a tile.
        dict(name="attn-bwd-4k-cap", op="attn", pass_="bwd", B=1, Tq=4001, Tk=4001, Hq=32, Hk=8,
             D=128, cap=30.0, bias=False, mode="prefix", docs=2, pad=5),
        # Norm and rotation of a short row (latency) and of 16k tokens, both
        # from one fused projection's output.
        dict(name="norm-fwd-64", op="norm", pass_="fwd", T=64, Hq=12, Hk=12, D=64, rd=64,
             inter=False, dtype="bf16", far=0),
        dict(name="norm-fwd-16k", op="norm", pass_="fwd", T=16384, Hq=32, Hk=8, D=128, rd=128,
             inter=False, dtype="bf16", far=1_000_000),
        dict(name="norm-bwd-8k", op="norm", pass_="bwd", T=8192, Hq=32, Hk=8, D=128, rd=128,
             inter=False, dtype="bf16", far=0),
        # fp32 activations, half of each head rotated, neighbouring pairs.
        dict(name="norm-bwd-4k-f32", op="norm", pass_="bwd", T=4097, Hq=12, Hk=3, D=96, rd=48,
             inter=True, dtype="f32", far=0),
        # The loss of one short sequence with its gradient, and of a
        # micro-batch of 8k tokens, at GPT-2's vocabulary (odd: rows start
        # misaligned).
        dict(name="distill-61", op="distill", pass_="both", N=61, V=50257, K=16, tau=2.0,
             tail=False, dtype="bf16"),
        dict(name="distill-8k", op="distill", pass_="both", N=8192, V=50257, K=64, tau=1.5,
             tail=True, dtype="bf16"),
        # The gradient alone, from the saved row statistics (forward and
        # backward as two calls), of a large vocabulary in fp32.
        dict(name="distill-bwd-131k-f32", op="distill", pass_="bwd", N=1024, V=131072, K=32,
             tau=1.0, tail=True, dtype="f32"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["attn", "attn", "norm", "distill"])
    if op == "attn":
        D = rng.choice([32, 64, 96, 128])
        Hk = rng.choice([1, 2, 4, 8, 12])
        Hq = Hk * rng.choice([1, 1, 2, 4])
        Tk = _log_int(rng, 24, 4096)
        one = rng.random() < 0.2
        Tq = rng.randint(1, min(8, Tk)) if one else Tk
        # at most the largest listed case's scores (32 heads, 4096 x 4096)
        B = _log_int(rng, 1, 16)
        # at most as many scores as the largest listed case sees
        while B * Hq * Tq * Tk > 8 * 4096 * 4096:
            if B > 1:
                B //= 2
            else:
                Tk = Tk * 3 // 4
                Tq = Tq if one else Tk
        bias = rng.random() < 0.5
        mode = "causal" if one else rng.choice(["full", "causal", "docs", "prefix"])
        docs = _log_int(rng, 1, max(1, min(16, Tk // 16))) if mode in ("docs", "prefix") else 0
        pad = rng.randint(0, min(40, Tk // 4)) if mode in ("docs", "prefix") else 0
        return dict(op="attn", pass_="fwd" if one else rng.choice(["fwd", "bwd"]), B=B, Tq=Tq,
                    Tk=Tk, Hq=Hq, Hk=Hk, D=D, cap=rng.choice([0.0, 0.0, 20.0, 30.0, 50.0]),
                    bias=bias, mode=mode, docs=docs, pad=pad)
    if op == "norm":
        D = rng.choice([32, 64, 96, 128, 192, 256])
        Hk = rng.choice([1, 2, 3, 4, 8, 16])
        Hq = Hk * rng.choice([1, 2, 4])
        T = _log_int(rng, 1, max(1, min(16384, 16384 * 40 * 128 // ((Hq + Hk) * D * 2))))
        return dict(op="norm", pass_=rng.choice(["fwd", "bwd"]), T=T, Hq=Hq, Hk=Hk, D=D,
                    rd=rng.choice([D, D, D // 2]), inter=rng.random() < 0.5,
                    dtype=rng.choice(["bf16", "bf16", "f32"]), far=rng.choice([0, 0, 1_000_000]))
    V = _log_int(rng, 500, 200_000)
    N = _log_int(rng, 1, max(1, min(8192, 8192 * 50257 // (2 * V))))
    return dict(op="distill", pass_=rng.choice(["fwd", "bwd", "both"]), N=N, V=V,
                K=_log_int(rng, 1, min(256, V)), tau=rng.choice([1.0, 1.5, 2.0, 4.0]),
                tail=rng.random() < 0.5, dtype=rng.choice(["bf16", "bf16", "f32"]))


# ------------------------------------------------- masks and position ids ---

def _documents(case):
    """(doc, start, end, prefix) per token, (B, T) int64 arrays on the host: a
    row holds `docs` documents of unlike lengths and `pad` padding tokens
    (doc -1).  A function of the case alone."""
    B, T, n, pad = case["B"], case["Tk"], max(1, case["docs"]), case["pad"]
    rng = random.Random(T * 1009 + n * 31 + B)
    doc = np.full((B, T), -1, np.int64)
    start, end, prefix = (np.zeros((B, T), np.int64) for _ in range(3))
    for b in range(B):
        room = T - pad
        cuts = sorted(rng.sample(range(1, room), min(n, room) - 1)) if room > 1 else []
        for d, (lo, hi) in enumerate(zip([0] + cuts, cuts + [room])):
            doc[b, lo:hi], start[b, lo:hi], end[b, lo:hi] = d, lo, hi
            prefix[b, lo:hi] = rng.randint(0, (hi - lo) // 2)
    return doc, start, end, prefix


def _ranges(case):
    """The keys [lo, hi) that each query sees, (B, Tq, 2) int64 on the host."""
    B, Tq, Tk, mode = case["B"], case["Tq"], case["Tk"], case["mode"]
    r = np.zeros((B, Tq, 2), np.int64)
    if mode == "full":
        r[..., 1] = Tk
    elif mode == "causal":
        r[..., 1] = np.arange(Tq) + 1 + Tk - Tq
    else:
        doc, start, end, prefix = _documents(case)
        hi = np.maximum(np.arange(Tk) + 1, start + prefix) if mode == "prefix" \
            else np.broadcast_to(np.arange(Tk) + 1, doc.shape)
        r[..., 0] = np.where(doc < 0, 0, start)
        r[..., 1] = np.where(doc < 0, 0, np.minimum(hi, end))
    return r


def _bucket_map():
    """Bucket of each key-minus-query distance in [-REACH, REACH], one-sided:
    one bucket for each of the nearest 16 distances behind the query, then 16
    that widen geometrically up to REACH; keys ahead share bucket 0."""
    half, out = BUCKETS // 2, []
    for rel in range(-REACH, REACH + 1):
        back = max(0, -rel)
        b = back
        if back >= half:
            steps = BUCKETS - half
            t = max(t for t in range(steps + 1)
                    if back ** steps >= half ** (steps - t) * REACH ** t)
            b = min(BUCKETS - 1, half + t)
        out.append(b)
    return np.array(out, np.int32)


# ------------------------------------------------------------------ inputs ---

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _normal(g, shape, dtype, scale=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)


def prepare(case, seed):
    g = _gen(seed)
    return {"attn": _prepare_attn, "norm": _prepare_norm,
            "distill": _prepare_distill}[case["op"]](case, g)


def _prepare_attn(case, g):
    B, Tq, Tk, Hq, Hk, D = (case[k] for k in ("B", "Tq", "Tk", "Hq", "Hk", "D"))
    bf = torch.bfloat16
    s = dict(case=case, scale=1.0 / math.sqrt(D), q=_normal(g, (B, Tq, Hq, D), bf, 3.0),
             k=_normal(g, (B, Tk, Hk, D), bf), v=_normal(g, (B, Tk, Hk, D), bf))
    # the mask as the path takes it: the range of keys that each query sees,
    # made once for a batch and used by every layer
    s["ranges"] = torch.from_numpy(_ranges(case).astype(np.int32)).cuda() \
        if case["mode"] in ("docs", "prefix") else None
    s["table"] = _normal(g, (BUCKETS, Hq), bf) if case["bias"] else None
    s["buckets"] = torch.from_numpy(_bucket_map()).cuda() if case["bias"] else None
    s["o"] = torch.empty((B, Tq, Hq, D), dtype=bf, device="cuda")
    s["lse"] = torch.empty((B, Hq, Tq), dtype=torch.float32, device="cuda")
    if case["pass_"] == "bwd":
        # what the forward pass of the same step left, and the gradient that
        # comes in
        o, lse = _attn_fwd_plain(s)
        s["o"].copy_(o)
        s["lse"].copy_(lse)
        s["do"] = _normal(g, (B, Tq, Hq, D), bf)
        for n, x in (("dq", "q"), ("dk", "k"), ("dv", "v"), ("dtable", "table")):
            s[n] = None if s[x] is None else torch.empty_like(s[x])
    # a row's statistics, a tile's share of the bias gradient, the parts of
    # rows whose keys are split, and each query head's share of its key head's
    # gradients
    s["ws"] = _workspace(4 * (B * Hq * Tq * 2 + B * Hq * (Tq // 32 + 1) * (BUCKETS + 4)
                              + B * (Tq + Tk + 64) + 1024 * 128 * (D + 2)
                              + (2 * B * Hq * Tk * D if case["pass_"] == "bwd" else 0)))
    return s


def _workspace(nbytes):
    """Scratch memory that a program keeps from step to step."""
    return torch.empty(nbytes + 4096, dtype=torch.uint8, device="cuda")


def _prepare_norm(case, g):
    T, Hq, Hk, D, rd = (case[k] for k in ("T", "Hq", "Hk", "D", "rd"))
    dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
    qkv = _normal(g, (T, (Hq + 2 * Hk) * D), dt, 1.7)      # one projection's output
    s = dict(case=case, q=qkv[:, :Hq * D].view(T, Hq, D),
             k=qkv[:, Hq * D:(Hq + Hk) * D].view(T, Hk, D),
             wq=_normal(g, (D,), torch.float32, 0.1).add_(1).to(dt),
             wk=_normal(g, (D,), torch.float32, 0.1).add_(1).to(dt), eps=1e-6,
             pos=torch.arange(T, device="cuda", dtype=torch.int32) + case["far"],
             inv_freq=torch.from_numpy(10000.0 ** (-np.arange(0, rd, 2) / rd)).cuda())
    if case["pass_"] == "fwd":
        s["yq"], s["yk"] = (torch.empty((T, h, D), dtype=dt, device="cuda") for h in (Hq, Hk))
    else:
        s["dyq"], s["dyk"] = (_normal(g, (T, h, D), dt) for h in (Hq, Hk))
        dqkv = torch.empty_like(qkv)
        s["dq"] = dqkv[:, :Hq * D].view(T, Hq, D)
        s["dk"] = dqkv[:, Hq * D:(Hq + Hk) * D].view(T, Hk, D)
        s["dwq"], s["dwk"] = torch.empty_like(s["wq"]), torch.empty_like(s["wk"])
        s["ws"] = _workspace(4 * 2 * D * 1024)
    return s


def _prepare_distill(case, g):
    N, V, K = case["N"], case["V"], case["K"]
    dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
    z = torch.randn((N, V), generator=g, device="cuda").mul_(2.0)
    # the teacher's logits: the student's with noise, of which it keeps the K
    # largest, and the log of its whole sum of exponentials
    t = torch.randn((N, V), generator=g, device="cuda").mul_(1.5).add_(z)
    val, idx = torch.topk(t, K, dim=1)
    tl = _logsumexp(t / case["tau"])
    s = dict(case=case, z=z.to(dt), idx=idx.to(torch.int32), val=val.to(dt),
             tlse=tl if case["tail"] else None)
    del t, z
    # a tenth of the rows carries no loss (prompt and padding tokens)
    s["w"] = (torch.rand(N, generator=g, device="cuda") > 0.1).float()
    s["gscale"] = 1.0 / N
    s["loss"] = torch.empty(N, dtype=torch.float32, device="cuda")
    s["stats"] = torch.empty((N, 2), dtype=torch.float32, device="cuda")
    if case["pass_"] != "fwd":
        s["dz"] = torch.empty_like(s["z"])
    if case["pass_"] == "bwd":
        lse, c = _distill_stats_plain(s)
        s["stats"].copy_(torch.stack([lse, c], 1))
    return s


# ------------------------------------------------------------- plain forms ---

def run(s):
    if own:
        return _run_own(s)
    case = s["case"]
    if case["op"] == "attn":
        return _attn_fwd_plain(s) if case["pass_"] == "fwd" else _attn_bwd_plain(s)
    if case["op"] == "norm":
        return _norm_fwd_plain(s) if case["pass_"] == "fwd" else _norm_bwd_plain(s)
    return _distill_plain(s)


def _heads(x, Hq):
    """(B, T, H, D) as fp32 (B, Hq, T, D), key heads repeated over their group."""
    x = x.float().permute(0, 2, 1, 3)
    return x.repeat_interleave(Hq // x.shape[1], dim=1)


def _distance_index(s):
    case = s["case"]
    i = torch.arange(case["Tq"], device="cuda") + case["Tk"] - case["Tq"]
    d = torch.arange(case["Tk"], device="cuda")[None, :] - i[:, None]
    return s["buckets"].long()[d.clamp(-REACH, REACH) + REACH]


def _scores_plain(s):
    """Scores (masked ones -inf), the tanh's value where there is a cap, and
    the heads' q and k."""
    case = s["case"]
    q, k = _heads(s["q"], case["Hq"]), _heads(s["k"], case["Hq"])
    x = torch.matmul(q, k.transpose(2, 3)).mul_(s["scale"])
    t = None
    if case["cap"]:
        t = x.div_(case["cap"]).tanh_()
        x = t * case["cap"]
    if case["bias"]:
        x = x + s["table"].float()[_distance_index(s)].permute(2, 0, 1)
    j = torch.arange(case["Tk"], device="cuda")
    if s["ranges"] is not None:
        seen = (j >= s["ranges"][:, None, :, :1]) & (j < s["ranges"][:, None, :, 1:])
        x = x.masked_fill(~seen, -math.inf)
    elif case["mode"] == "causal":
        last = torch.arange(case["Tq"], device="cuda") + case["Tk"] - case["Tq"]
        x = x.masked_fill(j[None, :] > last[:, None], -math.inf)
    return x, t, q, k


def _attn_fwd_plain(s):
    case = s["case"]
    x = _scores_plain(s)[0]
    m = x.amax(3, keepdim=True)
    m = torch.where(torch.isinf(m), torch.zeros_like(m), m)
    p = x.sub_(m).exp_()
    total = p.sum(3, keepdim=True)
    lse = (m + total.log())[..., 0]
    o = torch.matmul(p, _heads(s["v"], case["Hq"]))
    o = torch.where(total > 0, o / total, torch.zeros_like(o))
    return o.permute(0, 2, 1, 3).to(torch.bfloat16), lse


def _group_sum(x, Hk):
    """Gradients of shared heads: (B, Hq, T, D) summed to (B, T, Hk, D)."""
    B, Hq, T, D = x.shape
    return x.view(B, Hk, Hq // Hk, T, D).sum(2).permute(0, 2, 1, 3).to(torch.bfloat16)


def _dtable_plain(s, ds):
    """Sums of ds over each bucket: rows padded and flattened so that equal
    distances share a column, summed over the rows, then by bucket."""
    Tq, Tk, Hq = (s["case"][n] for n in ("Tq", "Tk", "Hq"))
    width = Tq + Tk
    d = torch.nn.functional.pad(ds.double().sum(0).flip(1), (0, Tq)).view(Hq, -1)
    d = d[:, :Tq * (width - 1)].view(Hq, Tq, width - 1).sum(1)
    dist = torch.arange(width - 1, device="cuda") - (Tq - 1) - (Tk - Tq)
    at = s["buckets"].long()[dist.clamp(-REACH, REACH) + REACH]
    member = (at[:, None] == torch.arange(BUCKETS, device="cuda")).double()
    return torch.matmul(member.t(), d.t()).to(s["table"].dtype)


def _attn_bwd_plain(s):
    case = s["case"]
    x, t, q, k = _scores_plain(s)
    lse = s["lse"][..., None]
    p = x.sub_(torch.where(torch.isinf(lse), torch.zeros_like(lse), lse)).exp_()
    do = _heads(s["do"], case["Hq"])
    delta = (do * _heads(s["o"], case["Hq"])).sum(3, keepdim=True)
    dv = torch.matmul(p.transpose(2, 3), do)
    ds = torch.matmul(do, _heads(s["v"], case["Hq"]).transpose(2, 3)).sub_(delta).mul_(p)
    dtable = None
    if case["bias"]:
        dtable = _dtable_plain(s, ds)
    if t is not None:
        ds = ds.mul_(t.mul_(t).neg_().add_(1))
    ds = ds.mul_(s["scale"])
    dq = torch.matmul(ds, k).permute(0, 2, 1, 3).to(torch.bfloat16)
    dk = _group_sum(torch.matmul(ds.transpose(2, 3), q), case["Hk"])
    out = {"dq": dq, "dk": dk, "dv": _group_sum(dv, case["Hk"])}
    if dtable is not None:
        out["dtable"] = dtable
    return out


def _angles_plain(s):
    a = s["pos"].double()[:, None, None] * s["inv_freq"]
    return a.cos().float(), a.sin().float()


def _pairs(x, case):
    """The two members of each rotated pair, and what is left unrotated."""
    rd = case["rd"]
    r, rest = x[..., :rd], x[..., rd:]
    if case["inter"]:
        return r[..., 0::2], r[..., 1::2], rest
    return r[..., :rd // 2], r[..., rd // 2:], rest


def _join(a, b, rest, case):
    r = torch.stack([a, b], -1).flatten(-2) if case["inter"] else torch.cat([a, b], -1)
    return torch.cat([r, rest], -1)


def _norm_fwd_plain(s):
    cos, sin = _angles_plain(s)

    def one(x, w):
        f = x.float()
        f = f * (f.square().mean(-1, keepdim=True) + s["eps"]).rsqrt() * w.float()
        a, b, rest = _pairs(f, s["case"])
        return _join(a * cos - b * sin, b * cos + a * sin, rest, s["case"]).to(x.dtype)

    return {"yq": one(s["q"], s["wq"]), "yk": one(s["k"], s["wk"])}


def _norm_bwd_plain(s):
    cos, sin = _angles_plain(s)

    def one(x, w, dy):
        f = x.float()
        r = (f.square().mean(-1, keepdim=True) + s["eps"]).rsqrt()
        f = f * r
        a, b, rest = _pairs(dy.float(), s["case"])
        gn = _join(a * cos + b * sin, b * cos - a * sin, rest, s["case"])
        dw = (gn * f).double().sum((0, 1))
        gn = gn * w.float()
        dx = (gn - f * (gn * f).mean(-1, keepdim=True)) * r
        return dx.to(x.dtype), dw.to(w.dtype)

    dq, dwq = one(s["q"], s["wq"], s["dyq"])
    dk, dwk = one(s["k"], s["wk"], s["dyk"])
    return {"dq": dq, "dk": dk, "dwq": dwq, "dwk": dwk}


def _logsumexp(x):
    m = x.amax(1)
    return m + (x - m[:, None]).exp().double().sum(1).log().float()


def _teacher_plain(s):
    """The teacher's probabilities of its K entries (64 bits: the mass of the
    tail is what is left of 1) and the mass of the tail."""
    t = s["val"].double() / s["case"]["tau"]
    if s["tlse"] is not None:
        p = (t - s["tlse"].double()[:, None]).exp()
        return p, (1 - p.sum(1)).clamp_min(0)
    e = (t - t.amax(1, keepdim=True)).exp()
    return e / e.sum(1, keepdim=True), None


def _distill_stats_plain(s):
    """Log of the row's sum of exponentials, and the factor of the student's
    probabilities in the gradient outside the teacher's entries."""
    x = s["z"].float() / s["case"]["tau"]
    lse = _logsumexp(x)
    if s["tlse"] is None:
        return lse, torch.ones_like(lse)
    rest = _logsumexp(x.scatter_(1, s["idx"].long(), -math.inf))
    tail = _teacher_plain(s)[1]
    return lse, (1 - tail * (lse.double() - rest.double()).exp()).float()


def _distill_plain(s):
    case, tau, out = s["case"], s["case"]["tau"], {}
    idx = s["idx"].long()
    p, tail = _teacher_plain(s)
    if case["pass_"] == "bwd":
        lse, c = s["stats"][:, 0], s["stats"][:, 1]
    else:
        x = s["z"].float() / tau
        m = x.amax(1)
        e = x.sub_(m[:, None]).exp_()
        zt = (s["z"].gather(1, idx).float() / tau).double()
        top = e.gather(1, idx)
        lse = m.double() + e.double().sum(1).log()
        loss = (p * (p.log() - zt + lse[:, None])).nan_to_num(nan=0.0).sum(1)
        c = torch.ones_like(m)
        if tail is not None:
            rest = m.double() + e.scatter_(1, idx, 0.0).double().sum(1).log()
            loss = loss + torch.where(tail > 0, tail * (tail.log() - rest + lse), 0.0)
            c = (1 - tail * (lse - rest).exp()).float()
            e.scatter_(1, idx, top)
        out["loss"] = (loss * tau * tau * s["w"].double()).float()
        out["stats"] = torch.stack([lse.float(), c], 1)
        if case["pass_"] == "fwd":
            return out
        lse = lse.float()
        del x, e
    q = (s["z"].float() / tau).sub_(lse[:, None]).exp_()
    qt = q.gather(1, idx)
    d = q.mul_(c[:, None]).scatter_(1, idx, qt - p.float())
    out["dz"] = d.mul_((s["w"] * (tau * s["gscale"]))[:, None]).to(s["z"].dtype)
    return out


# ------------------------------------------------------ through the package ---

def _run_own(s):
    import zero_sharded_mixed_step_amd as zs
    case = s["case"]
    if case["op"] == "attn":
        kw = dict(scale=s["scale"], cap=case["cap"], ranges=s["ranges"],
                  causal=case["mode"] == "causal", bias_table=s["table"],
                  bias_buckets=s["buckets"], workspace=s["ws"])
        if case["pass_"] == "fwd":
            zs.zero_attn_fwd(s["q"], s["k"], s["v"], s["o"], s["lse"], **kw)
            return s["o"], s["lse"]
        zs.zero_attn_bwd(s["q"], s["k"], s["v"], s["o"], s["lse"], s["do"], s["dq"], s["dk"],
                         s["dv"], dbias_table=s["dtable"], **kw)
        return {n: s[n] for n in ("dq", "dk", "dv", "dtable") if s[n] is not None}
    if case["op"] == "norm":
        kw = dict(wq=s["wq"], wk=s["wk"], eps=s["eps"], pos=s["pos"], inv_freq=s["inv_freq"],
                  interleaved=case["inter"])
        if case["pass_"] == "fwd":
            zs.zero_qk_norm_rope_fwd(s["q"], s["k"], s["yq"], s["yk"], **kw)
            return {n: s[n] for n in ("yq", "yk")}
        zs.zero_qk_norm_rope_bwd(s["q"], s["k"], s["dyq"], s["dyk"], s["dq"], s["dk"],
                                 dwq=s["dwq"], dwk=s["dwk"], workspace=s["ws"], **kw)
        return {n: s[n] for n in ("dq", "dk", "dwq", "dwk")}
    kw = dict(temperature=case["tau"], teacher_lse=s["tlse"], row_weight=s["w"],
              grad_scale=s["gscale"])
    if case["pass_"] == "bwd":
        zs.zero_distill_bwd(s["z"], s["idx"], s["val"], s["stats"], s["dz"], **kw)
        return {"dz": s["dz"]}
    zs.zero_distill_fwd(s["z"], s["idx"], s["val"], s["loss"], s["stats"],
                        dlogits=s.get("dz"), **kw)
    return {n: s[n] for n in ("loss", "stats", "dz") if n in s}


# -------------------------------------------------------------------- work ---

def work(case):
    if case["op"] == "attn":
        B, Tq, Tk, Hq, Hk, D = (case[k] for k in ("B", "Tq", "Tk", "Hq", "Hk", "D"))
        r = _ranges(case)
        pairs = float(np.maximum(r[..., 1] - r[..., 0], 0).sum()) * Hq
        rows = 2 * B * Tq * Hq * D                                 # one of q, o, do, dq
        cols = 2 * B * Tk * Hk * D                                 # one of k, v, dk, dv
        extra = 4 * B * Hq * Tq + (8 * B * Tq if case["docs"] else 0)
        if case["bias"]:
            extra += 2 * BUCKETS * Hq
        if case["pass_"] == "fwd":
            return {"bytes": 2 * rows + 2 * cols + extra, "flops": 4.0 * D * pairs}
        return {"bytes": 4 * rows + 4 * cols + extra, "flops": 10.0 * D * pairs}
    if case["op"] == "norm":
        n = case["T"] * (case["Hq"] + case["Hk"]) * case["D"]
        b = 2 if case["dtype"] == "bf16" else 4
        k = 2 if case["pass_"] == "fwd" else 3
        return {"bytes": k * n * b + 4 * case["T"] + 4 * case["rd"], "flops": 6.0 * k * n}
    N, V, K = case["N"], case["V"], case["K"]
    b = 2 if case["dtype"] == "bf16" else 4
    k = 1 if case["pass_"] == "fwd" else 2
    return {"bytes": k * N * V * b + N * K * (4 + b) + 20 * N, "flops": 4.0 * k * N * V}


# ------------------------------------------------------- the 64-bit answer ---

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "attn":
        return _attn_exact(case, s)
    if case["op"] == "norm":
        return _norm_exact(case, s)
    return _distill_exact(case, s)


def _attn_exact(case, s):
    B, Tq, Tk, Hq, Hk = (case[k] for k in ("B", "Tq", "Tk", "Hq", "Hk"))
    dev = "cuda"
    i = torch.arange(Tq, device=dev) + (Tk - Tq)
    j = torch.arange(Tk, device=dev)
    seen = torch.ones((B, Tq, Tk), dtype=torch.bool, device=dev)
    if case["mode"] == "causal":
        seen &= j[None, :] <= i[:, None]
    elif case["mode"] in ("docs", "prefix"):
        doc, start, _, prefix = (torch.from_numpy(a).to(dev) for a in _documents(case))
        same = (doc[:, :, None] == doc[:, None, :]) & (doc >= 0)[:, :, None]
        back = (j[None, :] <= i[:, None])[None]
        if case["mode"] == "prefix":
            back = back | (j < (start + prefix)[:, :, None])
        seen = same & back
    dist = (j[None, :] - i[:, None]).clamp(-REACH, REACH) + REACH
    bucket = s["buckets"].long()[dist] if case["bias"] else None
    bwd = case["pass_"] == "bwd"
    o = torch.zeros((B, Tq, Hq, case["D"]), dtype=torch.float64, device=dev)
    lse = torch.zeros((B, Hq, Tq), dtype=torch.float64, device=dev)
    if bwd:
        dq, dk, dv = (torch.zeros(s[n].shape, dtype=torch.float64, device=dev)
                      for n in ("q", "k", "v"))
        dtab = torch.zeros((BUCKETS, Hq), dtype=torch.float64, device=dev)
    for b in range(B):
        for h in range(Hq):
            kh = h // (Hq // Hk)
            q, k, v = s["q"][b, :, h].double(), s["k"][b, :, kh].double(), s["v"][b, :, kh].double()
            x = (q @ k.T) * s["scale"]
            slope = 1.0
            if case["cap"]:
                t = torch.tanh(x / case["cap"])
                x, slope = case["cap"] * t, 1 - t * t
            if bucket is not None:
                x = x + s["table"][:, h].double()[bucket]
            x = torch.where(seen[b], x, -math.inf)
            lse[b, h] = torch.logsumexp(x, 1)
            p = torch.where(seen[b], torch.exp(x - lse[b, h][:, None]), 0.0)
            o[b, :, h] = p @ v
            if bwd:
                do = s["do"][b, :, h].double()
                dv[b, :, kh] += p.T @ do
                dp = do @ v.T
                ds = p * (dp - (p * dp).sum(1, keepdim=True))
                if bucket is not None:
                    dtab[:, h].index_add_(0, bucket.reshape(-1), ds.reshape(-1))
                ds = ds * slope * s["scale"]
                dq[b, :, h] = ds @ k
                dk[b, :, kh] += ds.T @ q
    if not bwd:
        return o, lse
    out = {"dq": dq, "dk": dk, "dv": dv}
    if case["bias"]:
        out["dtable"] = dtab
    return out


def _norm_exact(case, s):
    rd, inter = case["rd"], case["inter"]
    a = s["pos"].double()[:, None] * s["inv_freq"][None, :]
    turn = torch.polar(torch.ones_like(a), a)[:, None, :]        # e^(i angle)

    def rotate(x, by):
        z = x[..., :rd]
        z = torch.view_as_complex(z.reshape(*z.shape[:-1], rd // 2, 2).contiguous()) if inter \
            else torch.complex(z[..., :rd // 2].contiguous(), z[..., rd // 2:].contiguous())
        z = torch.view_as_real(z * by)
        z = z.flatten(-2) if inter else z.transpose(-1, -2).flatten(-2)
        return torch.cat([z, x[..., rd:]], -1)

    out = {}
    for n in ("q", "k"):
        x, w = s[n].double(), s["w" + n].double()
        rms = torch.sqrt((x * x).sum(-1, keepdim=True) / case["D"] + s["eps"])
        if case["pass_"] == "fwd":
            out["y" + n] = rotate(x / rms * w, turn)
        else:
            gn = rotate(s["dy" + n].double(), turn.conj())
            out["dw" + n] = (gn * x / rms).sum((0, 1))
            gn = gn * w
            out["d" + n] = gn / rms - x * (gn * x).sum(-1, keepdim=True) / (case["D"] * rms ** 3)
    return out


def _distill_exact(case, s):
    tau, out = case["tau"], {}
    N, V = case["N"], case["V"]
    parts = {"loss": [], "stats": [], "dz": []}
    step = max(1, (1 << 27) // V)                                # rows at a time, 1 GiB of fp64
    for r in range(0, N, step):
        rows = slice(r, min(N, r + step))
        logq = torch.log_softmax(s["z"][rows].double() / tau, 1)
        lse = torch.logsumexp(s["z"][rows].double() / tau, 1)
        idx = s["idx"][rows].long()
        t, w = s["val"][rows].double() / tau, s["w"][rows].double()
        member = torch.zeros_like(logq, dtype=torch.bool).scatter_(1, idx, True)
        c = torch.ones_like(lse)
        if s["tlse"] is None:
            logp = torch.log_softmax(t, 1)
            loss = (logp.exp() * (logp - logq.gather(1, idx))).sum(1)
        else:
            logp = t - s["tlse"][rows].double()[:, None]
            rest = (-torch.expm1(torch.logsumexp(logp, 1))).clamp_min(0)
            logtail = torch.logsumexp(logq.masked_fill(member, -math.inf), 1)
            loss = (logp.exp() * (logp - logq.gather(1, idx))).sum(1) \
                + torch.special.xlogy(rest, rest) - rest * logtail
            c = 1 - rest / logtail.exp()
        parts["loss"].append(loss * tau * tau * w)
        parts["stats"].append(torch.stack([lse, c], 1))
        if case["pass_"] != "fwd":
            q = logq.exp()
            d = torch.where(member, q, q * c[:, None])
            d.scatter_add_(1, idx, -logp.exp())
            parts["dz"].append((d * (w * tau * s["gscale"])[:, None]).to(torch.float64))
    names = {"fwd": ("loss", "stats"), "both": ("loss", "stats", "dz"), "bwd": ("dz",)}
    for n in names[case["pass_"]]:
        out[n] = torch.cat(parts[n])
    return out
