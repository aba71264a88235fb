"""Workloads of the operators around a student's blocks: the embedding lookup
and its gradient, the norms before and after a block with its gate and
residual scale, the clipped policy loss with a KL term, and the global norm
and clipping of the gradients of many tensors.

Each case is one call a training program makes (norm and clipping are two).
`run` computes it either with elementary torch operations (`own` false) or
through this package's entry points (`own` true); `exact` computes it from the
definition in 64 bits.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
BYTES = {"bf16": 2, "f32": 4}


# --------------------------------------------------------------- the cases ---

def listed():
    return [
        # The rows of one micro-batch of 16k tokens looked up in a table of
        # GPT-2's vocabulary, with the factor sqrt(width) on the way.
        dict(name="embed-fwd-16k", op="embed", pass_="fwd", N=16384, V=50257, C=4096, dtype="bf16",
             grad="bf16", base="none", scale=64.0),
        # The table's gradient of one short sequence: a few rows, and zeros
        # for the whole rest of the table.
        dict(name="embed-bwd-61", op="embed", pass_="bwd", N=61, V=50257, C=768, dtype="bf16",
             grad="f32", base="none", scale=1.0),
        # A tied table's gradient: the rows' sums on top of the gradient that
        # the logits' product left in fp32, into the bf16 replica that the
        # optimizer step reduces.
        dict(name="embed-bwd-16k-tied", op="embed", pass_="bwd", N=16384, V=50257, C=4096,
             dtype="bf16", grad="bf16", base="f32", scale=64.0),
        # Residual sum and the next block's norm of a short row: latency.
        dict(name="block-norm-fwd-61", op="norm", pass_="fwd", T=61, C=768, dtype="bf16",
             res="bf16", post=False, gate="none", y=True, z=True, offset=0.0, res_scale=1.0,
             branch_scale=1.0),
        # 16k tokens of a larger student: the block's output normed, gated by
        # channel, added to the residual stream, normed for the next block.
        dict(name="block-norm-fwd-16k", op="norm", pass_="fwd", T=16384, C=4096, dtype="bf16",
             res="bf16", post=True, gate="channel", y=True, z=True, offset=0.0, res_scale=1.0,
             branch_scale=0.5),
        # The same in training, with the weights' and the gate's gradients.
        dict(name="block-norm-bwd-8k", op="norm", pass_="bwd", T=8192, C=4096, dtype="bf16",
             res="bf16", post=True, gate="channel", y=True, z=True, offset=0.0, res_scale=1.0,
             branch_scale=0.5),
        # An fp32 residual stream of an odd width, a gate of its own for each
        # token, weights kept as differences from 1.
        dict(name="block-norm-bwd-4k-res32", op="norm", pass_="bwd", T=4097, C=1000, dtype="bf16",
             res="f32", post=True, gate="token", y=True, z=True, offset=1.0, res_scale=0.9,
             branch_scale=1.0),
        # The policy loss of one short answer with its gradient, at GPT-2's
        # vocabulary (odd: rows start misaligned).
        dict(name="policy-61", op="policy", pass_="both", N=61, V=50257, tau=1.0, lo=0.2, hi=0.2,
             kl=0.05, old=True, dtype="bf16"),
        # A micro-batch of 8k sampled tokens.
        dict(name="policy-8k", op="policy", pass_="both", N=8192, V=50257, tau=0.8, lo=0.2, hi=0.28,
             kl=0.02, old=True, dtype="bf16"),
        # The gradient alone, from the saved row statistics, of a large
        # vocabulary in fp32.
        dict(name="policy-bwd-131k-f32", op="policy", pass_="bwd", N=1024, V=131072, tau=1.0, lo=0.2,
             hi=0.2, kl=0.05, old=True, dtype="f32"),
        # All gradients of a one-block student of odd width (latency, tensors
        # that start at any element).
        dict(name="clip-10-tensors", op="clip", blocks=1, width=129, vocab=512, norms="f32",
             loss_scale=1.0, max_norm=0.25),
        # All gradients of 24 blocks, norm weights in fp32, with a loss scale.
        dict(name="clip-194-tensors", op="clip", blocks=24, width=640, vocab=50257, norms="f32",
             loss_scale=1024.0, max_norm=1.0),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["embed", "norm", "policy", "clip"])
    if op == "embed":
        C = 8 * _log_int(rng, 4, 1024)
        V = _log_int(rng, 100, min(200_000, 50257 * 4096 // C))
        return dict(op="embed", pass_=rng.choice(["fwd", "bwd", "bwd"]),
                    N=_log_int(rng, 1, min(65536, 16384 * 4096 // C)), V=V, C=C,
                    dtype=rng.choice(["bf16", "bf16", "f32"]), grad=rng.choice(["bf16", "f32"]),
                    base=rng.choice(["none", "none", "f32", "bf16"]),
                    scale=rng.choice([1.0, 16.0, math.sqrt(C)]))
    if op == "norm":
        C = 8 * _log_int(rng, 4, 2048)
        dtype, res = rng.choice([("bf16", "bf16"), ("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")])
        y = rng.random() < 0.85
        return dict(op="norm", pass_=rng.choice(["fwd", "bwd"]),
                    T=_log_int(rng, 1, min(16384, 8192 * 4096 // C)), C=C, dtype=dtype, res=res,
                    post=y and rng.random() < 0.6,
                    gate=rng.choice(["none", "channel", "token"]) if y else "none", y=y,
                    z=not y or rng.random() < 0.85, offset=rng.choice([0.0, 0.0, 1.0]),
                    res_scale=rng.choice([1.0, 1.0, 0.9]) if y else 1.0,
                    branch_scale=rng.choice([1.0, 0.5, 0.22]) if y else 1.0)
    if op == "policy":
        V = _log_int(rng, 500, 200_000)
        return dict(op="policy", pass_=rng.choice(["fwd", "bwd", "both"]),
                    N=_log_int(rng, 1, max(1, min(8192, 8192 * 50257 // (2 * V)))), V=V,
                    tau=rng.choice([1.0, 0.7, 1.3]), lo=0.2, hi=rng.choice([0.2, 0.28]),
                    kl=rng.choice([0.0, 0.01, 0.1]), old=rng.random() < 0.7,
                    dtype=rng.choice(["bf16", "bf16", "f32"]))
    width = _log_int(rng, 33, 900)
    return dict(op="clip", blocks=_log_int(rng, 1, max(1, min(40, 24 * 640 * 640 // (width * width)))),
                width=width, vocab=_log_int(rng, 100, 50257), norms=rng.choice(["f32", "bf16"]),
                loss_scale=rng.choice([1.0, 1024.0]), max_norm=rng.choice([0.1, 1.0, 1e6]))


# ------------------------------------------------------------------ inputs ---

def _normal(g, shape, dtype, scale=1.0):
    return torch.randn(shape, generator=g, device="cuda").mul_(scale).to(DTYPES[dtype])


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return {"embed": _prepare_embed, "norm": _prepare_norm, "policy": _prepare_policy,
            "clip": _prepare_clip}[case["op"]](case, g)


def _package():
    import zero_sharded_mixed_step_amd as zs
    return zs


def _scratch(nbytes):
    """Scratch memory that a program keeps from step to step."""
    return torch.empty(max(nbytes, 16), dtype=torch.uint8, device="cuda")


def _prepare_embed(case, g):
    N, V, C = case["N"], case["V"], case["C"]
    # tokens of a text: a few words make up much of it, most of the table is
    # not met; every 33rd place is padding
    u = torch.rand(N, generator=g, device="cuda", dtype=torch.float64)
    at = torch.randint(V, (1,), generator=g, device="cuda")
    ids = ((u * math.log(V + 1)).exp().long() - 1).clamp(0, V - 1)
    ids = ((ids * 7919 + at) % V).to(torch.int32)
    ids[32::33] = -1
    s = dict(case=case, ids=ids)
    if case["pass_"] == "fwd":
        s["table"] = _normal(g, (V, C), case["dtype"], 0.5)
        s["out"] = torch.empty((N, C), dtype=DTYPES[case["dtype"]], device="cuda")
        return s
    s["dout"] = _normal(g, (N, C), case["dtype"], 1e-2)
    s["base"] = None if case["base"] == "none" else _normal(g, (V, C), case["base"], 1e-2)
    s["dtable"] = torch.empty((V, C), dtype=DTYPES[case["grad"]], device="cuda")
    if own:
        s["ws"] = _scratch(_package().zero_embed_workspace_bytes(N, C))
    return s


def _prepare_norm(case, g):
    T, C, dt, res = case["T"], case["C"], case["dtype"], case["res"]
    s = dict(case=case, eps=1e-6)
    s["x"] = _normal(g, (T, C), res, 2.0)
    s["y"] = _normal(g, (T, C), dt, 1.3) if case["y"] else None
    for n, on in (("w1", case["post"]), ("w2", case["z"])):
        s[n] = (torch.randn(C, generator=g, device="cuda") * 0.1 + 1 - case["offset"]).to(
            DTYPES[dt]) if on else None
    shape = {"none": None, "channel": (C,), "token": (T, C)}[case["gate"]]
    s["gate"] = None if shape is None else _normal(g, shape, dt, 0.6)
    if case["pass_"] == "fwd":
        s["h"] = torch.empty_like(s["x"]) if case["y"] else None
        s["z"] = torch.empty((T, C), dtype=DTYPES[dt], device="cuda") if case["z"] else None
        return s
    # the residual sum that the forward pass of the same step left
    s["h"] = _norm_fwd_plain(s)["h"] if case["y"] else s["x"]
    s["dh"] = _normal(g, (T, C), res)
    s["dz"] = _normal(g, (T, C), dt) if case["z"] else None
    s["dx"] = torch.empty_like(s["x"])
    for n, x in (("dy", "y"), ("dw1", "w1"), ("dw2", "w2"), ("dgate", "gate")):
        s[n] = None if s[x] is None else torch.empty_like(s[x])
    if own:
        s["ws"] = _scratch(_package().zero_block_norm_workspace_bytes(T, C))
    return s


def _prepare_policy(case, g):
    N, V, tau = case["N"], case["V"], case["tau"]
    z = _normal(g, (N, V), case["dtype"], 2.0)
    # the sampled tokens, their log probability when they were sampled (some
    # updates ago) and under the reference policy
    at = torch.rand(N, generator=g, device="cuda")
    act = torch.empty(N, dtype=torch.int64, device="cuda")
    lse = torch.empty(N, dtype=torch.float64, device="cuda")
    step = max(1, (1 << 26) // V)
    for r in range(0, N, step):
        x = z[r:r + step].double() / tau
        lse[r:r + step] = torch.logsumexp(x, 1)
        c = (x - lse[r:r + step, None]).exp_().cumsum_(1)
        act[r:r + step] = torch.searchsorted(c, at[r:r + step, None].double())[:, 0].clamp_(0, V - 1)
        del x, c
    lp = z.gather(1, act[:, None])[:, 0].double() / tau - lse
    noise = torch.randn((3, N), generator=g, device="cuda", dtype=torch.float64)
    s = dict(case=case, z=z, act=act.to(torch.int32), adv=noise[0].float(),
             old=(lp + 0.15 * noise[1]).float() if case["old"] else None,
             ref=(lp + 0.3 * noise[2]).float() if case["kl"] else None)
    # a tenth of the rows carries no loss (prompt and padding tokens)
    s["w"] = (torch.rand(N, generator=g, device="cuda") > 0.1).float()
    s["gscale"] = 1.0 / N
    s["loss"] = torch.empty(N, dtype=torch.float32, device="cuda")
    s["stats"] = torch.empty((N, 4), dtype=torch.float32, device="cuda")
    if case["pass_"] != "fwd":
        s["dz"] = torch.empty_like(z)
    if case["pass_"] == "bwd":
        s["stats"].copy_(_policy_rows_plain(s)["stats"])
    return s


def _tensors(case):
    """(elements, dtype) of every gradient: table, then of each block a norm,
    the three projections as one, the output's, a norm, the wide pair with the
    first one's bias, and the last norm."""
    w, n = case["width"], case["norms"]
    block = [(w, n), (3 * w * w, "bf16"), (w * w, "bf16"), (w, n), (4 * w * w, "bf16"),
             (4 * w, "bf16"), (4 * w * w, "bf16"), (w, "bf16")]
    return [(case["vocab"] * w, "bf16")] + block * case["blocks"] + [(w, n)]


def _prepare_clip(case, g):
    """The gradients as views of one buffer of each type, as a program that
    reduces them in buckets keeps them."""
    sizes = _tensors(case)
    s = dict(case=case, grads=[], outs=[], flat={}, out={})
    for dt in ("bf16", "f32"):
        n = sum(k for k, t in sizes if t == dt)
        if n:
            s["flat"][dt] = _normal(g, (n,), dt, 1e-3 * case["loss_scale"])
            s["out"][dt] = torch.empty_like(s["flat"][dt])
    at = {"bf16": 0, "f32": 0}
    for k, dt in sizes:
        for name, flat in (("grads", "flat"), ("outs", "out")):
            s[name].append(s[flat][dt][at[dt]:at[dt] + k])
        at[dt] += k
    s["inv"] = 1.0 / case["loss_scale"]
    s["norm"] = torch.empty(1, dtype=torch.float32, device="cuda")
    if own:
        # the table of the tensors that a program makes once for its gradients
        zs = _package()
        s["tensors"] = zs.GradTable(s["grads"], s["outs"])
        s["acc"], s["ws"] = zs.new_norm_acc(1), _scratch(zs.zero_grads_workspace_bytes())
    return s


# ------------------------------------------------------------- plain forms ---

def run(s):
    if own:
        return _run_own(s)
    case = s["case"]
    if case["op"] == "embed":
        return _embed_fwd_plain(s) if case["pass_"] == "fwd" else _embed_bwd_plain(s)
    if case["op"] == "norm":
        return _norm_outputs(s, _norm_fwd_plain(s)) if case["pass_"] == "fwd" else _norm_bwd_plain(s)
    return _policy_plain(s) if case["op"] == "policy" else _clip_plain(s)


def _embed_fwd_plain(s):
    ok = s["ids"] >= 0
    rows = s["table"][s["ids"].clamp_min(0).long()].float() * s["case"]["scale"]
    return torch.where(ok[:, None], rows, torch.zeros_like(rows)).to(s["table"].dtype)


def _embed_bwd_plain(s):
    case, ok = s["case"], s["ids"] >= 0
    out = torch.zeros(s["dtable"].shape, dtype=torch.float32, device="cuda")
    out.index_add_(0, s["ids"][ok].long(), s["dout"][ok].float())
    out = out * case["scale"]
    if s["base"] is not None:
        out = out + s["base"].float()
    return out.to(s["dtable"].dtype)


def _rms(x, eps):
    return (x.square().mean(-1, keepdim=True) + eps).rsqrt()


def _norm_parts(s):
    """Block output in fp32, its reciprocal norm, weight, normed output, gate times scale."""
    case = s["case"]
    y = s["y"].float()
    r = w = None
    u = y
    if case["post"]:
        r, w = _rms(y, s["eps"]), s["w1"].float() + case["offset"]
        u = y * r * w
    g = case["branch_scale"] if s["gate"] is None else s["gate"].float() * case["branch_scale"]
    return y, r, w, u, g


def _norm_fwd_plain(s):
    case = s["case"]
    h = s["x"].float() * case["res_scale"]
    if case["y"]:
        u, g = _norm_parts(s)[3:]
        h = h + u * g
    out = {"h": h.to(s["x"].dtype)}
    if case["z"]:
        out["z"] = (h * _rms(h, s["eps"]) * (s["w2"].float() + case["offset"])).to(DTYPES[case["dtype"]])
    return out


def _norm_outputs(s, out):
    return {n: out[n] for n in ("h", "z") if n in out and s[n] is not None}


def _norm_bwd_plain(s):
    case, out = s["case"], {}
    gh = s["dh"].float()
    if case["z"]:
        h, dz = s["h"].float(), s["dz"].float()
        r = _rms(h, s["eps"])
        hat = h * r
        out["dw2"] = (dz * hat).double().sum(0).to(s["w2"].dtype)
        u2 = dz * (s["w2"].float() + case["offset"])
        gh = gh + r * (u2 - hat * (u2 * hat).mean(-1, keepdim=True))
    out["dx"] = (gh * case["res_scale"]).to(s["dx"].dtype)
    if not case["y"]:
        return out
    y, r, w, u, g = _norm_parts(s)
    if s["gate"] is not None:
        dg = gh * u * case["branch_scale"]
        out["dgate"] = (dg.double().sum(0) if case["gate"] == "channel" else dg).to(s["gate"].dtype)
    du = gh * g
    if case["post"]:
        hat = y * r
        out["dw1"] = (du * hat).double().sum(0).to(s["w1"].dtype)
        v = du * w
        du = r * (v - hat * (v * hat).mean(-1, keepdim=True))
    out["dy"] = du.to(s["y"].dtype)
    return out


def _policy_rows_plain(s):
    """Losses and statistics of the rows; the sum of exponentials and all that
    follows from it in 64 bits (the ratio may lie next to its border)."""
    case = s["case"]
    x = s["z"].float() / case["tau"]
    m = x.amax(1)
    lse = m.double() + x.sub_(m[:, None]).exp_().double().sum(1).log()
    del x
    za = s["z"].gather(1, s["act"].long()[:, None])[:, 0].double()
    lp = za / case["tau"] - lse
    A = s["adv"].double()
    r = (lp - s["old"].double()).exp() if s["old"] is not None else torch.ones_like(lp)
    bound = r.clamp(1 - case["lo"], 1 + case["hi"])
    loss = -torch.minimum(r * A, bound * A)
    clipped = ((A > 0) & (r > 1 + case["hi"])) | ((A < 0) & (r < 1 - case["lo"]))
    g = torch.where(clipped, torch.zeros_like(r), -A * r)
    kl = torch.zeros_like(lp)
    if s["ref"] is not None:
        d = s["ref"].double() - lp
        kl = torch.expm1(d) - d
        loss = loss + case["kl"] * kl
        g = g - case["kl"] * torch.expm1(d)
    return {"loss": (loss * s["w"].double()).float(),
            "stats": torch.stack([lse, lp, g, kl], 1).float()}


def _policy_plain(s):
    case = s["case"]
    out = _policy_rows_plain(s) if case["pass_"] != "bwd" else {"stats": s["stats"]}
    if case["pass_"] == "fwd":
        return out
    lse, lp, g = out["stats"][:, 0], out["stats"][:, 1], out["stats"][:, 2]
    k = s["w"] * g * (s["gscale"] / case["tau"])
    d = (s["z"].float() / case["tau"]).sub_(lse[:, None]).exp_().mul_(-k[:, None])
    own_ = -torch.expm1(lp.double()).float() * k
    d.scatter_(1, s["act"].long()[:, None], own_[:, None])
    out = dict(out, dz=d.to(s["z"].dtype))
    if case["pass_"] == "bwd":
        del out["stats"]
    return out


def _clip_plain(s):
    case = s["case"]
    total = torch.zeros((), dtype=torch.float64, device="cuda")
    for x in s["grads"]:
        total = total + (x.float() * s["inv"]).double().square().sum()
    norm = total.sqrt()
    coef = (case["max_norm"] / (norm + 1e-6)).clamp_max(1.0).float()
    for x, y in zip(s["grads"], s["outs"]):
        y.copy_(x.float() * s["inv"] * coef)
    return dict(s["out"], norm=norm.float())


# ------------------------------------------------------ through the package ---

def _run_own(s):
    zs, case = _package(), s["case"]
    if case["op"] == "embed":
        if case["pass_"] == "fwd":
            zs.zero_embed_fwd(s["table"], s["ids"], s["out"], scale=case["scale"])
            return s["out"]
        zs.zero_embed_bwd(s["ids"], s["dout"], s["dtable"], scale=case["scale"], base=s["base"],
                          workspace=s["ws"])
        return s["dtable"]
    if case["op"] == "norm":
        kw = dict(post_norm=case["post"], post_weight=s["w1"], gate=s["gate"], pre_weight=s["w2"],
                  weight_offset=case["offset"], res_scale=case["res_scale"],
                  branch_scale=case["branch_scale"], eps=s["eps"])
        if case["pass_"] == "fwd":
            zs.zero_block_norm_fwd(s["x"], s["y"], s["h"], s["z"], **kw)
            return {n: s[n] for n in ("h", "z") if s[n] is not None}
        zs.zero_block_norm_bwd(s["y"], s["h"], s["dh"], s["dz"], s["dx"], s["dy"],
                               dpost_weight=s["dw1"], dgate=s["dgate"], dpre_weight=s["dw2"],
                               workspace=s["ws"], **kw)
        return {n: s[n] for n in ("dx", "dy", "dw1", "dgate", "dw2") if s[n] is not None}
    if case["op"] == "policy":
        kw = dict(row_weight=s["w"], temperature=case["tau"], grad_scale=s["gscale"])
        if case["pass_"] == "bwd":
            zs.zero_policy_bwd(s["z"], s["act"], s["stats"], s["dz"], **kw)
            return {"dz": s["dz"]}
        zs.zero_policy_fwd(s["z"], s["act"], s["adv"], s["loss"], s["stats"], dlogits=s.get("dz"),
                           old_logp=s["old"], ref_logp=s["ref"], clip_low=case["lo"],
                           clip_high=case["hi"], kl_coef=case["kl"], **kw)
        return {n: s[n] for n in ("loss", "stats", "dz") if n in s}
    zs.zero_grads_norm(s["tensors"], s["acc"], inv_scale=s["inv"], workspace=s["ws"])
    zs.zero_grads_clip(s["tensors"], s["acc"], max_norm=case["max_norm"], inv_scale=s["inv"],
                       norm_out=s["norm"])
    return dict(s["out"], norm=s["norm"][0])


# -------------------------------------------------------------------- work ---

def work(case):
    if case["op"] == "embed":
        N, V, C, b = case["N"], case["V"], case["C"], BYTES[case["dtype"]]
        if case["pass_"] == "fwd":
            return {"bytes": 2 * N * C * b + 4 * N, "flops": 1.0 * N * C}
        wide = V * C * (BYTES[case["grad"]] + (0 if case["base"] == "none" else BYTES[case["base"]]))
        return {"bytes": N * C * b + 4 * N + wide, "flops": 2.0 * N * C}
    if case["op"] == "norm":
        T, C, b, r = case["T"], case["C"], BYTES[case["dtype"]], BYTES[case["res"]]
        n, y, z = T * C, 1 if case["y"] else 0, 1 if case["z"] else 0
        vec = C * b * ((1 if case["post"] else 0) + z + (1 if case["gate"] == "channel" else 0))
        tok = n * b if case["gate"] == "token" else 0
        if case["pass_"] == "fwd":
            return {"bytes": n * (r + r * y + b * y + b * z) + vec + tok, "flops": 8.0 * n}
        # read dh, and h and dz where there is a norm after, and y; write dx, dy
        # (y itself is not needed where it is neither normed nor gated)
        reads_y = b * y if case["post"] or case["gate"] != "none" else 0
        return {"bytes": n * (2 * r + (r + b) * z + reads_y + b * y) + 2 * vec + 2 * tok,
                "flops": 20.0 * n}
    if case["op"] == "policy":
        N, V, b = case["N"], case["V"], BYTES[case["dtype"]]
        k = 1 if case["pass_"] == "fwd" else 2
        return {"bytes": k * N * V * b + 36 * N, "flops": 4.0 * k * N * V}
    n = {dt: sum(k for k, t in _tensors(case) if t == dt) for dt in ("bf16", "f32")}
    return {"bytes": 2 * (2 * n["bf16"] + 4 * n["f32"]), "flops": 4.0 * (n["bf16"] + n["f32"])}


# ------------------------------------------------------- the 64-bit answer ---

def exact(case, seed):
    s = prepare(case, seed)
    return {"embed": _embed_exact, "norm": _norm_exact, "policy": _policy_exact,
            "clip": _clip_exact}[case["op"]](case, s)


def _embed_exact(case, s):
    ids = s["ids"].long()
    if case["pass_"] == "fwd":
        out = torch.zeros((case["N"], case["C"]), dtype=torch.float64, device="cuda")
        out[ids >= 0] = s["table"].double()[ids[ids >= 0]] * case["scale"]
        return out
    out = torch.zeros((case["V"], case["C"]), dtype=torch.float64, device="cuda")
    out.index_add_(0, ids[ids >= 0], s["dout"].double()[ids >= 0], alpha=case["scale"])
    return out if s["base"] is None else out.add_(s["base"].double())


def _norm_exact(case, s):
    off = case["offset"]

    def root(x):
        return torch.sqrt((x * x).sum(-1, keepdim=True) / case["C"] + s["eps"])

    b = case["branch_scale"]
    y, gate = (None if s[n] is None else s[n].double() for n in ("y", "gate"))
    if case["y"]:
        ry = root(y)
        u = y / ry * (s["w1"].double() + off) if case["post"] else y
        scaled = b if gate is None else b * gate
    if case["pass_"] == "fwd":
        h = s["x"].double() * case["res_scale"] + (u * scaled if case["y"] else 0.0)
        out = {"h": h} if case["y"] else {}
        if case["z"]:
            out["z"] = h / root(h) * (s["w2"].double() + off)
        return out
    out, gh = {}, s["dh"].double()
    if case["z"]:
        h, dz = s["h"].double(), s["dz"].double()
        rh = root(h)
        out["dw2"] = (dz * h / rh).sum(0)
        v = dz * (s["w2"].double() + off)
        gh = gh + v / rh - h * (v * h).sum(-1, keepdim=True) / (case["C"] * rh ** 3)
    out["dx"] = gh * case["res_scale"]
    if case["y"]:
        if gate is not None:
            out["dgate"] = b * gh * u
            if case["gate"] == "channel":
                out["dgate"] = out["dgate"].sum(0)
        v = gh * scaled
        if case["post"]:
            out["dw1"] = (v * y / ry).sum(0)
            v = v * (s["w1"].double() + off)
            v = v / ry - y * (v * y).sum(-1, keepdim=True) / (case["C"] * ry ** 3)
        out["dy"] = v
    return out


def _policy_exact(case, s):
    N, V, tau = case["N"], case["V"], case["tau"]
    parts = {"loss": [], "stats": [], "dz": []}
    step = max(1, (1 << 27) // V)                          # rows at a time, 1 GiB of fp64
    for a in range(0, N, step):
        rows = slice(a, min(N, a + step))
        x = s["z"][rows].double() / tau
        act = s["act"][rows].long()[:, None]
        logq = torch.log_softmax(x, 1)
        lp, w, A = logq.gather(1, act)[:, 0], s["w"][rows].double(), s["adv"][rows].double()
        if case["pass_"] == "bwd":
            g = s["stats"][rows, 2].double()
        else:
            r = torch.exp(lp - s["old"][rows].double()) if s["old"] is not None \
                else torch.ones_like(lp)
            lo, hi = 1 - case["lo"], 1 + case["hi"]
            inside = torch.where(A > 0, r <= hi, r >= lo)
            loss = -A * torch.where(inside, r, torch.where(A > 0, hi, lo))
            g = -A * r * inside
            kl = torch.zeros_like(lp)
            if s["ref"] is not None:
                ratio = torch.exp(s["ref"][rows].double() - lp)
                kl = ratio - ratio.log() - 1
                loss, g = loss + case["kl"] * kl, g + case["kl"] * (1 - ratio)
            parts["loss"].append(loss * w)
            parts["stats"].append(torch.stack([torch.logsumexp(x, 1), lp, g, kl], 1))
        if case["pass_"] != "fwd":
            d = -logq.exp()
            d.scatter_add_(1, act, torch.ones_like(act, dtype=torch.float64))
            parts["dz"].append(d * (w * g * s["gscale"] / tau)[:, None])
    names = {"fwd": ("loss", "stats"), "both": ("loss", "stats", "dz"), "bwd": ("dz",)}
    return {n: torch.cat(parts[n]) for n in names[case["pass_"]]}


def _clip_exact(case, s):
    flat = {dt: x.double() * s["inv"] for dt, x in s["flat"].items()}
    norm = math.sqrt(sum(float(x.square().sum()) for x in flat.values()))
    coef = min(1.0, case["max_norm"] / (norm + 1e-6))
    out = {dt: x * coef for dt, x in flat.items()}
    return dict(out, norm=torch.tensor(norm, dtype=torch.float64))
