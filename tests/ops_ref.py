"""The training operators in 64 bits on the host, straight from their
formulas, with bounds on what a kernel of 32-bit sums and bf16 roundings may
differ by.  A bf16 rounding is off by at most 2^-8 of the value (half a step),
an fp32 one by 2^-24."""
import math

import torch

BF, F32R = 2.0 ** -8, 2.0 ** -24


def half_step(dtype):
    return BF if dtype == torch.bfloat16 else F32R


# -------------------------------------------------------------- attention ---

def visible(B, Tq, Tk, ranges=None, causal=False):
    """(B, Tq, Tk) truth values."""
    j = torch.arange(Tk)
    if ranges is not None:
        r = ranges.long()
        return (j >= r[..., :1]) & (j < r[..., 1:])
    if causal:
        i = torch.arange(Tq) + (Tk - Tq)
        return (j[None, :] <= i[:, None]).expand(B, Tq, Tk)
    return torch.ones((B, Tq, Tk), dtype=torch.bool)


def doc_ranges(doc, prefix=None, causal=True):
    """Key ranges of packed rows, token by token."""
    B, T = doc.shape
    out = torch.zeros((B, T, 2), dtype=torch.int32)
    for b in range(B):
        for t in range(T):
            if doc[b, t] < 0:
                continue
            lo = t
            while lo > 0 and doc[b, lo - 1] == doc[b, t]:
                lo -= 1
            hi = t + 1
            while hi < T and doc[b, hi] == doc[b, t]:
                hi += 1
            see = hi
            if causal:
                see = t + 1
                if prefix is not None:
                    see = min(hi, max(see, lo + int(prefix[b, t])))
            out[b, t, 0], out[b, t, 1] = lo, see
    return out


class Attention:
    """Forward and backward of one call, all heads at once."""

    def __init__(self, q, k, v, *, scale, cap=0.0, seen, table=None, buckets=None):
        self.dt = q.dtype
        B, Tq, Hq, D = q.shape
        Tk, Hk = k.shape[1], k.shape[2]
        self.shape, self.Hk, self.scale, self.cap = (B, Tq, Hq, D), Hk, scale, cap
        g = Hq // Hk
        self.q = q.double().permute(0, 2, 1, 3)
        self.k = k.double().permute(0, 2, 1, 3).repeat_interleave(g, 1)
        self.v = v.double().permute(0, 2, 1, 3).repeat_interleave(g, 1)
        seen = seen[:, None]
        # masked keys hold anything: their rows are taken as 0 where unseen by all
        x = torch.where(seen, self.q @ self.k.transpose(2, 3), 0.0) * scale
        mag = torch.where(seen, self.q.abs() @ self.k.abs().transpose(2, 3), 0.0) * scale
        self.th = torch.tanh(x / cap) if cap else torch.zeros_like(x)
        s = cap * self.th if cap else x
        self.bucket = None
        if table is not None:
            reach = buckets.shape[0] // 2
            dist = torch.arange(Tk)[None, :] - (torch.arange(Tq)[:, None] + Tk - Tq)
            self.bucket = buckets.long()[dist.clamp(-reach, reach) + reach].clamp(
                0, table.shape[0] - 1)
            s = s + table.double()[self.bucket].permute(2, 0, 1)
        self.table = table
        s = torch.where(seen, s, -math.inf)
        self.seen = seen
        big = s.abs()[torch.isfinite(s)]
        # error of a score: D products summed, then a few roundings of its parts
        self.e_s = D * F32R * float(mag.max()) + 16 * F32R * (
            cap + (float(big.max()) if big.numel() else 0.0) + 8)
        self.lse = torch.logsumexp(s, 3)
        self.lse = torch.where(seen.any(3).expand_as(self.lse), self.lse, -math.inf)
        self.p = torch.where(seen, torch.exp(s - torch.where(
            torch.isinf(self.lse), 0.0, self.lse)[..., None]), 0.0)

    def forward(self):
        """o (B, Tq, Hq, D), its bound, lse and its bound."""
        v = torch.where(self.seen.any(2)[..., None], self.v, 0.0)
        o, a = self.p @ v, self.p @ v.abs()
        bound = BF * (o.abs() + 1.02 * a) + 4 * self.e_s * a + 1e-30
        lse_bound = 2 * self.e_s + 4 * F32R * torch.where(
            torch.isinf(self.lse), 0.0, self.lse).abs() + 1e-7
        return (o.permute(0, 2, 1, 3), bound.permute(0, 2, 1, 3), self.lse, lse_bound)

    def backward(self, o, do):
        """{name: (value, bound)} given the forward's stored o."""
        B, Tq, Hq, D = self.shape
        live = self.seen.any(3)[..., None]
        keys = self.seen.any(2)[..., None]
        do = torch.where(live, do.double().permute(0, 2, 1, 3), 0.0)
        o = torch.where(live, o.double().permute(0, 2, 1, 3), 0.0)
        q = torch.where(live, self.q, 0.0)
        k, v = torch.where(keys, self.k, 0.0), torch.where(keys, self.v, 0.0)
        dp = do @ v.transpose(2, 3)
        delta = (do * o).sum(3, keepdim=True)
        e_dp = D * F32R * (float((do.abs() @ v.abs().transpose(2, 3)).max())
                           + float((do * o).abs().sum(3).max()))
        ds = self.p * (dp - delta)
        slope = (1 - self.th ** 2) if self.cap else torch.ones_like(ds)
        dx = ds * slope * self.scale
        rel = 6 * self.e_s + 8 * F32R * (1 + torch.where(
            torch.isinf(self.lse), 0.0, self.lse).abs().max().item())
        e_ds = rel * ds.abs() + self.p * e_dp + 16 * F32R * self.p * (dp.abs() + delta.abs())
        e_dx = (BF * dx.abs() + self.scale * (e_ds + 16 * F32R * ds.abs()))
        group = lambda x: x.view(B, self.Hk, Hq // self.Hk, -1, D).sum(2).permute(0, 2, 1, 3)
        out = {}
        dq, e = dx @ k, e_dx @ k.abs()
        out["dq"] = (dq.permute(0, 2, 1, 3), (BF * dq.abs() + 1.02 * e).permute(0, 2, 1, 3))
        dk, e = group(dx.transpose(2, 3) @ q), group(e_dx.transpose(2, 3) @ q.abs())
        out["dk"] = (dk, BF * dk.abs() + 1.02 * e)
        dv = group(self.p.transpose(2, 3) @ do)
        e = group(self.p.transpose(2, 3) @ do.abs()) * (BF + 2 * rel)
        out["dv"] = (dv, BF * dv.abs() + 1.02 * e)
        if self.table is not None:
            n = self.table.shape[0]
            n_sum = Tq + self.seen.shape[-1] + 64
            val, err = torch.zeros(n, Hq, dtype=torch.float64), torch.zeros(n, Hq,
                                                                            dtype=torch.float64)
            at = self.bucket.reshape(-1)
            val.index_add_(0, at, ds.sum(0).permute(1, 2, 0).reshape(-1, Hq))
            e_sum = e_ds + n_sum * F32R * ds.abs()
            err.index_add_(0, at, e_sum.sum(0).permute(1, 2, 0).reshape(-1, Hq))
            out["dtable"] = (val, half_step(self.table.dtype) * val.abs() + 1.02 * err)
        return {n: (x, b + 1e-30) for n, (x, b) in out.items()}


# ------------------------------------------------------- norm and rotation ---

def _rotate(x, ang, rd, inter, sign):
    """Pairs of the first rd values turned by sign * ang (T, rd / 2)."""
    if rd == 0:
        return x
    c, s = torch.cos(ang)[:, None], sign * torch.sin(ang)[:, None]
    y = x.clone()
    a, b = (x[..., 0:rd:2], x[..., 1:rd:2]) if inter else (x[..., :rd // 2], x[..., rd // 2:rd])
    u, v = a * c - b * s, b * c + a * s
    if inter:
        y[..., 0:rd:2], y[..., 1:rd:2] = u, v
    else:
        y[..., :rd // 2], y[..., rd // 2:rd] = u, v
    return y


def _spread(x, rd, inter):
    """|a| + |b| of each pair, at both members: what a rotation's error scales with."""
    y = x.abs().clone()
    if rd:
        a, b = (y[..., 0:rd:2], y[..., 1:rd:2]) if inter else (y[..., :rd // 2],
                                                               y[..., rd // 2:rd])
        t = a + b
        if inter:
            y[..., 0:rd:2], y[..., 1:rd:2] = t, t
        else:
            y[..., :rd // 2], y[..., rd // 2:rd] = t, t
    return y


def norm_forward(x, w, eps, pos, inv_freq, inter):
    """y and its bound, of one tensor (T, H, D)."""
    f = x.double()
    rd = 0 if inv_freq is None else 2 * inv_freq.shape[0]
    ang = None if rd == 0 else pos.double()[:, None] * inv_freq[None]
    n = f / torch.sqrt((f * f).mean(-1, keepdim=True) + eps)
    if w is not None:
        n = n * w.double()
    y = _rotate(n, ang, rd, inter, 1.0)
    # sum of D squares, root, quotient, products, the sine and cosine
    e = (f.shape[-1] / 2 + 24) * F32R * _spread(n, rd, inter)
    return y, half_step(x.dtype) * y.abs() + 1.02 * e + 1e-30


def norm_backward(x, w, dy, eps, pos, inv_freq, inter):
    """{dx, dw: (value, bound)}."""
    f, D = x.double(), x.shape[-1]
    rd = 0 if inv_freq is None else 2 * inv_freq.shape[0]
    ang = None if rd == 0 else pos.double()[:, None] * inv_freq[None]
    r = 1 / torch.sqrt((f * f).mean(-1, keepdim=True) + eps)
    g = _rotate(dy.double(), ang, rd, inter, -1.0)
    ga = _spread(dy.double(), rd, inter)
    wd = torch.ones(D, dtype=torch.float64) if w is None else w.double()
    u, ua, xh = g * wd, ga * wd.abs(), f * r
    dx = r * (u - xh * (u * xh).mean(-1, keepdim=True))
    e = (D + 40) * F32R * r * (ua + xh.abs() * (ua * xh.abs()).mean(-1, keepdim=True))
    dw = (g * xh).sum((0, 1))
    rows = x.shape[0] * x.shape[1]
    ew = (rows + D + 40) * F32R * (ga * xh.abs()).sum((0, 1))
    h = half_step(x.dtype)
    return {"dx": (dx, h * dx.abs() + 1.02 * e + 1e-30),
            "dw": (dw, h * dw.abs() + 1.02 * ew + 1e-30)}


# ----------------------------------------------------------------- distill ---

def distill(z, idx, val, tau, tlse=None, w=None, grad_scale=1.0):
    """{loss, stats, dz: (value, bound)}; entries outside [0, V) are absent."""
    N, V = z.shape
    x = z.double() / tau
    ok = (idx >= 0) & (idx < V)
    at = torch.where(ok, idx, 0).long()
    t = torch.where(ok, val.double() / tau, -math.inf)
    if tlse is None:
        base = torch.logsumexp(t, 1)
        base = torch.where(torch.isinf(base) & (base < 0), 0.0, base)
    else:
        base = tlse.double()
    p = torch.where(ok, torch.exp(t - base[:, None]), 0.0)
    mass = p.sum(1)
    lse = torch.logsumexp(x, 1)
    logq = x - lse[:, None]
    lq = logq.gather(1, at)
    loss = torch.where(p > 0, p * (torch.log(p) - lq), 0.0).sum(1)
    member = torch.zeros(N, V + 1, dtype=torch.bool)
    member.scatter_(1, torch.where(ok, at, V), True)
    member = member[:, :V]
    coef = torch.ones_like(lse)
    tail = torch.zeros_like(lse)
    if tlse is not None:
        tail = (1 - mass).clamp_min(0)
        logout = torch.logsumexp(torch.where(member, -math.inf, logq), 1)
        loss = loss + torch.where(tail > 0, tail * (torch.log(tail) - logout), 0.0)
        coef = torch.where(tail > 0, 1 - tail * torch.exp(-logout), 1.0)
    wd = torch.ones(N, dtype=torch.float64) if w is None else w.double()
    on = (wd != 0) & (ok.any(1) | (tlse is not None))
    q = torch.exp(logq)
    dz = q * torch.where(member, 1.0, coef[:, None].expand(N, V))
    add = torch.zeros(N, V + 1, dtype=torch.float64)
    add.scatter_add_(1, torch.where(ok, at, V), p)
    dz = (dz - add[:, :V]) * (grad_scale * tau * wd)[:, None]
    loss = loss * tau * tau * wd
    zero = lambda a: torch.where(on.view(-1, *[1] * (a.dim() - 1)), a, 0.0)
    # error of log-sums: the sums' roundings and the exponents' of the far terms
    fin = x[torch.isfinite(x)]
    span = float(fin.max() - fin.min()) if fin.numel() else 0.0
    e = (V / 256 + 64) * F32R + 4 * F32R * min(span, 100.0)
    top = float(fin.abs().max()) if fin.numel() else 0.0
    eq = 8 * F32R * (2 * top + 8 + (lse.abs().max().item() if torch.isfinite(lse).all() else 0))
    e_loss = tau * tau * wd.abs() * 4 * e + 4 * F32R * loss.abs() + 1e-30
    e_coef = (1 - coef).abs() * 4 * e + 4 * F32R * (1 + coef.abs())
    e_stats = torch.stack([e + 4 * F32R * lse.abs(), e_coef], 1) + 1e-30
    sc = (abs(grad_scale) * tau * wd.abs())[:, None]
    h = half_step(z.dtype)
    e_dz = h * dz.abs() + sc * (q * (torch.where(member, 1.0, coef.abs()[:, None]) * 1.02
                                     * (eq + 4 * e) + torch.where(member, 0.0, e_coef[:, None]))
                                + 16 * F32R * add[:, :V]) + 1e-30
    return {"loss": (zero(loss), e_loss), "stats": (torch.stack([lse, coef], 1), e_stats),
            "dz": (zero(dz), e_dz)}


def check(name, got, want, bound):
    """Every value within its bound; infinities and NaN where they are wanted."""
    got, want = got.detach().cpu().double(), want.double()
    assert got.shape == want.shape, (name, got.shape, want.shape)
    special = ~torch.isfinite(want)
    assert torch.equal(torch.isnan(got), torch.isnan(want)), f"{name}: NaN in other places"
    same = torch.isnan(want) | (got == want)
    assert bool(same[special].all()), f"{name}: infinities in other places"
    off = torch.where(special, 0.0, (got - torch.where(special, 0.0, want)).abs())
    bound = bound.expand_as(want) if isinstance(bound, torch.Tensor) else torch.full_like(want, bound)
    bad = off > bound
    assert not bool(bad.any()), (
        f"{name}: {int(bad.sum())} of {bad.numel()} values past their bound, worst "
        f"{float((off / bound)[bad].max()):.3g} times, at {bad.nonzero()[0].tolist()}")
