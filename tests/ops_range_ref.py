"""Bounds for the ends of the operators' ranges, beside ops_ref's: the error of a
capped score by the score's size and not by the cap's, and a loss's by its row's
outside entries too."""
import math

import torch

import ops_ref as R

# Up to this cap a score is formed as cap - 2 cap u, u = 1 / (exp(2 x / cap) + 1), of which
# u is off by two steps (exponential, sum, reciprocal); beyond, by its own size alone.
U_CAP = 64.0


class Attention(R.Attention):
    def __init__(self, q, k, v, *, scale, cap=0.0, seen, table=None, buckets=None):
        super().__init__(q, k, v, scale=scale, cap=cap, seen=seen, table=table, buckets=buckets)
        s = seen[:, None]
        mag = torch.where(s, self.q.abs() @ self.k.abs().transpose(2, 3), 0.0) * abs(scale)
        x = torch.where(s, self.q @ self.k.transpose(2, 3), 0.0) * scale
        x = cap * torch.tanh(x / cap) if cap else x
        big = float(x.abs().max())
        if table is not None:
            b = table.double()[self.bucket].permute(2, 0, 1).abs()
            big += float(torch.where(s & torch.isfinite(b), b, 0.0).max())
        # D products summed, the score's roundings, and of a small cap the u's
        self.e_s = q.shape[-1] * R.F32R * float(mag.max()) + 16 * R.F32R * (big + 8) \
            + 8 * R.F32R * min(cap, U_CAP)


def distill(z, idx, val, tau, tlse=None, w=None, grad_scale=1.0):
    """As ops_ref.distill, in logarithms throughout, so that the outside of the entries may
    be any size.  The statistics' second number is c = 1 - pT / qT down to -2^24, and
    log(pT / qT) beyond.  Distinct entries; every row has weight and an entry."""
    N, V = z.shape
    x = z.double() / tau
    ok = (idx >= 0) & (idx < V)
    at = torch.where(ok, idx, 0).long()
    t = torch.where(ok, val.double() / tau, -math.inf)
    base = torch.logsumexp(t, 1) if tlse is None else tlse.double()
    logp = t - base[:, None]
    p = torch.exp(logp)
    lse = torch.logsumexp(x, 1)
    logq = x - lse[:, None]
    loss = torch.where(p > 0, p * (logp - logq.gather(1, at)), 0.0).sum(1)
    member = torch.zeros(N, V + 1, dtype=torch.bool).scatter_(1, torch.where(ok, at, V), True)[:, :V]
    # pT / qT of the gradient outside, and what of it the statistics hold
    logr = torch.full_like(lse, -math.inf)
    if tlse is not None:
        tail = (1 - p.sum(1)).clamp_min(0)
        logout = torch.logsumexp(torch.where(member, -math.inf, logq), 1)
        dust = (1 + tlse.double().abs()) * 2.0 ** -23      # of teacher_lse's rounding
        tail = torch.where(member.all(1) | (torch.isinf(logout) & (tail <= dust)), 0.0, tail)
        loss = loss + torch.where(tail > 0, tail * (torch.log(tail) - logout), 0.0)
        logr = torch.where(tail > 0, torch.log(tail) - logout, -math.inf)
    wd = torch.ones(N, dtype=torch.float64) if w is None else w.double()
    far = logr > math.log(2.0 ** 24)
    second = torch.where(far, logr, 1 - torch.exp(torch.where(far, 0.0, logr)))
    q = torch.exp(logq)
    share = torch.where(member, 0.0, torch.exp(logq + logr[:, None]))      # pT of each outside
    share = torch.where(torch.isinf(logq), 0.0, share)
    add = torch.zeros(N, V + 1, dtype=torch.float64).scatter_add_(1, torch.where(ok, at, V), p)[:, :V]
    sc = (grad_scale * tau * wd)[:, None]
    dz = (q - share - add) * sc
    loss = loss * tau * tau * wd
    # errors: a sum's roundings and those of its terms' exponents (terms 2^-25 below the
    # largest count for nothing); exponents of the gradient's terms, of binary32 statistics
    e = (V / 256 + 64 + 50) * R.F32R
    fin = x[torch.isfinite(x)]
    top = float(fin.abs().max())
    reach = float(lse.abs().max()) + float(logr[torch.isfinite(logr)].abs().max()
                                           if bool(torch.isfinite(logr).any()) else 0.0)
    eq = 8 * R.F32R * (2 * top + 8 + reach)
    e_second = torch.where(far, 4 * e + 4 * R.F32R * second.abs(),
                           (1 - second).abs() * 4 * e + 4 * R.F32R * (1 + second.abs()))
    h = R.half_step(z.dtype)
    e_dz = h * dz.abs() + sc.abs() * ((q + share) * 1.02 * (eq + 8 * e) + 16 * R.F32R * add) + 1e-30
    return {"loss": (loss, tau * tau * wd * 4 * e + 4 * R.F32R * loss.abs() + 1e-30),
            "stats": (torch.stack([lse, second], 1),
                      torch.stack([e + 4 * R.F32R * lse.abs(), e_second], 1) + 1e-30),
            "dz": (dz, e_dz)}
