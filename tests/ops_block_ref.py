"""The operators around a student's blocks in 64 bits on the host, straight from
their formulas, with bounds on what a kernel of 32-bit sums and one rounding of every
output may differ by.  F is an fp32 rounding, half_step that of an output."""
import math

import torch

from ops_ref import F32R as F
from ops_ref import half_step

TINY = 1e-30


# -------------------------------------------------------------- embedding ---

def embed_forward(table, ids, scale):
    """out and its bound: one product, one rounding."""
    V = table.shape[0]
    ok = (ids >= 0) & (ids < V)
    rows = table.double()[torch.where(ok, ids, 0).long()] * scale
    out = torch.where(ok[:, None], rows, 0.0)
    return out, (half_step(table.dtype) + 2 * F) * out.abs() + TINY


def embed_backward(ids, dout, V, scale, base, grad_dtype):
    """dtable and its bound: as many additions as the row has terms, in any order,
    the product, the base's addition, one rounding."""
    ok = (ids >= 0) & (ids < V)
    at, d = ids[ok].long(), dout.double()[ok]
    out = torch.zeros(V, dout.shape[1], dtype=torch.float64)
    mag, n = out.clone(), torch.zeros(V, dtype=torch.float64)
    out.index_add_(0, at, d)
    mag.index_add_(0, at, d.abs())
    n.index_add_(0, at, torch.ones(at.shape[0], dtype=torch.float64))
    val = out * scale + (0.0 if base is None else base.double())
    e = (n[:, None] + 3) * F * mag * abs(scale) + 2 * F * val.abs()
    return val, half_step(grad_dtype) * val.abs() + 1.02 * e + TINY


# ------------------------------------------------------ norms round a block ---

# Of a row's sum of squares: 16 products a thread at most, then 10 joins; half of it in the
# root, whose own rounding, argument and product add 5.
E_ROOT = 18 * F


def _root(v, eps):
    return 1 / torch.sqrt((v * v).mean(-1, keepdim=True) + eps)


def _weight(w, offset):
    return 1.0 if w is None else w.double() + offset


class Block:
    """One call: inputs as tensors or None, numbers as the operator takes them."""

    def __init__(self, x, y, *, post=False, w1=None, gate=None, w2=None, offset=0.0, res=1.0,
                 branch=1.0, eps=1e-6, dt=None):
        self.x, self.rt, self.eps = x.double(), x.dtype, eps
        self.dt = dt or (x.dtype if y is None else y.dtype)
        self.y = None if y is None else y.double()
        self.post, self.res, self.branch = post, res, branch
        self.w1, self.w2, self.offset = w1, w2, offset
        self.g = branch * (1.0 if gate is None else gate.double())
        self.gate = gate
        if y is not None:
            self.r1 = _root(self.y, eps) if post else torch.ones(x.shape[0], 1, dtype=torch.float64)
            self.k1 = _weight(w1, offset) if post else 1.0
            self.u = self.y * self.r1 * self.k1

    def forward(self, want_z):
        h = self.res * self.x
        e = 2 * F * h.abs()
        if self.y is not None:
            part = self.g * self.u
            h = h + part
            e = e + (E_ROOT + 8 * F) * part.abs() + 2 * F * h.abs()
        out = {"h": (h, half_step(self.rt) * h.abs() + 1.02 * e + TINY)}
        if want_z:
            r = _root(h, self.eps)
            z = h * r * _weight(self.w2, self.offset)
            moved = torch.sqrt((e * e).mean(-1, keepdim=True)) * r
            ez = (z / h).nan_to_num(0.0).abs() * e + z.abs() * (E_ROOT + 6 * F + moved)
            out["z"] = (z, half_step(self.dt) * z.abs() + 1.02 * ez + TINY)
        return out

    def backward(self, h, dh, dz):
        """{name: (value, bound)} from the forward's stored h."""
        C, T = self.x.shape[1], self.x.shape[0]
        out, gh = {}, torch.zeros_like(self.x) if dh is None else dh.double()
        size = gh.abs()
        hd, hr = half_step(self.dt), half_step(self.rt)
        if dz is not None:
            h, dz = h.double(), dz.double()
            r = _root(h, self.eps)
            hh, u2 = h * r, dz * _weight(self.w2, self.offset)
            gh = gh + r * (u2 - hh * (u2 * hh).mean(-1, keepdim=True))
            size = size + r * (u2.abs() + hh.abs() * (u2 * hh).abs().mean(-1, keepdim=True))
            out["dw2"] = self._sum(dz * hh, (E_ROOT + 4 * F) * (dz * hh).abs(), T, hd)
        # two roots' errors, the mean's 26 joins and products, a few roundings of the parts
        e = (3 * E_ROOT + 40 * F) * size
        out["dx"] = (self.res * gh, hr * (self.res * gh).abs() + 1.02 * abs(self.res) * e + TINY)
        if self.y is None:
            return out
        if self.gate is not None:
            d = self.branch * gh * self.u
            ed = abs(self.branch) * self.u.abs() * e + (E_ROOT + 8 * F) * d.abs()
            out["dgate"] = self._sum(d, ed, T, hd) if self.gate.dim() == 1 \
                else (d, hd * d.abs() + 1.02 * ed + TINY)
        du = self.g * gh
        eu = abs(self.g) * e if isinstance(self.g, float) else self.g.abs() * e
        eu = eu + 4 * F * du.abs()
        if self.post:
            yy = self.y * self.r1
            out["dw1"] = self._sum(du * yy, eu * yy.abs() + (E_ROOT + 4 * F) * (du * yy).abs(), T, hd)
            v = du * self.k1
            ev = eu * (abs(self.k1) if isinstance(self.k1, float) else self.k1.abs()) + 3 * F * v.abs()
            du = self.r1 * (v - yy * (v * yy).mean(-1, keepdim=True))
            size = v.abs() + yy.abs() * (v * yy).abs().mean(-1, keepdim=True)
            eu = self.r1 * (ev + yy.abs() * (ev * yy.abs()).mean(-1, keepdim=True)
                            + (3 * E_ROOT + 40 * F) * size)
        out["dy"] = (du, hd * du.abs() + 1.02 * eu + TINY)
        return out

    @staticmethod
    def _sum(terms, e, T, half):
        """Summed over the tokens: at most T additions and 40 joins."""
        val = terms.sum(0)
        return val, half * val.abs() + 1.02 * (e.sum(0) + (T + 40) * F * terms.abs().sum(0)) + TINY


# ------------------------------------------------------------ policy loss ---

def policy(z, action, adv, *, tau=1.0, old=None, ref=None, w=None, lo=0.2, hi=0.2, kl_coef=0.0,
           grad_scale=1.0):
    """{loss, stats, dz: (value, bound)}; rows whose ratio is next to a border of the
    clipping, where a rounding decides, are counted in "near"."""
    N, V = z.shape
    x = z.double() / tau
    lse = torch.logsumexp(x, 1)
    named = (action >= 0) & (action < V)
    empty = torch.isinf(lse) & (lse < 0)
    live = named & ~empty
    at = torch.where(named, action, 0).long()[:, None]
    lp = torch.where(live, x.gather(1, at)[:, 0] - torch.where(empty, 0.0, lse), 0.0)
    A = adv.double()
    r = torch.exp(lp - old.double()) if old is not None else torch.ones_like(lp)
    free, held = r * A, r.clamp(1 - lo, 1 + hi) * A
    loss = -torch.minimum(free, held)
    clipped = ((A > 0) & (r > 1 + hi)) | ((A < 0) & (r < 1 - lo))
    g = torch.where(clipped, 0.0, -free)
    kl, ev = torch.zeros_like(lp), torch.zeros_like(lp)
    if ref is not None:
        ev = ref.double() - lp
        kl = torch.expm1(ev) - ev
        loss = loss + kl_coef * kl
        g = g - kl_coef * torch.expm1(ev)
    wd = torch.ones(N, dtype=torch.float64) if w is None else w.double()
    on = live & (wd != 0)
    q = torch.exp(x - lse[:, None]).nan_to_num(0.0)
    one = torch.zeros_like(q).scatter_(1, at, 1.0)
    sc = grad_scale * wd / tau
    dz = torch.where(on[:, None] & (g != 0)[:, None], (one - q) * (sc * g)[:, None], 0.0)
    # errors: the sum of the powers (a thread's share of the row in order, their exponents),
    # which is lp's; what lp's error does to the rest; the products' roundings
    fin = x[torch.isfinite(x)]
    span = float(fin.max() - fin.min()) if fin.numel() else 0.0
    top = float(fin.abs().max()) if fin.numel() else 0.0
    e = (V / 256 + 64) * F + 4 * F * min(span, 100.0)
    qa = torch.where(live, torch.exp(lp), 0.0)
    e_lp = e * (1 - qa).clamp_min(0) + 1e-11
    soft = torch.where(clipped, 0.0, free.abs()) + abs(kl_coef) * torch.expm1(ev).abs()
    e_g = (free.abs() * ~clipped + abs(kl_coef) * torch.exp(ev)) * e_lp * 1.1 + 2 * F * g.abs()
    out = {}
    out["loss"] = (torch.where(on, loss * wd, 0.0),
                   wd.abs() * (soft * e_lp * 1.1) + 4 * F * (loss * wd).abs() + 1e-11)
    stats = torch.stack([lse, lp, torch.where(live, g, 0.0), torch.where(live, kl, 0.0)], 1)
    bound = torch.stack([e + 2 * F * lse.abs().nan_to_num(0.0, posinf=0.0), e_lp + 2 * F * lp.abs(),
                         e_g, torch.expm1(ev).abs() * e_lp * 1.1 + 4 * F * kl], 1)
    out["stats"] = (stats, bound + 1e-11)
    eq = 8 * F * (2 * top + 8 + lse.abs().nan_to_num(0.0, posinf=0.0))[:, None] + 2 * e
    e_dz = sc.abs()[:, None] * (g.abs()[:, None] * (q * eq + one * (1 - qa)[:, None] * 6 * (e + F))
                                + e_g[:, None] * (one - q).abs())
    out["dz"] = (dz, half_step(z.dtype) * dz.abs() + 1.02 * torch.where(on[:, None], e_dz, 0.0) + TINY)
    near = ((r - (1 - lo)).abs() < 1e-4) | ((r - (1 + hi)).abs() < 1e-4)
    out["near"] = int((near & live).sum())
    return out
