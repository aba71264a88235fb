"""Bounds for the ends of the operators' ranges, beside ops_ref's: the error of a
capped score by the score's size and not by the cap's."""
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
