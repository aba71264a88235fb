"""The norm of heads on the GPU for rows whose inverse root is past binary32's ends, against its
formula in 64 bits."""
import math

import pytest

import ops_ref as R
from gpu_util import gpu_or_skip

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D", [32, 64, 96, 128, 256])
@pytest.mark.parametrize("size", [2.0 ** -126, 2.0 ** -128, 2.0 ** -131, 2.0 ** -140, 1.2e38])
def test_norm_of_heads_at_the_ends(size, D, dtype):
    """Beside ordinary rows, heads of subnormal values and of the largest, without eps: normed as any
    other, and so are the gradients."""
    torch = gpu_or_skip()
    import zero_sharded_mixed_step_amd as zs
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    if dt == torch.bfloat16:
        size = max(size, 2.0 ** -131)          # (its smallest number is 2^-133)
    g = torch.Generator()
    g.manual_seed(D)
    T, H = 7, 3
    x = torch.randn(T, H, D, generator=g).clamp(-2, 2)
    x[1::2] *= size
    x[0, 1] *= size
    x = x.to(dt)
    dy = (torch.randn(T, H, D, generator=g) * (2.0 ** -60 if size < 1 else 1.0)).to(dt)
    w = torch.randn(D, generator=g).to(dt)
    pos, freq = torch.randint(0, 1000, (T,), generator=g, dtype=torch.int32), zs.rope_inv_freq(D)
    kw = dict(wq=w.cuda(), eps=0.0, pos=pos.cuda(), inv_freq=freq.cuda())
    y, dx = torch.full_like(x, math.nan).cuda(), torch.full_like(x, math.nan).cuda()
    dw = torch.full_like(w, math.nan).cuda()
    ws = torch.empty(zs.zero_qk_norm_rope_workspace_bytes(T, D), dtype=torch.uint8, device="cuda")
    zs.zero_qk_norm_rope_fwd(x.cuda(), None, y, None, **kw)
    assert bool(torch.isfinite(y).all())
    R.check("y", y, *R.norm_forward(x, w, 0.0, pos, freq, False))
    zs.zero_qk_norm_rope_bwd(x.cuda(), None, dy.cuda(), None, dx, None, dwq=dw, workspace=ws, **kw)
    want = R.norm_backward(x, w, dy, 0.0, pos, freq, False)
    assert bool(torch.isfinite(dx).all() and torch.isfinite(dw).all())
    value, bound = want["dx"]
    # (gradients near the smallest numbers are off by those' steps)
    R.check("dx", dx, value, bound + 2.0 ** -126 * (R.half_step(dt) if dt == torch.float32 else 2.0 ** -7))
    R.check("dw", dw, *want["dw"])
