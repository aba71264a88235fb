"""The operators around a student's blocks on the GPU where test_gpu_ops_block does not reach:
arrays that lie between one another, the ends of binary32, long sums of one sign."""
import math

import pytest

import ops_block_ref as B
import ops_ref as R
from gpu_util import gpu_or_skip
from test_gpu_ops_block import _gen, _rand, _same, _types, _ws

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def zs():
    gpu_or_skip()
    import zero_sharded_mixed_step_amd as zs
    zs.ops_lib()
    return zs


@pytest.fixture(scope="module")
def torch():
    return gpu_or_skip()


@pytest.mark.parametrize("T,C", [(1, 64), (37, 64), (300, 1000)])
def test_columns_of_one_buffer(zs, torch, T, C):
    """Inputs and outputs that are columns of one buffer, or its rows in turn, are apart: the same
    bits as in buffers of their own."""
    bf = torch.bfloat16
    g = _gen(torch, T)
    x, y, dh, dz, d = (_rand(torch, g, (T, C), bf).cuda() for _ in range(5))
    w = _rand(torch, g, (C,), bf, 0.3).cuda()
    ids = torch.randint(-1, T, (T,), generator=g, dtype=torch.int32).cuda()
    kw = dict(post_norm=True, post_weight=w, gate=w, pre_weight=w)
    ws = _ws(torch, max(zs.zero_block_norm_workspace_bytes(T, C), zs.zero_embed_workspace_bytes(T, C)))[0]

    def run(x, y, dh, dz, d, h, z, dx, dy, dt):
        zs.zero_block_norm_fwd(x, y, h, z, **kw)
        zs.zero_block_norm_bwd(y, h, dh, dz, dx, dy, **kw)
        zs.zero_embed_bwd(ids, d, dt, workspace=ws)
        return h, z, dx, dy, dt

    want = run(x, y, dh, dz, d, *(torch.empty_like(x) for _ in range(5)))
    columns = torch.full((T, 10 * C), math.nan, dtype=bf, device="cuda").view(T, 10, C).unbind(1)
    turns = torch.full((T, 10, C), math.nan, dtype=bf, device="cuda").unbind(1)
    for v in (columns, turns):
        for to, of in zip(v, (x, y, dh, dz, d)):
            to.copy_(of)
        for a, b in zip(run(*v), want):
            assert _same(a, b)


def _ends(torch, g, T, C, dtype, size):
    """Rows 0 and 2 of about `size`, the others ordinary."""
    x = torch.randn(T, C, generator=g).clamp(-2, 2)
    x[0::2] *= size
    return x.to(dtype)


@pytest.mark.parametrize("C", [64, 1000, 2048, 4096, 8192, 16384])
@pytest.mark.parametrize("types", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")], ids=str)
@pytest.mark.parametrize("size", [2.0 ** -126, 2.0 ** -128, 2.0 ** -130, 2.0 ** -140, 1.2e38])
def test_block_norm_rows_at_the_ends(zs, torch, C, types, size):
    """Rows whose inverse root is past binary32's ends, from subnormal values to the largest: normed as
    any other, and so are their gradients.  (Bounds: every row's own; the powers of 2 round nothing.)"""
    dt, rt = _types(torch, *types)
    if size < 2.0 ** -133 and (dt, rt) != (torch.float32, torch.float32):
        size = 2.0 ** -131                     # (bf16's smallest number is 2^-133)
    T, g = 3, _gen(torch, C)
    small = size < 1.0
    ws, behind = _ws(torch, zs.zero_block_norm_workspace_bytes(T, C))
    w1, w2, gate_c = (_rand(torch, g, (C,), dt, 0.5) for _ in range(3))
    dz = _rand(torch, g, (T, C), dt, 2.0 ** -60 if small else 1.0)
    dh = _rand(torch, g, (T, C), rt, 2.0 ** 60 if small else 1.0)

    def both(x, y, post, gate, branch, dh):
        ref = B.Block(x, y, post=post, w1=w1 if post else None, gate=gate, w2=w2, branch=branch, eps=0.0, dt=dt)
        d = [None if t is None else t.cuda() for t in (x, y, w1 if post else None, gate, w2, dh, dz)]
        kw = dict(post_norm=post, post_weight=d[2], gate=d[3], pre_weight=d[4], branch_scale=branch, eps=0.0)
        h = torch.full((T, C), math.nan, dtype=rt, device="cuda")
        z = torch.full((T, C), math.nan, dtype=dt, device="cuda")
        zs.zero_block_norm_fwd(d[0], d[1], h, z, **kw)
        want = ref.forward(True)
        R.check("h", h, *want["h"])
        R.check("z", z, *want["z"])
        assert bool(torch.isfinite(z).all())
        got = dict(dx=torch.full_like(h, math.nan), dw2=torch.full_like(d[4], math.nan))
        if y is not None:
            got.update(dy=torch.full_like(z, math.nan), dw1=torch.full_like(d[4], math.nan),
                       dgate=torch.full_like(d[3], math.nan))
        zs.zero_block_norm_bwd(d[1], h, d[5], d[6], got["dx"], got.get("dy"), dpost_weight=got.get("dw1"),
                               dgate=got.get("dgate"), dpre_weight=got["dw2"], workspace=ws, **kw)
        want = ref.backward(h.cpu(), dh, dz)
        for n, t in got.items():
            assert bool(torch.isfinite(t).all()), n
            R.check(n, t, *want[n])

    # the stream itself is at the end; then a block's output that is normed into an ordinary stream
    both(_ends(torch, g, T, C, rt, size), None, False, None, 1.0, dh)
    for gate in (gate_c, _rand(torch, g, (T, C), dt, 0.5)):
        both(_rand(torch, g, (T, C), rt), _ends(torch, g, T, C, dt, size), True, gate,
             2.0 ** -60 if small else 1.0, _rand(torch, g, (T, C), rt))
    assert bool((behind == 0xFF).all())


# |lse| up to which the backward's probabilities are formed from it, beyond from the token's logit
FAR_LSE = {"f32": 32.0, "bf16": 2048.0}


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V,tau", [(300, 1.0), (20011, 0.7)])
@pytest.mark.parametrize("centre", [0.0, 20.0, -25.0, 45.0, 1000.0, -3000.0, 30000.0, -60000.0, 65000.0, 4e6])
def test_policy_gradients_keep_their_digits_far_from_0(zs, torch, dtype, V, tau, centre):
    """A row's gradient depends on differences of its logits alone: the forward's is as good wherever the
    row lies, the backward's but for the rounding of the statistic that it is formed from."""
    dt, = _types(torch, dtype)
    g, N, F = _gen(torch, V + int(abs(centre))), 8, R.F32R
    z = ((torch.randn(N, V, generator=g) * 2 + centre) * tau).to(dt)
    act = torch.randint(0, V, (N,), generator=g, dtype=torch.int32)
    act[:2] = z[:2].float().argmax(1).to(torch.int32)
    z[2, act[2]] = (centre - 40.0) * tau                       # a token of little probability
    adv = torch.tensor([1.0, -0.5, 2.0, 0.7, -1.0, 1.5, -2.0, 0.3])
    x = z.double() / tau
    lse = torch.logsumexp(x, 1)
    lp = x.gather(1, act.long()[:, None])[:, 0] - lse
    old, ref = (lp - 0.05).float(), (lp + 0.3).float()
    kw = dict(tau=tau, old=old, ref=ref, kl_coef=0.1, grad_scale=0.5)
    want = B.policy(z, act, adv, **kw)
    assert want["near"] == 0
    d = [t.cuda() for t in (z, act, adv, old, ref)]
    loss, stats = torch.empty(N, device="cuda"), torch.empty(N, 4, device="cuda")
    dz, back, place = torch.empty_like(d[0]), torch.empty_like(d[0]), d[0].clone()
    bkw = dict(grad_scale=0.5, temperature=tau)
    zs.zero_policy_fwd(*d[:3], loss, stats, dlogits=dz, old_logp=d[3], ref_logp=d[4], kl_coef=0.1, **bkw)
    zs.zero_policy_bwd(d[0], d[1], stats, back, **bkw)
    zs.zero_policy_bwd(place, d[1], stats, place, **bkw)
    assert _same(back, place)
    # Errors of q, relative: of the row's sum (as in ops_block_ref); of an exponent, which is below
    # `span` and takes three roundings and those of 1 / tau and log2 e; of the power and three products.
    span = (x.max(1, keepdim=True).values - x).clamp(max=100.0)
    e = (V / 256 + 64) * F + 4 * F * span.max(1, keepdim=True).values
    q, one = torch.exp(x - lse[:, None]), torch.zeros_like(x).scatter_(1, act.long()[:, None], 1.0)
    val, g_row, g_off = want["dz"][0], want["stats"][0][:, 2:3].abs(), want["stats"][1][:, 2:3]

    def bound(eq):
        off = g_row * (q * eq + one * (1 - q) * 6 * (e + F)) + g_off * (one - q).abs()
        return R.half_step(dt) * val.abs() + 1.02 * 0.5 / tau * off + B.TINY

    R.check("dz", dz, val, bound(F * (6 * span + 16) + e))
    # Backward besides: lse's or lp's own rounding, and of the exponent's parts that are as large
    # (z / tau, or the difference from the token's logit, twice).
    far = (lse.abs() > FAR_LSE[dtype]) & (lp.abs() < lse.abs())
    large = torch.where(far, lp.abs(), lse.abs())[:, None]
    arg = (x - lse[:, None]).abs().clamp(max=200.0)
    R.check("dz of the backward", back, val, bound(F * (3 * large + 6 * arg + 16) + e))


@pytest.mark.parametrize("C", [64, 1000, 4096])
@pytest.mark.parametrize("T", [20011, 262144])
def test_block_norm_sums_of_one_sign(zs, torch, T, C):
    """Weights' and gate's gradients whose terms all have one sign.  A thread adds the rows of its
    workgroup that it walks, of 256 workgroups at least and up to four rows of each at a time; then come
    four rows' parts, 32 workgroups' in order and 16 waves'."""
    T = min(T, (1 << 25) // C)
    F, f32 = R.F32R, torch.float32
    g = torch.Generator(device="cuda")
    g.manual_seed(C)
    r = lambda *s: torch.rand(*s, generator=g, device="cuda") + 0.25
    y, h, dh, dz, w, gate = r(T, C), r(T, C), r(T, C), r(T, C), r(C), r(C)
    dw1, dgate, dw2 = (torch.full((C,), math.nan, device="cuda") for _ in range(3))
    ws = torch.empty(zs.zero_block_norm_workspace_bytes(T, C), dtype=torch.uint8, device="cuda")
    kw = dict(post_norm=True, post_weight=w, gate=gate, eps=0.0, workspace=ws)
    zs.zero_block_norm_bwd(y, None, dh, None, None, None, dpost_weight=dw1, dgate=dgate, **kw)
    zs.zero_block_norm_bwd(None, h, None, dz, dh, None, pre_weight=w, dpre_weight=dw2, eps=0.0, workspace=ws)
    # (in pieces: 64-bit copies of everything would be 16 times as large)
    t = torch.zeros(C, dtype=torch.float64, device="cuda")
    s = t.clone()
    g.manual_seed(C)
    y, h, dh = r(T, C), r(T, C), r(T, C)
    for i in range(0, T, 16384):
        a, b = y[i:i + 16384].double(), h[i:i + 16384].double()
        t += (dh[i:i + 16384].double() * a / a.square().mean(1, keepdim=True).sqrt()).sum(0)
        s += (dz[i:i + 16384].double() * b / b.square().mean(1, keepdim=True).sqrt()).sum(0)
    chain = T / (256 * (4 if C <= 1024 else 1)) + 1 + 4 + 32 + 16
    for name, got, want in (("dw1", dw1, t * gate.double()), ("dgate", dgate, t * w.double()), ("dw2", dw2, s)):
        off = float(((got.double() - want) / want).abs().max())
        assert off <= (chain + 10) * F + B.E_ROOT, (name, off / F, chain)


@pytest.mark.parametrize("grad", ["f32", "bf16"])
@pytest.mark.parametrize("N", [300, 16390, 1 << 17, 1 << 20])
def test_embed_sums_of_one_sign(zs, torch, N, grad):
    """All tokens one row, all terms of one sign: 64 places of a chunk in order at most, every 16th
    of the chunks', the 16 waves'."""
    gt, = _types(torch, grad)
    g = torch.Generator(device="cuda")
    g.manual_seed(N)
    C = 24
    d = torch.rand(N, C, generator=g, device="cuda") + 0.25
    ids = torch.full((N,), 2, dtype=torch.int32, device="cuda")
    got = torch.full((5, C), math.nan, dtype=gt, device="cuda")
    zs.zero_embed_bwd(ids, d, got, workspace=_ws(torch, zs.zero_embed_workspace_bytes(N, C))[0])
    want = d.double().sum(0)
    places = max(4, min(64, (N + 255) // 256))
    chain = places + N / places / 16 + 1 + 16
    off = float(((got[2].double() - want) / want).abs().max())
    assert off <= (chain + 3) * R.F32R + R.half_step(gt), (off / R.F32R, chain)
    assert bool((got[[0, 1, 3, 4]] == 0).all())
