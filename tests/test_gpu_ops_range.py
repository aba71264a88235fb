"""The training operators at the ends of what they accept: large and tiny caps, empty
batches, rows that a teacher is sure of, infinities in masked places, and the paths
that only larger shapes take."""
import math

import pytest

import ops_ref as R
import ops_range_ref as X
from gpu_util import gpu_or_skip

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


def _gen(torch, seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


def _rand(torch, g, shape, dtype, scale=1.0):
    return (torch.randn(shape, generator=g) * scale).to(dtype)


def _attn_inputs(torch, B, Tq, Tk, Hq, Hk, D, seed, qscale=2.0):
    g = _gen(torch, seed)
    bf = torch.bfloat16
    return [_rand(torch, g, (B, Tq, Hq, D), bf, qscale), _rand(torch, g, (B, Tk, Hk, D), bf),
            _rand(torch, g, (B, Tk, Hk, D), bf), _rand(torch, g, (B, Tq, Hq, D), bf)]


def _attn(zs, torch, q, k, v, do, table=None, **kw):
    """o, lse and the gradients {name: tensor} of one call of each direction."""
    B, Tq, Hq, D = q.shape
    n = 0 if table is None else table.shape[0]
    ws = [torch.full((max(16, zs.zero_attn_workspace_bytes(B, Tq, k.shape[1], Hq, k.shape[2], D, n, b)),),
                     0x7F, dtype=torch.uint8, device="cuda") for b in (False, True)]
    o = torch.full_like(q, math.nan)
    lse = torch.full((B, Hq, Tq), math.nan, dtype=torch.float32, device="cuda")
    zs.zero_attn_fwd(q, k, v, o, lse, bias_table=table, workspace=ws[0], **kw)
    g = {name: torch.full_like(x, math.nan) for name, x in (("dv", v), ("dk", k), ("dq", q))}
    if table is not None:
        g["dtable"] = torch.full_like(table, math.nan)
    zs.zero_attn_bwd(q, k, v, o, lse, do, g["dq"], g["dk"], g["dv"], dbias_table=g.get("dtable"),
                     bias_table=table, workspace=ws[1], **kw)
    return o, lse, g


def _attn_check(zs, torch, q, k, v, do, *, scale=None, cap=0.0, ranges=None, causal=False, table=None,
                buckets=None, ref=X.Attention):
    """Both directions against the 64-bit formula."""
    scale = q.shape[-1] ** -0.5 if scale is None else scale
    seen = R.visible(q.shape[0], q.shape[1], k.shape[1], ranges, causal)
    want = ref(q, k, v, scale=scale, cap=cap, seen=seen, table=table, buckets=buckets)
    dev = lambda t: None if t is None else t.cuda()
    o, lse, g = _attn(zs, torch, *(dev(t) for t in (q, k, v, do)), dev(table), scale=scale, cap=cap,
                      ranges=dev(ranges), causal=causal, bias_buckets=dev(buckets))
    want_o, bound_o, want_l, bound_l = want.forward()
    R.check("lse", lse, want_l, bound_l)
    R.check("o", o, want_o, bound_o)
    grads = want.backward(o.cpu(), do)
    for name, got in g.items():
        R.check(name, got, *grads[name])


# -------------------------------------------------------------------- caps ---

@pytest.mark.parametrize("cap", [50.0, 64.0, 65.0, 1e3, 1e5, 1e6, 1e9, 1e30])
@pytest.mark.parametrize("D,bias", [(64, False), (64, True), (128, False), (128, True), (96, True),
                                    (32, False)])
def test_attention_caps_of_any_size(zs, torch, D, bias, cap):
    """A cap far above the scores leaves them as they are."""
    q, k, v, do = _attn_inputs(torch, 1, 140, 140, 4, 2, D, seed=D)
    table = buckets = None
    if bias:
        table = _rand(torch, _gen(torch, 3), (8, 4), torch.float32)
        buckets = zs.relpos_buckets(8, 20)
    _attn_check(zs, torch, q, k, v, do, causal=True, cap=cap, table=table, buckets=buckets)


@pytest.mark.parametrize("cap", [100.0, 2000.0])
def test_attention_caps_beside_large_scores(zs, torch, cap):
    """Scores on both sides of the place where the tanh's two forms meet, and past the cap."""
    q, k, v, do = _attn_inputs(torch, 1, 150, 150, 2, 2, 64, seed=12, qscale=60.0)
    _attn_check(zs, torch, q, k, v, do, causal=True, cap=cap)


def test_attention_split_keys_large_cap(zs, torch):
    q, k, v, do = _attn_inputs(torch, 1, 3, 2500, 2, 2, 64, seed=8)
    assert zs.zero_attn_workspace_bytes(1, 3, 2500, 2, 2, 64) > 0
    _attn_check(zs, torch, q, k, v, do, causal=True, cap=1e6)


@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("cap", [1e-10, 1e-40])
def test_attention_tiny_caps(zs, torch, cap, bias):
    """Scores that a cap takes to nothing: the softmax of the bias alone; a score of
    exactly 0 stays one."""
    q, k, v, do = _attn_inputs(torch, 1, 70, 70, 2, 2, 64, seed=4)
    q[:, 5] = 0
    table = buckets = None
    if bias:
        table = _rand(torch, _gen(torch, 3), (8, 2), torch.float32)
        buckets = zs.relpos_buckets(8, 20)
    dev = lambda t: None if t is None else t.cuda()
    o, lse, g = _attn(zs, torch, *(dev(t) for t in (q, k, v, do)), dev(table), scale=0.125, cap=cap,
                      causal=True, bias_buckets=dev(buckets))
    seen = R.visible(1, 70, 70, causal=True)
    want = X.Attention(torch.zeros_like(q), k, v, scale=0.125, seen=seen, table=table, buckets=buckets)
    want_o, bound_o, want_l, bound_l = want.forward()
    R.check("lse", lse, want_l, bound_l)
    R.check("o", o, want_o, bound_o)
    grads = want.backward(o.cpu(), do)
    R.check("dv", g["dv"], *grads["dv"])
    if bias:
        R.check("dtable", g["dtable"], *grads["dtable"])
    for name in ("dq", "dk"):
        assert bool(torch.isfinite(g[name]).all()), name


def test_attention_sum_of_many_equal_weights(zs, torch):
    """2^17 keys of one weight, 0.7 of the largest: sums whose roundings all go one way."""
    T, Tq, H, D = 1 << 17, 129, 160, 32
    bf = torch.bfloat16
    q = torch.zeros(1, Tq, H, D, device="cuda", dtype=bf)
    q[..., 0] = 1
    k = torch.zeros(1, T, 1, D, device="cuda", dtype=bf)
    k[0, 0, 0, 0] = 0.357
    v = torch.ones(1, T, 1, D, device="cuda", dtype=bf)
    o, lse = torch.empty_like(q), torch.empty(1, H, Tq, device="cuda")
    assert zs.zero_attn_workspace_bytes(1, Tq, T, H, 1, D) == 0              # (not split)
    zs.zero_attn_fwd(q, k, v, o, lse, scale=1.0)
    want = math.log(math.exp(float(k[0, 0, 0, 0])) + T - 1)
    # a lane takes 32 of a tile's 64 keys: 32 + 2048 sums, and the score's own roundings
    bound = (32 + T / 64) * R.F32R + 32 * R.F32R + 4 * R.F32R * want
    assert float((lse.double() - want).abs().max()) <= bound
    # the products' sums: 4 of 16 keys a tile
    assert float((o.double() - 1).abs().max()) <= 2 * R.BF + 4 * T / 64 * R.F32R


# ----------------------------------------------------------- empty batches ---

@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,Tq,Tk", [(0, 5, 5), (2, 0, 0), (0, 0, 0), (2, 0, 5), (2, 5, 0)])
def test_attention_bias_gradient_of_an_empty_batch(zs, torch, B, Tq, Tk, dtype):
    """The sum over nothing is 0, and is written."""
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    bf = torch.bfloat16
    q = torch.ones(B, Tq, 4, 64, device="cuda", dtype=bf)
    k = torch.ones(B, Tk, 2, 64, device="cuda", dtype=bf)
    o, lse = torch.zeros_like(q), torch.full((B, 4, Tq), -math.inf, device="cuda")
    table = torch.ones(8, 4, device="cuda", dtype=dt)
    dtable = torch.full_like(table, math.nan)
    gq, gk, gv = (torch.full_like(x, math.nan) for x in (q, k, k))
    ws = torch.full((max(16, zs.zero_attn_workspace_bytes(B, Tq, Tk, 4, 2, 64, 8, True)),), 0x7F,
                    dtype=torch.uint8, device="cuda")
    zs.zero_attn_bwd(q, k, k, o, lse, q, gq, gk, gv, dbias_table=dtable, bias_table=table,
                     bias_buckets=zs.relpos_buckets(8, 20, device="cuda"), workspace=ws)
    assert bool((dtable == 0).all())
    assert all(bool((x == 0).all()) for x in (gq, gk, gv))


# ----------------------------------------------- masked places, sure masks ---

@pytest.mark.parametrize("D", [64, 96, 128])
@pytest.mark.parametrize("cap", [0.0, 30.0])
def test_attention_infinite_bias_in_masked_places(zs, torch, D, cap):
    """A causal mask leaves no key ahead of its query: what the bias says there, +inf or NaN,
    has no part in either direction."""
    T = 200
    q, k, v, do = _attn_inputs(torch, 1, T, T, 2, 2, D, seed=D)
    g = _gen(torch, 6)
    table = _rand(torch, g, (4, 2), torch.float32)
    buckets = torch.tensor([1, 1, 2, 2, 0, 3, 3, 3, 3], dtype=torch.int32)     # 3: ahead
    clean = table.clone()
    clean[3] = 0
    seen = R.visible(1, T, T, causal=True)
    want = X.Attention(q, k, v, scale=D ** -0.5, cap=cap, seen=seen, table=clean, buckets=buckets)
    for value in (math.inf, -math.inf, math.nan):
        table[3] = value
        o, lse, got = _attn(zs, torch, q.cuda(), k.cuda(), v.cuda(), do.cuda(), table.cuda(),
                            scale=D ** -0.5, cap=cap, causal=True, bias_buckets=buckets.cuda())
        want_o, bound_o, want_l, bound_l = want.forward()
        R.check("lse", lse, want_l, bound_l)
        R.check("o", o, want_o, bound_o)
        grads = want.backward(o.cpu(), do)
        for name in ("dv", "dk", "dq", "dtable"):
            R.check(name, got[name], *grads[name])


@pytest.mark.parametrize("D", [64, 96, 128])
@pytest.mark.parametrize("cap", [0.0, 30.0])
def test_attention_products_past_binary32_in_masked_places(zs, torch, D, cap):
    """Documents whose products overflow with each other's rows, but not with their
    own: q . k, do . v of masked pairs."""
    T, cut = 190, 70
    q, k, v, do = _attn_inputs(torch, 1, T, T, 2, 2, D, seed=D + 1)
    big = 2.0 ** 66
    # document 0: small q and do, large k and v; document 1 the other way round
    for x, y in ((q, k), (do, v)):
        x[:, :cut] /= big
        y[:, :cut] *= big
        x[:, cut:] *= big
        y[:, cut:] /= big
    doc = torch.zeros((1, T), dtype=torch.int32)
    doc[:, cut:] = 1
    ranges = R.doc_ranges(doc)
    seen = R.visible(1, T, T, ranges)
    o, lse, got = _attn(zs, torch, q.cuda(), k.cuda(), v.cuda(), do.cuda(), scale=D ** -0.5, cap=cap,
                        ranges=ranges.cuda())
    # (bounds a document at a time: theirs are of unlike size)
    for lo, hi in ((0, cut), (cut, T)):
        one = [x[:, lo:hi] for x in (q, k, v, do)]
        part = X.Attention(*one[:3], scale=D ** -0.5, cap=cap, seen=seen[:, lo:hi, lo:hi])
        want_o, bound_o, want_l, bound_l = part.forward()
        R.check("lse", lse[:, :, lo:hi], want_l, bound_l)
        R.check("o", o[:, lo:hi], want_o, bound_o)
        grads = part.backward(o.cpu()[:, lo:hi], one[3])
        for name in ("dv", "dk", "dq"):
            R.check(name, got[name][:, lo:hi], *grads[name])


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("value", ["lowest", "-inf"])
def test_attention_backward_of_masking_biases(zs, torch, D, value):
    """A bias of the type's lowest value, or -inf, at distances beside others that are
    seen: both directions are those of a mask."""
    T = 150
    q, k, v, do = _attn_inputs(torch, 1, T, T, 2, 2, D, seed=D + 2)
    low = torch.finfo(torch.bfloat16).min if value == "lowest" else -math.inf
    table = _rand(torch, _gen(torch, 6), (4, 2), torch.bfloat16)
    buckets = torch.tensor([3, 3, 1, 0, 2, 3, 3], dtype=torch.int32)           # 3: 2 and further
    dist = torch.arange(T)[None] - torch.arange(T)[:, None]
    seen = ((dist <= 1) & (dist >= -1))[None]
    want = X.Attention(q, k, v, scale=D ** -0.5, seen=seen, table=table, buckets=buckets)
    table[3] = low
    o, lse, got = _attn(zs, torch, q.cuda(), k.cuda(), v.cuda(), do.cuda(), table.cuda(),
                        scale=D ** -0.5, bias_buckets=buckets.cuda())
    want_o, bound_o, want_l, bound_l = want.forward()
    R.check("lse", lse, want_l, bound_l)
    R.check("o", o, want_o, bound_o)
    grads = want.backward(o.cpu(), do)
    for name in ("dv", "dk", "dq"):
        R.check(name, got[name], *grads[name])
    val, bound = grads["dtable"]
    R.check("dtable", got["dtable"][:3], val[:3], bound[:3])
    assert bool((got["dtable"][3] == 0).all())


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("value", ["lowest", -1e9, -1e20])
def test_attention_rows_with_no_normaliser_left(zs, torch, D, value):
    """Queries of which every key has a bias of the type's lowest value or -1e9: their lse
    has no room for the log of a sum, and the backward pass takes them as queries
    that see nothing.  The others' gradients are as without them."""
    T = 150
    q, k, v, do = _attn_inputs(torch, 1, T, T, 2, 2, D, seed=D + 3)
    low = torch.finfo(torch.bfloat16).min if value == "lowest" else value
    table = _rand(torch, _gen(torch, 6), (3, 2), torch.bfloat16)
    table[0] = low
    buckets = torch.tensor([1, 2, 0, 1, 1], dtype=torch.int32)                 # 0: the query's own key
    seen = R.visible(1, T, T, causal=True)
    o, lse, got = _attn(zs, torch, q.cuda(), k.cuda(), v.cuda(), do.cuda(), table.cuda(),
                        scale=D ** -0.5, causal=True, bias_buckets=buckets.cuda())
    # the first query sees its own key alone; the others see what is behind them
    R.check("first", o[:, :1], v[:, :1].double(), R.BF * v[:, :1].double().abs())
    strict = seen & ~torch.eye(T, dtype=torch.bool)[None]
    want = X.Attention(q, k, v, scale=D ** -0.5, seen=strict, table=torch.where(
        torch.arange(3)[:, None] == 0, 0.0, table.float()), buckets=buckets)
    want_o, bound_o, want_l, bound_l = want.forward()
    R.check("o", o[:, 1:], want_o[:, 1:], bound_o[:, 1:])
    R.check("lse", lse[:, :, 1:], want_l[:, :, 1:], bound_l[:, :, 1:])
    grads = want.backward(o.cpu(), do)
    for name in ("dv", "dk", "dq"):
        R.check(name, got[name], *grads[name])
    val, bound = grads["dtable"]
    R.check("dtable", got["dtable"][1:], val[1:], bound[1:])
    assert bool((got["dtable"][0] == 0).all())


# ------------------------------------------- paths that larger shapes take ---

@pytest.mark.parametrize("B,T,Hq,Hk,D,cap", [
    (4, 1100, 32, 8, 128, 30.0),      # 288 groups of keys: two parts of two heads each
    (8, 1100, 16, 8, 128, 0.0),       # 576: one part of two heads
    (4, 1100, 32, 8, 64, 0.0),        # the same in one launch with the queries' kernel
    (8, 1100, 16, 8, 32, 0.0),
    (8, 1100, 16, 8, 96, 0.0)])
def test_attention_backward_of_several_heads_a_workgroup(zs, torch, B, T, Hq, Hk, D, cap):
    """Key heads that a workgroup walks for more than one query head, in documents that
    begin inside tiles.  (One batch row against the formula, the others are its copies.)"""
    q, k, v, do = _attn_inputs(torch, 1, T, T, Hq, Hk, D, seed=T + D)
    doc = torch.zeros((1, T), dtype=torch.int32)
    cuts = [0, 300, 411, 900, T - 9]
    for n, (lo, hi) in enumerate(zip(cuts, cuts[1:])):
        doc[0, lo:hi] = n
    doc[0, cuts[-1]:] = -1
    ranges = R.doc_ranges(doc)
    all_ = [x.expand(B, *x.shape[1:]).contiguous().cuda() for x in (q, k, v, do)]
    o, lse, got = _attn(zs, torch, *all_, cap=cap,
                        ranges=ranges.expand(B, T, 2).contiguous().cuda())
    for name, x in [("o", o), ("lse", lse)] + list(got.items()):
        assert all(torch.equal(x[0], x[b]) for b in range(1, B)), name
    # the formula a few key heads at a time (64 bits on the host)
    G = Hq // Hk
    seen = R.visible(1, T, T, ranges)
    for hk in (0, Hk - 1):
        one = [q[:, :, hk * G:(hk + 1) * G], k[:, :, hk:hk + 1], v[:, :, hk:hk + 1],
               do[:, :, hk * G:(hk + 1) * G]]
        ref = X.Attention(*one[:3], scale=D ** -0.5, cap=cap, seen=seen)
        want_o, bound_o, _, _ = ref.forward()
        oh = o[:1, :, hk * G:(hk + 1) * G].cpu()
        R.check("o", oh, want_o, bound_o)
        grads = ref.backward(oh, one[3])
        R.check("dq", got["dq"][:1, :, hk * G:(hk + 1) * G], *grads["dq"])
        R.check("dk", got["dk"][:1, :, hk:hk + 1], *grads["dk"])
        R.check("dv", got["dv"][:1, :, hk:hk + 1], *grads["dv"])


@pytest.mark.parametrize("D,Hq,Hk", [(64, 2, 2), (64, 4, 1), (32, 2, 1), (96, 2, 2), (128, 4, 2)])
def test_attention_cap_and_bias(zs, torch, D, Hq, Hk):
    q, k, v, do = _attn_inputs(torch, 2, 210, 210, Hq, Hk, D, seed=D + Hq)
    table = _rand(torch, _gen(torch, 3), (16, Hq), torch.bfloat16)
    _attn_check(zs, torch, q, k, v, do, causal=True, cap=10.0, table=table,
                buckets=zs.relpos_buckets(16, 40))


@pytest.mark.parametrize("cap,bias", [(0.0, False), (0.0, True), (8.0, False), (500.0, True)])
@pytest.mark.parametrize("D", [64, 128])
def test_attention_scales_of_any_sign(zs, torch, D, cap, bias):
    """A negative scale, which is a positive one of -q (whose bounds count the scale's
    size), and one of 0 (the softmax of the bias alone)."""
    q, k, v, do = _attn_inputs(torch, 1, 130, 130, 4, 2, D, seed=D + 5)
    table = buckets = None
    if bias:
        table = _rand(torch, _gen(torch, 3), (8, 4), torch.float32)
        buckets = zs.relpos_buckets(8, 20, bidirectional=True)
    dev = lambda t: None if t is None else t.cuda()
    o, lse, g = _attn(zs, torch, *(dev(t) for t in (q, k, v, do)), dev(table), scale=-D ** -0.5, cap=cap,
                      bias_buckets=dev(buckets))
    want = X.Attention(-q, k, v, scale=D ** -0.5, cap=cap, seen=R.visible(1, 130, 130), table=table,
                       buckets=buckets)
    want_o, bound_o, want_l, bound_l = want.forward()
    R.check("lse", lse, want_l, bound_l)
    R.check("o", o, want_o, bound_o)
    grads = want.backward(o.cpu(), do)
    for name, got in g.items():
        R.check(name, -got if name == "dq" else got, *grads[name])
    _attn_check(zs, torch, q, k, v, do, scale=0.0, cap=cap, table=table, buckets=buckets)


def test_distill_backward_of_many_rows(zs, torch):
    """More rows than one launch takes."""
    N, V, K = 65535 + 70, 24, 3
    g = _gen(torch, 5)
    z = _rand(torch, g, (N, V), torch.float32, 2.0)
    t = z + torch.randn(N, V, generator=g)
    val, idx = torch.topk(t, K, dim=1)
    idx, tlse = idx.to(torch.int32), torch.logsumexp(t.double(), 1).float()
    w = torch.rand(N, generator=g) + 0.5
    want = R.distill(z, idx, val, 1.0, tlse, w, 0.5)
    loss, stats = torch.empty(N, device="cuda"), torch.empty(N, 2, device="cuda")
    kw = dict(teacher_lse=tlse.cuda(), row_weight=w.cuda(), grad_scale=0.5)
    zs.zero_distill_fwd(z.cuda(), idx.cuda(), val.cuda(), loss, stats, **kw)
    R.check("loss", loss, *want["loss"])
    dz = torch.full((N, V), math.nan, device="cuda")
    zs.zero_distill_bwd(z.cuda(), idx.cuda(), val.cuda(), stats, dz, **kw)
    R.check("dz", dz, *want["dz"])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D", [32, 64, 128, 256])
@pytest.mark.parametrize("size", [1e-36, 1e-25, 1e-20, 1e-16, 1e16, 1e20, 1e30])
def test_norm_of_values_of_any_size(zs, torch, size, D, dtype):
    """Rows whose mean square is past binary32's ends, beside ordinary ones: without eps,
    the norm is the same at every size."""
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    g = _gen(torch, D)
    T, H = 7, 3
    x = torch.randn(T, H, D, generator=g)
    x[1::2] *= size
    x = x.to(dt)
    dy = torch.randn(T, H, D, generator=g)
    dy[1::2] *= min(1.0, size)                            # (dx = dy / size stays in range)
    dy, w = dy.to(dt), _rand(torch, g, (D,), dt)
    pos, freq = torch.randint(0, 1000, (T,), generator=g, dtype=torch.int32), zs.rope_inv_freq(D)
    kw = dict(wq=w.cuda(), eps=0.0, pos=pos.cuda(), inv_freq=freq.cuda())
    y, dx = torch.full_like(x, math.nan).cuda(), torch.full_like(x, math.nan).cuda()
    zs.zero_qk_norm_rope_fwd(x.cuda(), None, y, None, **kw)
    R.check("y", y, *R.norm_forward(x, w, 0.0, pos, freq, False))
    zs.zero_qk_norm_rope_bwd(x.cuda(), None, dy.cuda(), None, dx, None, **kw)
    want, bound = R.norm_backward(x, w, dy, 0.0, pos, freq, False)["dx"]
    # (gradients near the smallest numbers are off by those' steps)
    tiny = 2.0 ** -126 * (R.half_step(dt) if dt == torch.float32 else 2.0 ** -7)
    R.check("dx", dx, want, bound + tiny)


# --------------------------------------------- rows a model is sure of, tails ---

def _distill_check(zs, torch, z, idx, val, tau, tlse, w=None, grad_scale=0.25):
    """Loss, statistics and gradient, in one pass, from the statistics, and in place."""
    want = X.distill(z, idx, val, tau, tlse, w, grad_scale)
    dev = lambda t: None if t is None else t.cuda()
    N = z.shape[0]
    zd, di, dv = z.cuda(), idx.cuda(), val.cuda()
    loss, stats = torch.full((N,), math.nan, device="cuda"), torch.full((N, 2), math.nan, device="cuda")
    kw = dict(temperature=tau, teacher_lse=dev(tlse), row_weight=dev(w), grad_scale=grad_scale)
    dz = torch.full_like(zd, math.nan)
    zs.zero_distill_fwd(zd, di, dv, loss, stats, dlogits=dz, **kw)
    R.check("loss", loss, *want["loss"])
    R.check("stats", stats, *want["stats"])
    R.check("dz", dz, *want["dz"])
    alone, stats2 = torch.full_like(loss, math.nan), torch.full_like(stats, math.nan)
    zs.zero_distill_fwd(zd, di, dv, alone, stats2, **kw)
    assert torch.equal(alone, loss) and torch.equal(stats2, stats)
    back = torch.full_like(zd, math.nan)
    zs.zero_distill_bwd(zd, di, dv, stats, back, **kw)
    R.check("dz from stats", back, *want["dz"])
    place = zd.clone()
    zs.zero_distill_bwd(place, di, dv, stats, place, **kw)
    assert torch.equal(place, back)
    zs.zero_distill_fwd(zd, di, dv, alone, stats2, dlogits=zd, **kw)
    assert torch.equal(zd, dz)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("V,tau", [(40, 1.0), (1000, 2.0), (20011, 1.0), (140003, 1.0)])
@pytest.mark.parametrize("gap", [10, 14, 60, 95, 110, 300, 10000])
def test_distill_tail_of_a_sure_student(zs, torch, gap, V, tau, dtype):
    """The teacher's entries lead every other logit by `gap` temperatures, and the teacher
    leaves a hundredth to the tail: the outside's sum is far below the row's."""
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    N, K = 5, 8
    g = _gen(torch, V + gap)
    z = torch.randn(N, V, generator=g)
    idx = torch.stack([torch.randperm(V, generator=g)[:K] for _ in range(N)]).to(torch.int32)
    lead = torch.randn(N, K, generator=g) + gap * tau
    lead[0] -= gap * tau                                  # an ordinary row among them
    z.scatter_(1, idx.long(), lead)
    z[1, ::3] = torch.where(z[1, ::3] > gap * tau / 2, z[1, ::3], -math.inf)   # a masked vocabulary
    z = z.to(dt)
    val = torch.randn(N, K, generator=g).to(dt)
    tlse = (torch.logsumexp(val.double() / tau, 1) - math.log(0.99)).float()
    _distill_check(zs, torch, z, idx, val, tau, tlse, torch.rand(N, generator=g) + 0.5)


@pytest.mark.parametrize("V,K", [(1, 1), (5, 5), (6, 9), (300, 300)])
def test_distill_entries_of_the_whole_vocabulary(zs, torch, V, K):
    """No token is left for a tail, whatever teacher_lse's rounding leaves of 1."""
    N = 40
    g = _gen(torch, V)
    z = torch.randn(N, V, generator=g) * 2
    idx = torch.stack([torch.randperm(V, generator=g) for _ in range(N)]).to(torch.int32)
    idx = torch.nn.functional.pad(idx, (0, K - V), value=-1)
    val = torch.randn(N, K, generator=g) + 9
    tlse = torch.logsumexp(val[:, :V].double(), 1).float()
    _distill_check(zs, torch, z, idx, val, 1.0, tlse)


def test_distill_entries_of_all_that_is_allowed(zs, torch):
    """The vocabulary outside the entries is masked for teacher and student: what
    teacher_lse's rounding leaves of 1 is no tail; a real one makes the loss infinite."""
    N, V, K = 40, 500, 30
    g = _gen(torch, 3)
    idx = torch.stack([torch.randperm(V, generator=g)[:K] for _ in range(N)]).to(torch.int32)
    z = torch.full((N, V), -math.inf)
    z.scatter_(1, idx.long(), torch.randn(N, K, generator=g) * 2)
    val = torch.randn(N, K, generator=g) + 9
    tlse = torch.logsumexp(val.double(), 1).float()
    assert bool((torch.exp(val.double() - tlse.double()[:, None]).sum(1) < 1).any())
    _distill_check(zs, torch, z, idx, val, 1.0, tlse)
    loss, stats = torch.empty(N, device="cuda"), torch.empty(N, 2, device="cuda")
    zs.zero_distill_fwd(z.cuda(), idx.cuda(), val.cuda(), loss, stats, teacher_lse=(tlse + 0.1).cuda())
    assert bool((loss == math.inf).all())


@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("V", [900, 20011])
@pytest.mark.parametrize("offset", [1e3, 1e4, -1e4])
def test_distill_logits_far_from_zero(zs, torch, offset, V, tail):
    """Only differences of logits count: far from 0 the loss is as near to the formula."""
    N, K = 6, 12
    g = _gen(torch, V)
    z = torch.randn(N, V, generator=g) * 2
    t = z + torch.randn(N, V, generator=g)
    val, idx = torch.topk(t, K, dim=1)
    tlse = torch.logsumexp(t.double() / 1.3, 1).float() if tail else None
    z = z + offset
    want = X.distill(z, idx.to(torch.int32), val, 1.3, tlse)
    loss, stats = torch.empty(N, device="cuda"), torch.empty(N, 2, device="cuda")
    dz = torch.empty(N, V, device="cuda")
    zs.zero_distill_fwd(z.cuda(), idx.to(torch.int32).cuda(), val.cuda(), loss, stats, dlogits=dz,
                        temperature=1.3, teacher_lse=None if tlse is None else tlse.cuda())
    R.check("loss", loss, *want["loss"])
    R.check("stats", stats, *want["stats"])
    R.check("dz", dz, *want["dz"])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_distill_longest_row_with_most_entries(zs, torch, dtype):
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    N, V, K = 2, zs._ops_binding.DISTILL_MAX_V, zs._ops_binding.DISTILL_MAX_K
    g = _gen(torch, 9)
    z = (torch.randn(N, V, generator=g) * 2).to(dt)
    t = z.float() + torch.randn(N, V, generator=g)
    val, idx = torch.topk(t, K, dim=1)
    tlse = torch.logsumexp(t.double(), 1).float()
    _distill_check(zs, torch, z, idx.to(torch.int32), val.to(dt), 1.0, tlse)
