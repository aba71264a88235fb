"""The training operators (libzero_ops.so) on the GPU against their formulas
in 64 bits on the host (ops_ref)."""
import math

import pytest

import ops_ref as R
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


# -------------------------------------------------------------- attention ---

def _attn_inputs(torch, B, Tq, Tk, Hq, Hk, D, seed, qscale=2.0):
    g = _gen(torch, seed)
    bf = torch.bfloat16
    return [_rand(torch, g, (B, Tq, Hq, D), bf, qscale), _rand(torch, g, (B, Tk, Hk, D), bf),
            _rand(torch, g, (B, Tk, Hk, D), bf), _rand(torch, g, (B, Tq, Hq, D), bf)]


def _dev(*ts):
    return [None if t is None else t.cuda() for t in ts]


def _ws(zs, torch, q, k, table, backward):
    n = zs.zero_attn_workspace_bytes(q.shape[0], q.shape[1], k.shape[1], q.shape[2], k.shape[2],
                                     q.shape[3], 0 if table is None else table.shape[0], backward)
    return torch.full((max(n, 16),), 0x7F, dtype=torch.uint8, device="cuda")


def _attn_both(zs, torch, q, k, v, do, *, scale=None, cap=0.0, ranges=None, causal=False,
               table=None, buckets=None, backward=True):
    """Runs both directions on the GPU and checks them."""
    B, Tq, Hq, D = q.shape
    Tk = k.shape[1]
    scale = D ** -0.5 if scale is None else scale
    seen = R.visible(B, Tq, Tk, ranges, causal)
    ref = R.Attention(q, k, v, scale=scale, cap=cap, seen=seen, table=table, buckets=buckets)
    dq_, dk_, dv_, ddo, dr, dt, db = _dev(q, k, v, do, ranges, table, buckets)
    o = torch.full_like(dq_, math.nan)
    lse = torch.full((B, Hq, Tq), math.nan, dtype=torch.float32, device="cuda")
    kw = dict(scale=scale, cap=cap, ranges=dr, causal=causal, bias_table=dt, bias_buckets=db)
    zs.zero_attn_fwd(dq_, dk_, dv_, o, lse, workspace=_ws(zs, torch, q, k, table, False), **kw)
    want_o, bound_o, want_l, bound_l = ref.forward()
    R.check("lse", lse, want_l, bound_l)
    R.check("o", o, want_o, bound_o)
    if not backward:
        return o, lse
    gq, gk, gv = (torch.full_like(x, math.nan) for x in (dq_, dk_, dv_))
    gt = None if dt is None else torch.full_like(dt, math.nan)
    zs.zero_attn_bwd(dq_, dk_, dv_, o, lse, ddo, gq, gk, gv, dbias_table=gt,
                     workspace=_ws(zs, torch, q, k, table, True), **kw)
    want = ref.backward(o.cpu(), do)
    for name, got in (("dv", gv), ("dk", gk), ("dq", gq), ("dtable", gt)):
        if got is not None:
            R.check(name, got, *want[name])
    return o, lse


SHAPES = [(1, 1, 1, 1, 1), (2, 3, 3, 2, 1), (1, 31, 31, 4, 4), (2, 64, 64, 2, 2),
          (1, 65, 65, 6, 2), (1, 129, 129, 2, 1), (1, 200, 200, 3, 3), (1, 33, 260, 2, 2),
          (2, 1, 300, 4, 2), (1, 140, 70, 2, 2)]


@pytest.mark.parametrize("D", [32, 64, 96, 128])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_attention_causal_and_full(zs, torch, shape, D):
    B, Tq, Tk, Hq, Hk = shape
    q, k, v, do = _attn_inputs(torch, B, Tq, Tk, Hq, Hk, D, seed=Tq * 7 + D)
    for causal in (False, True):
        _attn_both(zs, torch, q, k, v, do, causal=causal)


@pytest.mark.parametrize("D,cap,bias", [(64, 5.0, None), (128, 30.0, "bf16"), (32, 0.0, "f32"),
                                        (96, 20.0, "f32"), (64, 0.0, "bf16")])
@pytest.mark.parametrize("T,docs", [(1, 1), (47, 3), (130, 2), (257, 5)])
def test_attention_cap_bias_documents(zs, torch, T, docs, D, cap, bias):
    """Caps, the learned bias with its gradient, documents with prefixes and
    padding between and after them (rows that see nothing, holding NaN)."""
    B, Hq, Hk = 2, 4, 2
    q, k, v, do = _attn_inputs(torch, B, T, T, Hq, Hk, D, seed=T + D)
    g = _gen(torch, T)
    doc = torch.zeros((B, T), dtype=torch.int32)
    prefix = torch.zeros((B, T), dtype=torch.int32)
    for b in range(B):
        cut = sorted(torch.randint(0, T, (docs,), generator=g).tolist())
        for n, (lo, hi) in enumerate(zip([0] + cut, cut + [T])):
            pad = n % 3 == 2
            doc[b, lo:hi] = -1 if pad else n + 5
            prefix[b, lo:hi] = (hi - lo) // 3
            if pad:
                for x in (q, k, v, do):
                    x[b, lo:hi] = math.nan
    table = buckets = None
    if bias:
        table = _rand(torch, g, (8, Hq), torch.bfloat16 if bias == "bf16" else torch.float32)
        buckets = zs.relpos_buckets(8, 20, bidirectional=T == 130)
    ranges = R.doc_ranges(doc, prefix)
    dr = torch.full((B, T, 2), 77, dtype=torch.int32, device="cuda")
    zs.zero_attn_ranges(doc.cuda(), dr, prefix=prefix.cuda(), causal=True)
    assert torch.equal(dr.cpu(), ranges)
    nan_free = [torch.nan_to_num(x) for x in (q, k, v, do)]
    seen = R.visible(B, T, T, ranges)
    ref = R.Attention(*nan_free[:3], scale=D ** -0.5, cap=cap, seen=seen, table=table,
                      buckets=buckets)
    dq_, dk_, dv_, ddo, dt, db = _dev(q, k, v, do, table, buckets)
    o = torch.full_like(dq_, math.nan)
    lse = torch.full((B, Hq, T), math.nan, dtype=torch.float32, device="cuda")
    kw = dict(cap=cap, ranges=dr, bias_table=dt, bias_buckets=db)
    zs.zero_attn_fwd(dq_, dk_, dv_, o, lse, workspace=_ws(zs, torch, q, k, table, False), **kw)
    want_o, bound_o, want_l, bound_l = ref.forward()
    R.check("lse", lse, want_l, bound_l)
    R.check("o", o, want_o, bound_o)
    gq, gk, gv = (torch.full_like(x, math.nan) for x in (dq_, dk_, dv_))
    gt = None if dt is None else torch.full_like(dt, math.nan)
    zs.zero_attn_bwd(dq_, dk_, dv_, o, lse, ddo, gq, gk, gv, dbias_table=gt,
                     workspace=_ws(zs, torch, q, k, table, True), **kw)
    want = ref.backward(o.cpu(), nan_free[3])
    for name, got in (("dv", gv), ("dk", gk), ("dq", gq), ("dtable", gt)):
        if got is not None:
            R.check(name, got, *want[name])


def test_attention_ranges_of_any_shape(zs, torch):
    """Intervals that no document gives: unsorted, past the ends, empty,
    single keys."""
    B, T, D = 1, 190, 64
    q, k, v, do = _attn_inputs(torch, B, T, T, 2, 2, D, seed=3)
    g = _gen(torch, 4)
    a = torch.randint(-20, T + 20, (B, T, 2), generator=g, dtype=torch.int32)
    a[0, 5] = torch.tensor([7, 8])
    a[0, 6] = torch.tensor([9, 9])
    a[0, 7] = torch.tensor([-2 ** 31, 2 ** 31 - 1])
    a[0, 8] = torch.tensor([2 ** 31 - 1, -2 ** 31])
    a[0, 64:128] = torch.tensor([50, 50])          # a whole tile of queries sees nothing
    _attn_both(zs, torch, q, k, v, do, ranges=a)


def test_attention_nothing_visible(zs, torch):
    q, k, v, do = _attn_inputs(torch, 1, 70, 70, 2, 1, 32, seed=5)
    for x in (q, k, v, do):
        x.fill_(math.nan)
    r = torch.zeros((1, 70, 2), dtype=torch.int32, device="cuda")
    dq_, dk_, dv_, ddo = _dev(q, k, v, do)
    o, lse = torch.empty_like(dq_), torch.empty(1, 2, 70, device="cuda")
    zs.zero_attn_fwd(dq_, dk_, dv_, o, lse, ranges=r)
    assert float(o.float().abs().max()) == 0 and bool((lse == -math.inf).all())
    gq, gk, gv = (torch.full_like(x, 3.0) for x in (dq_, dk_, dv_))
    zs.zero_attn_bwd(dq_, dk_, dv_, o, lse, ddo, gq, gk, gv, ranges=r,
                     workspace=_ws(zs, torch, q, k, None, True))
    for x in (gq, gk, gv):
        assert float(x.float().abs().max()) == 0


def test_attention_no_keys_and_no_queries(zs, torch):
    bf = torch.bfloat16
    q = torch.randn(1, 5, 2, 64, device="cuda").to(bf)
    none = torch.empty(1, 0, 2, 64, device="cuda", dtype=bf)
    o, lse = torch.empty_like(q), torch.empty(1, 2, 5, device="cuda")
    zs.zero_attn_fwd(q, none, none, o, lse)
    assert float(o.float().abs().max()) == 0 and bool((lse == -math.inf).all())
    gq = torch.full_like(q, 3.0)
    ws = torch.empty(zs.zero_attn_workspace_bytes(1, 5, 0, 2, 2, 64, 0, True), dtype=torch.uint8,
                     device="cuda")
    zs.zero_attn_bwd(q, none, none, o, lse, q, gq, none, none, workspace=ws)
    assert float(gq.float().abs().max()) == 0
    k = torch.randn(1, 5, 2, 64, device="cuda").to(bf)
    gk, gv = torch.full_like(k, 3.0), torch.full_like(k, 3.0)
    l0 = torch.empty(1, 2, 0, device="cuda")
    zs.zero_attn_fwd(none, k, k, none, l0)
    zs.zero_attn_bwd(none, k, k, none, l0, none, none, gk, gv)
    assert float(gk.float().abs().max()) == 0 and float(gv.float().abs().max()) == 0


def test_attention_lowest_value_and_infinite_scores(zs, torch):
    """A bias of the type's lowest value masks like -inf beside others and
    leaves a uniform softmax where every key has it; -inf in the bias masks."""
    T, D, Hq = 40, 64, 2
    q, k, v, do = _attn_inputs(torch, 1, T, T, Hq, Hq, D, seed=9, qscale=0.5)
    low = torch.finfo(torch.bfloat16).min
    for value in (low, -math.inf):
        table = torch.tensor([[0.0, 0.0], [value, value]]).to(torch.bfloat16)
        buckets = torch.tensor([1, 1, 0, 0, 1], dtype=torch.int32)  # near distances only
        seen = R.visible(1, T, T)
        ref = R.Attention(q, k, v, scale=0.125, seen=seen & (
            (torch.arange(T)[None] - torch.arange(T)[:, None]).clamp(-2, 2) >= 0)[None]
            & ((torch.arange(T)[None] - torch.arange(T)[:, None]) <= 1)[None])
        dq_, dk_, dv_, dt, db = _dev(q, k, v, table, buckets)
        o, lse = torch.empty_like(dq_), torch.empty(1, Hq, T, device="cuda")
        zs.zero_attn_fwd(dq_, dk_, dv_, o, lse, scale=0.125, bias_table=dt, bias_buckets=db)
        want_o, bound_o, want_l, bound_l = ref.forward()
        R.check("o", o, want_o, bound_o)
        R.check("lse", lse, want_l, bound_l)
    table = torch.full((1, Hq), low, dtype=torch.bfloat16, device="cuda")
    zs.zero_attn_fwd(dq_, dk_, dv_, o, lse, scale=0.125, bias_table=table,
                     bias_buckets=torch.zeros(1, dtype=torch.int32, device="cuda"))
    mean = v.double().mean(1, keepdim=True).expand(1, T, Hq, D)
    R.check("uniform", o, mean, R.BF * (mean.abs() + 1.1 * v.double().abs().mean(1, keepdim=True)))


@pytest.mark.parametrize("cap", [0.0, 4.0])
def test_attention_large_scores(zs, torch, cap):
    """Scores of several hundred: the maximum is subtracted, the cap saturates."""
    q, k, v, do = _attn_inputs(torch, 1, 150, 150, 2, 2, 64, seed=11, qscale=60.0)
    _attn_both(zs, torch, q, k, v, do, causal=True, cap=cap)


def test_attention_split_keys(zs, torch):
    """Few queries against many keys: the keys are split over workgroups."""
    for B, Tq, Tk, Hq, Hk, D in ((1, 1, 3001, 2, 1, 64), (2, 7, 2500, 4, 4, 128),
                                 (1, 3, 1100, 1, 1, 96)):
        assert zs.zero_attn_workspace_bytes(B, Tq, Tk, Hq, Hk, D) > 0
        q, k, v, do = _attn_inputs(torch, B, Tq, Tk, Hq, Hk, D, seed=Tk)
        g = _gen(torch, Tk)
        table = _rand(torch, g, (32, Hq), torch.bfloat16)
        _attn_both(zs, torch, q, k, v, do, causal=True, table=table,
                   buckets=zs.relpos_buckets(32, 128))
        r = torch.tensor([[[5, 6]] * Tq] * B, dtype=torch.int32)      # one part has all of it
        r[0, 0] = 0
        _attn_both(zs, torch, q, k, v, do, ranges=r, backward=False)


@pytest.mark.parametrize("reach,buckets", [(0, 1), (1, 3), (512, 256)])
def test_attention_bias_reach(zs, torch, reach, buckets):
    T, Hq = 150, 3
    q, k, v, do = _attn_inputs(torch, 1, T, T, Hq, 1, 32, seed=reach)
    g = _gen(torch, 1)
    table = _rand(torch, g, (buckets, Hq), torch.float32)
    b = torch.randint(-2, buckets + 2, (2 * reach + 1,), generator=g, dtype=torch.int32)
    _attn_both(zs, torch, q, k, v, do, table=table, buckets=b)


def test_attention_strides(zs, torch):
    """Heads before tokens, one packed projection, gaps between rows."""
    B, T, Hq, Hk, D = 2, 75, 4, 2, 64
    g = _gen(torch, 21)
    bf = torch.bfloat16
    qkv = _rand(torch, g, (B, T, Hq + 2 * Hk, D), bf)
    q, k, v = qkv[:, :, :Hq], qkv[:, :, Hq:Hq + Hk], qkv[:, :, Hq + Hk:]
    do = _rand(torch, g, (B, Hq, T, D), bf).transpose(1, 2)
    ref = R.Attention(q, k, v, scale=0.125, seen=R.visible(B, T, T, causal=True))
    dqkv, ddo = qkv.cuda(), torch.empty(B, Hq, T + 3, D, device="cuda", dtype=bf)[:, :, :T]
    ddo.copy_(do.transpose(1, 2))
    ddo = ddo.transpose(1, 2)
    gq = lambda x: (x[:, :, :Hq], x[:, :, Hq:Hq + Hk], x[:, :, Hq + Hk:])
    o = torch.zeros(B, Hq, T, D + 8, device="cuda", dtype=bf)[..., :D].transpose(1, 2)
    lse = torch.empty(B, Hq, T, device="cuda")
    grad = torch.full_like(dqkv, 9.0)
    a, b, c = gq(dqkv)
    zs.zero_attn_fwd(a, b, c, o, lse, scale=0.125, causal=True)
    R.check("o", o, *ref.forward()[:2])
    zs.zero_attn_bwd(a, b, c, o, lse, ddo, *gq(grad), scale=0.125, causal=True,
                     workspace=_ws(zs, torch, q, k, None, True))
    want = ref.backward(o.cpu(), do)
    for name, got in zip(("dq", "dk", "dv"), gq(grad)):
        R.check(name, got, *want[name])


def test_attention_offsets_past_32_bits(zs, torch):
    """Rows more than 2^31 elements from the base (and 2^32 bytes)."""
    bf = torch.bfloat16
    T, D, stride = 70, 64, 1 << 25
    big = torch.empty(T * stride, dtype=bf, device="cuda")            # 4.7 GB
    q, k, v, do = _attn_inputs(torch, 1, T, T, 1, 1, D, seed=2)
    kk = big.as_strided((1, T, 1, D), (T * stride, stride, D, 1))
    vv = big[4096:].as_strided((1, T, 1, D), (T * stride, stride, D, 1))
    kk.copy_(k)
    vv.copy_(v)
    dq_ = q.cuda()
    o, lse = torch.empty_like(dq_), torch.empty(1, 1, T, device="cuda")
    zs.zero_attn_fwd(dq_, kk, vv, o, lse, causal=True)
    ref = R.Attention(q, k, v, scale=D ** -0.5, seen=R.visible(1, T, T, causal=True))
    R.check("o", o, *ref.forward()[:2])
    gk = big[8192:].as_strided((1, T, 1, D), (T * stride, stride, D, 1))
    gv = big[12288:].as_strided((1, T, 1, D), (T * stride, stride, D, 1))
    gq = torch.empty_like(dq_)
    zs.zero_attn_bwd(dq_, kk, vv, o, lse, do.cuda(), gq, gk, gv, causal=True,
                     workspace=_ws(zs, torch, q, k, None, True))
    want = ref.backward(o.cpu(), do)
    for name, got in (("dq", gq), ("dk", gk), ("dv", gv)):
        R.check(name, got, *want[name])


@pytest.mark.parametrize("D", [96, 128])
def test_attention_far_query_rows(zs, torch, D):
    """Rows of q and do, and keys and values, 16 MiB apart: further than a staged
    tile's 32-bit offsets go."""
    bf = torch.bfloat16
    T, stride = 70, 1 << 23
    q, k, v, do = _attn_inputs(torch, 1, T, T, 1, 1, D, seed=D)
    big = torch.empty(T * stride, dtype=bf, device="cuda")            # 1.2 GB
    far = [big[4096 * n:].as_strided((1, T, 1, D), (T * stride, stride, D, 1)) for n in range(4)]
    for x, y in zip(far, (q, k, v, do)):
        x.copy_(y)
    near = _dev(q, k, v, do)
    ws = _ws(zs, torch, q, k, None, True)
    results = []
    for a in (far, near):
        o, lse = torch.empty_like(near[0]), torch.empty(1, 1, T, device="cuda")
        zs.zero_attn_fwd(*a[:3], o, lse, causal=True)
        g = [torch.empty_like(x) for x in near[:3]]
        zs.zero_attn_bwd(*a[:3], o, lse, a[3], *g, causal=True, workspace=ws)
        results.append((o, lse, *g))
    # the same sums in the same order, whichever way a tile was fetched
    assert all(torch.equal(x, y) for x, y in zip(*results))


@pytest.mark.parametrize("T,H,D,cap", [(517, 2, 128, 30.0), (517, 2, 96, 0.0), (2060, 16, 128, 0.0)])
def test_attention_many_tiles_of_documents(zs, torch, T, H, D, cap):
    """Several tiles each way: whole and partly masked tiles in turn, documents that
    begin inside a tile, and (17 tiles of 16 heads) tiles taken by cost."""
    q, k, v, do = _attn_inputs(torch, 1, T, T, H, H, D, seed=T + D)
    doc = torch.zeros((1, T), dtype=torch.int32)
    prefix = torch.zeros((1, T), dtype=torch.int32)
    cuts = [0, T // 3 + 5, T // 3 + 40, T - 9]
    for n, (lo, hi) in enumerate(zip(cuts, cuts[1:])):
        doc[0, lo:hi] = n
        prefix[0, lo:hi] = (hi - lo) // 2
    doc[0, cuts[-1]:] = -1
    _attn_both(zs, torch, q, k, v, do, ranges=R.doc_ranges(doc, prefix), cap=cap)


def test_attention_gradient_by_differences(zs, torch):
    """dtable, and dq, dk, dv along random directions, against central
    differences of the 64-bit forward (1e-4 steps: their error is below 1e-6
    of the values'), within the 64-bit gradient's bounds."""
    B, T, Hq, Hk, D, cap = 1, 40, 2, 1, 32, 6.0
    q, k, v, do = _attn_inputs(torch, B, T, T, Hq, Hk, D, seed=17)
    g = _gen(torch, 5)
    table = _rand(torch, g, (6, Hq), torch.float32)
    buckets = zs.relpos_buckets(6, 10)
    seen = R.visible(B, T, T, causal=True)
    dq_, dk_, dv_, ddo, dt, db = _dev(q, k, v, do, table, buckets)
    o, lse = torch.empty_like(dq_), torch.empty(B, Hq, T, device="cuda")
    kw = dict(cap=cap, causal=True, bias_table=dt, bias_buckets=db)
    zs.zero_attn_fwd(dq_, dk_, dv_, o, lse, **kw)
    out = [torch.empty_like(x) for x in (dq_, dk_, dv_, dt)]
    zs.zero_attn_bwd(dq_, dk_, dv_, o, lse, ddo, *out[:3], dbias_table=out[3],
                     workspace=_ws(zs, torch, q, k, table, True), **kw)

    def loss(*x):
        a = R.Attention(x[0], x[1], x[2], scale=D ** -0.5, cap=cap, seen=seen, table=x[3],
                        buckets=buckets)
        return float((a.forward()[0] * do.double()).sum())

    base = [x.double() for x in (q, k, v, table)]
    bounds = R.Attention(q, k, v, scale=D ** -0.5, cap=cap, seen=seen, table=table,
                         buckets=buckets).backward(o.cpu(), do)
    # the stored o is rounded to bf16: delta, and with it ds, moves by p times this
    slack = float((do.double().abs() * o.cpu().double().abs()).sum(3).max()) * R.BF
    for n, name in enumerate(("dq", "dk", "dv", "dtable")):
        way = torch.randn(base[n].shape, generator=g, dtype=torch.float64)
        h = 1e-4
        plus, minus = list(base), list(base)
        plus[n], minus[n] = base[n] + h * way, base[n] - h * way
        diff = (loss(*plus) - loss(*minus)) / (2 * h)
        got = float((out[n].cpu().double() * way).sum())
        tol = float((bounds[name][1] * way.abs()).sum()) + slack * float(way.abs().sum())
        assert abs(got - diff) <= tol + 1e-6 * abs(diff), (name, got, diff, tol)


# -------------------------------------------------------------------- norm ---

NORMS = [(1, 1, 1, 64, 64, False), (5, 3, 2, 32, 16, True), (33, 12, 3, 96, 48, True),
         (7, 8, 8, 128, 128, False), (130, 2, 1, 256, 128, False), (19, 5, 0, 192, 192, True),
         (9, 0, 4, 8, 8, True), (17, 4, 4, 40, 0, False), (4500, 2, 1, 64, 32, False)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,Hq,Hk,D,rd,inter", NORMS)
def test_norm_rotation(zs, torch, T, Hq, Hk, D, rd, inter, dtype):
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    g = _gen(torch, T + D)
    pos = torch.randint(0, 1 << 24, (T,), generator=g, dtype=torch.int32)
    freq = zs.rope_inv_freq(rd) if rd else None
    qkv = _rand(torch, g, (T, Hq + Hk, D), dt, 3.0)
    dy = _rand(torch, g, (T, Hq + Hk, D), dt)
    wq = _rand(torch, g, (D,), dt) if T != 33 else None
    wk = _rand(torch, g, (D,), dt)
    dqkv, ddy, dwq_, dwk_, dpos, dfreq = _dev(qkv, dy, wq, wk, pos if rd else None, freq)
    cut = lambda t: (t[:, :Hq] if Hq else None, t[:, Hq:] if Hk else None)
    out = torch.full_like(dqkv, math.nan)
    kw = dict(wq=dwq_ if Hq else None, wk=dwk_ if Hk else None, eps=1e-5, pos=dpos,
              inv_freq=dfreq, interleaved=inter)
    zs.zero_qk_norm_rope_fwd(*cut(dqkv), *cut(out), **kw)
    for x, w, y in ((qkv[:, :Hq], wq, out[:, :Hq]), (qkv[:, Hq:], wk, out[:, Hq:])):
        if x.shape[1]:
            R.check("y", y, *R.norm_forward(x, w, 1e-5, pos, freq, inter))
    grad = torch.full_like(dqkv, math.nan)
    ws = torch.empty(max(16, zs.zero_qk_norm_rope_workspace_bytes(T, D)), dtype=torch.uint8,
                     device="cuda").fill_(0x7F)
    gw = [torch.full_like(w, math.nan) if w is not None else None for w in (kw["wq"], kw["wk"])]
    zs.zero_qk_norm_rope_bwd(*cut(dqkv), *cut(ddy), *cut(grad), dwq=gw[0], dwk=gw[1],
                             workspace=ws, **kw)
    for x, w, d, y, got in ((qkv[:, :Hq], wq, dy[:, :Hq], grad[:, :Hq], gw[0]),
                            (qkv[:, Hq:], wk, dy[:, Hq:], grad[:, Hq:], gw[1])):
        if x.shape[1]:
            want = R.norm_backward(x, w, d, 1e-5, pos, freq, inter)
            R.check("dx", y, *want["dx"])
            if got is not None:
                R.check("dw", got, *want["dw"])
    # in place: y over x, dx over dy
    zs.zero_qk_norm_rope_bwd(*cut(dqkv), *cut(ddy), *cut(ddy), **kw)
    assert torch.equal(ddy.view(torch.uint8), grad.view(torch.uint8))
    zs.zero_qk_norm_rope_fwd(*cut(dqkv), *cut(dqkv), **kw)
    assert torch.equal(dqkv.view(torch.uint8), out.view(torch.uint8))


def test_norm_zero_rows_and_specials(zs, torch):
    """A row of zeros with eps (gives zeros) and without (NaN, as 0/0); a NaN
    stays in its row."""
    x = torch.ones(4, 2, 64, device="cuda")
    x[1] = 0
    x[2, 0, 5] = math.nan
    y = torch.empty_like(x)
    zs.zero_qk_norm_rope_fwd(x, None, y, None, eps=1e-6)
    assert bool((y[1] == 0).all()) and bool(y[2, 0].isnan().all())
    assert bool(y[2, 1].isfinite().all()) and bool(y[3].isfinite().all())
    zs.zero_qk_norm_rope_fwd(x, None, y, None, eps=0.0)
    assert bool(y[1].isnan().all()) and bool(y[0].isfinite().all())


def test_norm_empty(zs, torch):
    x = torch.empty(0, 3, 64, device="cuda")
    zs.zero_qk_norm_rope_fwd(x, None, x, None)
    w, dw = torch.ones(64, device="cuda"), torch.full((64,), 5.0, device="cuda")
    zs.zero_qk_norm_rope_bwd(x, None, x, None, x, None, wq=w, dwq=dw)
    assert bool((dw == 0).all())


# ----------------------------------------------------------------- distill ---

def _distill_inputs(torch, N, V, K, dt, tau, seed):
    g = _gen(torch, seed)
    z = torch.randn(N, V, generator=g) * 2
    t = torch.randn(N, V, generator=g) + z
    val, idx = torch.topk(t, K, dim=1)
    tlse = torch.logsumexp(t.double() / tau, 1).float()
    w = torch.rand(N, generator=g) + 0.5
    return z.to(dt), idx.to(torch.int32), val.to(dt), tlse, w


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N,V,K,tau,tail", [
    (3, 1, 1, 1.0, False), (4, 7, 3, 2.0, True), (5, 513, 16, 1.0, True), (3, 5000, 300, 4.0, False),
    (6, 9001, 64, 1.5, True), (2, 50257, 64, 1.0, True), (3, 70001, 1024, 2.0, True),
    (2, 140003, 5, 0.7, False), (300, 100, 8, 1.0, True)])
def test_distill(zs, torch, N, V, K, tau, tail, dtype):
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    z, idx, val, tlse, w = _distill_inputs(torch, N, V, K, dt, tau, V)
    if N > 2:
        w[1] = 0.0
        z[1] = math.nan                                   # a row without weight holds anything
        idx[2, K // 2:] = -1                              # fewer entries
        idx[2, K - 1] = V                                 # out of range: absent too
    if not tail:
        tlse = None
    want = R.distill(torch.where(torch.isnan(z), 0, z), idx, val, tau, tlse, w, 0.25)
    dz_, di, dv_, dl, dw = _dev(z, idx, val, tlse, w)
    loss = torch.full((N,), math.nan, device="cuda")
    stats = torch.full((N, 2), math.nan, device="cuda")
    kw = dict(temperature=tau, teacher_lse=dl, row_weight=dw, grad_scale=0.25)
    zs.zero_distill_fwd(dz_, di, dv_, loss, stats, **kw)
    R.check("loss", loss, *want["loss"])
    rows = ~torch.isnan(z).any(1)                         # (stats are formed for every row)
    R.check("stats", stats.cpu()[rows], *(x[rows] for x in want["stats"]))
    out = torch.full_like(dz_, math.nan)
    loss2, stats2 = torch.empty_like(loss), torch.empty_like(stats)
    zs.zero_distill_fwd(dz_, di, dv_, loss2, stats2, dlogits=out, **kw)
    assert torch.equal(loss2, loss)
    assert torch.equal(stats2.view(torch.int32), stats.view(torch.int32))
    R.check("dz", out, *want["dz"])
    out2 = torch.full_like(dz_, math.nan)
    zs.zero_distill_bwd(dz_, di, dv_, stats, out2, **kw)
    R.check("dz from stats", out2, *want["dz"])
    # in place, both ways; rows that start elsewhere than their gradients do
    spare = dz_.clone()
    zs.zero_distill_bwd(spare, di, dv_, stats, spare, **kw)
    assert torch.equal(spare, out2)
    zs.zero_distill_fwd(dz_, di, dv_, loss2, stats2, dlogits=dz_, **kw)
    assert torch.equal(dz_, out)


def test_distill_strides(zs, torch):
    """Padded rows, and gradient rows that start at another alignment."""
    z, idx, val, tlse, w = _distill_inputs(torch, 5, 777, 9, torch.bfloat16, 1.0, 1)
    want = R.distill(z, idx, val, 1.0, tlse, None, 1.0)
    wide = torch.full((5, 790), math.nan, device="cuda", dtype=torch.bfloat16)
    zin = wide[:, 3:780]
    zin.copy_(z)
    guard = torch.full((5, 785), 42.0, device="cuda", dtype=torch.bfloat16)
    out = guard[:, 1:778]
    loss, stats = torch.empty(5, device="cuda"), torch.empty(5, 2, device="cuda")
    for _ in range(2):
        out.fill_(math.nan)
        if _ == 0:
            zs.zero_distill_fwd(zin, idx.cuda(), val.cuda(), loss, stats, dlogits=out,
                                teacher_lse=tlse.cuda())
        else:
            zs.zero_distill_bwd(zin, idx.cuda(), val.cuda(), stats, out, teacher_lse=tlse.cuda())
        R.check("dz", out, *want["dz"])
        assert bool((guard[:, 0] == 42).all()) and bool((guard[:, 778:] == 42).all())


def test_distill_infinities(zs, torch):
    """-inf logits (a masked vocabulary) have no probability; a teacher entry
    there makes the loss infinite; teacher entries of -inf have no part."""
    z = torch.zeros(4, 40)
    z[:, 30:] = -math.inf
    z[3, :] = -math.inf
    idx = torch.tensor([[0, 1], [0, 35], [0, 1], [0, 1]], dtype=torch.int32)
    val = torch.tensor([[1.0, 0.0], [1.0, 0.0], [1.0, -math.inf], [1.0, 0.0]])
    loss, stats = torch.empty(4, device="cuda"), torch.empty(4, 2, device="cuda")
    dz = torch.empty(4, 40, device="cuda")
    zs.zero_distill_fwd(z.cuda(), idx.cuda(), val.cuda(), loss, stats, dlogits=dz)
    want = R.distill(z[:1], idx[:1], val[:1], 1.0)
    R.check("loss", loss[:1], *want["loss"])
    R.check("dz", dz[:1], *want["dz"])
    got = loss.cpu()
    assert got[1] == math.inf and abs(got[2] - math.log(30)) < 1e-5
    assert abs(float(dz[2, 1]) - 1 / 30) < 1e-7 and abs(float(dz[2, 0]) - (1 / 30 - 1)) < 1e-6


def test_distill_gradient_by_differences(zs, torch):
    """dz along random directions against central differences of the 64-bit
    loss."""
    for tail in (False, True):
        z, idx, val, tlse, w = _distill_inputs(torch, 3, 60, 7, torch.float32, 1.3, 8)
        tlse = tlse if tail else None
        dz = torch.empty(3, 60, device="cuda")
        loss, stats = torch.empty(3, device="cuda"), torch.empty(3, 2, device="cuda")
        dl = None if tlse is None else tlse.cuda()
        zs.zero_distill_fwd(z.cuda(), idx.cuda(), val.cuda(), loss, stats, dlogits=dz,
                            temperature=1.3, teacher_lse=dl, row_weight=w.cuda())
        f = lambda x: float(R.distill(x, idx, val, 1.3, tlse, w)["loss"][0].sum())
        g = _gen(torch, 2)
        bound = R.distill(z, idx, val, 1.3, tlse, w)["dz"][1]
        for _ in range(4):
            way = torch.randn(3, 60, generator=g, dtype=torch.float64)
            h = 1e-5
            diff = (f(z.double() + h * way) - f(z.double() - h * way)) / (2 * h)
            got = float((dz.cpu().double() * way).sum())
            tol = float((bound * way.abs()).sum()) + 1e-8
            assert abs(got - diff) <= tol + 1e-7 * abs(diff), (got, diff, tol)


# ------------------------------------------- streams, graphs, repeatability ---

def _student_pass(zs, torch, s):
    """norm -> attention -> loss, forward and backward, on the current stream."""
    zs.zero_qk_norm_rope_fwd(s["q0"], s["k0"], s["q"][0], s["k"][0], wq=s["w"], wk=s["w"],
                             pos=s["pos"], inv_freq=s["freq"])
    kw = dict(cap=20.0, ranges=s["ranges"], bias_table=s["table"], bias_buckets=s["buckets"],
              workspace=s["ws"])
    zs.zero_attn_fwd(s["q"], s["k"], s["v"], s["o"], s["lse"], **kw)
    zs.zero_attn_bwd(s["q"], s["k"], s["v"], s["o"], s["lse"], s["do"], s["dq"], s["dk"], s["dv"],
                     dbias_table=s["dt"], **kw)
    zs.zero_qk_norm_rope_bwd(s["q0"], s["k0"], s["dq"][0], s["dk"][0], s["dq0"], s["dk0"],
                             wq=s["w"], wk=s["w"], dwq=s["dw"], dwk=s["dw2"], pos=s["pos"],
                             inv_freq=s["freq"], workspace=s["ws"])
    zs.zero_distill_fwd(s["z"], s["idx"], s["val"], s["loss"], s["stats"], dlogits=s["dz"],
                        teacher_lse=s["tl"])
    return [s[n] for n in ("o", "lse", "dq0", "dk0", "dv", "dt", "dw", "dw2", "loss", "stats",
                           "dz")]


def _student_state(zs, torch, T=210, Hq=4, Hk=2, D=64, V=1003):
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    bf = torch.bfloat16
    r = lambda *sh: torch.randn(*sh, generator=g, device="cuda").to(bf)
    s = dict(q0=r(T, Hq, D), k0=r(T, Hk, D), v=r(1, T, Hk, D), do=r(1, T, Hq, D), w=r(D),
             q=torch.empty(1, T, Hq, D, device="cuda", dtype=bf),
             k=torch.empty(1, T, Hk, D, device="cuda", dtype=bf), table=r(16, Hq), z=r(T, V))
    s["pos"] = torch.arange(T, device="cuda", dtype=torch.int32)
    s["freq"] = zs.rope_inv_freq(D).cuda()
    s["buckets"] = zs.relpos_buckets(16, 40, device="cuda")
    doc = torch.zeros(1, T, dtype=torch.int32, device="cuda")
    doc[:, 90:] = 1
    doc[:, 200:] = -1
    s["ranges"] = torch.empty(1, T, 2, dtype=torch.int32, device="cuda")
    zs.zero_attn_ranges(doc, s["ranges"])
    for n, like in (("o", "do"), ("dq", "do"), ("dk", "k"), ("dv", "v"), ("dt", "table"),
                    ("dq0", "q0"), ("dk0", "k0"), ("dw", "w"), ("dw2", "w"), ("dz", "z")):
        s[n] = torch.empty_like(s[like])
    s["lse"] = torch.empty(1, Hq, T, device="cuda")
    val, idx = torch.topk(r(T, V).float(), 12, dim=1)
    s["val"], s["idx"] = val.to(bf), idx.to(torch.int32)
    s["tl"] = torch.full((T,), 8.0, device="cuda")
    s["loss"], s["stats"] = torch.empty(T, device="cuda"), torch.empty(T, 2, device="cuda")
    n = max(zs.zero_attn_workspace_bytes(1, T, T, Hq, Hk, D, 16, b) for b in (False, True))
    s["ws"] = torch.empty(max(n, zs.zero_qk_norm_rope_workspace_bytes(T, D)), dtype=torch.uint8,
                          device="cuda")
    return s


def test_ops_repeat_bitwise_on_streams_and_in_graphs(zs, torch):
    """The same bits on every run, on another stream, and from every replay of
    a recorded graph, with eager work between the replays."""
    s = _student_state(zs, torch)
    torch.cuda.synchronize()
    want = [t.clone() for t in _student_pass(zs, torch, s)]
    torch.cuda.synchronize()
    same = lambda: all(torch.equal(a.view(torch.uint8), b.view(torch.uint8))
                       for a, b in zip(want, outs))
    outs = _student_pass(zs, torch, s)
    torch.cuda.synchronize()
    assert same()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for t in outs:
        t.zero_()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        _student_pass(zs, torch, s)
    side.synchronize()
    assert same()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        _student_pass(zs, torch, s)
    for _ in range(4):
        for t in outs:
            t.zero_()
        s["ws"].fill_(0x55)
        graph.replay()
        torch.cuda.synchronize()
        assert same()
        _student_pass(zs, torch, s)
        torch.cuda.synchronize()
        assert same()
