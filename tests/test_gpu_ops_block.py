"""The operators around a student's blocks (embedding, norms with gate and residual
sum, policy loss, the gradients' norm and clipping) on the GPU against their formulas
in 64 bits on the host (ops_block_ref)."""
import math

import pytest

import ops_block_ref as B
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


def _types(torch, *names):
    return [dict(bf16=torch.bfloat16, f32=torch.float32)[n] for n in names]


def _ws(torch, nbytes):
    """A workspace of that many bytes, full of NaN, with a page behind it to stay as it was."""
    t = torch.full((nbytes + 4096,), 0xFF, dtype=torch.uint8, device="cuda")
    return t[:nbytes], t[nbytes:]


def _bits(t):
    return t.contiguous().view(-1).view(dtype=__import__("torch").uint8)


def _same(a, b):
    import torch
    return torch.equal(_bits(a), _bits(b))


def _strided(torch, t, pad=16):
    """The same values as a view with `pad` more columns behind each row, which hold 7."""
    wide = torch.full((t.shape[0], t.shape[1] + pad), 7.0, dtype=t.dtype, device=t.device)
    view = wide[:, :t.shape[1]]
    view.copy_(t)
    return view, wide[:, t.shape[1]:]


# -------------------------------------------------------------- embedding ---

@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N,V,C", [(1, 1, 8), (3, 5, 24), (65, 300, 520), (130, 17, 2056),
                                   (7, 40, 4104), (2, 9, 16384)])
def test_embed_forward(zs, torch, N, V, C, dtype):
    dt, = _types(torch, dtype)
    g = _gen(torch, N + C)
    table = _rand(torch, g, (V, C), dt)
    ids = torch.randint(-2, V + 2, (N,), generator=g, dtype=torch.int32)
    ids[0] = V - 1
    if N > 2:
        ids[1], ids[2] = -2 ** 31, 2 ** 31 - 1
    for scale in (1.0, -3.7):
        want, bound = B.embed_forward(table, ids, scale)
        view, _ = _strided(torch, table.cuda())
        out, rest = _strided(torch, torch.full((N, C), math.nan, dtype=dt, device="cuda"), 8)
        zs.zero_embed_fwd(view, ids.cuda(), out, scale=scale)
        R.check("out", out, want, bound)
        assert bool((rest == 7).all())


def _ids(torch, kind, N, V, g):
    if kind == "same":
        return torch.full((N,), V // 2, dtype=torch.int32)
    if kind == "none":
        return torch.full((N,), -1, dtype=torch.int32)
    if kind == "down":
        return torch.arange(N - 1, -1, -1, dtype=torch.int32) % (V + 3)
    if kind == "few":
        return (torch.randint(0, 3, (N,), generator=g) * (V // 3)).to(torch.int32)
    u = torch.rand(N, generator=g, dtype=torch.float64)
    ids = ((u * math.log(V + 1)).exp().long() - 1).clamp(0, V - 1).to(torch.int32)
    ids[::7] = -5
    return ids


def _embed_bwd(zs, torch, ids, dout, V, scale, base, grad_dtype, in_place=False):
    N, C = dout.shape
    want, bound = B.embed_backward(ids, dout, V, scale, base, grad_dtype)
    got, rest = _strided(torch, torch.full((V, C), math.nan, dtype=grad_dtype, device="cuda"), 8)
    dbase = None if base is None else base.cuda()
    if in_place:
        got.copy_(dbase)
        dbase = got
    ws, behind = _ws(torch, zs.zero_embed_workspace_bytes(N, C))
    d, _ = _strided(torch, dout.cuda())
    zs.zero_embed_bwd(ids.cuda(), d, got, scale=scale, base=dbase, workspace=ws)
    R.check("dtable", got, want, bound)
    assert bool((rest == 7).all()) and bool((behind == 0xFF).all())
    return got


@pytest.mark.parametrize("kind", ["zipf", "same", "few", "down", "none"])
@pytest.mark.parametrize("N", [1, 2, 61, 64, 65, 255, 256, 257, 1000, 1023, 1024, 1025, 2047, 2048, 2049, 4099, 16390])
def test_embed_backward_tokens(zs, torch, N, kind):
    """Numbers of tokens about every border of the sort, and how they are spread: one
    row for all, runs over many chunks, rows that no token names."""
    g = _gen(torch, N)
    V, C = (40, 24) if N > 300 else (301, 24)
    ids = _ids(torch, kind, N, V, g)
    dout = _rand(torch, g, (N, C), torch.bfloat16)
    got = _embed_bwd(zs, torch, ids, dout, V, 1.0, None, torch.float32)
    absent = torch.ones(V, dtype=torch.bool)
    absent[ids[(ids >= 0) & (ids < V)].long()] = False
    assert bool((got.cpu()[absent] == 0).all())


@pytest.mark.parametrize("kind", ["zipf", "same", "few", "down"])
@pytest.mark.parametrize("N", [16384, 16385, 40003, 262144, 262145, 2 ** 21])
def test_embed_backward_many_tokens(zs, torch, N, kind):
    """Lists that are joined in one, two and three passes, the last ones short; runs over more
    chunks than a wave has lanes, and than it finds in two steps."""
    g = _gen(torch, N)
    V, C = 5003, 8
    ids = _ids(torch, kind, N, V, g)
    # whole numbers, whose sums binary32 holds exactly
    dout = torch.randint(-4, 5, (N, C), generator=g).to(torch.bfloat16)
    want = torch.zeros(V + 1, C, dtype=torch.float64)
    want.index_add_(0, torch.where((ids >= 0) & (ids < V), ids, V).long(), dout.double())
    ws, behind = _ws(torch, zs.zero_embed_workspace_bytes(N, C))
    got = torch.full((V, C), math.nan, device="cuda")
    zs.zero_embed_bwd(ids.cuda(), dout.cuda(), got, workspace=ws)
    assert torch.equal(got.cpu().double(), want[:V]) and bool((behind == 0xFF).all())


@pytest.mark.parametrize("kind", ["zipf", "same", "few", "down", "beside", "none"])
@pytest.mark.parametrize("N", [257, 4097, 70001])
@pytest.mark.parametrize("V,C", [(20011, 8), (300007, 8), (9001, 2048), (8209, 4104)])
def test_embed_backward_runs_in_large_tables(zs, torch, V, C, N, kind):
    """Runs that fill the keys a wave looks at for the rows that no id names, with a row beside them."""
    if N * C > 1 << 24:
        N = 4097
    g = _gen(torch, V + N)
    ids = _ids(torch, kind if kind != "beside" else "same", N, V, g)
    if kind == "beside":
        ids[3], ids[4] = V // 2 - 1, V // 2 + 2
    dout = torch.randint(-4, 5, (N, C), generator=g).to(torch.bfloat16)
    want = torch.zeros(V + 1, C, dtype=torch.float64)
    want.index_add_(0, torch.where((ids >= 0) & (ids < V), ids, V).long(), dout.double())
    ws, _ = _ws(torch, zs.zero_embed_workspace_bytes(N, C))
    got = torch.full((V, C), math.nan, device="cuda")
    zs.zero_embed_bwd(ids.cuda(), dout.cuda(), got, workspace=ws)
    assert torch.equal(got.cpu().double(), want[:V])


@pytest.mark.parametrize("types", [("bf16", "bf16", None), ("bf16", "f32", "bf16"), ("f32", "f32", "f32"),
                                   ("bf16", "bf16", "f32"), ("f32", "bf16", "bf16")], ids=str)
@pytest.mark.parametrize("N,V,C", [(1, 1, 8), (37, 12, 520), (500, 90, 1000), (2100, 70, 1544)])
def test_embed_backward_types(zs, torch, N, V, C, types):
    dt, gt = _types(torch, *types[:2])
    g = _gen(torch, C)
    ids = _ids(torch, "zipf", N, V, g)
    dout = _rand(torch, g, (N, C), dt)
    base = None if types[2] is None else _rand(torch, g, (V, C), _types(torch, types[2])[0], 3.0)
    _embed_bwd(zs, torch, ids, dout, V, -0.37, base, gt)


@pytest.mark.parametrize("base", [None, "bf16", "f32"])
@pytest.mark.parametrize("N", [5, 400])
@pytest.mark.parametrize("V,C", [(20011, 8), (300007, 8), (9001, 104), (4099, 1528), (33, 8200)])
def test_embed_backward_rows_without_tokens(zs, torch, V, C, N, base):
    """Several table rows to a wave, one, and parts of one; the shortest pieces."""
    g = _gen(torch, V)
    ids = _ids(torch, "zipf", N, V, g)
    ids[N // 2] = V - 1
    b = None if base is None else _rand(torch, g, (V, C), _types(torch, base)[0])
    for grad in (torch.bfloat16, torch.float32):
        _embed_bwd(zs, torch, ids, _rand(torch, g, (N, C), torch.bfloat16), V, 1.0, b, grad)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N", [0, 1, 70, 3000])
def test_embed_backward_adds_in_place(zs, torch, N, dtype):
    """Rows that no token names keep their bits, NaN and all."""
    dt, = _types(torch, dtype)
    V, C = 97, 72
    g = _gen(torch, 5)
    ids = _ids(torch, "zipf", N, V - 10, g)
    base = _rand(torch, g, (V, C), dt)
    got = _embed_bwd(zs, torch, ids, _rand(torch, g, (N, C), dt), V, 2.0, base, dt, in_place=True)
    got[V - 10:] = math.nan
    keep = got.clone()
    ws, _ = _ws(torch, zs.zero_embed_workspace_bytes(N, C))
    zs.zero_embed_bwd(ids.cuda(), torch.zeros(N, C, dtype=dt, device="cuda"), got, base=got,
                      workspace=ws)
    assert _same(got, keep)


def test_embed_backward_of_no_tokens(zs, torch):
    ids, dout = torch.empty(0, dtype=torch.int32, device="cuda"), torch.empty(0, 16, device="cuda")
    got = torch.full((33, 16), math.nan, device="cuda")
    zs.zero_embed_bwd(ids, dout, got)
    assert bool((got == 0).all())
    base = torch.randn(33, 16, device="cuda")
    zs.zero_embed_bwd(ids, dout, got, base=base)
    assert _same(got, base)


def test_embed_backward_keeps_nan_to_its_row(zs, torch):
    """A padding token's gradient is not read into the sums, a NaN stays in its row."""
    N, V, C = 300, 50, 16
    ids = torch.arange(N, dtype=torch.int32) % V
    ids[::9] = -1
    dout = torch.ones(N, C)
    dout[::9] = math.nan
    hit = int(ids[1])
    dout[1] = math.inf
    ws, _ = _ws(torch, zs.zero_embed_workspace_bytes(N, C))
    got = torch.empty(V, C, device="cuda")
    zs.zero_embed_bwd(ids.cuda(), dout.cuda(), got, workspace=ws)
    assert bool(torch.isinf(got[hit]).all())
    got[hit] = 0
    assert bool(torch.isfinite(got).all())


def test_embed_gradient_against_differences(zs, torch):
    """d/dtable of sum(weights * out), by differences of the forward in fp32."""
    g = _gen(torch, 8)
    N, V, C, scale = 40, 11, 16, 1.5
    table = _rand(torch, g, (V, C), torch.float32)
    ids = torch.randint(-1, V, (N,), generator=g, dtype=torch.int32).cuda()
    k = _rand(torch, g, (N, C), torch.float32).cuda()
    ws, _ = _ws(torch, zs.zero_embed_workspace_bytes(N, C))
    got = torch.empty(V, C, device="cuda")
    zs.zero_embed_bwd(ids, k, got, scale=scale, workspace=ws)
    f = lambda t: _embed_sum(zs, torch, t, ids, k, scale)
    for _ in range(3):
        way = _rand(torch, g, (V, C), torch.float32)
        # (linear in the table: a whole step, its products' roundings of 2^-23 of some 640 terms)
        diff = f((table + way).cuda()) - f((table - way).cuda())
        want = 2 * float((got.cpu().double() * way.double()).sum())
        assert abs(diff - want) < 2e-3


def _embed_sum(zs, torch, table, ids, k, scale):
    out = torch.empty_like(k)
    zs.zero_embed_fwd(table, ids, out, scale=scale)
    return float((out.double() * k.double()).sum())


# ------------------------------------------------------ norms round a block ---

def _block_inputs(torch, T, C, dt, rt, seed, post, gate, block=True, scale=1.0, gate_scale=0.7):
    g = _gen(torch, seed)
    s = dict(x=_rand(torch, g, (T, C), rt, 2.0 * scale), y=None, w1=None, gate=None)
    if block:
        s["y"] = _rand(torch, g, (T, C), dt, 1.5 * scale)
        s["w1"] = _rand(torch, g, (C,), dt, 0.3) if post else None
        s["gate"] = {"none": None, "channel": _rand(torch, g, (C,), dt, gate_scale),
                     "token": _rand(torch, g, (T, C), dt, gate_scale)}[gate]
    s["w2"] = _rand(torch, g, (C,), dt, 0.3)
    s["dh"], s["dz"] = _rand(torch, g, (T, C), rt), _rand(torch, g, (T, C), dt)
    return s


def _block_both(zs, torch, s, *, post, offset=0.0, res=1.0, branch=1.0, eps=1e-6, want_z=True,
                use_dh=True, check_h=True):
    T, C = s["x"].shape
    rt, dt = s["x"].dtype, s["dz"].dtype
    w2 = s["w2"] if want_z else None
    ref = B.Block(s["x"], s["y"], post=post, w1=s["w1"], gate=s["gate"], w2=w2, offset=offset, res=res,
                  branch=branch, eps=eps, dt=dt)
    d = {n: None if t is None else t.cuda() for n, t in s.items()}
    kw = dict(post_norm=post, post_weight=d["w1"], gate=d["gate"], weight_offset=offset, res_scale=res,
              branch_scale=branch, eps=eps, pre_weight=d["w2"] if want_z else None)
    x, _ = _strided(torch, d["x"])
    y = None if d["y"] is None else _strided(torch, d["y"], 24)[0]
    if d["gate"] is not None and d["gate"].dim() == 2:
        kw["gate"] = _strided(torch, d["gate"], 8)[0]
    h, h_rest = _strided(torch, torch.full((T, C), math.nan, dtype=rt, device="cuda"), 32)
    z, z_rest = _strided(torch, torch.full((T, C), math.nan, dtype=dt, device="cuda"), 8)
    zs.zero_block_norm_fwd(x, y, h, z if want_z else None, **kw)
    want = ref.forward(want_z)
    if check_h:
        R.check("h", h, *want["h"])
    if want_z:
        R.check("z", z, *want["z"])
    assert bool((h_rest == 7).all()) and bool((z_rest == 7).all())
    # backward, from the h that is stored
    ws, behind = _ws(torch, zs.zero_block_norm_workspace_bytes(T, C))
    dx, dx_rest = _strided(torch, torch.full((T, C), math.nan, dtype=rt, device="cuda"), 8)
    got = dict(dx=dx)
    if y is not None:
        got["dy"] = torch.full((T, C), math.nan, dtype=dt, device="cuda")
    for n, of in (("dw1", "w1"), ("dgate", "gate"), ("dw2", "w2")):
        got[n] = None if d[of] is None or (n == "dw2" and not want_z) \
            else torch.full_like(d[of], math.nan)
    dh = d["dh"] if use_dh else None
    zs.zero_block_norm_bwd(y, h if want_z else None, dh, d["dz"] if want_z else None, got["dx"],
                           got.get("dy"), dpost_weight=got["dw1"], dgate=got["dgate"],
                           dpre_weight=got["dw2"], workspace=ws, **kw)
    want = ref.backward(h.cpu(), s["dh"] if use_dh else None, s["dz"] if want_z else None)
    for n, t in got.items():
        if t is not None:
            R.check(n, t, *want[n])
    assert bool((behind == 0xFF).all()) and bool((dx_rest == 7).all())
    return h, z, got


WIDTHS = [8, 40, 512, 520, 1000, 1024, 1032, 2048, 2056, 4096, 4104, 8192, 8200, 16384]


@pytest.mark.parametrize("C", WIDTHS)
@pytest.mark.parametrize("types", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")], ids=str)
def test_block_norm_widths(zs, torch, C, types):
    """Every width's kernel, the last row of a workgroup's alone too."""
    dt, rt = _types(torch, *types)
    for T, gate in ((1, "channel"), (6, "token")):
        s = _block_inputs(torch, T, C, dt, rt, C + T, True, gate)
        _block_both(zs, torch, s, post=True, offset=1.0, res=0.9, branch=0.5)


@pytest.mark.parametrize("C", [24, 1000, 1288])
@pytest.mark.parametrize("post", [False, True])
@pytest.mark.parametrize("gate", ["none", "channel", "token"])
@pytest.mark.parametrize("want_z,use_dh", [(True, True), (False, True), (True, False)])
def test_block_norm_forms(zs, torch, C, post, gate, want_z, use_dh):
    s = _block_inputs(torch, 5, C, torch.bfloat16, torch.bfloat16, 3, post, gate)
    _block_both(zs, torch, s, post=post, res=-1.5, branch=0.22, want_z=want_z, use_dh=use_dh)


@pytest.mark.parametrize("C", [64, 1000, 2056])
def test_block_norm_without_weights(zs, torch, C):
    s = _block_inputs(torch, 7, C, torch.bfloat16, torch.float32, 4, True, "none")
    s["w1"] = s["w2"] = None
    _block_both(zs, torch, s, post=True, offset=3.0)


@pytest.mark.parametrize("C", [64, 1000, 2056])
def test_block_norm_without_a_block(zs, torch, C):
    """The plain norm of the residual stream, h wanted and not."""
    s = _block_inputs(torch, 9, C, torch.bfloat16, torch.float32, 5, False, "none", block=False)
    h, z, _ = _block_both(zs, torch, s, post=False, res=0.5)
    _, z, _ = _block_both(zs, torch, s, post=False)
    z2 = torch.empty_like(z)
    zs.zero_block_norm_fwd(s["x"].cuda(), None, None, z2, pre_weight=s["w2"].cuda())
    assert _same(z.contiguous(), z2)


@pytest.mark.parametrize("C,T", [(40, 2100), (1000, 2051), (2048, 515), (4096, 530), (8200, 1030)])
def test_block_norm_many_rows(zs, torch, C, T):
    """More rows than one walk of the backward's workgroups: the sums over the tokens."""
    s = _block_inputs(torch, T, C, torch.bfloat16, torch.bfloat16, 6, True, "channel")
    _block_both(zs, torch, s, post=True, branch=0.5)


@pytest.mark.parametrize("gate", ["channel", "token"])
@pytest.mark.parametrize("C,types", [(1288, ("bf16", "f32")), (2048, ("bf16", "bf16")), (5128, ("f32", "f32")),
                                     (8192, ("bf16", "bf16")), (9000, ("bf16", "f32"))], ids=str)
def test_block_norm_backward_walks(zs, torch, C, types, gate):
    """Three rows and more to a workgroup, two rows side by side and the next row's loads ahead of
    this one's end among them; over its own input, and without the branch's gradient."""
    dt, rt = _types(torch, *types)
    T = 2051 if C <= 2048 else 774
    s = _block_inputs(torch, T, C, dt, rt, C, True, gate)
    h, _, got = _block_both(zs, torch, s, post=True, offset=0.5, branch=0.3)
    d = {n: None if t is None else t.cuda() for n, t in s.items()}
    kw = dict(post_norm=True, post_weight=d["w1"], gate=d["gate"], pre_weight=d["w2"], weight_offset=0.5,
              branch_scale=0.3)
    ws, _ = _ws(torch, zs.zero_block_norm_workspace_bytes(T, C))
    dw2 = torch.empty_like(d["w2"])
    zs.zero_block_norm_bwd(d["y"], h, d["dh"], d["dz"], d["dh"], None, dpre_weight=dw2, workspace=ws, **kw)
    assert _same(d["dh"], got["dx"].contiguous()) and _same(dw2, got["dw2"])


@pytest.mark.parametrize("C,types", [(1024, ("bf16", "bf16")), (2056, ("f32", "f32")), (4096, ("bf16", "f32")),
                                     (8192, ("bf16", "bf16")), (16384, ("bf16", "f32"))], ids=str)
def test_block_norm_outputs_past_the_caches(zs, torch, C, types):
    """Outputs of more than 192 MiB: the rows of the same call on 256 of them, to the bit."""
    dt, rt = _types(torch, *types)
    T = -(-(200 << 20) // (C * ((torch.finfo(dt).bits + torch.finfo(rt).bits) // 8)))
    s = {n: None if t is None else t.cuda()
         for n, t in _block_inputs(torch, 256, C, dt, rt, C, True, "channel").items()}
    some = torch.arange(T, device="cuda") % 251
    big = {n: s[n][some].contiguous() for n in ("x", "y", "dh", "dz")}
    kw = dict(post_norm=True, post_weight=s["w1"], gate=s["gate"], pre_weight=s["w2"], res_scale=0.9)
    out = []
    for d in (s, big):
        h, z, dx, dy = (torch.full_like(d[n], math.nan) for n in ("x", "y", "x", "y"))
        zs.zero_block_norm_fwd(d["x"], d["y"], h, z, **kw)
        zs.zero_block_norm_bwd(d["y"], h, d["dh"], d["dz"], dx, dy, **kw)
        out.append((h, z, dx, dy))
    for a, b in zip(*out):
        assert _same(a[some], b)


@pytest.mark.parametrize("C", [64, 1000, 4096, 16384])
@pytest.mark.parametrize("scale,eps", [(1e25, 1e-6), (1e-20, 0.0), (1e15, 1e-6), (3e-16, 1e-32)])
def test_block_norm_far_rows(zs, torch, C, scale, eps):
    """Rows whose mean square leaves binary32's range are normed as any other.  The branch is
    gated by fp32 numbers of the stream's size where it is added unnormed."""
    s = _block_inputs(torch, 3, C, torch.float32, torch.float32, 7, True, "none", scale=scale)
    s["dh"] = s["dh"] / scale
    s["x"][1] /= scale                          # one ordinary row among them
    _block_both(zs, torch, s, post=True, eps=eps, branch=scale)


@pytest.mark.parametrize("C", [64, 1000, 2056, 16384])
def test_block_norm_nan_stays_in_its_row(zs, torch, C):
    s = _block_inputs(torch, 6, C, torch.bfloat16, torch.bfloat16, 8, True, "token")
    clean, zc, gc = _block_both(zs, torch, s, post=True)
    clean, zc = clean.clone(), zc.clone()
    for n in ("x", "y", "dh", "dz"):
        s[n][2, 3] = math.nan if n != "y" else math.inf
    d = {n: None if t is None else t.cuda() for n, t in s.items()}
    h, z = torch.empty_like(d["x"]), torch.empty_like(d["x"])
    kw = dict(post_norm=True, post_weight=d["w1"], gate=d["gate"], pre_weight=d["w2"])
    zs.zero_block_norm_fwd(d["x"], d["y"], h, z, **kw)
    rows = [0, 1, 3, 4, 5]
    assert _same(h[rows], clean[rows]) and _same(z[rows], zc[rows])
    dx, dy = torch.empty_like(h), torch.empty_like(h)
    zs.zero_block_norm_bwd(d["y"], h, d["dh"], d["dz"], dx, dy, **kw)
    assert _same(dx[rows], gc["dx"][rows]) and _same(dy[rows], gc["dy"][rows])


@pytest.mark.parametrize("C", [64, 1000, 4096, 16384])
def test_block_norm_in_place(zs, torch, C):
    """h over x and dx over dh, to the bit."""
    s = _block_inputs(torch, 9, C, torch.bfloat16, torch.float32, 9, True, "channel")
    h, z, got = _block_both(zs, torch, s, post=True, res=0.8)
    d = {n: None if t is None else t.cuda() for n, t in s.items()}
    kw = dict(post_norm=True, post_weight=d["w1"], gate=d["gate"], pre_weight=d["w2"], res_scale=0.8)
    z2 = torch.empty_like(z.contiguous())
    zs.zero_block_norm_fwd(d["x"], d["y"], d["x"], z2, **kw)
    assert _same(d["x"], h) and _same(z2, z)
    zs.zero_block_norm_bwd(d["y"], d["x"], d["dh"], d["dz"], d["dh"], None, **kw)
    assert _same(d["dh"], got["dx"])


def test_block_norm_no_rows(zs, torch):
    e = torch.empty(0, 64, device="cuda")
    w = torch.ones(64, device="cuda")
    dw = torch.full_like(w, math.nan)
    zs.zero_block_norm_fwd(e, e, e.clone(), e.clone(), pre_weight=w)
    zs.zero_block_norm_bwd(e, e, e, e, e.clone(), e.clone(), pre_weight=w, dpre_weight=dw)
    assert bool((dw == 0).all())


def test_block_norm_gradient_against_differences(zs, torch):
    """All gradients by differences of the 64-bit forward, weighted by dh and dz."""
    s = _block_inputs(torch, 6, 48, torch.float32, torch.float32, 10, True, "channel")
    kw = dict(post=True, offset=0.5, res=0.9, branch=0.7)
    _, _, got = _block_both(zs, torch, s, **kw)

    def f(v):
        b = B.Block(v["x"], v["y"], w1=v["w1"], gate=v["gate"], w2=v["w2"], eps=1e-6, **kw)
        o = b.forward(True)
        return float((o["h"][0] * s["dh"].double()).sum() + (o["z"][0] * s["dz"].double()).sum())

    g = _gen(torch, 11)
    for n, dn in (("x", "dx"), ("y", "dy"), ("w1", "dw1"), ("gate", "dgate"), ("w2", "dw2")):
        way = torch.randn(s[n].shape, generator=g, dtype=torch.float64)
        step = lambda k: f({**{m: t.double() for m, t in s.items()}, n: s[n].double() + k * way})
        diff = (step(1e-5) - step(-1e-5)) / 2e-5
        grad = float((got[dn].cpu().double() * way).sum())
        # h enters the backward as stored in fp32: 2^-24 of gradients of some units, 300 terms
        assert abs(grad - diff) < 1e-4 * (1 + abs(diff)), (n, grad, diff)


# ------------------------------------------------------------ policy loss ---

def _policy_inputs(torch, N, V, dt, seed, scale=2.0, tau=1.0):
    g = _gen(torch, seed)
    z = _rand(torch, g, (N, V), dt, scale)
    act = torch.randint(0, V, (N,), generator=g, dtype=torch.int32)
    act[::3] = z.float().argmax(1)[::3].to(torch.int32)
    x = z.double() / tau
    lp = (x - torch.logsumexp(x, 1, keepdim=True)).gather(1, act.long()[:, None])[:, 0]
    # ratios clear of the borders: inside, and far outside on both sides
    r = torch.tensor([1.0, 0.9, 1.15, 0.5, 1.9, 0.05, 30.0])[torch.arange(N) % 7].double()
    adv = torch.randn(N, generator=g)
    ref = lp + 0.4 * torch.randn(N, generator=g, dtype=torch.float64)
    w = torch.rand(N, generator=g) + 0.2
    return z, act, adv, (lp - r.log()).float(), ref.float(), w


def _policy_all(zs, torch, z, act, adv, old, ref, w, *, tau=1.0, lo=0.2, hi=0.2, kl=0.0, gs=1.0,
                tight=True):
    """Forward alone, forward with the gradient, backward from the statistics, and in
    place."""
    N, V = z.shape
    want = B.policy(z, act, adv, tau=tau, old=old, ref=ref, w=w, lo=lo, hi=hi, kl_coef=kl,
                    grad_scale=gs)
    assert not tight or want["near"] == 0
    d = [None if t is None else t.cuda() for t in (act, adv, old, ref, w)]
    zd = z.cuda()
    kw = dict(old_logp=d[2], ref_logp=d[3], row_weight=d[4], temperature=tau, clip_low=lo, clip_high=hi,
              kl_coef=kl, grad_scale=gs)
    new = lambda *sh: torch.full(sh, math.nan, device="cuda")
    loss, stats = new(N), new(N, 4)
    zs.zero_policy_fwd(zd, d[0], d[1], loss, stats, **kw)
    R.check("loss", loss, *want["loss"])
    R.check("stats", stats, *want["stats"])
    l2, s2, dz = new(N), new(N, 4), torch.full_like(zd, math.nan)
    zs.zero_policy_fwd(zd, d[0], d[1], l2, s2, dlogits=dz, **kw)
    assert _same(loss, l2) and _same(stats, s2)
    R.check("dz", dz, *want["dz"])
    bkw = dict(row_weight=d[4], temperature=tau, grad_scale=gs)
    back = torch.full_like(zd, math.nan)
    zs.zero_policy_bwd(zd, d[0], stats, back, **bkw)
    R.check("dz of the backward", back, *want["dz"])
    inplace = zd.clone()
    zs.zero_policy_fwd(inplace, d[0], d[1], l2, s2, dlogits=inplace, **kw)
    assert _same(inplace, dz)
    inplace = zd.clone()
    zs.zero_policy_bwd(inplace, d[0], stats, inplace, **bkw)
    assert _same(inplace, back)
    return loss, stats, dz


# rows of every kernel: in registers, in shared memory too, and partly read again
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("V", [1, 2, 7, 500, 1031, 2047, 4001, 8185, 12001, 16400, 33333, 65540,
                               131071, 200003])
def test_policy_lengths(zs, torch, V, dtype):
    dt, = _types(torch, dtype)
    N = 7 if V < 50000 else 3
    s = _policy_inputs(torch, N, V, dt, V, tau=0.8)
    _policy_all(zs, torch, *s, tau=0.8, kl=0.1, gs=0.25)


@pytest.mark.parametrize("V,dtype", [(4088, "bf16"), (4090, "bf16"), (8200, "bf16"), (16370, "bf16"),
                                     (32761, "bf16"), (65521, "bf16"), (65529, "bf16"), (103921, "bf16"),
                                     (103937, "bf16"), (2045, "f32"), (32765, "f32"), (51973, "f32"),
                                     (262147, "f32")])
def test_policy_lengths_next_to_the_kernels(zs, torch, V, dtype):
    """The last row of one form and the first of the next; the sampled token in what is kept in
    shared memory or read again; rows that rise to their end, so that every piece has a new maximum."""
    dt, = _types(torch, dtype)
    z, act, adv, old, ref, w = _policy_inputs(torch, 3, V, dt, V)
    z[1] = (z[1].float() + torch.linspace(0, 40, V)).to(dt)
    z[2] = (z[2].float() - torch.linspace(0, 40, V)).to(dt)
    z[2, V // 2:] = -math.inf
    act = torch.tensor([V - 1, V - 2, 5], dtype=torch.int32)
    lp = torch.log_softmax(z.double(), 1).gather(1, act.long()[:, None])[:, 0]
    _policy_all(zs, torch, z, act, adv, (lp + 0.05).float(), (lp - 0.2).float(), w, kl=0.1)


@pytest.mark.parametrize("V,dtype", [(2001, "bf16"), (50257, "bf16"), (90001, "bf16"), (131072, "f32"),
                                     (200003, "bf16")])
def test_policy_masked_stretches(zs, torch, V, dtype):
    """Stretches of the vocabulary at the type's lowest value or -inf: the end, the middle, all but a
    few tokens, whichever pass or piece of the row they fall into."""
    dt, = _types(torch, dtype)
    lowest = torch.finfo(dt).min
    g = _gen(torch, V)
    z = _rand(torch, g, (6, V), dt, 2.0)
    act = torch.tensor([1, V // 3, V - 1, 7, V // 2, 0], dtype=torch.int32)
    z[0, V // 2:] = lowest
    z[1, V // 2:] = -math.inf
    z[2, :V - 5] = lowest
    z[3, 9:] = torch.where(torch.arange(V - 9) % 2 == 0, lowest, -math.inf).to(dt)
    z[4, : V // 2 - 3] = lowest
    z[4, V // 2 + 3:] = -math.inf
    z[5, 1:] = lowest                           # one token alone
    # (the same rows for the oracle: 64 bits need no lowest value, and its bounds take none)
    same = torch.where(z == lowest, -math.inf, z.float()).to(dt)
    lp = torch.log_softmax(same.double(), 1).gather(1, act.long()[:, None])[:, 0]
    adv = torch.tensor([1.0, -0.5, 2.0, -1.0, 0.3, 1.0])
    old, ref = (lp - 0.05).float(), (lp + 0.2).float()
    want = B.policy(same, act, adv, old=old, ref=ref, kl_coef=0.1)
    d = [t.cuda() for t in (z, act, adv, old, ref)]
    loss, stats, dz = torch.empty(6, device="cuda"), torch.empty(6, 4, device="cuda"), torch.empty_like(d[0])
    zs.zero_policy_fwd(*d[:3], loss, stats, dlogits=dz, old_logp=d[3], ref_logp=d[4], kl_coef=0.1)
    R.check("loss", loss, *want["loss"])
    R.check("stats", stats, *want["stats"])
    R.check("dz", dz, *want["dz"])
    zs.zero_policy_bwd(d[0], d[1], stats, dz)
    R.check("dz of the backward", dz, *want["dz"])


@pytest.mark.parametrize("tau,lo,hi", [(1.0, 0.2, 0.28), (0.5, 0.0, 0.0), (3.0, 1.0, 5.0)])
@pytest.mark.parametrize("forms", ["old", "ref", "both", "neither"])
def test_policy_forms(zs, torch, forms, tau, lo, hi):
    z, act, adv, old, ref, w = _policy_inputs(torch, 21, 333, torch.float32, 2, tau=tau)
    if lo == 0.0:                               # (a border at 1 itself: ratios away from it)
        old = old + torch.where(torch.arange(21) % 7 == 0, 0.3, 0.0)
    if forms in ("ref", "neither"):
        old = None
        adv = torch.where(torch.arange(21) % 5 == 0, 0.0, adv)
    if forms in ("old", "neither"):
        ref = None
    _policy_all(zs, torch, z, act, adv, old, ref, None if forms == "old" else w, tau=tau, lo=lo, hi=hi,
                kl=0.3, tight=forms in ("old", "both"))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_policy_strides_and_absent_rows(zs, torch, dtype):
    """Rows that start at any element, rows without an action, without weight, of -inf
    alone and with NaN in them, and what lies between the rows."""
    dt, = _types(torch, dtype)
    N, V = 12, 1003
    z, act, adv, old, ref, w = _policy_inputs(torch, N, V, dt, 3)
    act[2], act[3], act[4] = -1, V, -2 ** 31
    w[5] = 0.0
    z[6] = -math.inf
    z[7, ::2] = -math.inf                       # half of the vocabulary masked
    z[7, act[7]] = 1.0
    x = z[7].double()
    old[7] = float(x[act[7]] - torch.logsumexp(x, 0))
    ref[7] = old[7] + 0.1
    clean = z.clone()
    clean[5] = 0.0
    want = B.policy(clean, act, adv, old=old, ref=ref, w=w, kl_coef=0.1)
    z[5] = math.nan
    wide = torch.full((N, V + 10), 7.0, dtype=dt, device="cuda")
    wide[:, 3:3 + V] = z.cuda()
    dwide = torch.full((N, V + 12), 7.0, dtype=dt, device="cuda")
    zv, dv = wide[:, 3:3 + V], dwide[:, 5:5 + V]
    loss, stats = torch.empty(N, device="cuda"), torch.empty(N, 4, device="cuda")
    d = [t.cuda() for t in (act, adv, old, ref, w)]
    for back in (False, True):
        dv.fill_(math.nan)
        if back:
            zs.zero_policy_bwd(zv, d[0], stats, dv, row_weight=d[4])
        else:
            zs.zero_policy_fwd(zv, d[0], d[1], loss, stats, dlogits=dv, old_logp=d[2], ref_logp=d[3],
                               row_weight=d[4], kl_coef=0.1)
        R.check("dz", dv, *want["dz"])
        assert bool((dwide[:, :5] == 7).all()) and bool((dwide[:, 5 + V:] == 7).all())
    # a NaN beside nothing but -inf is not an absent row, wherever it stands
    for at in (0, int(act[8])):
        z2 = torch.full((1, V), -math.inf, dtype=dt)
        z2[0, at] = math.nan
        l2, s2 = torch.empty(1, device="cuda"), torch.empty(1, 4, device="cuda")
        zs.zero_policy_fwd(z2.cuda(), d[0][8:9], d[1][8:9], l2, s2)
        assert math.isnan(float(l2)) and math.isnan(float(s2[0, 0]))
    R.check("loss", loss, *want["loss"])
    keep = [n for n in range(N) if n != 5]
    R.check("stats", stats[keep], want["stats"][0][keep], want["stats"][1][keep])
    assert bool((dv[2:6] == 0).all()) and bool((loss[2:7] == 0).all())


@pytest.mark.parametrize("V", [300, 33333])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_policy_rows_far_from_0(zs, torch, dtype, V):
    """Rows of the type's lowest value alone, or with -inf; logits that agree where binary32 holds
    no logarithm of a sum beside them: as the same rows next to 0."""
    dt, = _types(torch, dtype)
    g = _gen(torch, 21)
    lowest = torch.finfo(dt).min
    place = torch.arange(V)
    # (what the row is, the same row with its largest value at 0)
    rows = [(torch.full((V,), lowest), torch.zeros(V)),
            (torch.where(place % 3 == 0, -math.inf, lowest), torch.where(place % 3 == 0, -math.inf, 0.0)),
            (torch.full((V,), -1e30), torch.zeros(V)),
            (torch.where(place % 5 == 2, 1e35, torch.randn(V, generator=g)),
             torch.where(place % 5 == 2, 0.0, -math.inf)),
            (torch.where(place == 7, lowest, -1e38), torch.where(place == 7, -math.inf, 0.0))]
    tau = 1.0
    if dt == torch.float32:                     # (differences of some temperatures beside 2^23 of them)
        k = torch.randint(-12, 1, (V,), generator=g).float()
        k[5] = 0.0
        rows.append((2.0 ** 23 + k, k))
        rows.append((-2.0 ** 23 + k, k))
    z, near = (torch.stack([r[i] for r in rows]).to(dt) for i in (0, 1))
    N = len(rows)
    act = torch.tensor([3, 7, 299, 2, 11, 5, 6][:N], dtype=torch.int32)
    adv = torch.tensor([1.0, -0.5, 2.0, 0.7, -1.0, 1.5, -2.0][:N])
    lp = torch.log_softmax(near.double(), 1).gather(1, act.long()[:, None])[:, 0]
    old, ref = (lp - 0.1).float(), (lp + 0.3).float()
    want = B.policy(near, act, adv, tau=tau, old=old, ref=ref, kl_coef=0.2, grad_scale=0.5)
    d = [t.cuda() for t in (z, act, adv, old, ref)]
    loss, stats = torch.empty(N, device="cuda"), torch.empty(N, 4, device="cuda")
    dz, back, inplace = torch.empty_like(d[0]), torch.empty_like(d[0]), d[0].clone()
    zs.zero_policy_fwd(*d[:3], loss, stats, dlogits=dz, old_logp=d[3], ref_logp=d[4], kl_coef=0.2,
                       grad_scale=0.5, temperature=tau)
    zs.zero_policy_bwd(d[0], d[1], stats, back, grad_scale=0.5, temperature=tau)
    zs.zero_policy_bwd(inplace, d[1], stats, inplace, grad_scale=0.5, temperature=tau)
    R.check("loss", loss, *want["loss"])
    R.check("stats", stats[:, 1:], want["stats"][0][:, 1:], want["stats"][1][:, 1:])
    lse = z.double().max(1).values / tau + want["stats"][0][:, 0]
    R.check("lse", stats[:, 0], lse, want["stats"][1][:, 0] + 2 ** -23 * lse.abs())
    R.check("dz", dz, *want["dz"])
    R.check("dz of the backward", back, *want["dz"])
    assert _same(back, inplace)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_policy_ends_of_the_range(zs, torch, dtype):
    """Sure tokens (1 - q far below a rounding of 1), tokens of no probability, logits far
    from 0, ratios that leave binary32 and binary64."""
    dt, = _types(torch, dtype)
    V = 300
    g = _gen(torch, 4)
    z = _rand(torch, g, (8, V), dt, 1.0)
    act = torch.arange(8, dtype=torch.int32) * 3
    for n, lead in ((0, 20.0), (1, 60.0), (2, -30.0), (3, -90.0)):
        z[n, act[n]] = lead
    z[4] = (z[4].float() * 4 + 1000).to(dt)
    z[5] = (z[5].float() * 4 - 5000).to(dt)
    x = z.double()
    lp = (x - torch.logsumexp(x, 1, keepdim=True)).gather(1, act.long()[:, None])[:, 0]
    adv = torch.tensor([1.0, -1.0, 2.0, -0.5, 1.0, 1.0, -1.0, 1.0])
    old = (lp + 0.05).float()
    ref = (lp - 0.2).float()
    _policy_all(zs, torch, z, act, adv, old, ref, None, kl=0.1)
    # a ratio past binary32 with a negative advantage: an infinite loss, the gradient's
    # coefficient its largest number; past binary64 with a positive one: clipped
    old[6], old[7] = float(lp[6]) - 200.0, float(lp[7]) - 2000.0
    d = [t.cuda() for t in (z, act, adv, old)]
    loss, stats = torch.empty(8, device="cuda"), torch.empty(8, 4, device="cuda")
    dz, back = torch.empty_like(d[0]), torch.empty_like(d[0])
    zs.zero_policy_fwd(d[0], d[1], d[2], loss, stats, dlogits=dz, old_logp=d[3])
    zs.zero_policy_bwd(d[0], d[1], stats, back)
    assert float(loss[6]) == math.inf and float(stats[6, 2]) == math.inf
    assert float(loss[7]) == -1.2000000476837158 and float(stats[7, 2]) == 0.0
    assert bool((dz[7] == 0).all()) and bool((back[7] == 0).all())
    for t in (dz, back):
        assert not bool(torch.isnan(t).any())
        assert float(t[6, act[6]]) > 1e38 and bool((t[6] < 0).sum() == V - 1)


def test_policy_gradient_against_differences(zs, torch):
    z, act, adv, old, ref, w = _policy_inputs(torch, 5, 40, torch.float32, 6)
    _, _, dz = _policy_all(zs, torch, z, act, adv, old, ref, w, kl=0.2)
    f = lambda t: float(B.policy(t, act, adv, old=old, ref=ref, w=w, kl_coef=0.2)["loss"][0].sum())
    g = _gen(torch, 7)
    for _ in range(4):
        way = torch.randn(5, 40, generator=g, dtype=torch.float64)
        diff = (f(z.double() + 1e-5 * way) - f(z.double() - 1e-5 * way)) / 2e-5
        grad = float((dz.cpu().double() * way).sum())
        assert abs(grad - diff) < 1e-4 * (1 + abs(diff)), (grad, diff)


# ------------------------------------------- norm and clipping of gradients ---

def _tensors(torch, sizes, types, seed, scale=1.0, offset=0):
    """Views of one buffer of each type, one after another from element `offset` on."""
    g = _gen(torch, seed)
    n = sum(sizes) + offset + 64
    flat = {t: (torch.randn(n, generator=g) * scale).to(t).cuda() for t in set(types)}
    at = {t: offset for t in flat}
    out = []
    for k, t in zip(sizes, types):
        out.append(flat[t][at[t]:at[t] + k])
        at[t] += k
    return out


def _one_by_one(zs, torch, grads, inv):
    acc = zs.new_norm_acc(1)
    for t in grads:
        if t.numel():
            zs.zero_grad_norm(t.clone(), inv, acc)     # (aligned)
    return acc


def _clipped(torch, grads, outs, inv, coef):
    return [((g.float() * inv) * coef).to(o.dtype) for g, o in zip(grads, outs)]


SIZES = [1, 2, 7, 31, 32, 33, 255, 2048, 8191, 8192, 8193, 0, 16400, 100003]


@pytest.mark.parametrize("offset", [0, 1, 3])
@pytest.mark.parametrize("inv", [1.0, 1 / 3])
def test_grads_norm_and_clip(zs, torch, inv, offset):
    """Sizes about every border, both types, any alignment: the norm's accumulator is that
    of the tensors one by one, the clipped tensors the product of binary32, to the bit."""
    bf, f32 = torch.bfloat16, torch.float32
    types = [(bf, f32)[i % 2] for i in range(len(SIZES))]
    grads = _tensors(torch, SIZES, types, offset, offset=offset)
    outs = _tensors(torch, SIZES, [(bf, bf, f32)[i % 3] for i in range(len(SIZES))], 9,
                    offset=offset + 1)
    keep = [t.clone() for t in grads]
    table = zs.GradTable(grads, outs)
    acc = torch.full_like(zs.new_norm_acc(1), -1)
    ws, behind = _ws(torch, zs.zero_grads_workspace_bytes())
    zs.zero_grads_norm(table, acc, inv_scale=inv, workspace=ws)
    want = _one_by_one(zs, torch, grads, inv)
    assert zs.read_norm_acc(acc) == zs.read_norm_acc(want)
    total = sum(float((t.float() * inv).double().square().sum()) for t in grads)
    for max_norm in (0.0, 1.0, 1e9):
        coef, skip = torch.empty(1, device="cuda"), torch.empty(1, dtype=torch.int32, device="cuda")
        zs.zero_step_gate(acc, max_norm, False, coef, skip)
        norm, got_coef = torch.empty(1, device="cuda"), torch.empty(1, device="cuda")
        got_skip = torch.full((1,), 5, dtype=torch.int32, device="cuda")
        zs.zero_grads_clip(table, acc, max_norm=max_norm, inv_scale=inv, norm_out=norm,
                           coef_out=got_coef, skipped_out=got_skip)
        assert abs(float(norm) - math.sqrt(total)) <= 2.0 ** -23 * math.sqrt(total)
        assert _same(coef, got_coef) and int(got_skip) == int(skip) == 0
        for a, b in zip(outs, _clipped(torch, grads, outs, inv, float(coef))):
            assert _same(a, b)
    assert all(_same(a, b) for a, b in zip(grads, keep)) and bool((behind == 0xFF).all())
    # added to, and what lies between the tensors
    zs.zero_grads_norm(table, acc, inv_scale=inv, add=True, workspace=ws)
    twice = _one_by_one(zs, torch, grads + grads, inv)
    assert zs.read_norm_acc(acc) == zs.read_norm_acc(twice)


def test_grads_clip_writes_nothing_else(zs, torch):
    flat = torch.full((5000,), 7.0, dtype=torch.bfloat16, device="cuda")
    grads = [torch.randn(n, device="cuda") for n in (3, 1000, 33)]
    outs = [flat[1:4], flat[11:1011], flat[2001:2034]]
    acc = zs.new_norm_acc(1)
    ws, _ = _ws(torch, zs.zero_grads_workspace_bytes())
    table = zs.GradTable(grads, outs)
    zs.zero_grads_norm(table, acc, workspace=ws)
    zs.zero_grads_clip(table, acc, max_norm=0.5)
    hit = torch.zeros(5000, dtype=torch.bool, device="cuda")
    for a, b in ((1, 4), (11, 1011), (2001, 2034)):
        hit[a:b] = True
    assert bool((flat[~hit] == 7).all()) and not bool((flat[hit] == 7).any())


@pytest.mark.parametrize("count", [1, 159, 160, 161, 239, 240, 241, 255, 256, 257, 520])
def test_grads_more_tensors_than_a_launch(zs, torch, count):
    sizes = [(i * 37) % 300 + 1 for i in range(count)]
    types = [(torch.bfloat16, torch.float32)[i % 3 == 0] for i in range(count)]
    grads = _tensors(torch, sizes, types, count)
    want = _one_by_one(zs, torch, grads, 1.0)
    table = zs.GradTable(grads)
    acc = zs.new_norm_acc(1)
    ws, _ = _ws(torch, zs.zero_grads_workspace_bytes())
    zs.zero_grads_norm(table, acc, workspace=ws)
    assert zs.read_norm_acc(acc) == zs.read_norm_acc(want)
    coef = torch.empty(1, device="cuda")
    before = [t.clone() for t in grads]
    zs.zero_grads_clip(table, acc, max_norm=0.25, coef_out=coef)       # in place
    assert 0 < float(coef) < 1
    for a, b in zip(grads, _clipped(torch, before, grads, 1.0, float(coef))):
        assert _same(a, b)


@pytest.mark.parametrize("n", [8188, 8192, 8195, 24576, 40001])
@pytest.mark.parametrize("offset", [0, 1])
def test_grads_clip_types_of_whole_tiles(zs, torch, n, offset):
    """Every pair of types, whole tiles and cut ones, beside each other in one call."""
    pairs = [(a, b) for a in (torch.bfloat16, torch.float32) for b in (torch.bfloat16, torch.float32)]
    grads = _tensors(torch, [n] * 4, [a for a, _ in pairs], 21, offset=offset)
    outs = _tensors(torch, [n] * 4, [b for _, b in pairs], 22, offset=1 - offset)
    acc = zs.new_norm_acc(1)
    ws, _ = _ws(torch, zs.zero_grads_workspace_bytes())
    table, coef = zs.GradTable(grads, outs), torch.empty(1, device="cuda")
    zs.zero_grads_norm(table, acc, inv_scale=0.3, workspace=ws)
    zs.zero_grads_clip(table, acc, max_norm=2.0, inv_scale=0.3, coef_out=coef)
    inv = float(torch.tensor(0.3))
    for a, b in zip(outs, _clipped(torch, grads, outs, inv, float(coef))):
        assert _same(a, b)


def test_grads_many_tiles(zs, torch):
    """More tiles than workgroups, in both calls, over several tensors."""
    sizes = [8192 * 700 + 5, 8192 * 4100, 11, 8192 * 900 + 8191]
    types = [torch.bfloat16, torch.bfloat16, torch.float32, torch.float32]
    grads = [torch.randn(n, device="cuda").to(t) for n, t in zip(sizes, types)]
    table, acc = zs.GradTable(grads), zs.new_norm_acc(1)
    ws, _ = _ws(torch, zs.zero_grads_workspace_bytes())
    zs.zero_grads_norm(table, acc, workspace=ws)
    assert zs.read_norm_acc(acc) == zs.read_norm_acc(_one_by_one(zs, torch, grads, 1.0))
    coef, before = torch.empty(1, device="cuda"), [t.clone() for t in grads]
    zs.zero_grads_clip(table, acc, max_norm=3.0, coef_out=coef)
    for a, b in zip(grads, _clipped(torch, before, grads, 1.0, float(coef))):
        assert _same(a, b)


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_grads_not_finite(zs, torch, bad):
    """Skipped with the check; without it the coefficient is 0, as the step's."""
    g = [torch.randn(50, device="cuda"), torch.randn(9000, device="cuda").bfloat16()]
    g[1][8999] = bad
    g[0][0] = 3e38
    keep = [t.clone() for t in g]
    table, acc = zs.GradTable(g), zs.new_norm_acc(1)
    ws, _ = _ws(torch, zs.zero_grads_workspace_bytes())
    zs.zero_grads_norm(table, acc, workspace=ws)
    assert zs.read_norm_acc(acc) == zs.read_norm_acc(_one_by_one(zs, torch, g, 1.0))
    norm, coef = torch.empty(1, device="cuda"), torch.empty(1, device="cuda")
    skip = torch.zeros(1, dtype=torch.int32, device="cuda")
    kw = dict(max_norm=1.0, norm_out=norm, coef_out=coef, skipped_out=skip)
    zs.zero_grads_clip(table, acc, check_overflow=True, **kw)
    assert int(skip) == 1 and float(coef) == 0 and float(norm) == math.inf
    assert all(_same(a, b) for a, b in zip(g, keep))
    zs.zero_grads_clip(table, acc, **kw)
    assert int(skip) == 0 and float(coef) == 0 and float(norm) == math.inf
    assert bool((g[0] == 0).all()) and bool(torch.isnan(g[1][8999])) and bool((g[1][:8999] == 0).all())


def test_grads_of_ranks_add_up(zs, torch):
    """The accumulators of two ranks' tensors as one argument, and no accumulator at all."""
    a, b = torch.randn(5000, device="cuda"), torch.randn(777, device="cuda")
    accs = zs.new_norm_acc(2)
    ws, _ = _ws(torch, zs.zero_grads_workspace_bytes())
    for i, t in enumerate((a, b)):
        zs.zero_grads_norm(zs.GradTable([t]), accs.view(2, -1)[i], workspace=ws)
    out, norm = torch.empty_like(a), torch.empty(1, device="cuda")
    zs.zero_grads_clip(zs.GradTable([a], [out]), accs, max_norm=2.0, norm_out=norm)
    want = math.sqrt(float(a.double().square().sum() + b.double().square().sum()))
    assert abs(float(norm) - want) <= 2.0 ** -23 * want
    assert float(out.norm()) < float(a.norm())
    zs.zero_grads_clip(zs.GradTable([a], [out]), None, max_norm=2.0, norm_out=norm)
    assert _same(a, out) and float(norm) == 0.0
    empty = zs.GradTable([])
    acc = torch.full_like(zs.new_norm_acc(1), -1)
    zs.zero_grads_norm(empty, acc, workspace=ws)
    assert int(acc.abs().sum()) == 0
    zs.zero_grads_clip(empty, acc, max_norm=1.0, norm_out=norm)
    assert float(norm) == 0.0


def test_grads_feed_the_step(zs, torch):
    """The norm of many tensors as the gate of the sharded step's update: the same bits as
    from the flat gradient's own norm."""
    n = 4096
    flat = torch.randn(n, device="cuda")
    cuts = [0, 32, 96, 1024, 4096]                # (whole groups of 32)
    table = zs.GradTable([flat[a:b] for a, b in zip(cuts, cuts[1:])])
    acc, want = zs.new_norm_acc(1), zs.new_norm_acc(1)
    ws, _ = _ws(torch, zs.zero_grads_workspace_bytes())
    zs.zero_grads_norm(table, acc, workspace=ws)
    zs.zero_grad_norm(flat, 1.0, want)
    assert zs.read_norm_acc(acc) == zs.read_norm_acc(want)


def test_grad_table_notices_what_moved(zs, torch):
    t = torch.randn(100, device="cuda")
    table, acc = zs.GradTable([t]), zs.new_norm_acc(1)
    ws, _ = _ws(torch, zs.zero_grads_workspace_bytes())
    zs.zero_grads_norm(table, acc, workspace=ws)
    t.data = torch.randn(100, device="cuda")
    with pytest.raises(ValueError):
        zs.zero_grads_norm(table, acc, workspace=ws)
    with pytest.raises(ValueError):
        zs.zero_grads_clip(table, acc, max_norm=1.0)
    g, o = torch.randn(100, device="cuda"), torch.randn(100, device="cuda")
    table = zs.GradTable([g], [o])
    o.data = torch.randn(100, device="cuda")
    with pytest.raises(ValueError):
        zs.zero_grads_clip(table, acc, max_norm=1.0)
    with pytest.raises(ValueError):
        zs.GradTable([t.view(10, 10).t()])
    with pytest.raises(ValueError):
        zs.GradTable([t], [t[:50]])
    with pytest.raises(TypeError):
        zs.GradTable([t.half()])
    # the same tensor twice, neighbours that overlap, an output on another's gradient
    u = torch.randn(200, device="cuda")
    for grads, outs in (([t, t], None), ([u[:100], u[99:]], None), ([u[:100], u[100:]], [u[100:], t]),
                        ([t, u[:100]], [u[50:150], u[:100]])):
        with pytest.raises(ValueError):
            zs.GradTable(grads, outs)
    zs.GradTable([t, t], [u[:100], u[100:]])           # read twice, written apart
    zs.GradTable([u[:100], u[100:]])


# ------------------------------------------- streams, graphs, repeatability ---

def _state(zs, torch, N=333, V=1003, C=1000, seed=3):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    bf = torch.bfloat16
    r = lambda *sh: torch.randn(*sh, generator=g, device="cuda").to(bf)
    s = dict(table=r(V, C), x=r(N, C), y=r(N, C), w1=r(C), gate=r(C), w2=r(C), dh=r(N, C), dz=r(N, C),
             logits=r(N, V))
    s["ids"] = torch.randint(-1, 60, (N,), generator=g, device="cuda", dtype=torch.int32)
    s["adv"] = torch.randn(N, generator=g, device="cuda")
    for n, like in (("emb", "x"), ("dtable", "table"), ("h", "x"), ("z", "x"), ("dx", "x"), ("dy", "x"),
                    ("dw1", "w1"), ("dgate", "gate"), ("dw2", "w2"), ("dl", "logits")):
        s[n] = torch.empty_like(s[like])
    s["loss"], s["stats"] = torch.empty(N, device="cuda"), torch.empty(N, 4, device="cuda")
    s["norm"] = torch.empty(1, device="cuda")
    s["acc"] = zs.new_norm_acc(1)
    s["clipped"] = torch.empty_like(s["dtable"])
    s["grads"] = zs.GradTable([s["dtable"], s["dw1"]], [s["clipped"], s["dw1"]])
    s["ws"] = torch.empty(max(zs.zero_embed_workspace_bytes(N, C),
                              zs.zero_block_norm_workspace_bytes(N, C),
                              zs.zero_grads_workspace_bytes()), dtype=torch.uint8, device="cuda")
    return s


def _pass(zs, s):
    """Every call once, all on one workspace, on the current stream."""
    zs.zero_embed_fwd(s["table"], s["ids"], s["emb"], scale=3.0)
    kw = dict(post_norm=True, post_weight=s["w1"], gate=s["gate"], pre_weight=s["w2"])
    zs.zero_block_norm_fwd(s["emb"], s["y"], s["h"], s["z"], **kw)
    zs.zero_policy_fwd(s["logits"], s["ids"], s["adv"], s["loss"], s["stats"], dlogits=s["dl"])
    zs.zero_policy_bwd(s["logits"], s["ids"], s["stats"], s["dl"])
    zs.zero_block_norm_bwd(s["y"], s["h"], s["dh"], s["dz"], s["dx"], s["dy"], dpost_weight=s["dw1"],
                           dgate=s["dgate"], dpre_weight=s["dw2"], workspace=s["ws"], **kw)
    zs.zero_embed_bwd(s["ids"], s["dx"], s["dtable"], scale=3.0, workspace=s["ws"])
    zs.zero_grads_norm(s["grads"], s["acc"], workspace=s["ws"])
    zs.zero_grads_clip(s["grads"], s["acc"], max_norm=1.0, norm_out=s["norm"])
    return [s[n] for n in ("emb", "h", "z", "loss", "stats", "dl", "dx", "dy", "dw1", "dgate", "dw2",
                           "dtable", "acc", "clipped", "norm")]


@pytest.mark.parametrize("N", [61, 333, 2500])
def test_block_ops_repeat_bitwise_on_streams_and_in_graphs(zs, torch, N):
    """The same bits on every run, on another stream, and from every replay of two recorded
    graphs that share a workspace, with eager work between the replays."""
    s = _state(zs, torch, N)
    torch.cuda.synchronize()
    want = [t.clone() for t in _pass(zs, s)]
    torch.cuda.synchronize()
    outs = _pass(zs, s)
    torch.cuda.synchronize()
    same = lambda: all(_same(a, b) for a, b in zip(want, outs))
    assert same()
    side = torch.cuda.Stream()
    for t in outs:
        t.zero_()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        _pass(zs, s)
    side.synchronize()
    assert same()
    graphs = []
    other = _state(zs, torch, N, seed=4)
    other["ws"] = s["ws"]
    for st in (s, other):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            _pass(zs, st)
    for _ in range(4):
        for t in outs:
            t.zero_()
        s["ws"].fill_(0x55)
        graphs[1].replay()
        graphs[0].replay()
        graphs[1].replay()
        torch.cuda.synchronize()
        assert same()
        _pass(zs, other)
        _pass(zs, s)
        torch.cuda.synchronize()
        assert same()


def test_large_forms_in_a_graph(zs, torch):
    """Long rows of logits, wide rows backward and tokens whose lists are joined in two passes, which
    take other kernels than the pass above: replayed with eager calls between."""
    g = _gen(torch, 31)
    V, N, width, tokens = 90001, 3, 9000, 20000
    z = _rand(torch, g, (N, V), torch.bfloat16, 2.0).cuda()
    act = torch.tensor([5, V - 1, 70000], dtype=torch.int32).cuda()
    adv = torch.tensor([1.0, -0.5, 2.0]).cuda()
    loss, stats, dz = torch.empty(N, device="cuda"), torch.empty(N, 4, device="cuda"), torch.empty_like(z)
    rows = [_rand(torch, g, (600, width), torch.bfloat16).cuda() for _ in range(4)]
    w = _rand(torch, g, (width,), torch.bfloat16).cuda()
    dx, dy, dw = torch.empty_like(rows[0]), torch.empty_like(rows[0]), torch.empty_like(w)
    ws = torch.empty(zs.zero_block_norm_workspace_bytes(600, width), dtype=torch.uint8, device="cuda")
    ids = torch.randint(0, 500, (tokens,), generator=g, dtype=torch.int32).cuda()
    dout = _rand(torch, g, (tokens, 64), torch.bfloat16).cuda()
    dtable = torch.empty(500, 64, device="cuda")
    ews = torch.empty(zs.zero_embed_workspace_bytes(tokens, 64), dtype=torch.uint8, device="cuda")

    def run():
        zs.zero_policy_fwd(z, act, adv, loss, stats, dlogits=dz)
        zs.zero_block_norm_bwd(*rows, dx, dy, dpost_weight=dw, post_norm=True, post_weight=w, workspace=ws)
        zs.zero_embed_bwd(ids, dout, dtable, workspace=ews)

    outs = (loss, stats, dz, dx, dy, dw, dtable)
    run()
    torch.cuda.synchronize()
    want = [t.clone() for t in outs]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    for _ in range(4):
        for t in (*outs, ws, ews):
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(_same(a, b) for a, b in zip(outs, want))
        run()
        torch.cuda.synchronize()
        assert all(_same(a, b) for a, b in zip(outs, want))


def test_block_ops_with_other_memory_between_streams(zs, torch):
    """A call on a stream of its own, given as an argument."""
    s = _state(zs, torch, 100)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    zs.zero_embed_fwd(s["table"], s["ids"], s["emb"], scale=3.0)
    torch.cuda.synchronize()
    want = s["emb"].clone()
    s["emb"].zero_()
    torch.cuda.synchronize()
    zs.zero_embed_fwd(s["table"], s["ids"], s["emb"], scale=3.0, stream=side)
    side.synchronize()
    assert _same(want, s["emb"])


def test_long_rows_past_32_bits(zs, torch):
    """Rows whose offsets pass 32 bits: a table and logits of more than 4 GiB."""
    free = torch.cuda.mem_get_info()[0]
    if free < 40 << 30:
        pytest.skip("needs 40 GiB")
    V, C = 140000, 16384                           # 4.6 GB in bf16
    table = torch.zeros(V, C, dtype=torch.bfloat16, device="cuda")
    table[V - 1] = 1.5
    ids = torch.tensor([V - 1, 0, V - 1, 70001], dtype=torch.int32, device="cuda")
    out = torch.empty(4, C, dtype=torch.bfloat16, device="cuda")
    zs.zero_embed_fwd(table, ids, out, scale=2.0)
    assert bool((out[0] == 3).all()) and bool((out[1] == 0).all()) and bool((out[2] == 3).all())
    table.fill_(9.0)
    ws = torch.empty(zs.zero_embed_workspace_bytes(4, C), dtype=torch.uint8, device="cuda")
    zs.zero_embed_bwd(ids, out, table, workspace=ws)
    assert bool((table[V - 1] == 6).all()) and float(table[:V - 1].float().abs().max()) == 0
    del table
    N, V = 60, 200003                              # rows 80 MB apart
    wide = torch.zeros(N, 40 << 20, dtype=torch.bfloat16, device="cuda")
    z = wide[:, :V]
    z[:, 5] = 3.0
    act = torch.full((N,), 5, dtype=torch.int32, device="cuda")
    loss, stats = torch.empty(N, device="cuda"), torch.empty(N, 4, device="cuda")
    dz = torch.empty(N, V, dtype=torch.bfloat16, device="cuda")
    zs.zero_policy_fwd(z, act, torch.ones(N, device="cuda"), loss, stats, dlogits=dz)
    q = math.exp(3) / (math.exp(3) + V - 1)
    assert float((stats[:, 1] - math.log(q)).abs().max()) < 1e-5
    assert float((dz[:, 5].float() + (1 - q)).abs().max()) < 2.0 ** -8


def test_clip_coefficient_of_any_accumulator(zs, torch):
    """The coefficient of zero_step_gate to the bit, and the norm, for sums from a single
    unit of 2^-128 to the top digit, with carries pending, of one accumulator and of three."""
    g = torch.Generator()
    g.manual_seed(12)
    coef, want = torch.empty(1, device="cuda"), torch.empty(1, device="cuda")
    skip, norm = torch.empty(1, dtype=torch.int32, device="cuda"), torch.empty(1, device="cuda")
    table = zs.GradTable([])
    for case in range(120):
        words = torch.zeros(3, 16, dtype=torch.int64)
        n = 1 if case % 3 else 3
        for a in range(n):
            for k in range(13):
                if case < 13 and k != case:
                    continue
                if torch.rand(1, generator=g) < (1.0 if case < 13 else 0.4):
                    bits = int(torch.randint(1, 50, (1,), generator=g))
                    words[a, k] = int(torch.randint(0, 1 << bits, (1,), generator=g)) + (case % 2)
        if case == 14:                          # a tie: 2^53 + 1 units, and the next up
            words.zero_()
            words[0, 0], words[0, 1] = 1, 1 << 21
        if case == 16:
            words.zero_()
            words[0, 0], words[0, 1] = 3, 1 << 21
        accs = words[:n].cuda()
        X = sum(x for x, _ in zs.read_norm_acc(accs))
        true = math.sqrt(X / 2 ** 128) if X < 2 ** 1000 else 0.0
        for max_norm in (true * 0.7 + 1e-300, 1e-6, 1.0):
            zs.zero_step_gate(accs, max_norm, True, want, skip)
            zs.zero_grads_clip(table, accs, max_norm=max_norm, check_overflow=True, norm_out=norm,
                               coef_out=coef)
            assert _same(coef, want), case
        if true < 3.4e38:
            assert abs(float(norm) - true) <= 2.0 ** -23 * true + 1e-45, case
