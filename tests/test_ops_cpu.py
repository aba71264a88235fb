"""libzero_ops.so without a GPU: its exports, its argument checks (every case is
rejected or has nothing to do, so nothing is launched), the binding's view of
the argument structs, the host helpers, and the 64-bit reference itself
against differences."""
import ctypes as C
import math
import os
import re
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "zero_ops.h")
PKG = os.path.join(ROOT, "zero_sharded_mixed_step_amd")
LIB = os.path.join(PKG, "libzero_ops.so")
FAKE = 0x10000                                   # aligned, never dereferenced
OK, EINVAL, EALIGN, ESIZE = 0, -1, -2, -3

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(LIB):
        pytest.fail("libzero_ops.so is not built (run __graft_entry__.build())")
    from zero_sharded_mixed_step_amd import _ops_binding as B
    return B.ops_lib()


def _text():
    return re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)


def _fields(name):
    """[(type, field, count)] of a struct of the header."""
    body = re.search(r"typedef struct " + name + r" \{(.*?)\} " + name + ";", _text(), re.S).group(1)
    out = []
    for decl in body.split(";"):
        decl = " ".join(decl.split())
        if not decl:
            continue
        m = re.match(r"(const )?(\w+) (.*)", decl)
        for f in m.group(3).split(","):
            f = f.strip()
            n = re.search(r"\[(\d+)\]", f)
            kind = "ptr" if "*" in decl.split(",")[0] or f.startswith("*") else m.group(2)
            out.append((kind, re.sub(r"[\*\s]|\[\d+\]", "", f), int(n.group(1)) if n else 1))
    return out


CODES = {"ptr": "Q", "size_t": "Q", "int64_t": "q", "int32_t": "i", "double": "d"}
STRUCTS = {"zero_qk_norm_rope_args": "_NORM_ARGS", "zero_attn_args": "_ATTN_ARGS",
           "zero_distill_args": "_DISTILL_ARGS"}


class Args:
    """A struct of the header as named values; call() packs them."""

    def __init__(self, name, **values):
        from zero_sharded_mixed_step_amd import _ops_binding as B
        self.packer, self.fields = getattr(B, STRUCTS[name]), _fields(name)
        self.v = {f: ([0] * n if n > 1 else 0.0 if k == "double" else 0)
                  for k, f, n in self.fields}
        self.v["struct_bytes"] = self.packer.size
        self.v.update(values)

    def call(self, fn, **change):
        flat = []
        for _, f, n in self.fields:
            x = change.get(f, self.v[f])
            flat += list(x) if n > 1 else [x]
        return fn(self.packer.pack(*flat), None)


def test_binding_structs_follow_the_header():
    from zero_sharded_mixed_step_amd import _ops_binding as B
    for name, packer in STRUCTS.items():
        want = "".join(CODES[k] * n for k, _, n in _fields(name))
        got = "".join(c * int(n or 1) for n, c in
                      re.findall(r"(\d*)([Qqid])", getattr(B, packer).format))
        assert got == want, name
    consts = dict(re.findall(r"#define (ZERO_\w+) (.+)", open(HEADER).read()))
    assert int(consts["ZERO_OPS_ABI_VERSION"]) == B.OPS_ABI_VERSION
    assert int(consts["ZERO_ATTN_MAX_REACH"]) == B.ATTN_MAX_REACH
    assert int(consts["ZERO_ATTN_MAX_BUCKETS"]) == B.ATTN_MAX_BUCKETS
    assert int(consts["ZERO_DISTILL_MAX_K"]) == B.DISTILL_MAX_K
    assert consts["ZERO_DISTILL_MAX_V"] == "(1 << 20)" and B.DISTILL_MAX_V == 1 << 20


def test_exports_every_declared_symbol(lib):
    names = set(re.findall(r"\b(zero_[a-z0-9_]+)\s*\(", _text()))
    assert {"zero_attn_fwd", "zero_attn_bwd", "zero_attn_ranges", "zero_distill_fwd",
            "zero_distill_bwd", "zero_qk_norm_rope_fwd", "zero_qk_norm_rope_bwd"} <= names
    assert not [n for n in names if not hasattr(lib, n)]
    import zero_sharded_mixed_step_amd as zs
    assert not [n for n in names if not hasattr(zs, n)]


def test_header_compiles_as_c11_and_agrees_on_sizes(tmp_path):
    from zero_sharded_mixed_step_amd import _ops_binding as B
    src = tmp_path / "t.c"
    src.write_text('#include "zero_ops.h"\n' + "".join(
        f"_Static_assert(sizeof({n}) == {getattr(B, p).size}, \"size\");\n"
        for n, p in STRUCTS.items()) + "int main(void) { return 0; }\n")
    r = subprocess.run(["gcc", "-std=c11", "-pedantic", "-Werror", "-Wall", "-Wextra",
                        "-fsyntax-only", "-I", os.path.join(ROOT, "include"), str(src)],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr


def test_status_strings(lib):
    texts = {lib.zero_ops_strerror(s) for s in (0, -1, -2, -3, -4, 7)}
    assert len(texts) == 6 and all(texts)


def test_norm_argument_checks(lib):
    a = Args("zero_qk_norm_rope_args", T=8, Hq=2, Hk=1, D=64, rot_dim=64, dtype=1, eps=1e-6,
             q=FAKE, k=FAKE, wq=FAKE, wk=FAKE, pos=FAKE, inv_freq=FAKE, yq=FAKE, yk=FAKE, dyq=FAKE,
             dyk=FAKE, dq=FAKE, dk=FAKE, workspace=FAKE, workspace_bytes=1 << 20,
             **{s + "_stride": [128, 64] for s in ("q", "k", "yq", "yk", "dyq", "dyk", "dq", "dk")})
    for fn, fwd in ((lib.zero_qk_norm_rope_fwd, True), (lib.zero_qk_norm_rope_bwd, False)):
        assert fn(None, None) == EINVAL
        bad = [(dict(struct_bytes=8), EINVAL), (dict(dtype=2), EINVAL), (dict(T=-1), EINVAL),
               (dict(Hq=-1), EINVAL), (dict(eps=-1.0), EINVAL), (dict(eps=math.nan), EINVAL),
               (dict(D=60), ESIZE), (dict(D=264), ESIZE), (dict(D=0), ESIZE),
               (dict(rot_dim=72), ESIZE), (dict(rot_dim=40), ESIZE), (dict(rot_dim=-8), ESIZE),
               (dict(rot_dim=36, interleaved=1), ESIZE), (dict(T=1 << 40), ESIZE),
               (dict(pos=0), EINVAL), (dict(inv_freq=0), EINVAL), (dict(pos=FAKE + 2), EALIGN),
               (dict(inv_freq=FAKE + 4), EALIGN), (dict(wq=FAKE + 8), EALIGN),
               (dict(q=0), EINVAL), (dict(k=FAKE + 8), EALIGN), (dict(q_stride=[129, 64]), EALIGN)]
        if fwd:
            bad += [(dict(yq=0), EINVAL), (dict(yk=FAKE + 2), EALIGN),
                    (dict(yk_stride=[128, 60]), EALIGN)]
        else:
            bad += [(dict(dyq=0), EINVAL), (dict(dq=FAKE + 2), EALIGN),
                    (dict(dwq=FAKE, wq=0), EINVAL), (dict(dwk=FAKE + 1), EALIGN),
                    (dict(dwq=FAKE, workspace=0), EINVAL),
                    (dict(dwq=FAKE, workspace=FAKE + 8), EALIGN),
                    (dict(dwq=FAKE, workspace_bytes=16), ESIZE)]
        for change, status in bad:
            assert a.call(fn, **change) == status, change
        assert a.call(fn, T=0) == OK
        assert a.call(fn, Hq=0, Hk=0) == OK
    assert lib.zero_qk_norm_rope_workspace_bytes(8, 64) >= 2 * 64 * 4
    assert lib.zero_qk_norm_rope_workspace_bytes(1 << 20, 128) <= 1 << 20


def test_attention_argument_checks(lib):
    strides = {s + "_stride": [8192, 128, 64] for s in ("q", "k", "v", "o", "do", "dq", "dk", "dv")}
    a = Args("zero_attn_args", B=1, Tq=16, Tk=16, Hq=2, Hk=1, D=64, scale=0.1, q=FAKE, k=FAKE,
             v=FAKE, o=FAKE, lse=FAKE, d_o=FAKE, dq=FAKE, dk=FAKE, dv=FAKE, workspace=FAKE,
             workspace_bytes=1 << 24, **strides)
    bias = dict(bias_table=FAKE, bias_buckets=FAKE, n_buckets=8, reach=4, bias_dtype=1)
    for fn, fwd in ((lib.zero_attn_fwd, True), (lib.zero_attn_bwd, False)):
        assert fn(None, None) == EINVAL
        bad = [(dict(struct_bytes=1), EINVAL), (dict(Hk=0), EINVAL), (dict(Hq=3, Hk=2), EINVAL),
               (dict(B=-1), EINVAL), (dict(D=48), ESIZE), (dict(D=256), ESIZE),
               (dict(Tq=1 << 22), ESIZE), (dict(B=1 << 23, Hq=4), ESIZE),
               (dict(scale=math.inf), EINVAL), (dict(cap=-1.0), EINVAL), (dict(cap=math.nan), EINVAL),
               (dict(cap=1e-60), EINVAL), (dict(q=0), EINVAL), (dict(k=FAKE + 8), EALIGN),
               (dict(v_stride=[8192, 132, 64]), EALIGN), (dict(lse=0), EINVAL),
               (dict(lse=FAKE + 1), EALIGN), (dict(ranges=FAKE + 4), EALIGN),
               (dict(bias, bias_buckets=0), EINVAL), (dict(bias, n_buckets=0), EINVAL),
               (dict(bias, n_buckets=257), ESIZE), (dict(bias, reach=513), ESIZE),
               (dict(bias, reach=-1), EINVAL), (dict(bias, bias_dtype=2), EINVAL),
               (dict(bias, bias_table=FAKE + 1), EALIGN)]
        if not fwd:
            bad += [(dict(d_o=0), EINVAL), (dict(dq=FAKE + 8), EALIGN), (dict(dk=0), EINVAL),
                    (dict(dv_stride=[1, 128, 64]), EALIGN), (dict(dbias_table=FAKE), EINVAL),
                    (dict(bias, dbias_table=FAKE + 1), EALIGN), (dict(workspace=0), EINVAL),
                    (dict(workspace=FAKE + 8), EALIGN), (dict(workspace_bytes=100), ESIZE)]
        else:
            many = dict(Tk=65536, k_stride=[0, 128, 64])
            bad += [(dict(many, workspace=0), EINVAL), (dict(many, workspace_bytes=64), ESIZE),
                    (dict(many, workspace=FAKE + 4), EALIGN)]
        for change, status in bad:
            assert a.call(fn, **change) == status, change
        assert a.call(fn, B=0) == OK
    assert a.call(lib.zero_attn_fwd, Tq=0, q=0, o=0, lse=0) == OK
    w = lib.zero_attn_workspace_bytes
    assert w(1, 16, 16, 2, 3, 64, 0, 1) == 0 and w(8, 1024, 1024, 12, 12, 64, 0, 0) == 0
    assert w(1, 16, 16, 2, 1, 64, 8, 1) >= 4 * 2 * 32
    rng = lib.zero_attn_ranges
    assert rng(FAKE, None, -1, 4, 1, FAKE, None) == EINVAL
    assert rng(None, None, 1, 4, 1, FAKE, None) == EINVAL
    assert rng(FAKE, None, 1, 4, 1, FAKE + 4, None) == EALIGN
    assert rng(FAKE, FAKE + 1, 1, 4, 1, FAKE, None) == EALIGN
    assert rng(FAKE, None, 1, 1 << 22, 1, FAKE, None) == ESIZE
    assert rng(None, None, 0, 4, 1, None, None) == OK


def test_distill_argument_checks(lib):
    a = Args("zero_distill_args", N=4, V=100, K=8, dtype=1, temperature=2.0, grad_scale=1.0,
             logits=FAKE, teacher_idx=FAKE, teacher_val=FAKE, loss=FAKE, stats=FAKE, dlogits=FAKE,
             logits_stride=100, dlogits_stride=100)
    for fn, fwd in ((lib.zero_distill_fwd, True), (lib.zero_distill_bwd, False)):
        assert fn(None, None) == EINVAL
        bad = [(dict(struct_bytes=1), EINVAL), (dict(dtype=2), EINVAL), (dict(N=-1), EINVAL),
               (dict(V=0), EINVAL), (dict(K=0), EINVAL), (dict(K=1025), ESIZE),
               (dict(V=(1 << 20) + 1), ESIZE), (dict(N=1 << 22), ESIZE),
               (dict(temperature=0.0), EINVAL), (dict(temperature=math.nan), EINVAL),
               (dict(temperature=-1.0), EINVAL), (dict(grad_scale=math.inf), EINVAL),
               (dict(logits=0), EINVAL), (dict(teacher_idx=0), EINVAL), (dict(teacher_val=0), EINVAL),
               (dict(stats=0), EINVAL), (dict(logits=FAKE + 1), EALIGN),
               (dict(teacher_idx=FAKE + 2), EALIGN), (dict(teacher_lse=FAKE + 2), EALIGN),
               (dict(row_weight=FAKE + 1), EALIGN), (dict(stats=FAKE + 2), EALIGN),
               (dict(dlogits=FAKE + 1), EALIGN), (dict(dlogits_stride=99), EINVAL)]
        bad += [(dict(loss=0), EINVAL)] if fwd else [(dict(dlogits=0), EINVAL)]
        for change, status in bad:
            assert a.call(fn, **change) == status, change
        assert a.call(fn, N=0) == OK


def test_binding_refuses_host_tensors_and_wrong_shapes():
    """Checked before the library is called: no GPU is needed."""
    import zero_sharded_mixed_step_amd as zs
    x = torch.zeros(1, 4, 2, 64, dtype=torch.bfloat16)
    lse = torch.zeros(1, 2, 4)
    with pytest.raises(TypeError):
        zs.zero_attn_fwd(x, x, x, x, lse)
    with pytest.raises(ValueError):
        zs.zero_attn_fwd(x[0], x, x, x, lse)
    with pytest.raises(TypeError):
        zs.zero_attn_bwd(x, x, x, x, lse, None, x, x, x)
    with pytest.raises(TypeError):
        zs.zero_qk_norm_rope_fwd(x[0], None, x[0], None)
    with pytest.raises(ValueError):
        zs.zero_qk_norm_rope_fwd(None, None, None, None)
    with pytest.raises(TypeError):
        zs.zero_qk_norm_rope_fwd(x[0].half(), None, x[0], None)
    z = torch.zeros(2, 10)
    with pytest.raises(TypeError):
        zs.zero_distill_fwd(z, torch.zeros(2, 3, dtype=torch.int32), z[:, :3], z[:, 0], z[:, :2])
    with pytest.raises(TypeError):
        zs.zero_distill_bwd(z, torch.zeros(2, 3, dtype=torch.int32), z[:, :3], z[:, :2], None)


def test_no_kernel_uses_scratch():
    from test_kernel_resources import _kernels
    path = LIB + ".resources.txt"
    if not os.path.exists(path):
        pytest.skip("libzero_ops.so was built without its resource report")
    kernels = _kernels(path)
    assert kernels
    assert not {k for k, v in kernels.items() if v.get("ScratchSize [bytes/lane]", 0) != 0
                or v.get("VGPRs Spill", 0) != 0}


@pytest.mark.parametrize("n,reach,both", [(32, 128, False), (32, 128, True), (8, 20, False),
                                          (2, 2, False), (6, 7, True), (64, 512, False)])
def test_relpos_buckets(n, reach, both):
    """Against the formula in 64 bits wherever that is clear of a border, and
    its shape: one distance to a bucket, then widening, saturating at the reach."""
    import zero_sharded_mixed_step_amd as zs
    b = zs.relpos_buckets(n, reach, bidirectional=both)
    assert b.dtype == torch.int32 and b.shape == (2 * reach + 1,)
    m = n // 2 if both else n
    exact = m // 2
    for d in range(0, reach + 1):
        got = int(b[reach - d])
        if d < exact:
            assert got == d
            continue
        x = math.log(d / exact) / math.log(reach / exact) * (m - exact)
        if abs(x - round(x)) > 1e-9:
            assert got == min(m - 1, exact + int(x))
        else:
            assert got == min(m - 1, exact + round(x))
    back = b[:reach + 1].flip(0)
    assert bool((back.diff() >= 0).all()) and int(back[-1]) == m - 1
    ahead = b[reach + 1:]
    assert torch.equal(ahead, back[1:] + m) if both else bool((ahead == 0).all())
    with pytest.raises(ValueError):
        zs.relpos_buckets(1, 8)


def test_rope_frequencies():
    import zero_sharded_mixed_step_amd as zs
    f = zs.rope_inv_freq(8, 100.0)
    assert f.dtype == torch.float64 and f.tolist() == pytest.approx(
        [1.0, 100 ** -0.25, 100 ** -0.5, 100 ** -0.75], rel=1e-15)


# ------------------------------------- the 64-bit reference, by differences ---

def _directional(f, x, grad, gen, h=1e-5, rel=1e-6):
    way = torch.randn(x.shape, generator=gen, dtype=torch.float64)
    diff = float(f(x + h * way) - f(x - h * way)) / (2 * h)
    got = float((grad * way).sum())
    scale = float((grad.abs() * way.abs()).sum())
    assert abs(got - diff) <= rel * scale + 1e-9, (got, diff)


def test_reference_attention_gradients():
    import ops_ref as R
    g = torch.Generator().manual_seed(1)
    B, T, Hq, Hk, D = 2, 9, 4, 2, 8
    q, k, v, do = (torch.randn(B, T, h, D, generator=g, dtype=torch.float64)
                   for h in (Hq, Hk, Hk, Hq))
    table = torch.randn(5, Hq, generator=g, dtype=torch.float64)
    buckets = torch.tensor([0, 1, 2, 3, 4, 4, 9], dtype=torch.int32)
    doc = torch.tensor([[0, 0, 0, 1, 1, 1, 1, -1, -1], [3] * 9])
    seen = R.visible(B, T, T, R.doc_ranges(doc, torch.full((B, T), 2)))
    at = [q, k, v, table]

    def run(x):
        return R.Attention(x[0], x[1], x[2], scale=0.4, cap=2.0, seen=seen, table=x[3],
                           buckets=buckets)

    a = run(at)
    o = a.forward()[0]
    got = a.backward(o, do)
    for n, name in enumerate(("dq", "dk", "dv", "dtable")):
        def f(x, n=n):
            return (run(at[:n] + [x] + at[n + 1:]).forward()[0] * do).sum()
        _directional(f, at[n], got[name][0], g)


def test_reference_norm_gradients():
    import ops_ref as R
    g = torch.Generator().manual_seed(2)
    pos, freq = torch.tensor([0, 3, 70000]), torch.tensor([1.0, 0.1, 0.01, 0.001]).double()
    for inter in (False, True):
        x, dy = (torch.randn(3, 2, 16, generator=g, dtype=torch.float64) for _ in range(2))
        w = torch.randn(16, generator=g, dtype=torch.float64)
        f = lambda x, w: (R.norm_forward(x, w, 1e-3, pos, freq, inter)[0] * dy).sum()
        got = R.norm_backward(x, w, dy, 1e-3, pos, freq, inter)
        _directional(lambda x: f(x, w), x, got["dx"][0], g)
        _directional(lambda w: f(x, w), w, got["dw"][0], g)


def test_reference_distill_gradients():
    import ops_ref as R
    g = torch.Generator().manual_seed(3)
    z = torch.randn(3, 12, generator=g, dtype=torch.float64)
    idx = torch.tensor([[3, 1, 7], [0, -1, 11], [5, 6, 12]], dtype=torch.int32)
    val = torch.randn(3, 3, generator=g, dtype=torch.float64)
    w = torch.tensor([1.0, 0.5, 2.0])
    for tlse in (None, torch.tensor([2.5, 2.0, 3.0])):
        f = lambda z: R.distill(z, idx, val, 1.7, tlse, w)["loss"][0].sum() * 0.3
        _directional(f, z, R.distill(z, idx, val, 1.7, tlse, w, 0.3)["dz"][0], g)


def test_reference_document_ranges():
    import ops_ref as R
    doc = torch.tensor([[4, 4, 4, -1, 2, 2, 4]])
    want = [[0, 2], [0, 2], [0, 3], [0, 0], [4, 6], [4, 6], [6, 7]]
    assert R.doc_ranges(doc, torch.full((1, 7), 2))[0].tolist() == want
    assert R.doc_ranges(doc, causal=False)[0].tolist()[0] == [0, 3]
