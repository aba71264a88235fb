"""The operators around a student's blocks without a GPU: argument checks (every case is
rejected or has nothing to do, so nothing is launched), the binding's view of the
structs, its own checks, and the 64-bit reference against differences."""
import math
import os
import re
import subprocess

import pytest

torch = pytest.importorskip("torch")

import ops_block_ref as B  # noqa: E402
import test_ops_cpu as base  # noqa: E402
from test_ops_cpu import CODES, EALIGN, EINVAL, ESIZE, FAKE, OK, ROOT, lib  # noqa: E402,F401

STRUCTS = {"zero_embed_args": "_EMBED_ARGS", "zero_block_norm_args": "_BLOCK_NORM_ARGS",
           "zero_policy_args": "_POLICY_ARGS", "zero_grads_args": "_GRADS_ARGS"}


def _fields(name):
    return [(k, re.sub("^const", "", f), n) for k, f, n in base._fields(name)]


class Args:
    """A struct of the header as named values; call() packs them."""

    def __init__(self, name, **values):
        from zero_sharded_mixed_step_amd import _ops_binding as ops
        self.packer, self.fields = getattr(ops, STRUCTS[name]), _fields(name)
        self.v = {f: 0.0 if k == "double" else 0 for k, f, _ in self.fields}
        self.v["struct_bytes"] = self.packer.size
        self.v.update(values)

    def call(self, fn, **change):
        assert not set(change) - set(self.v), change
        return fn(self.packer.pack(*(change.get(f, self.v[f]) for _, f, _ in self.fields)), None)


def _check(args, fn, cases):
    assert fn(None, None) == EINVAL
    for change, status in cases:
        assert args.call(fn, **change) == status, change


def test_binding_structs_and_limits_follow_the_header():
    from zero_sharded_mixed_step_amd import _ops_binding as ops
    for name, packer in STRUCTS.items():
        want = "".join(CODES[k] * n for k, _, n in _fields(name))
        got = "".join(c * int(n or 1) for n, c in
                      re.findall(r"(\d*)([Qqid])", getattr(ops, packer).format))
        assert got == want, name
    text = open(base.HEADER).read()
    for c, v in (("ROW_MAX_C", ops.ROW_MAX_C), ("EMBED_MAX_V", ops.EMBED_MAX_V),
                 ("POLICY_MAX_V", ops.POLICY_MAX_V), ("GRADS_MAX_COUNT", ops.GRADS_MAX_COUNT)):
        shift = re.search(r"#define ZERO_%s \(1 << (\d+)\)" % c, text)
        assert v == 1 << int(shift.group(1)), c


def test_header_agrees_on_sizes(tmp_path):
    from zero_sharded_mixed_step_amd import _ops_binding as ops
    src = tmp_path / "t.c"
    src.write_text('#include "zero_ops.h"\n' + "".join(
        f"_Static_assert(sizeof({n}) == {getattr(ops, p).size}, \"size\");\n"
        for n, p in STRUCTS.items()) + "int main(void) { return 0; }\n")
    r = subprocess.run(["gcc", "-std=c11", "-pedantic", "-Werror", "-Wall", "-Wextra",
                        "-fsyntax-only", "-I", os.path.join(ROOT, "include"), str(src)],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr


def test_embed_argument_checks(lib):  # noqa: F811
    a = Args("zero_embed_args", N=8, V=20, C=64, dtype=1, grad_dtype=0, base_dtype=1, scale=1.0,
             ids=FAKE, table=FAKE, out=FAKE, dout=FAKE, dtable=FAKE, table_stride=64, out_stride=64,
             dout_stride=64, base_stride=64, dtable_stride=64, workspace=FAKE,
             workspace_bytes=1 << 20)
    both = [(dict(struct_bytes=8), EINVAL), (dict(dtype=2), EINVAL), (dict(N=-1), EINVAL),
            (dict(V=0), EINVAL), (dict(scale=math.inf), EINVAL), (dict(scale=math.nan), EINVAL),
            (dict(scale=1e39), EINVAL), (dict(N=(1 << 21) + 1), ESIZE), (dict(V=(1 << 24) + 1), ESIZE),
            (dict(C=0), ESIZE), (dict(C=12), ESIZE), (dict(C=(1 << 14) + 8), ESIZE),
            (dict(ids=0), EINVAL), (dict(ids=FAKE + 2), EALIGN)]
    _check(a, lib.zero_embed_fwd, both + [
        (dict(table=0), EINVAL), (dict(table=FAKE + 8), EALIGN), (dict(table_stride=65), EALIGN),
        (dict(out=0), EINVAL), (dict(out=FAKE + 2), EALIGN), (dict(out_stride=68), EALIGN),
        (dict(out_stride=56), EINVAL), (dict(out_stride=0), EINVAL), (dict(N=0, table=0), OK)])
    _check(a, lib.zero_embed_bwd, both + [
        (dict(grad_dtype=2), EINVAL), (dict(base=FAKE, base_dtype=3), EINVAL), (dict(dtable=0), EINVAL),
        (dict(dtable=FAKE + 8), EALIGN), (dict(dtable_stride=60), EINVAL), (dict(dout=0), EINVAL),
        (dict(dout=FAKE + 4), EALIGN), (dict(dout_stride=65), EALIGN), (dict(base=FAKE + 8), EALIGN),
        (dict(base=FAKE), EINVAL), (dict(base=FAKE, base_dtype=0, base_stride=128), EINVAL),
        (dict(N=300, workspace=0), EINVAL), (dict(N=300, workspace=FAKE + 8), EALIGN),
        (dict(N=300, workspace_bytes=64), ESIZE)])
    w = lib.zero_embed_workspace_bytes
    assert w(0, 64) == 0 and w(-1, 64) == 0 and w(300, 64) >= 4 * 1200 + 2 * 75 * 64 * 4
    # (less than the gradient itself takes, beside the lists)
    assert w(1 << 20, 4096) < (1 << 20) * 4096 * 2 // 4


def test_block_norm_argument_checks(lib):  # noqa: F811
    strides = {s + "_stride": 64 for s in ("x", "y", "gate", "h", "z", "dh", "dz", "dx", "dy", "dgate")}
    a = Args("zero_block_norm_args", T=8, C=64, dtype=1, res_dtype=0, post_norm=1, gate_tokens=1,
             eps=1e-6, res_scale=1.0, branch_scale=1.0, x=FAKE, y=FAKE, post_w=FAKE, gate=FAKE,
             pre_w=FAKE, h=FAKE + 4096, z=FAKE, dh=FAKE, dz=FAKE, dx=FAKE + 4096, dy=FAKE, dpost_w=FAKE,
             dgate=FAKE, dpre_w=FAKE, workspace=FAKE, workspace_bytes=1 << 20, **strides)
    both = [(dict(struct_bytes=1), EINVAL), (dict(dtype=2), EINVAL), (dict(res_dtype=2), EINVAL),
            (dict(dtype=0, res_dtype=1), EINVAL), (dict(T=-1), EINVAL), (dict(eps=-1.0), EINVAL),
            (dict(eps=math.nan), EINVAL), (dict(weight_offset=math.inf), EINVAL),
            (dict(res_scale=math.nan), EINVAL), (dict(branch_scale=1e39), EINVAL),
            (dict(T=(1 << 21) + 1), ESIZE), (dict(C=60), ESIZE), (dict(C=0), ESIZE),
            (dict(C=(1 << 14) + 8), ESIZE), (dict(post_norm=0), EINVAL),
            (dict(y=0, post_w=0, post_norm=0), EINVAL), (dict(y=0, post_w=0, gate=0), EINVAL),
            (dict(post_w=FAKE + 8), EALIGN), (dict(pre_w=FAKE + 2), EALIGN),
            (dict(gate=FAKE + 8), EALIGN), (dict(gate_stride=65), EALIGN), (dict(y=FAKE + 8), EALIGN),
            (dict(y_stride=4), EALIGN)]
    _check(a, lib.zero_block_norm_fwd, both + [
        (dict(x=0), EINVAL), (dict(x=FAKE + 8), EALIGN), (dict(x_stride=65), EALIGN),
        (dict(h=0, z=0), EINVAL), (dict(z=0), EINVAL), (dict(h=FAKE, h_stride=128), EINVAL),
        (dict(h=FAKE + 8), EALIGN), (dict(h_stride=60), EINVAL), (dict(z=FAKE + 8), EALIGN),
        (dict(z_stride=56), EINVAL), (dict(T=0, x=0), OK)])
    _check(a, lib.zero_block_norm_bwd, both + [
        (dict(post_w=0), EINVAL), (dict(gate=0), EINVAL), (dict(pre_w=0), EINVAL), (dict(dz=0), EINVAL),
        (dict(dz=0, dpre_w=0, dh=0), EINVAL), (dict(h=0), EINVAL), (dict(dh=FAKE + 8), EALIGN),
        (dict(dh=FAKE + 4096, dh_stride=128), EINVAL), (dict(dx_stride=60), EINVAL),
        (dict(dy_stride=0), EINVAL), (dict(dgate_stride=8), EINVAL), (dict(dgate=FAKE + 8), EALIGN),
        (dict(dpost_w=FAKE + 1), EALIGN), (dict(dpre_w=FAKE + 1), EALIGN),
        (dict(gate_tokens=0, dgate=FAKE + 1), EALIGN), (dict(workspace=0), EINVAL),
        (dict(workspace=FAKE + 4), EALIGN), (dict(workspace_bytes=256), ESIZE),
        (dict(y=0, post_w=0, post_norm=0, gate=0, dgate=0, dpost_w=0), EINVAL)])
    w = lib.zero_block_norm_workspace_bytes
    assert w(0, 64) == 0 and w(8, 64) >= 3 * 64 * 4 and w(1 << 20, 4096) <= 512 * 3 * 4096 * 4


def test_policy_argument_checks(lib):  # noqa: F811
    a = Args("zero_policy_args", N=4, V=100, dtype=1, temperature=2.0, clip_low=0.2, clip_high=0.2,
             grad_scale=1.0, logits=FAKE, action=FAKE, advantage=FAKE, loss=FAKE, stats=FAKE,
             dlogits=FAKE, logits_stride=100, dlogits_stride=100)
    both = [(dict(struct_bytes=1), EINVAL), (dict(dtype=2), EINVAL), (dict(N=-1), EINVAL),
            (dict(V=0), EINVAL), (dict(V=(1 << 20) + 1), ESIZE), (dict(N=(1 << 21) + 1), ESIZE),
            (dict(temperature=0.0), EINVAL), (dict(temperature=math.nan), EINVAL),
            (dict(temperature=1e31), EINVAL), (dict(grad_scale=math.inf), EINVAL),
            (dict(logits=0), EINVAL), (dict(action=0), EINVAL), (dict(stats=0), EINVAL),
            (dict(logits=FAKE + 1), EALIGN), (dict(action=FAKE + 2), EALIGN),
            (dict(stats=FAKE + 2), EALIGN), (dict(row_weight=FAKE + 1), EALIGN),
            (dict(dlogits=FAKE + 1), EALIGN), (dict(dlogits_stride=99), EINVAL),
            (dict(logits_stride=101), EINVAL), (dict(N=0, logits=0), OK)]
    _check(a, lib.zero_policy_fwd, both + [
        (dict(clip_low=-0.1), EINVAL), (dict(clip_low=1.1), EINVAL), (dict(clip_low=math.nan), EINVAL),
        (dict(clip_high=-0.1), EINVAL), (dict(clip_high=math.inf), EINVAL),
        (dict(kl_coef=math.nan), EINVAL), (dict(advantage=0), EINVAL), (dict(loss=0), EINVAL),
        (dict(advantage=FAKE + 2), EALIGN), (dict(loss=FAKE + 1), EALIGN),
        (dict(old_logp=FAKE + 2), EALIGN), (dict(ref_logp=FAKE + 2), EALIGN)])
    _check(a, lib.zero_policy_bwd, both + [(dict(dlogits=0), EINVAL)])


def test_grads_argument_checks(lib):  # noqa: F811
    import ctypes as C

    def host(kind, *values):
        return (kind * len(values))(*values)

    at = lambda x: C.addressof(x)
    keep = dict(ptrs=host(C.c_uint64, FAKE, FAKE + 64), off=host(C.c_uint64, FAKE, FAKE + 1),
                none=host(C.c_uint64, FAKE, 0), sizes=host(C.c_int64, 5, 7), neg=host(C.c_int64, 5, -1),
                huge=host(C.c_int64, 1 << 37, 1), types=host(C.c_int32, 1, 0), bad=host(C.c_int32, 1, 2))
    p = {n: at(x) for n, x in keep.items()}
    a = Args("zero_grads_args", count=2, grads=p["ptrs"], outs=p["ptrs"], sizes=p["sizes"],
             dtypes=p["types"], out_dtypes=p["types"], inv_scale=1.0, acc=FAKE, n_accs=1, accs=FAKE,
             max_norm=1.0, workspace=FAKE, workspace_bytes=1 << 20)
    both = [(dict(struct_bytes=1), EINVAL), (dict(count=-1), EINVAL), (dict(count=(1 << 16) + 1), ESIZE),
            (dict(inv_scale=math.inf), EINVAL), (dict(grads=0), EINVAL), (dict(sizes=0), EINVAL),
            (dict(dtypes=0), EINVAL), (dict(dtypes=p["bad"]), EINVAL), (dict(sizes=p["neg"]), EINVAL),
            (dict(sizes=p["huge"]), ESIZE), (dict(grads=p["none"]), EINVAL),
            (dict(grads=p["off"]), EALIGN)]
    _check(a, lib.zero_grads_norm, both + [
        (dict(acc=0), EINVAL), (dict(acc=FAKE + 8), EALIGN), (dict(workspace=0), EINVAL),
        (dict(workspace=FAKE + 4), EALIGN), (dict(workspace_bytes=128), ESIZE),
        (dict(count=0, add=1), OK)])
    swapped = host(C.c_int32, 0, 1)
    _check(a, lib.zero_grads_clip, both + [
        (dict(outs=0), EINVAL), (dict(out_dtypes=0), EINVAL), (dict(out_dtypes=p["bad"]), EINVAL),
        (dict(outs=p["none"]), EINVAL), (dict(outs=p["off"]), EALIGN),
        (dict(out_dtypes=at(swapped)), EINVAL), (dict(n_accs=-1), EINVAL), (dict(accs=0), EINVAL),
        (dict(accs=FAKE + 8), EALIGN), (dict(max_norm=math.nan), EINVAL),
        (dict(norm_out=FAKE + 2), EALIGN), (dict(coef_out=FAKE + 2), EALIGN),
        (dict(skipped_out=FAKE + 1), EALIGN)])
    assert lib.zero_grads_workspace_bytes() == 1024 * 14 * 8


def test_binding_refuses_host_tensors_and_wrong_shapes():
    """Checked before the library is called: no GPU is needed."""
    import zero_sharded_mixed_step_amd as zs
    x, ids = torch.zeros(4, 64), torch.zeros(4, dtype=torch.int32)
    for bad, call in (
            (TypeError, lambda: zs.zero_embed_fwd(x, ids, x)),
            (TypeError, lambda: zs.zero_embed_fwd(x.half(), ids, x)),
            (ValueError, lambda: zs.zero_embed_fwd(x[0], ids, x)),
            (ValueError, lambda: zs.zero_embed_fwd(x, ids.view(2, 2), x)),
            (TypeError, lambda: zs.zero_embed_bwd(ids, x, x)),
            (TypeError, lambda: zs.zero_embed_bwd(ids, x.half(), x)),
            (TypeError, lambda: zs.zero_embed_bwd(ids, None, x)),
            (TypeError, lambda: zs.zero_block_norm_fwd(x, x, x, x)),
            (ValueError, lambda: zs.zero_block_norm_fwd(x[0], x, x, x)),
            (TypeError, lambda: zs.zero_block_norm_fwd(x.half(), None, x, x)),
            (ValueError, lambda: zs.zero_block_norm_bwd(x, None, None, x, None, x)),
            (TypeError, lambda: zs.zero_block_norm_bwd(x, x, x, x, x, x)),
            (TypeError, lambda: zs.zero_policy_fwd(x, ids, x[:, 0], x[:, 0], x[:, :4])),
            (ValueError, lambda: zs.zero_policy_fwd(x[0], ids, x[:, 0], x[:, 0], x[:, :4])),
            (TypeError, lambda: zs.zero_policy_bwd(x, ids, x[:, :4], None)),
            (TypeError, lambda: zs.zero_policy_bwd(x.half(), ids, x[:, :4], x)),
            (TypeError, lambda: zs.GradTable([x])),
            (ValueError, lambda: zs.GradTable([x], []))):
        with pytest.raises(bad):
            call()
    table = zs.GradTable([])
    with pytest.raises(TypeError):
        zs.zero_grads_norm(table, torch.zeros(1, 16, dtype=torch.int64))


def _gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


def test_block_reference_against_differences():
    """The 64-bit reference's own gradients, from its own forward."""
    g = _gen(1)
    T, C = 4, 12
    r = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)
    for post, gate in ((True, r(C)), (False, r(T, C)), (True, None)):
        s = dict(x=r(T, C), y=r(T, C), w1=r(C) if post else None, gate=gate, w2=r(C))
        dh, dz = r(T, C), r(T, C)
        make = lambda v: B.Block(v["x"], v["y"], post=post, w1=v["w1"], gate=v["gate"], w2=v["w2"],
                                 offset=0.3, res=0.8, branch=1.3)
        f = lambda v: float((make(v).forward(True)["h"][0] * dh).sum()
                            + (make(v).forward(True)["z"][0] * dz).sum())
        got = make(s).backward(make(s).forward(False)["h"][0], dh, dz)
        for n, dn in (("x", "dx"), ("y", "dy"), ("w1", "dw1"), ("gate", "dgate"), ("w2", "dw2")):
            if s[n] is None:
                continue
            way = r(*s[n].shape)
            diff = (f({**s, n: s[n] + 1e-6 * way}) - f({**s, n: s[n] - 1e-6 * way})) / 2e-6
            assert abs(diff - float((got[dn][0] * way).sum())) < 1e-6 * (1 + abs(diff)), n


def test_policy_reference_against_differences_and_plain_cases():
    g = _gen(2)
    z = torch.randn(6, 9, generator=g, dtype=torch.float64)
    act = torch.tensor([0, 3, 8, 5, 1, 2], dtype=torch.int32)
    adv = torch.tensor([1.0, -1.0, 2.0, -0.5, 0.3, 0.0])
    lp = (z / 0.7 - torch.logsumexp(z / 0.7, 1, keepdim=True)).gather(1, act.long()[:, None])[:, 0]
    old = lp - torch.tensor([1.0, 1.0, 1.5, 0.5, 0.5, 1.1]).log()
    kw = dict(tau=0.7, old=old, ref=lp + 0.3, w=torch.tensor([1.0, 2.0, 1.0, 1.0, 0.5, 1.0]), kl_coef=0.2)
    out = B.policy(z, act, adv, **kw)
    for _ in range(3):
        way = torch.randn(6, 9, generator=g, dtype=torch.float64)
        f = lambda k: float(B.policy(z + k * way, act, adv, **kw)["loss"][0].sum())
        diff = (f(1e-6) - f(-1e-6)) / 2e-6
        assert abs(diff - float((out["dz"][0] * way).sum())) < 1e-7 * (1 + abs(diff))
    # clipped above with a positive advantage, below with a negative one: the KL term alone
    g_kl = -0.2 * math.expm1(0.3)
    assert abs(float(out["stats"][0][2, 2]) - g_kl) < 1e-12
    assert abs(float(out["stats"][0][3, 2]) - g_kl) < 1e-12
    assert abs(float(out["stats"][0][0, 2]) - (-1.0 + g_kl)) < 1e-12


def test_embed_reference_sums_rows():
    ids = torch.tensor([2, 0, -1, 2, 9], dtype=torch.int32)
    d = torch.arange(10.0).view(5, 2)
    val, _ = B.embed_backward(ids, d, 4, 0.5, None, torch.float32)
    assert val.tolist() == [[1.0, 1.5], [0.0, 0.0], [3.0, 4.0], [0.0, 0.0]]
    out, _ = B.embed_forward(torch.tensor([[1.0], [2.0], [3.0], [4.0]]), ids, 2.0)
    assert out[:, 0].tolist() == [6.0, 2.0, 0.0, 6.0, 0.0]
