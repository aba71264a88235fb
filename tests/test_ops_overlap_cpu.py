"""Calls of the operators around a student's blocks whose outputs lie where they may not, without
a GPU: each is refused before anything is launched, while the same calls with every array in
a place of its own, in place where the header says so, or with rows between one another's, pass
the checks (and end at the launch, as there is no device)."""
import ctypes as C
import os
import subprocess

import pytest

torch = pytest.importorskip("torch")

from test_ops_block_cpu import Args  # noqa: E402
from test_ops_cpu import EINVAL, ROOT, lib  # noqa: E402,F401

EHIP = -4
MB = 1 << 20


def place(n):
    """The n-th place of 1 MB; never dereferenced."""
    return (n + 1) * MB


def _passes(args, fn, **change):
    if not torch.cuda.is_available():          # (with a device it would be launched)
        assert args.call(fn, **change) == EHIP, change


def _refused(args, fn, cases):
    _passes(args, fn)
    for change in cases:
        assert args.call(fn, **change) == EINVAL, change


def test_spans_against_all_pairs_of_rows(tmp_path):
    exe = str(tmp_path / "span_checks")
    subprocess.run(["g++", "-O1", "-g", "-std=c++17", "-fsanitize=address,undefined",
                    "-fno-sanitize-recover=all", "-I",
                    os.path.join(ROOT, "zero_sharded_mixed_step_amd", "csrc"),
                    os.path.join(ROOT, "tests", "sanitize", "span_checks.cpp"), "-o", exe], check=True)
    r = subprocess.run([exe], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.startswith("ok"), (r.returncode, r.stdout, r.stderr[-4000:])


def test_embed_refuses_overlaps(lib):  # noqa: F811
    N, V, W = 300, 50, 64                      # rows of 128 bytes (bf16)
    a = Args("zero_embed_args", N=N, V=V, C=W, dtype=1, scale=1.0, ids=place(0), table=place(1),
             out=place(2), table_stride=W, out_stride=W)
    _refused(a, lib.zero_embed_fwd, [
        dict(out=place(1)), dict(out=place(1) + (V - 1) * 128), dict(out=place(1) - (N - 1) * 128 - 112),
        dict(out=place(0) + 16), dict(table_stride=2 * W, out_stride=2 * W, out=place(1) + 112)])
    # columns of one buffer, and rows in turn
    _passes(a, lib.zero_embed_fwd, table_stride=2 * W, out_stride=2 * W, out=place(1) + 128)
    _passes(a, lib.zero_embed_fwd, table_stride=3 * W, out_stride=6 * W, out=place(1) + 256)
    ws = lib.zero_embed_workspace_bytes(N, W)
    b = Args("zero_embed_args", N=N, V=V, C=W, dtype=1, grad_dtype=1, base_dtype=1, scale=1.0,
             ids=place(0), dout=place(1), base=place(2), dtable=place(3), workspace=place(4),
             workspace_bytes=ws, dout_stride=W, base_stride=W, dtable_stride=W)
    _passes(b, lib.zero_embed_bwd, base=place(3))
    _passes(b, lib.zero_embed_bwd, base=0)
    _passes(b, lib.zero_embed_bwd, N=0, dtable=place(1), workspace=place(1))
    _refused(b, lib.zero_embed_bwd, [
        dict(dtable=place(2) + 128), dict(dtable=place(2) - 128), dict(dtable=place(1)),
        dict(dtable=place(0)), dict(dtable=place(4)), dict(workspace=place(1)), dict(workspace=place(2)),
        dict(workspace=place(0)), dict(dtable=place(4) + ws - 16), dict(base=place(3) + 16)])


def test_block_norm_refuses_overlaps(lib):  # noqa: F811
    T, W = 40, 64
    rows = ("x", "y", "gate", "h", "z", "dh", "dz", "dx", "dy", "dgate")
    kw = {s + "_stride": W for s in rows}
    kw.update({s: place(n) for n, s in enumerate(rows)})
    kw.update(post_w=place(20), pre_w=place(21), dpost_w=place(22), dpre_w=place(23), workspace=place(24),
              workspace_bytes=lib.zero_block_norm_workspace_bytes(T, W))
    a = Args("zero_block_norm_args", T=T, C=W, dtype=1, res_dtype=1, post_norm=1, gate_tokens=1, eps=1e-6,
             res_scale=1.0, branch_scale=1.0, **kw)
    fwd, bwd = lib.zero_block_norm_fwd, lib.zero_block_norm_bwd
    last = (T - 1) * 128
    _passes(a, fwd, h=place(0))
    _refused(a, fwd, [
        dict(z=kw["h"]), dict(z=kw["x"]), dict(z=kw["y"]), dict(h=kw["y"]), dict(h=kw["gate"]),
        dict(z=kw["gate"] + last), dict(h=kw["x"] + 128), dict(h=kw["x"] - 128), dict(z=place(20)),
        dict(z=place(21) + 112), dict(h=place(0), z=place(0)), dict(z=kw["h"] + last + 112)])
    _passes(a, bwd, dx=kw["dh"])
    _passes(a, bwd, dz=0, pre_w=0, dpre_w=0, dx=kw["h"])          # (h is not read)
    _passes(a, bwd, gate_tokens=0, gate=place(25), dgate=place(26))
    _refused(a, bwd, [
        dict(dx=kw["h"]), dict(dx=kw["dz"]), dict(dx=kw["y"]), dict(dx=kw["dh"] + 128), dict(dy=kw["dz"]),
        dict(dy=kw["y"]), dict(dy=kw["h"]), dict(dy=kw["dh"]), dict(dy=kw["dx"]), dict(dgate=kw["gate"]),
        dict(dgate=kw["dy"]), dict(dpost_w=place(20)), dict(dpre_w=place(21)), dict(dpre_w=place(22)),
        dict(dpost_w=kw["dy"]), dict(workspace=kw["dh"]), dict(workspace=kw["dx"]),
        dict(workspace=place(22)), dict(gate_tokens=0, dgate=place(22)),
        dict(gate_tokens=0, dgate=kw["gate"])])
    # x's and the block's halves of one buffer: z beside y, h beside x
    wide = {s + "_stride": 2 * W for s in ("x", "y", "h", "z")}
    _passes(a, fwd, h=kw["x"] + 128, z=kw["y"] + 128, **wide)
    assert a.call(fwd, h=kw["x"] + 112, z=kw["y"] + 128, **wide) == EINVAL


def test_policy_refuses_overlaps(lib):  # noqa: F811
    N, V = 30, 101
    names = ("logits", "dlogits", "action", "advantage", "old_logp", "ref_logp", "row_weight", "loss",
             "stats")
    kw = {s: place(n) for n, s in enumerate(names)}
    a = Args("zero_policy_args", N=N, V=V, dtype=1, temperature=1.0, clip_low=0.2, clip_high=0.2,
             grad_scale=1.0, logits_stride=V, dlogits_stride=V, **kw)
    fwd, bwd = lib.zero_policy_fwd, lib.zero_policy_bwd
    shifted = [dict(dlogits=kw["logits"] + 2), dict(dlogits=kw["logits"] - 2 * V),
               dict(dlogits=kw["logits"] + 2 * (N * V - 1)), dict(dlogits=kw["action"]),
               dict(dlogits=kw["row_weight"]), dict(dlogits=kw["stats"] + 16 * N - 4)]
    for fn in (fwd, bwd):
        _passes(a, fn, dlogits=kw["logits"])
        # one element behind each row belongs to the other
        _passes(a, fn, logits_stride=2 * V, dlogits_stride=2 * V, dlogits=kw["logits"] + 2 * V)
        _refused(a, fn, shifted + [dict(logits_stride=2 * V, dlogits_stride=2 * V,
                                        dlogits=kw["logits"] + 2 * V - 2)])
    _passes(a, fwd, dlogits=0)
    _refused(a, fwd, [dict(loss=kw["advantage"]), dict(loss=kw["stats"] + 4), dict(stats=kw["old_logp"]),
                      dict(stats=kw["logits"]), dict(loss=kw["dlogits"]), dict(stats=kw["ref_logp"]),
                      dict(loss=kw["row_weight"] + 4 * N - 4), dict(stats=kw["action"])])


def test_grads_refuse_overlaps(lib):  # noqa: F811
    n = 3
    sizes = (C.c_int64 * n)(100, 0, 50)
    types = (C.c_int32 * n)(0, 1, 0)           # fp32, bf16, fp32: 400 and 200 bytes
    keep = []

    def table(*at):
        keep.append((C.c_uint64 * n)(*at))
        return C.addressof(keep[-1])

    g = (place(0), place(0) + 16, place(1))
    grads, apart = table(*g), table(place(2), place(0) + 16, place(3))
    a = Args("zero_grads_args", count=n, grads=grads, outs=apart, sizes=C.addressof(sizes),
             dtypes=C.addressof(types), out_dtypes=C.addressof(types), inv_scale=1.0, acc=place(4),
             n_accs=2, accs=place(4), max_norm=1.0, norm_out=place(5), coef_out=place(5) + 4,
             skipped_out=place(5) + 8, workspace=place(6), workspace_bytes=MB)
    norm, clip = lib.zero_grads_norm, lib.zero_grads_clip
    _passes(a, norm, grads=table(place(0), 0, place(0) + 40))      # tensors that are only read
    _refused(a, norm, [dict(acc=place(6)), dict(acc=place(0)), dict(acc=place(1) + 192),
                       dict(workspace=place(1) - MB // 16), dict(workspace=place(4))])
    # in place; into the next tensor; one tensor twice, but to places apart
    _passes(a, clip, outs=grads)
    _passes(a, clip, outs=table(place(2), 0, place(2) + 400))
    _passes(a, clip, grads=table(place(0), 0, place(0)))
    bad = [dict(outs=table(place(2), 0, place(2) + 396)), dict(outs=table(place(0) + 4, 0, place(3))),
           dict(outs=table(place(1), 0, place(3))), dict(outs=table(place(2), 0, place(0) + 396)),
           dict(outs=table(place(2), 0, place(2))), dict(grads=table(place(0), 0, place(0)), outs=grads),
           dict(grads=table(place(0), 0, place(0)), outs=table(place(0), 0, place(0)))]
    _refused(a, clip, bad)
    for change in bad:                         # (a caller that has seen to it itself)
        _passes(a, clip, outs_apart=1, **change)
    small = [dict(norm_out=place(0) + 396), dict(coef_out=place(2)), dict(skipped_out=place(4) + 252),
             dict(norm_out=place(5) + 4), dict(skipped_out=place(5)), dict(accs=place(3)),
             dict(accs=place(2) - 128, n_accs=2)]
    for change in small:
        assert a.call(clip, **change) == EINVAL, change
        assert a.call(clip, outs_apart=1, **change) == EINVAL, change
    _passes(a, clip, norm_out=0, coef_out=0, skipped_out=0, n_accs=0, accs=0)
