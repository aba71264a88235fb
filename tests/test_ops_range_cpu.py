"""More of libzero_ops.so's argument checks without a GPU: numbers that the kernels
cannot take.  Every case is rejected, so nothing is launched."""
import math

import pytest

from test_ops_cpu import EINVAL, FAKE, Args, lib  # noqa: F401  (the fixture)

torch = pytest.importorskip("torch")


def _norm(**kw):
    strides = {s + "_stride": [128, 64] for s in ("q", "k", "yq", "yk", "dyq", "dyk", "dq", "dk")}
    at = {n: FAKE + 0x1000 * i for i, n in enumerate(("q", "k", "yq", "yk", "dyq", "dyk", "dq", "dk"))}
    return Args("zero_qk_norm_rope_args", **dict(dict(T=8, Hq=2, Hk=1, D=64, rot_dim=64, dtype=1,
                                                      eps=1e-6, wq=FAKE, wk=FAKE, pos=FAKE,
                                                      inv_freq=FAKE, **at, **strides), **kw))


def _attn(**kw):
    strides = {s + "_stride": [8192, 128, 64] for s in ("q", "k", "v", "o", "do", "dq", "dk", "dv")}
    return Args("zero_attn_args", **dict(dict(B=1, Tq=16, Tk=16, Hq=2, Hk=1, D=64, scale=0.1, q=FAKE,
                                              k=FAKE, v=FAKE, o=FAKE, lse=FAKE, d_o=FAKE, dq=FAKE,
                                              dk=FAKE, dv=FAKE, workspace=FAKE,
                                              workspace_bytes=1 << 24, **strides), **kw))


def _distill(**kw):
    return Args("zero_distill_args", **dict(dict(N=4, V=100, K=8, dtype=1, temperature=2.0,
                                                 grad_scale=1.0, logits=FAKE, teacher_idx=FAKE,
                                                 teacher_val=FAKE, loss=FAKE, stats=FAKE,
                                                 dlogits=FAKE + 0x1000, logits_stride=100,
                                                 dlogits_stride=100), **kw))


def test_numbers_past_binary32(lib):  # noqa: F811
    for fn in (lib.zero_qk_norm_rope_fwd, lib.zero_qk_norm_rope_bwd):
        assert _norm().call(fn, eps=1e40) == EINVAL
    for fn in (lib.zero_attn_fwd, lib.zero_attn_bwd):
        for scale in (1e39, -1e300, math.nan):
            assert _attn().call(fn, scale=scale) == EINVAL
        for cap in (2e30, 1e300):
            assert _attn().call(fn, cap=cap) == EINVAL
    for fn in (lib.zero_distill_fwd, lib.zero_distill_bwd):
        for change in (dict(temperature=1e-31), dict(temperature=1e-300), dict(temperature=1e31),
                       dict(temperature=1e300), dict(grad_scale=1e39), dict(grad_scale=-1e300),
                       dict(grad_scale=math.nan)):
            assert _distill().call(fn, **change) == EINVAL, change


def test_in_place_with_other_strides(lib):  # noqa: F811
    """An output that is its input has to be laid out as it is: with other strides rows
    would be written before they are read."""
    same, wide = [128, 64], [256, 64]
    f, b = lib.zero_qk_norm_rope_fwd, lib.zero_qk_norm_rope_bwd
    for fn, x, y in ((f, "q", "yq"), (f, "k", "yk"), (b, "dyq", "dq"), (b, "dyk", "dk")):
        for strides in ((wide, same), (same, wide)):
            a = _norm(Hk=2, **{x: FAKE, y: FAKE, x + "_stride": strides[0], y + "_stride": strides[1]})
            assert a.call(fn) == EINVAL, (x, y)
        a = _norm(Hk=2, **{x: FAKE, y: FAKE, x + "_stride": [512, 64], y + "_stride": [512, 128]})
        assert a.call(fn) == EINVAL, (x, y)
    for fn in (lib.zero_distill_fwd, lib.zero_distill_bwd):
        for strides in ((128, 100), (100, 128)):
            assert _distill(dlogits=FAKE, logits_stride=strides[0],
                            dlogits_stride=strides[1]).call(fn) == EINVAL
