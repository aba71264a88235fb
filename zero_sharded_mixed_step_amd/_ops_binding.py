"""ctypes binding of libzero_ops.so (include/zero_ops.h), with the C entry
points' names: the training operators whose gradients the sharded step reduces.

Argument marshalling only, as in `_binding`: tensors become device pointers
and element strides, the current torch stream becomes the hipStream_t, and a
nonzero status raises ZeroOpsError.  The caller owns every buffer, outputs
and workspaces included, so every call can be recorded into a HIP graph.
There is no host or fallback path.
"""
import ctypes as C
import os
import struct

import torch

from . import build as _build
from ._binding import ZERO_BF16, ZERO_F32, ZeroStepError, _stream

OPS_ABI_VERSION = 2
ATTN_MAX_REACH = 512
ATTN_MAX_BUCKETS = 256
DISTILL_MAX_K = 1024
DISTILL_MAX_V = 1 << 20
ROW_MAX_C = 1 << 14
EMBED_MAX_V = 1 << 24
POLICY_MAX_V = 1 << 20
GRADS_MAX_COUNT = 1 << 16

# The argument structs of zero_ops.h, field by field (native alignment).
_NORM_ARGS = struct.Struct("@Qq6id14Q16q2Q")
_ATTN_ARGS = struct.Struct("@Q10i2d13Q24q2Q")
_DISTILL_ARGS = struct.Struct("@Q2q2i2d8Q2q")
_EMBED_ARGS = struct.Struct("@Q2q4id6Q5q2Q")
_BLOCK_NORM_ARGS = struct.Struct("@Qq6i4d14Q10q2Q")
_POLICY_ARGS = struct.Struct("@Q2q2i5d9Q2q")
_GRADS_ARGS = struct.Struct("@Qq5QdQ2iQd2i5Q")

_BF16 = torch.bfloat16
_CODES = {torch.float32: ZERO_F32, torch.bfloat16: ZERO_BF16}

_lib = None


class ZeroOpsError(ZeroStepError):
    """A status of libzero_ops.so; `status` as of the step's own library."""

    def __init__(self, status, fn):
        RuntimeError.__init__(self, f"{fn}: {zero_ops_strerror(status)} (status {status})")
        self.status = status


def ops_lib():
    """Load libzero_ops.so; fails loudly when it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(_build.OPS_LIB):
            raise RuntimeError(f"{_build.OPS_LIB} is not built: run __graft_entry__.build() "
                               "(there is no non-HIP implementation)")
        L = C.CDLL(_build.OPS_LIB)
        vp, i, i64 = C.c_void_p, C.c_int, C.c_int64
        L.zero_ops_abi_version.restype = i
        L.zero_ops_strerror.argtypes = [i]
        L.zero_ops_strerror.restype = C.c_char_p
        for name in ("zero_qk_norm_rope_fwd", "zero_qk_norm_rope_bwd", "zero_attn_fwd",
                     "zero_attn_bwd", "zero_distill_fwd", "zero_distill_bwd", "zero_embed_fwd",
                     "zero_embed_bwd", "zero_block_norm_fwd", "zero_block_norm_bwd",
                     "zero_policy_fwd", "zero_policy_bwd", "zero_grads_norm",
                     "zero_grads_clip"):
            f = getattr(L, name)
            f.argtypes, f.restype = [C.c_char_p, vp], i
        L.zero_qk_norm_rope_workspace_bytes.argtypes = [i64, i]
        L.zero_qk_norm_rope_workspace_bytes.restype = C.c_size_t
        L.zero_attn_workspace_bytes.argtypes = [i] * 8
        L.zero_attn_workspace_bytes.restype = C.c_size_t
        L.zero_attn_ranges.argtypes = [vp, vp, i, i, i, vp, vp]
        L.zero_attn_ranges.restype = i
        for name in ("zero_embed_workspace_bytes", "zero_block_norm_workspace_bytes"):
            f = getattr(L, name)
            f.argtypes, f.restype = [i64, i], C.c_size_t
        L.zero_grads_workspace_bytes.argtypes = []
        L.zero_grads_workspace_bytes.restype = C.c_size_t
        if L.zero_ops_abi_version() != OPS_ABI_VERSION:
            raise RuntimeError(f"{_build.OPS_LIB} has ABI version {L.zero_ops_abi_version()}, the "
                               f"binding expects {OPS_ABI_VERSION}: rebuild it")
        _lib = L
    return _lib


def zero_ops_abi_version() -> int:
    return ops_lib().zero_ops_abi_version()


def zero_ops_strerror(status: int) -> str:
    return ops_lib().zero_ops_strerror(int(status)).decode()


def _device():
    """The current device, asked once a call (the checks and packing below are
    what a small call costs: some 10 us of host time for 10 tensors)."""
    if torch.cuda.is_initialized():
        return torch._C._cuda_getDevice()
    return torch.cuda.current_device() if torch.cuda.is_available() else -1


def _call(fn, args, stream, dev):
    if stream is None:
        s = torch._C._cuda_getCurrentRawStream(dev)
    else:
        s = _stream(stream)
    status = getattr(_lib or ops_lib(), fn)(args, s)
    if status != 0:
        raise ZeroOpsError(status, fn)


def _refuse(t, name, shape, dtype, dev):
    """Says what is wrong with a tensor that is not on device `dev`, of `dtype` and `shape`."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA (HIP) tensor")
    if t.get_device() != dev:
        raise ValueError(f"{name} is on {t.device}; the library launches on the current "
                         f"device, cuda:{dev}")
    if t.dtype is not dtype:
        raise TypeError(f"{name}: dtype {t.dtype}, the call needs {dtype}")
    raise ValueError(f"{name} has shape {tuple(t.shape)}, the call needs {tuple(shape)}")


# (These three look at each tensor with as few calls as say all: some 0.5 us a tensor, of
# which a small call has time for few.)

def _tensor(t, name, shape, dtype, dev, Tensor=torch.Tensor):
    """Address and strides of a tensor on device `dev` with the given shape
    and dtype, whose last dimension is contiguous."""
    if not isinstance(t, Tensor) or t.get_device() != dev or dev < 0 or \
            t.dtype is not dtype or t.shape != shape:
        _refuse(t, name, shape, dtype, dev)
    st = t.stride()
    if st and st[-1] != 1 and shape[-1] > 1:
        raise ValueError(f"{name}: the last dimension must be contiguous")
    return t.data_ptr(), st


def _flat(t, name, shape, dtype, dev, Tensor=torch.Tensor):
    """Address of a contiguous tensor; 0 for None."""
    if t is None:
        return 0
    if not isinstance(t, Tensor) or t.get_device() != dev or dev < 0 or \
            t.dtype is not dtype or t.shape != shape:
        _refuse(t, name, shape, dtype, dev)
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _used(shape, strides):
    """Strides of all dimensions but the last, 0 where the size is 1: a stride
    that nothing uses need not be aligned."""
    if 1 in shape:
        return tuple(0 if n == 1 else s for n, s in zip(shape[:-1], strides))
    return strides[:-1]


def _workspace(ws, dev):
    if ws is None:
        return 0, 0
    if not isinstance(ws, torch.Tensor) or not ws.is_cuda or not ws.is_contiguous():
        raise TypeError("workspace must be a contiguous CUDA (HIP) tensor")
    if ws.get_device() != dev:
        raise ValueError(f"workspace is on {ws.device}, not on the current device")
    return ws.data_ptr(), ws.numel() * ws.element_size()


# ------------------------------------------------------------------- norm ---

def rope_inv_freq(rot_dim: int, base: float = 10000.0) -> torch.Tensor:
    """base^(-2i / rot_dim), i < rot_dim / 2, as float64 on the host: the usual
    frequencies of the rotation.  Move it to the device once."""
    return float(base) ** (-torch.arange(0, rot_dim, 2, dtype=torch.float64) / rot_dim)


def zero_qk_norm_rope_workspace_bytes(T: int, D: int) -> int:
    return ops_lib().zero_qk_norm_rope_workspace_bytes(int(T), int(D))


_NO_STRIDE = (0, 0)


def _heads(x, name, T, like, dtype, dev):
    """Address and two strides of one tensor of rows of heads shaped as `like`."""
    if like is None:
        if x is not None:
            raise ValueError(f"{name} without its input")
        return 0, _NO_STRIDE
    p, st = _tensor(x, name, like.shape, dtype, dev)
    return p, _used(like.shape, st)


def _norm_call(fn, q, k, outs, grads, wq, wk, dwq, dwk, eps, pos, inv_freq, interleaved,
               workspace, stream):
    x = q if q is not None else k
    if x is None:
        raise ValueError("one of q and k must be given")
    if not isinstance(x, torch.Tensor) or x.dim() != 3:
        raise ValueError("q and k are (T, H, D) tensors")
    T, _, D = x.shape
    dt = x.dtype
    code = _CODES.get(dt)
    if code is None:
        raise TypeError(f"q and k are float32 or bfloat16, not {dt}")
    if k is not None and (k.dim() != 3 or k.shape[0] != T or k.shape[2] != D):
        raise ValueError(f"k has shape {tuple(k.shape)}, the call needs ({T}, H, {D})")
    dev = _device()
    pq, sq = _heads(q, "q", T, q, dt, dev)
    pk, sk = _heads(k, "k", T, k, dt, dev)
    poq, soq = _heads(outs[0], "the output of q", T, q, dt, dev)
    pok, sok = _heads(outs[1], "the output of k", T, k, dt, dev)
    pairs = pos_p = freq_p = 0
    if inv_freq is not None:
        pairs = inv_freq.shape[0]
        pos_p = _flat(pos, "pos", (T,), torch.int32, dev)
        freq_p = _flat(inv_freq, "inv_freq", (pairs,), torch.float64, dev)
        if pos is None:
            raise ValueError("inv_freq needs pos")
    wqp, wkp = _flat(wq, "wq", (D,), dt, dev), _flat(wk, "wk", (D,), dt, dev)
    head = (_NORM_ARGS.size, T, 0 if q is None else q.shape[1], 0 if k is None else k.shape[1], D,
            2 * pairs, code, 1 if interleaved else 0, eps, pq, pk, wqp, wkp, pos_p, freq_p)
    if grads is None:
        args = _NORM_ARGS.pack(*head, poq, pok, 0, 0, 0, 0, 0, 0, *sq, *sk, *soq, *sok, 0, 0, 0, 0,
                               0, 0, 0, 0, 0, 0)
    else:
        pgq, sgq = _heads(grads[0], "dyq", T, q, dt, dev)
        pgk, sgk = _heads(grads[1], "dyk", T, k, dt, dev)
        args = _NORM_ARGS.pack(*head, 0, 0, pgq, pgk, poq, pok, _flat(dwq, "dwq", (D,), dt, dev),
                               _flat(dwk, "dwk", (D,), dt, dev), *sq, *sk, 0, 0, 0, 0, *sgq, *sgk,
                               *soq, *sok, *_workspace(workspace, dev))
    _call(fn, args, stream, dev)


def zero_qk_norm_rope_fwd(q, k, yq, yk, *, wq=None, wk=None, eps=1e-6, pos=None, inv_freq=None,
                          interleaved=False, stream=None) -> None:
    """RMS norm of every head of q (T, Hq, D) and k (T, Hk, D) with the weights
    wq and wk (D), and the rotation by pos (T, int32) times inv_freq (float64,
    half the rotated width): yq and yk.  q or k may be None, views of one
    projection's output are fine, and yq may be q."""
    _norm_call("zero_qk_norm_rope_fwd", q, k, (yq, yk), None, wq, wk, None, None, eps,
               pos, inv_freq, interleaved, None, stream)


def zero_qk_norm_rope_bwd(q, k, dyq, dyk, dq, dk, *, wq=None, wk=None, dwq=None, dwk=None,
                          eps=1e-6, pos=None, inv_freq=None, interleaved=False, workspace=None,
                          stream=None) -> None:
    """Gradients of zero_qk_norm_rope_fwd from its inputs and dyq, dyk: dq, dk
    and, where given, dwq and dwk (which need a workspace of
    zero_qk_norm_rope_workspace_bytes(T, D) bytes)."""
    _norm_call("zero_qk_norm_rope_bwd", q, k, (dq, dk), (dyq, dyk), wq, wk,
               dwq, dwk, eps, pos, inv_freq, interleaved, workspace, stream)


# -------------------------------------------------------------- attention ---

def relpos_buckets(num_buckets: int, max_distance: int, bidirectional: bool = False,
                   device=None) -> torch.Tensor:
    """The usual map of key-minus-query distances in [-max_distance,
    max_distance] to buckets (int32, 2 max_distance + 1 entries), for
    zero_attn_fwd's bias_buckets: of the buckets of one direction the first
    half holds one distance each, the rest widen geometrically up to
    max_distance.  Keys ahead of the query share bucket 0, or with
    `bidirectional` have the second half of the buckets.  Borders are decided
    in whole numbers."""
    n = num_buckets // 2 if bidirectional else num_buckets
    exact = n // 2
    if exact < 1 or max_distance <= exact or num_buckets > ATTN_MAX_BUCKETS \
            or max_distance > ATTN_MAX_REACH:
        raise ValueError("relpos_buckets: 2 or more buckets a direction, half as many < "
                         f"max_distance <= {ATTN_MAX_REACH}, at most {ATTN_MAX_BUCKETS} buckets")
    steps = n - exact

    def one(d):
        if d < exact:
            return d
        # the largest t with d >= exact * (max_distance / exact)^(t / steps)
        t = 0
        while t < steps and d ** steps >= exact ** (steps - t - 1) * max_distance ** (t + 1):
            t += 1
        return min(n - 1, exact + t)

    out = []
    for rel in range(-max_distance, max_distance + 1):
        if bidirectional:
            out.append(one(abs(rel)) + (n if rel > 0 else 0))
        else:
            out.append(one(max(0, -rel)))
    return torch.tensor(out, dtype=torch.int32, device=device)


def zero_attn_workspace_bytes(B: int, Tq: int, Tk: int, Hq: int, Hk: int, D: int,
                              n_buckets: int = 0, backward: bool = False) -> int:
    return ops_lib().zero_attn_workspace_bytes(int(B), int(Tq), int(Tk), int(Hq), int(Hk), int(D),
                                               int(n_buckets), int(bool(backward)))


def zero_attn_ranges(doc, ranges, *, prefix=None, causal=True, stream=None) -> None:
    """The key ranges (B, T, 2) int32 of packed rows: doc (B, T) int32 names each
    token's document (negative: padding), prefix (B, T) int32 the length of its
    document's prefix."""
    if not isinstance(doc, torch.Tensor) or doc.dim() != 2:
        raise ValueError("doc is a (B, T) tensor")
    B, T = doc.shape
    dev, i32 = _device(), torch.int32
    p = (_flat(doc, "doc", (B, T), i32, dev), _flat(prefix, "prefix", (B, T), i32, dev),
         _flat(ranges, "ranges", (B, T, 2), i32, dev))
    if ranges is None:
        raise TypeError("ranges must be a CUDA (HIP) tensor")
    status = ops_lib().zero_attn_ranges(p[0], p[1] or None, B, T, int(bool(causal)), p[2],
                                        _stream(stream))
    if status != 0:
        raise ZeroOpsError(status, "zero_attn_ranges")


def _attn_call(fn, q, k, v, o, lse, do, dq, dk, dv, dtable, scale, cap, ranges, causal, table,
               buckets, workspace, stream):
    if not isinstance(q, torch.Tensor) or q.dim() != 4:
        raise ValueError("q is a (B, Tq, Hq, D) tensor")
    if not isinstance(k, torch.Tensor) or k.dim() != 4:
        raise ValueError("k is a (B, Tk, Hk, D) tensor")
    B, Tq, Hq, D = qs = q.shape
    ks = k.shape
    Tk, Hk = ks[1], ks[2]
    if ks[0] != B or ks[3] != D:
        raise ValueError(f"k has shape {tuple(ks)}, the call needs ({B}, Tk, Hk, {D})")
    dev, bf, f32 = _device(), _BF16, torch.float32
    q_, sq = _tensor(q, "q", qs, bf, dev)
    k_, sk = _tensor(k, "k", ks, bf, dev)
    v_, sv = _tensor(v, "v", ks, bf, dev)
    o_, so = _tensor(o, "o", qs, bf, dev)
    n_buckets = reach = code = table_ = buckets_ = 0
    if table is not None:
        n_buckets = table.shape[0]
        if buckets is None or buckets.dim() != 1 or buckets.shape[0] % 2 == 0:
            raise ValueError("bias_buckets is an int32 tensor of 2 * reach + 1 entries")
        reach = buckets.shape[0] // 2
        if table.dtype not in _CODES:
            raise TypeError(f"bias_table is float32 or bfloat16, not {table.dtype}")
        code = _CODES[table.dtype]
        table_ = _flat(table, "bias_table", (n_buckets, Hq), table.dtype, dev)
        buckets_ = _flat(buckets, "bias_buckets", (2 * reach + 1,), torch.int32, dev)
    elif dtable is not None:
        raise ValueError("dbias_table without bias_table")
    ptr = (q_, k_, v_, _flat(ranges, "ranges", (B, Tq, 2), torch.int32, dev), table_, buckets_, o_,
           _flat(lse, "lse", (B, Hq, Tq), f32, dev))
    strides = _used(qs, sq) + _used(ks, sk) + _used(ks, sv) + _used(qs, so)
    if do is not None:
        do_, sdo = _tensor(do, "do", qs, bf, dev)
        dq_, sdq = _tensor(dq, "dq", qs, bf, dev)
        dk_, sdk = _tensor(dk, "dk", ks, bf, dev)
        dv_, sdv = _tensor(dv, "dv", ks, bf, dev)
        ptr += (do_, dq_, dk_, dv_,
                0 if dtable is None else
                _flat(dtable, "dbias_table", (n_buckets, Hq), table.dtype, dev))
        strides += _used(qs, sdo) + _used(qs, sdq) + _used(ks, sdk) + _used(ks, sdv)
    else:
        ptr += (0, 0, 0, 0, 0)
        strides += (0,) * 12
    args = _ATTN_ARGS.pack(_ATTN_ARGS.size, B, Tq, Tk, Hq, Hk, D, 1 if causal else 0, code,
                           n_buckets, reach, D ** -0.5 if scale is None else scale, cap, *ptr,
                           *strides, *_workspace(workspace, dev))
    _call(fn, args, stream, dev)


def zero_attn_fwd(q, k, v, o, lse, *, scale=None, cap=0.0, ranges=None, causal=False,
                  bias_table=None, bias_buckets=None, workspace=None, stream=None) -> None:
    """Attention of q (B, Tq, Hq, D) over k and v (B, Tk, Hk, D), bf16, into o
    (as q) and lse (B, Hq, Tq) float32.  scale defaults to D^-0.5; cap > 0 caps
    the scores; ranges (B, Tq, 2) int32 are the keys [lo, hi) that each query
    sees, or `causal` (aligned at the ends), or all; bias_table
    (buckets, Hq) with bias_buckets (2 reach + 1, int32) is the learned distance
    bias.  workspace: zero_attn_workspace_bytes(...) bytes (0 for many sizes)."""
    _attn_call("zero_attn_fwd", q, k, v, o, lse, None, None, None, None, None, scale, cap, ranges,
               causal, bias_table, bias_buckets, workspace, stream)


def zero_attn_bwd(q, k, v, o, lse, do, dq, dk, dv, *, dbias_table=None, scale=None, cap=0.0,
                  ranges=None, causal=False, bias_table=None, bias_buckets=None, workspace=None,
                  stream=None) -> None:
    """Gradients of zero_attn_fwd from its inputs, its o and lse, and do: dq, dk,
    dv and, if given, dbias_table (as bias_table).  The same scale, cap, mask
    and bias; workspace: zero_attn_workspace_bytes(..., backward=True) bytes."""
    if do is None:
        raise TypeError("do must be a CUDA (HIP) tensor")
    _attn_call("zero_attn_bwd", q, k, v, o, lse, do, dq, dk, dv, dbias_table, scale, cap, ranges,
               causal, bias_table, bias_buckets, workspace, stream)


# ---------------------------------------------------------------- distill ---

def _distill_call(fn, z, idx, val, loss, stats, dz, temperature, tlse, weight, grad_scale, stream):
    if not isinstance(z, torch.Tensor) or z.dim() != 2:
        raise ValueError("logits is an (N, V) tensor")
    if not isinstance(idx, torch.Tensor) or idx.dim() != 2:
        raise ValueError("teacher_idx is an (N, K) tensor")
    N, V = z.shape
    K = idx.shape[1]
    code = _CODES.get(z.dtype)
    if code is None:
        raise TypeError(f"logits are float32 or bfloat16, not {z.dtype}")
    dev, dt, f32 = _device(), z.dtype, torch.float32
    z_, sz = _tensor(z, "logits", z.shape, dt, dev)
    dz_, sdz = (0, (V, 1)) if dz is None else _tensor(dz, "dlogits", z.shape, dt, dev)
    args = _DISTILL_ARGS.pack(
        _DISTILL_ARGS.size, N, V, K, code, temperature, grad_scale, z_,
        _flat(idx, "teacher_idx", (N, K), torch.int32, dev),
        _flat(val, "teacher_val", (N, K), dt, dev), _flat(tlse, "teacher_lse", (N,), f32, dev),
        _flat(weight, "row_weight", (N,), f32, dev), _flat(loss, "loss", (N,), f32, dev),
        _flat(stats, "stats", (N, 2), f32, dev), dz_, sz[0], sdz[0])
    _call(fn, args, stream, dev)


def zero_distill_fwd(logits, teacher_idx, teacher_val, loss, stats, *, dlogits=None,
                     temperature=1.0, teacher_lse=None, row_weight=None, grad_scale=1.0,
                     stream=None) -> None:
    """Distillation loss of logits (N, V) against the teacher's top entries
    teacher_idx (N, K) int32 and teacher_val (N, K): loss (N) and stats (N, 2),
    float32, and, if given, dlogits (N, V) = the gradient of
    grad_scale * sum(loss), in the same pass (it may be `logits`).  With
    teacher_lse (N) the rest of the teacher's mass is a tail bucket;
    row_weight (N) weights the rows (0: no part in it)."""
    _distill_call("zero_distill_fwd", logits, teacher_idx, teacher_val, loss, stats, dlogits,
                  temperature, teacher_lse, row_weight, grad_scale, stream)


def zero_distill_bwd(logits, teacher_idx, teacher_val, stats, dlogits, *, temperature=1.0,
                     teacher_lse=None, row_weight=None, grad_scale=1.0, stream=None) -> None:
    """dlogits of zero_distill_fwd from its saved stats; row_weight (times what
    the rows' losses were weighted with afterwards) is the incoming gradient."""
    if dlogits is None:
        raise TypeError("dlogits must be a CUDA (HIP) tensor")
    _distill_call("zero_distill_bwd", logits, teacher_idx, teacher_val, None, stats, dlogits,
                  temperature, teacher_lse, row_weight, grad_scale, stream)


# -------------------------------------------------------------- embedding ---

def _matrix(t, name, shape, dtype, dev, Tensor=torch.Tensor):
    """Address and row stride (0 where there is one row) of a matrix; 0, 0 for None."""
    if t is None:
        return 0, 0
    if not isinstance(t, Tensor) or t.get_device() != dev or dev < 0 or \
            t.dtype is not dtype or t.shape != shape:
        _refuse(t, name, shape, dtype, dev)
    row, last = t.stride()
    if last != 1 and shape[1] > 1:
        raise ValueError(f"{name}: the last dimension must be contiguous")
    return t.data_ptr(), row if shape[0] > 1 else 0


def _given(t, name, shape, dtype, dev):
    if t is None:
        raise TypeError(f"{name} must be a CUDA (HIP) tensor")
    return _matrix(t, name, shape, dtype, dev)


def zero_embed_workspace_bytes(N: int, C: int) -> int:
    return ops_lib().zero_embed_workspace_bytes(int(N), int(C))


def zero_embed_fwd(table, ids, out, *, scale=1.0, stream=None) -> None:
    """out (N, C) = scale * table[ids]: table (V, C), float32 or bfloat16, ids (N)
    int32; ids outside [0, V) give rows of zeros."""
    if not isinstance(table, torch.Tensor) or table.dim() != 2:
        raise ValueError("table is a (V, C) tensor")
    if not isinstance(ids, torch.Tensor) or ids.dim() != 1:
        raise ValueError("ids is an (N) tensor")
    V, width = table.shape
    N, dt = ids.shape[0], table.dtype
    code = _CODES.get(dt)
    if code is None:
        raise TypeError(f"the table is float32 or bfloat16, not {dt}")
    dev = _device()
    table_, st = _matrix(table, "table", (V, width), dt, dev)
    out_, so = _given(out, "out", (N, width), dt, dev)
    args = _EMBED_ARGS.pack(_EMBED_ARGS.size, N, V, width, code, 0, 0, scale,
                            _flat(ids, "ids", (N,), torch.int32, dev), table_, out_, 0, 0, 0, st, so,
                            0, 0, 0, 0, 0)
    _call("zero_embed_fwd", args, stream, dev)


def zero_embed_bwd(ids, dout, dtable, *, scale=1.0, base=None, workspace=None,
                   stream=None) -> None:
    """The gradient of zero_embed_fwd by the table: dtable (V, C) = base + scale * the
    sums of dout's (N, C) rows by id.  base (V, C) is 0 where None, and may be dtable:
    the sums are then added to it.  dout, base and dtable are float32 or bfloat16 each;
    workspace: zero_embed_workspace_bytes(N, C) bytes (0 for few tokens)."""
    if not isinstance(dtable, torch.Tensor) or dtable.dim() != 2:
        raise ValueError("dtable is a (V, C) tensor")
    if not isinstance(ids, torch.Tensor) or ids.dim() != 1:
        raise ValueError("ids is an (N) tensor")
    if not isinstance(dout, torch.Tensor):
        raise TypeError("dout must be a CUDA (HIP) tensor")
    V, width = dtable.shape
    N = ids.shape[0]
    codes = [0 if x is None else _CODES.get(x.dtype) for x in (dout, dtable, base)]
    if None in codes:
        raise TypeError("dout, dtable and base are float32 or bfloat16")
    dev = _device()
    dout_, sd = _matrix(dout, "dout", (N, width), dout.dtype, dev)
    dt_, st = _matrix(dtable, "dtable", (V, width), dtable.dtype, dev)
    base_, sb = (0, 0) if base is None else _matrix(base, "base", (V, width), base.dtype, dev)
    args = _EMBED_ARGS.pack(_EMBED_ARGS.size, N, V, width, *codes, scale,
                            _flat(ids, "ids", (N,), torch.int32, dev), 0, 0, dout_, base_, dt_, 0, 0,
                            sd, sb, st, *_workspace(workspace, dev))
    _call("zero_embed_bwd", args, stream, dev)


# ---------------------------------------------------- norms around a block ---

def zero_block_norm_workspace_bytes(T: int, C: int) -> int:
    return ops_lib().zero_block_norm_workspace_bytes(int(T), int(C))


def _block_types(res, others, what):
    """T, C and the codes of a call's tensors: `res` one of the residual stream, `others`
    those of the block's type."""
    T, width = res.shape
    dt = rt = res.dtype
    for x in others:
        if x is not None:
            dt = x.dtype
            break
    code, rcode = _CODES.get(dt), _CODES.get(rt)
    if code is None or rcode is None:
        raise TypeError(f"{what}: float32 or bfloat16, not {dt} and {rt}")
    return T, width, dt, code, rcode


def _gate(gate, T, width, dt, dev, name="gate"):
    """Whether it is a gate of each token, its address and its stride."""
    if gate is None:
        return 0, 0, 0
    if isinstance(gate, torch.Tensor) and gate.dim() == 2:
        return 1, *_matrix(gate, name, (T, width), dt, dev)
    return 0, _flat(gate, name, (width,), dt, dev), 0


def zero_block_norm_fwd(x, y, h, z, *, post_norm=False, post_weight=None, gate=None,
                        pre_weight=None, weight_offset=0.0, res_scale=1.0, branch_scale=1.0,
                        eps=1e-6, stream=None) -> None:
    """The residual sum around a block and the next block's norm, over rows of C values:
    h = res_scale * x + branch_scale * gate * u with u = y, or, with post_norm,
    y / rms(y) * (post_weight + weight_offset); z = h / rms(h) * (pre_weight +
    weight_offset).  x and h are (T, C) of the residual stream's type, y and z (T, C) and the
    weights (C) of the block's (the same, or x and h are float32); gate is (C) or (T, C).  y
    None: no block; h or z None: not wanted; weights None: 1.  h may be x."""
    if not isinstance(x, torch.Tensor) or x.dim() != 2:
        raise ValueError("x is a (T, C) tensor")
    T, width, dt, code, rcode = _block_types(x, (y, z, post_weight, gate, pre_weight), "x, y and z")
    dev, rt = _device(), x.dtype
    x_, sx = _matrix(x, "x", (T, width), rt, dev)
    y_, sy = _matrix(y, "y", (T, width), dt, dev)
    h_, sh = _matrix(h, "h", (T, width), rt, dev)
    z_, sz = _matrix(z, "z", (T, width), dt, dev)
    tokens, gate_, sg = _gate(gate, T, width, dt, dev)
    args = _BLOCK_NORM_ARGS.pack(
        _BLOCK_NORM_ARGS.size, T, width, code, rcode, 1 if post_norm else 0, tokens, 0, eps,
        weight_offset, res_scale, branch_scale, x_, y_,
        _flat(post_weight, "post_weight", (width,), dt, dev), gate_,
        _flat(pre_weight, "pre_weight", (width,), dt, dev), h_, z_, 0, 0, 0, 0, 0, 0, 0,
        sx, sy, sg, sh, sz, 0, 0, 0, 0, 0, 0, 0)
    _call("zero_block_norm_fwd", args, stream, dev)


def zero_block_norm_bwd(y, h, dh, dz, dx, dy, *, dpost_weight=None, dgate=None, dpre_weight=None,
                        post_norm=False, post_weight=None, gate=None, pre_weight=None,
                        weight_offset=0.0, res_scale=1.0, branch_scale=1.0, eps=1e-6,
                        workspace=None, stream=None) -> None:
    """Gradients of zero_block_norm_fwd from its y, h, weights and gate and the gradients dh
    and dz that come in (None: 0; without dz, h may be None): dx, dy and, where given,
    dpost_weight, dgate and dpre_weight, each of which may be None.  dx may be dh.  workspace:
    zero_block_norm_workspace_bytes(T, C) bytes where a gradient is summed over the tokens."""
    res = dh if dh is not None else dx if dx is not None else h
    if not isinstance(res, torch.Tensor) or res.dim() != 2:
        raise ValueError("dh, dx and h are (T, C) tensors, one of them given")
    T, width, dt, code, rcode = _block_types(res, (y, dz, dy, post_weight, gate, pre_weight),
                                             "the gradients")
    dev, rt = _device(), res.dtype
    y_, sy = _matrix(y, "y", (T, width), dt, dev)
    h_, sh = _matrix(h, "h", (T, width), rt, dev)
    dh_, sdh = _matrix(dh, "dh", (T, width), rt, dev)
    dz_, sdz = _matrix(dz, "dz", (T, width), dt, dev)
    dx_, sdx = _matrix(dx, "dx", (T, width), rt, dev)
    dy_, sdy = _matrix(dy, "dy", (T, width), dt, dev)
    tokens, gate_, sg = _gate(gate, T, width, dt, dev)
    dgate_ = sdg = 0
    if dgate is not None:
        own, dgate_, sdg = _gate(dgate, T, width, dt, dev, "dgate")
        if gate is None or own != tokens:
            raise ValueError("dgate has the gate's shape")
    args = _BLOCK_NORM_ARGS.pack(
        _BLOCK_NORM_ARGS.size, T, width, code, rcode, 1 if post_norm else 0, tokens, 0, eps,
        weight_offset, res_scale, branch_scale, 0, y_,
        _flat(post_weight, "post_weight", (width,), dt, dev), gate_,
        _flat(pre_weight, "pre_weight", (width,), dt, dev), h_, 0, dh_, dz_, dx_, dy_,
        _flat(dpost_weight, "dpost_weight", (width,), dt, dev), dgate_,
        _flat(dpre_weight, "dpre_weight", (width,), dt, dev),
        0, sy, sg, sh, 0, sdh, sdz, sdx, sdy, sdg, *_workspace(workspace, dev))
    _call("zero_block_norm_bwd", args, stream, dev)


# ------------------------------------------------------------ policy loss ---

def _policy_call(fn, z, action, adv, old, ref, weight, loss, stats, dz, temperature, low, high,
                 kl_coef, grad_scale, stream):
    if not isinstance(z, torch.Tensor) or z.dim() != 2:
        raise ValueError("logits is an (N, V) tensor")
    N, V = z.shape
    code = _CODES.get(z.dtype)
    if code is None:
        raise TypeError(f"logits are float32 or bfloat16, not {z.dtype}")
    dev, dt, f32 = _device(), z.dtype, torch.float32
    z_, sz = _tensor(z, "logits", z.shape, dt, dev)
    dz_, sdz = (0, (V, 1)) if dz is None else _tensor(dz, "dlogits", z.shape, dt, dev)
    args = _POLICY_ARGS.pack(
        _POLICY_ARGS.size, N, V, code, 0, temperature, low, high, kl_coef, grad_scale, z_,
        _flat(action, "action", (N,), torch.int32, dev), _flat(adv, "advantage", (N,), f32, dev),
        _flat(old, "old_logp", (N,), f32, dev), _flat(ref, "ref_logp", (N,), f32, dev),
        _flat(weight, "row_weight", (N,), f32, dev), _flat(loss, "loss", (N,), f32, dev),
        _flat(stats, "stats", (N, 4), f32, dev), dz_, sz[0], sdz[0])
    _call(fn, args, stream, dev)


def zero_policy_fwd(logits, action, advantage, loss, stats, *, dlogits=None, old_logp=None,
                    ref_logp=None, row_weight=None, temperature=1.0, clip_low=0.2, clip_high=0.2,
                    kl_coef=0.0, grad_scale=1.0, stream=None) -> None:
    """The clipped policy loss of the sampled tokens action (N, int32) under logits
    (N, V), with their advantage (N): loss (N) and stats (N, 4) = the row's logsumexp, the
    token's log probability, the loss's derivative by it (before the row's weight) and the
    KL term; all float32.  If given, dlogits (N, V) = the gradient of grad_scale *
    sum(loss), in the same pass (it may be `logits`).  old_logp (N) are the log
    probabilities when sampled (None: now), ref_logp (N) the reference policy's, whose KL
    term counts kl_coef; row_weight (N) weights the rows (0: no part in it)."""
    _policy_call("zero_policy_fwd", logits, action, advantage, old_logp, ref_logp, row_weight, loss,
                 stats, dlogits, temperature, clip_low, clip_high, kl_coef, grad_scale, stream)


def zero_policy_bwd(logits, action, stats, dlogits, *, row_weight=None, temperature=1.0,
                    grad_scale=1.0, stream=None) -> None:
    """dlogits of zero_policy_fwd from its saved stats; row_weight (times what the rows'
    losses were weighted with afterwards) is the incoming gradient."""
    if dlogits is None:
        raise TypeError("dlogits must be a CUDA (HIP) tensor")
    _policy_call("zero_policy_bwd", logits, action, None, None, None, row_weight, None, stats,
                 dlogits, temperature, 0.0, 0.0, 0.0, grad_scale, stream)


# ------------------------------------------- norm and clipping of gradients ---

class GradTable:
    """The gradients of a model as zero_grads_norm and zero_grads_clip take them: their
    addresses, sizes and types, laid out once for tensors that keep their memory from step
    to step.  `outs` are where the clipped gradients go (float32 or bfloat16 each); None: in
    place.  The tensors and their memory are held, with the sizes that they have here, and a
    call raises if one that it reads or writes has moved since."""

    def __init__(self, grads, outs=None):
        self.grads = list(grads)
        self.outs = self.grads if outs is None else list(outs)
        if len(self.outs) != len(self.grads):
            raise ValueError("as many outs as grads")
        if len(self.grads) > GRADS_MAX_COUNT:
            raise ValueError(f"at most {GRADS_MAX_COUNT} tensors")
        self.device = None
        for g, o in zip(self.grads, self.outs):
            for name, t in (("grads", g), ("outs", o)):
                if not isinstance(t, torch.Tensor) or not t.is_cuda:
                    raise TypeError(f"{name} are CUDA (HIP) tensors")
                if t.dtype not in _CODES:
                    raise TypeError(f"{name} are float32 or bfloat16, not {t.dtype}")
                if not t.is_contiguous():
                    raise ValueError(f"{name} must be contiguous")
                if self.device is None:
                    self.device = t.get_device()
                if t.get_device() != self.device:
                    raise ValueError("the tensors are on one device")
            if o.numel() != g.numel():
                raise ValueError(f"an output of {o.numel()} elements for {g.numel()}")
        self._refuse_overlaps()
        n = len(self.grads)
        self._grads_at = self._out_at = list(map(torch.Tensor.data_ptr, self.grads))
        if self.outs is not self.grads:
            self._out_at = list(map(torch.Tensor.data_ptr, self.outs))
        # (a tensor that is given other memory leaves what the addresses name in place)
        self._memory = [t.untyped_storage() for t in self.grads + self.outs]
        flat = [(C.c_uint64 * n)(*self._grads_at), (C.c_uint64 * n)(*self._out_at),
                (C.c_int64 * n)(*(t.numel() for t in self.grads)),
                (C.c_int32 * n)(*(_CODES[t.dtype] for t in self.grads)),
                (C.c_int32 * n)(*(_CODES[t.dtype] for t in self.outs))]
        self._arrays = flat
        self._ptrs = tuple(C.addressof(a) for a in flat)

    def _refuse_overlaps(self):
        """An output lies on no other tensor but its own gradient."""
        spans = []
        for g, o in zip(self.grads, self.outs):
            for t, written in ((g, False), (o, True)):
                if t.numel() and (written or g.data_ptr() != o.data_ptr()):
                    at = t.data_ptr()
                    spans.append((at, at + t.numel() * t.element_size(), written))
        ends = {False: 0, True: 0}                 # of what was read, of what was written
        for at, end, written in sorted(spans):
            if at < ends[True] or (written and at < ends[False]):
                raise ValueError("outputs overlap one another or other gradients")
            ends[written] = max(ends[written], end)

    def _checked(self, dev, written):
        """The table's arrays, after a look at where its tensors are now (the outputs too if they are
        `written`: 40 ns a tensor, most of what a call on hundreds of small ones costs)."""
        at = torch.Tensor.data_ptr
        if list(map(at, self.grads)) != self._grads_at or (
                written and self.outs is not self.grads and list(map(at, self.outs)) != self._out_at):
            raise ValueError("a tensor of the table has moved: make a new table")
        if self.grads and self.device != dev:
            raise ValueError(f"the table is on cuda:{self.device}; the library launches on the "
                             f"current device, cuda:{dev}")
        return self._ptrs


def zero_grads_workspace_bytes() -> int:
    return ops_lib().zero_grads_workspace_bytes()


def _accs(acc, name, dev):
    """Address and number of norm accumulators (zero_step.h)."""
    if acc is None:
        return 0, 0
    if not isinstance(acc, torch.Tensor) or not acc.is_cuda or not acc.is_contiguous():
        raise TypeError(f"{name} must be a contiguous CUDA (HIP) tensor")
    if acc.get_device() != dev:
        raise ValueError(f"{name} is on {acc.device}, not on the current device")
    nbytes = acc.numel() * acc.element_size()
    if nbytes == 0 or nbytes % 128:
        raise ValueError(f"{name} holds accumulators of 128 bytes, not {nbytes} bytes")
    return acc.data_ptr(), nbytes // 128


def _scalar(t, name, dtype, dev):
    if t is None:
        return 0
    if isinstance(t, torch.Tensor) and t.numel() != 1:
        raise ValueError(f"{name} has one element")
    return _flat(t, name, t.shape if isinstance(t, torch.Tensor) else (1,), dtype, dev)


def zero_grads_norm(table, acc, *, inv_scale=1.0, add=False, workspace=None,
                    stream=None) -> None:
    """The norm state of grads * inv_scale of a GradTable's tensors into the accumulator acc
    (new_norm_acc(1)), added to what it holds if `add`: as zero_grad_norm's of the tensors one
    by one, so that it may be given to zero_adamw_step, or summed over ranks that each hold a
    shard of the reduced gradient.  workspace:
    zero_grads_workspace_bytes() bytes."""
    dev = _device()
    grads, _, sizes, types, _ = table._checked(dev, False)
    acc_, n = _accs(acc, "acc", dev)
    if n > 1:
        raise ValueError("acc is one accumulator")
    args = _GRADS_ARGS.pack(_GRADS_ARGS.size, len(table.grads), grads, 0, sizes, types, 0, inv_scale,
                            acc_, 1 if add else 0, 0, 0, 0.0, 0, 0, 0, 0, 0,
                            *_workspace(workspace, dev))
    _call("zero_grads_norm", args, stream, dev)


def zero_grads_clip(table, accs, *, max_norm, inv_scale=1.0, check_overflow=False, norm_out=None,
                    coef_out=None, skipped_out=None, stream=None) -> None:
    """outs = grads * inv_scale * coef of a GradTable's tensors, with coef and the skip as
    zero_step_gate gives them for the accumulators accs, max_norm (0: no clipping) and
    check_overflow; a skipped call writes no tensor.  norm_out and coef_out (float32) and
    skipped_out (int32), one element each, get the global norm, the coefficient and whether
    it was skipped."""
    dev, f32 = _device(), torch.float32
    grads, outs, sizes, types, out_types = table._checked(dev, True)
    accs_, n = _accs(accs, "accs", dev)
    args = _GRADS_ARGS.pack(_GRADS_ARGS.size, len(table.grads), grads, outs, sizes, types, out_types,
                            inv_scale, 0, 0, n, accs_, max_norm, 1 if check_overflow else 0, 1,
                            _scalar(norm_out, "norm_out", f32, dev),
                            _scalar(coef_out, "coef_out", f32, dev),
                            _scalar(skipped_out, "skipped_out", torch.int32, dev), 0, 0)
    _call("zero_grads_clip", args, stream, dev)
