// zo_abi.hip -- the extern "C" entry points of libzero_ops.so: argument
// checks, then the launches.  No allocation, no synchronisation, and no C++
// exception crosses this boundary.
#include <hip/hip_runtime.h>

#include <cfloat>
#include <cmath>
#include <cstdint>

#include "zero_ops.h"
#include "zo_internal.h"

namespace {

hipStream_t as_stream(void* s) { return static_cast<hipStream_t>(s); }

int status_of(hipError_t e) { return e == hipSuccess ? ZERO_OK : ZERO_EHIP; }

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// Limits of a launch's grid: a dimension holds 65535 workgroups (64 tokens of a
// row to each) or 2^32 threads.
constexpr int kMaxLen = 1 << 21;           // tokens of a batch row
constexpr int64_t kMaxTokens = 1 << 25;    // of a norm call, 64 threads each
constexpr int64_t kMaxHeads = 1 << 23;     // batch rows times heads, 256 threads each
constexpr int64_t kMaxRows = 1 << 21;      // batch rows of ranges, rows of logits: 1024 each

// A strided array of rows of 16-byte pieces.
int check_rows(const void* p, const int64_t* stride, int n, int elem_bytes) {
  if (p == nullptr) return ZERO_EINVAL;
  if (!aligned(p, 16)) return ZERO_EALIGN;
  for (int i = 0; i < n; ++i)
    if ((stride[i] * elem_bytes) % 16 != 0) return ZERO_EALIGN;
  return ZERO_OK;
}

// An output y that is its input x: rows have to be written where they were read.
int check_in_place(const void* x, const int64_t* xs, const void* y, const int64_t* ys, int64_t T,
                   int64_t H) {
  return x == y && ((T > 1 && xs[0] != ys[0]) || (H > 1 && xs[1] != ys[1])) ? ZERO_EINVAL : ZERO_OK;
}

#define ZO_CHECK(expr)              \
  do {                              \
    const int rc_ = (expr);         \
    if (rc_ != ZERO_OK) return rc_; \
  } while (0)

// Numbers that the kernels take in binary32.
bool fits_f32(double x) { return std::fabs(x) <= FLT_MAX; }

// ------------------------------------------------------------------- norm ---

int check_norm(const zero_qk_norm_rope_args* a, bool fwd) {
  if (a == nullptr || a->struct_bytes != sizeof(*a)) return ZERO_EINVAL;
  if (a->dtype != ZERO_BF16 && a->dtype != ZERO_F32) return ZERO_EINVAL;
  if (a->T < 0 || a->Hq < 0 || a->Hk < 0 || !(a->eps >= 0.0) || !fits_f32(a->eps))
    return ZERO_EINVAL;
  if (a->D < 8 || a->D > 256 || a->D % 8 != 0) return ZERO_ESIZE;
  if (a->rot_dim < 0 || a->rot_dim > a->D || a->rot_dim % (a->interleaved ? 8 : 16) != 0)
    return ZERO_ESIZE;
  if (a->T > kMaxTokens || a->Hq > (1 << 20) || a->Hk > (1 << 20)) return ZERO_ESIZE;
  const int eb = a->dtype == ZERO_BF16 ? 2 : 4;
  if (a->rot_dim > 0 && a->T > 0) {
    if (a->pos == nullptr || a->inv_freq == nullptr) return ZERO_EINVAL;
    if (!aligned(a->pos, 4) || !aligned(a->inv_freq, 8)) return ZERO_EALIGN;
  }
  if ((a->wq && !aligned(a->wq, 16)) || (a->wk && !aligned(a->wk, 16))) return ZERO_EALIGN;
  if (fwd) {
    if (a->T > 0 && a->Hq > 0) {
      ZO_CHECK(check_rows(a->q, a->q_stride, 2, eb));
      ZO_CHECK(check_rows(a->yq, a->yq_stride, 2, eb));
      ZO_CHECK(check_in_place(a->q, a->q_stride, a->yq, a->yq_stride, a->T, a->Hq));
    }
    if (a->T > 0 && a->Hk > 0) {
      ZO_CHECK(check_rows(a->k, a->k_stride, 2, eb));
      ZO_CHECK(check_rows(a->yk, a->yk_stride, 2, eb));
      ZO_CHECK(check_in_place(a->k, a->k_stride, a->yk, a->yk_stride, a->T, a->Hk));
    }
    return ZERO_OK;
  }
  if (a->T > 0 && a->Hq > 0) {
    ZO_CHECK(check_rows(a->q, a->q_stride, 2, eb));
    ZO_CHECK(check_rows(a->dyq, a->dyq_stride, 2, eb));
    ZO_CHECK(check_rows(a->dq, a->dq_stride, 2, eb));
    ZO_CHECK(check_in_place(a->dyq, a->dyq_stride, a->dq, a->dq_stride, a->T, a->Hq));
  }
  if (a->T > 0 && a->Hk > 0) {
    ZO_CHECK(check_rows(a->k, a->k_stride, 2, eb));
    ZO_CHECK(check_rows(a->dyk, a->dyk_stride, 2, eb));
    ZO_CHECK(check_rows(a->dk, a->dk_stride, 2, eb));
    ZO_CHECK(check_in_place(a->dyk, a->dyk_stride, a->dk, a->dk_stride, a->T, a->Hk));
  }
  if ((a->dwq && !a->wq) || (a->dwk && !a->wk)) return ZERO_EINVAL;
  if ((a->dwq && !aligned(a->dwq, eb)) || (a->dwk && !aligned(a->dwk, eb))) return ZERO_EALIGN;
  if ((a->dwq || a->dwk) && a->T > 0) {
    if (a->workspace == nullptr) return ZERO_EINVAL;
    if (!aligned(a->workspace, 16)) return ZERO_EALIGN;
    if (a->workspace_bytes < zo::qk_norm_rope_workspace(a->T, a->D)) return ZERO_ESIZE;
  }
  return ZERO_OK;
}

// -------------------------------------------------------------- attention ---

int check_attn_sizes(int B, int Tq, int Tk, int Hq, int Hk, int D) {
  if (B < 0 || Tq < 0 || Tk < 0 || Hq < 1 || Hk < 1 || Hq % Hk != 0) return ZERO_EINVAL;
  if (D != 32 && D != 64 && D != 96 && D != 128) return ZERO_ESIZE;
  if (Tq > kMaxLen || Tk > (1 << 30) || Hq > (1 << 20) ||
      static_cast<int64_t>(B) * Hq > kMaxHeads)
    return ZERO_ESIZE;
  return ZERO_OK;
}

int check_attn(const zero_attn_args* a, bool fwd) {
  if (a == nullptr || a->struct_bytes != sizeof(*a)) return ZERO_EINVAL;
  ZO_CHECK(check_attn_sizes(a->B, a->Tq, a->Tk, a->Hq, a->Hk, a->D));
  if (!fwd && a->Tk > kMaxLen) return ZERO_ESIZE;
  if (!fits_f32(a->scale) || !std::isfinite(a->cap) || a->cap < 0.0) return ZERO_EINVAL;
  if (a->cap != 0.0 && !(static_cast<float>(a->cap) > 0.f && a->cap <= 1e30)) return ZERO_EINVAL;
  if (a->bias_table != nullptr) {
    if (a->bias_buckets == nullptr || a->n_buckets < 1 || a->reach < 0) return ZERO_EINVAL;
    if (a->bias_dtype != ZERO_F32 && a->bias_dtype != ZERO_BF16) return ZERO_EINVAL;
    if (a->n_buckets > ZERO_ATTN_MAX_BUCKETS || a->reach > ZERO_ATTN_MAX_REACH) return ZERO_ESIZE;
    const uintptr_t eb = a->bias_dtype == ZERO_F32 ? 4 : 2;
    if (!aligned(a->bias_table, eb) || !aligned(a->bias_buckets, 4)) return ZERO_EALIGN;
    if (a->dbias_table && !aligned(a->dbias_table, eb)) return ZERO_EALIGN;
  } else if (!fwd && a->dbias_table != nullptr) {
    return ZERO_EINVAL;
  }
  if (a->ranges && !aligned(a->ranges, 8)) return ZERO_EALIGN;
  const bool queries = a->B > 0 && a->Tq > 0, keys = a->B > 0 && a->Tk > 0;
  if (queries) {
    ZO_CHECK(check_rows(a->q, a->q_stride, 3, 2));
    ZO_CHECK(check_rows(a->o, a->o_stride, 3, 2));
    if (a->lse == nullptr) return ZERO_EINVAL;
    if (!aligned(a->lse, 4)) return ZERO_EALIGN;
  }
  if (keys) {
    ZO_CHECK(check_rows(a->k, a->k_stride, 3, 2));
    ZO_CHECK(check_rows(a->v, a->v_stride, 3, 2));
  }
  if (!fwd) {
    if (queries) {
      ZO_CHECK(check_rows(a->d_o, a->do_stride, 3, 2));
      ZO_CHECK(check_rows(a->dq, a->dq_stride, 3, 2));
    }
    if (keys) {
      ZO_CHECK(check_rows(a->dk, a->dk_stride, 3, 2));
      ZO_CHECK(check_rows(a->dv, a->dv_stride, 3, 2));
    }
  }
  const size_t need =
      zero_attn_workspace_bytes(a->B, a->Tq, a->Tk, a->Hq, a->Hk, a->D,
                                a->bias_table ? a->n_buckets : 0, fwd ? 0 : 1);
  if (need > 0) {
    if (a->workspace == nullptr) return ZERO_EINVAL;
    if (!aligned(a->workspace, 16)) return ZERO_EALIGN;
    if (a->workspace_bytes < need) return ZERO_ESIZE;
  }
  return ZERO_OK;
}

// ---------------------------------------------------------------- distill ---

int check_distill(const zero_distill_args* a, bool fwd) {
  if (a == nullptr || a->struct_bytes != sizeof(*a)) return ZERO_EINVAL;
  if (a->dtype != ZERO_BF16 && a->dtype != ZERO_F32) return ZERO_EINVAL;
  if (a->N < 0 || a->V < 1 || a->K < 1) return ZERO_EINVAL;
  if (a->N > kMaxRows || a->V > ZERO_DISTILL_MAX_V || a->K > ZERO_DISTILL_MAX_K)
    return ZERO_ESIZE;
  if (!(a->temperature >= 1e-30 && a->temperature <= 1e30) || !fits_f32(a->grad_scale))
    return ZERO_EINVAL;
  if (a->N == 0) return ZERO_OK;
  if (!a->logits || !a->teacher_idx || !a->teacher_val || !a->stats) return ZERO_EINVAL;
  if (fwd ? a->loss == nullptr : a->dlogits == nullptr) return ZERO_EINVAL;
  const uintptr_t eb = a->dtype == ZERO_BF16 ? 2 : 4;
  if (!aligned(a->logits, eb) || !aligned(a->teacher_val, eb) || !aligned(a->teacher_idx, 4) ||
      !aligned(a->stats, 4) || !aligned(a->loss, 4) || !aligned(a->dlogits, eb) ||
      !aligned(a->teacher_lse, 4) || !aligned(a->row_weight, 4))
    return ZERO_EALIGN;
  if (a->dlogits && a->dlogits_stride < a->V && a->N > 1) return ZERO_EINVAL;
  if (a->dlogits == a->logits && a->dlogits_stride != a->logits_stride && a->N > 1)
    return ZERO_EINVAL;
  return ZERO_OK;
}

}  // namespace

extern "C" {

int zero_ops_abi_version(void) { return ZERO_OPS_ABI_VERSION; }

const char* zero_ops_strerror(int status) {
  switch (status) {
    case ZERO_OK: return "ok";
    case ZERO_EINVAL:
      return "invalid argument (null pointer, struct size, dtype, head counts, scale, cap, "
             "temperature, bias map, in place with other strides or missing workspace)";
    case ZERO_EALIGN:
      return "pointer or stride misaligned (head rows and workspaces need 16 bytes, ranges 8, "
             "other arrays their element)";
    case ZERO_ESIZE:
      return "size not supported (head dimension, rotation, lengths, reach, buckets, K, V) or "
             "workspace too small";
    case ZERO_EHIP: return "HIP runtime error at launch";
    default: return "unknown status";
  }
}

int zero_qk_norm_rope_fwd(const zero_qk_norm_rope_args* a, void* stream) {
  try {
    ZO_CHECK(check_norm(a, true));
    if (a->T == 0 || a->Hq + a->Hk == 0) return ZERO_OK;
    return status_of(zo::launch_qk_norm_rope_fwd(*a, as_stream(stream)));
  } catch (...) {
    return ZERO_EHIP;
  }
}

int zero_qk_norm_rope_bwd(const zero_qk_norm_rope_args* a, void* stream) {
  try {
    ZO_CHECK(check_norm(a, false));
    if ((a->T == 0 || a->Hq + a->Hk == 0) && !a->dwq && !a->dwk) return ZERO_OK;
    return status_of(zo::launch_qk_norm_rope_bwd(*a, as_stream(stream)));
  } catch (...) {
    return ZERO_EHIP;
  }
}

size_t zero_qk_norm_rope_workspace_bytes(int64_t T, int D) {
  return T < 0 || D < 0 ? 0 : zo::qk_norm_rope_workspace(T, D);
}

int zero_attn_fwd(const zero_attn_args* a, void* stream) {
  try {
    ZO_CHECK(check_attn(a, true));
    if (a->B == 0 || a->Tq == 0) return ZERO_OK;
    return status_of(zo::launch_attn_fwd(*a, as_stream(stream)));
  } catch (...) {
    return ZERO_EHIP;
  }
}

int zero_attn_bwd(const zero_attn_args* a, void* stream) {
  try {
    ZO_CHECK(check_attn(a, false));
    if (a->B == 0 && a->dbias_table == nullptr) return ZERO_OK;
    return status_of(zo::launch_attn_bwd(*a, as_stream(stream)));
  } catch (...) {
    return ZERO_EHIP;
  }
}

size_t zero_attn_workspace_bytes(int B, int Tq, int Tk, int Hq, int Hk, int D, int n_buckets,
                                 int backward) {
  if (check_attn_sizes(B, Tq, Tk, Hq, Hk, D) != ZERO_OK || n_buckets < 0) return 0;
  return backward ? zo::attn_bwd_workspace(B, Tq, Tk, Hq, Hk, D, n_buckets)
                  : zo::attn_fwd_workspace(B, Tq, Tk, Hq, Hk, D);
}

int zero_attn_ranges(const int32_t* doc, const int32_t* prefix, int B, int T, int causal,
                     int32_t* ranges, void* stream) {
  try {
    if (B < 0 || T < 0) return ZERO_EINVAL;
    if (T > kMaxLen || B > kMaxRows) return ZERO_ESIZE;
    if (B == 0 || T == 0) return ZERO_OK;
    if (doc == nullptr || ranges == nullptr) return ZERO_EINVAL;
    if (!aligned(doc, 4) || !aligned(prefix, 4) || !aligned(ranges, 8)) return ZERO_EALIGN;
    return status_of(
        zo::launch_attn_ranges(doc, prefix, B, T, causal, ranges, as_stream(stream)));
  } catch (...) {
    return ZERO_EHIP;
  }
}

int zero_distill_fwd(const zero_distill_args* a, void* stream) {
  try {
    ZO_CHECK(check_distill(a, true));
    if (a->N == 0) return ZERO_OK;
    return status_of(zo::launch_distill(*a, true, as_stream(stream)));
  } catch (...) {
    return ZERO_EHIP;
  }
}

int zero_distill_bwd(const zero_distill_args* a, void* stream) {
  try {
    ZO_CHECK(check_distill(a, false));
    if (a->N == 0) return ZERO_OK;
    return status_of(zo::launch_distill(*a, false, as_stream(stream)));
  } catch (...) {
    return ZERO_EHIP;
  }
}

}  // extern "C"
