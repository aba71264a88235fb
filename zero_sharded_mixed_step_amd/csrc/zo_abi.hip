// zo_abi.hip -- the extern "C" entry points of libzero_ops.so: argument
// checks, then the launches.  No allocation, no synchronisation, and no C++
// exception crosses this boundary.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cfloat>
#include <cmath>
#include <cstdint>
#include <vector>

#include "zero_ops.h"
#include "zo_internal.h"
#include "zo_spans.h"

namespace {

using zo::Span;

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

// -------------------------------------------------------------- embedding ---

bool known_dtype(int dtype) { return dtype == ZERO_BF16 || dtype == ZERO_F32; }
int bytes_of(int dtype) { return dtype == ZERO_BF16 ? 2 : 4; }

// A matrix of n rows: a row of one has a stride that nothing uses.
int check_matrix(const void* p, int64_t stride, int64_t n, int dtype) {
  const int64_t s = n > 1 ? stride : 0;
  return check_rows(p, &s, 1, bytes_of(dtype));
}

// Rows of C values that do not overlap one another: of an output, or of a gradient.
bool rows_apart(int64_t stride, int64_t n, int64_t C) {
  return n <= 1 || stride >= C || stride <= -C;
}

int check_row_width(int C) {
  return C < 8 || C > ZERO_ROW_MAX_C || C % 8 != 0 ? ZERO_ESIZE : ZERO_OK;
}

// Whether what a call writes meets nothing else of it; `need` bytes of its workspace are used.
bool embed_apart(const zero_embed_args* a, bool fwd, size_t need) {
  const int eb = bytes_of(a->dtype);
  zo::Arrays<2, 3> m;
  if (a->N > 0) m.reads(Span(a->ids, a->N * 4));
  if (fwd) {
    m.writes(Span(a->out, a->N, a->out_stride, a->C, eb));
    m.reads(Span(a->table, a->V, a->table_stride, a->C, eb));
    return m.apart();
  }
  m.writes(Span(a->dtable, a->V, a->dtable_stride, a->C, bytes_of(a->grad_dtype)));
  if (need > 0) m.writes(Span(a->workspace, static_cast<int64_t>(need)));
  if (a->N > 0) m.reads(Span(a->dout, a->N, a->dout_stride, a->C, eb));
  if (a->base != a->dtable)
    m.reads(Span(a->base, a->V, a->base_stride, a->C, bytes_of(a->base_dtype)));
  return m.apart();
}

int check_embed(const zero_embed_args* a, bool fwd) {
  if (a == nullptr || a->struct_bytes != sizeof(*a)) return ZERO_EINVAL;
  if (!known_dtype(a->dtype)) return ZERO_EINVAL;
  if (a->N < 0 || a->V < 1 || !fits_f32(a->scale)) return ZERO_EINVAL;
  if (a->N > kMaxRows || a->V > ZERO_EMBED_MAX_V) return ZERO_ESIZE;
  ZO_CHECK(check_row_width(a->C));
  if (a->N > 0) {
    if (a->ids == nullptr) return ZERO_EINVAL;
    if (!aligned(a->ids, 4)) return ZERO_EALIGN;
  }
  if (fwd) {
    if (a->N == 0) return ZERO_OK;
    ZO_CHECK(check_matrix(a->table, a->table_stride, a->V, a->dtype));
    ZO_CHECK(check_matrix(a->out, a->out_stride, a->N, a->dtype));
    return rows_apart(a->out_stride, a->N, a->C) && embed_apart(a, true, 0) ? ZERO_OK : ZERO_EINVAL;
  }
  if (!known_dtype(a->grad_dtype) || (a->base && !known_dtype(a->base_dtype))) return ZERO_EINVAL;
  ZO_CHECK(check_matrix(a->dtable, a->dtable_stride, a->V, a->grad_dtype));
  if (!rows_apart(a->dtable_stride, a->V, a->C)) return ZERO_EINVAL;
  if (a->base != nullptr) {
    ZO_CHECK(check_matrix(a->base, a->base_stride, a->V, a->base_dtype));
    if (a->base == a->dtable && (a->base_dtype != a->grad_dtype ||
                                 (a->V > 1 && a->base_stride != a->dtable_stride)))
      return ZERO_EINVAL;
  }
  size_t need = 0;
  if (a->N > 0) {
    ZO_CHECK(check_matrix(a->dout, a->dout_stride, a->N, a->dtype));
    need = zo::embed_workspace(a->N, a->C);
    if (need > 0) {
      if (a->workspace == nullptr) return ZERO_EINVAL;
      if (!aligned(a->workspace, 16)) return ZERO_EALIGN;
      if (a->workspace_bytes < need) return ZERO_ESIZE;
    }
  }
  return embed_apart(a, false, need) ? ZERO_OK : ZERO_EINVAL;
}

// ------------------------------------------------------ norms round a block ---

int check_vector(const void* p) { return p && !aligned(p, 16) ? ZERO_EALIGN : ZERO_OK; }

// (Of calls that have rows.)
bool block_apart(const zero_block_norm_args* a, bool fwd, bool parts) {
  const int eb = bytes_of(a->dtype), rb = bytes_of(a->res_dtype);
  const auto rows = [&](const void* p, int64_t stride, int bytes) {
    return Span(p, a->T, stride, a->C, bytes);
  };
  const auto vector = [&](const void* p) { return Span(p, static_cast<int64_t>(a->C) * eb); };
  const auto gate = [&](const void* p, int64_t stride) {
    return a->gate_tokens ? rows(p, stride, eb) : vector(p);
  };
  zo::Arrays<6, 7> m;
  m.reads(rows(a->y, a->y_stride, eb));
  m.reads(vector(a->post_w));
  m.reads(gate(a->gate, a->gate_stride));
  if (fwd || a->dz != nullptr) m.reads(vector(a->pre_w));
  if (fwd) {
    m.writes(rows(a->h, a->h_stride, rb));
    m.writes(rows(a->z, a->z_stride, eb));
    if (a->x != a->h) m.reads(rows(a->x, a->x_stride, rb));
    return m.apart();
  }
  m.writes(rows(a->dx, a->dx_stride, rb));
  m.writes(rows(a->dy, a->dy_stride, eb));
  m.writes(vector(a->dpost_w));
  m.writes(gate(a->dgate, a->dgate_stride));
  m.writes(vector(a->dpre_w));
  if (parts)
    m.writes(Span(a->workspace, static_cast<int64_t>(zo::block_norm_workspace(a->T, a->C))));
  if (a->dh != a->dx) m.reads(rows(a->dh, a->dh_stride, rb));
  m.reads(rows(a->dz, a->dz_stride, eb));
  if (a->dz != nullptr) m.reads(rows(a->h, a->h_stride, rb));
  return m.apart();
}

int check_block(const zero_block_norm_args* a, bool fwd) {
  if (a == nullptr || a->struct_bytes != sizeof(*a)) return ZERO_EINVAL;
  if (!known_dtype(a->dtype) || (a->res_dtype != a->dtype && a->res_dtype != ZERO_F32))
    return ZERO_EINVAL;
  if (a->T < 0 || !(a->eps >= 0.0) || !fits_f32(a->eps) || !fits_f32(a->weight_offset) ||
      !fits_f32(a->res_scale) || !fits_f32(a->branch_scale))
    return ZERO_EINVAL;
  if (a->T > kMaxRows) return ZERO_ESIZE;
  ZO_CHECK(check_row_width(a->C));
  // a weight without its norm, a norm or a gate without its block (without rows their
  // arrays may be NULL)
  const bool rows = a->T > 0;
  if ((a->post_w && !a->post_norm) || (rows && !a->y && (a->post_norm || a->gate)))
    return ZERO_EINVAL;
  ZO_CHECK(check_vector(a->post_w));
  ZO_CHECK(check_vector(a->pre_w));
  const int dt = a->dtype, rt = a->res_dtype;
  if (a->gate != nullptr) {
    if (a->gate_tokens && rows) ZO_CHECK(check_matrix(a->gate, a->gate_stride, a->T, dt));
    else ZO_CHECK(check_vector(a->gate));
  }
  if (a->y != nullptr && rows) ZO_CHECK(check_matrix(a->y, a->y_stride, a->T, dt));
  if (fwd) {
    if (!rows) return ZERO_OK;
    if ((!a->h && !a->z) || (a->pre_w && !a->z)) return ZERO_EINVAL;
    ZO_CHECK(check_matrix(a->x, a->x_stride, a->T, rt));
    if (a->h != nullptr) {
      ZO_CHECK(check_matrix(a->h, a->h_stride, a->T, rt));
      if (!rows_apart(a->h_stride, a->T, a->C)) return ZERO_EINVAL;
      if (a->h == a->x && a->T > 1 && a->h_stride != a->x_stride) return ZERO_EINVAL;
    }
    if (a->z != nullptr) {
      ZO_CHECK(check_matrix(a->z, a->z_stride, a->T, dt));
      if (!rows_apart(a->z_stride, a->T, a->C)) return ZERO_EINVAL;
    }
    return block_apart(a, true, false) ? ZERO_OK : ZERO_EINVAL;
  }
  if ((a->dpost_w && !a->post_w) || (a->dpre_w && !a->pre_w)) return ZERO_EINVAL;
  if (rows && ((a->dgate && !a->gate) || (a->dy && !a->y) || (a->dpre_w && !a->dz) ||
               (!a->dh && !a->dz)))
    return ZERO_EINVAL;
  const uintptr_t eb = bytes_of(dt);
  if ((a->dpost_w && !aligned(a->dpost_w, eb)) || (a->dpre_w && !aligned(a->dpre_w, eb)) ||
      (a->dgate && !aligned(a->dgate, a->gate_tokens ? 16 : eb)))
    return ZERO_EALIGN;
  if (!rows) return ZERO_OK;
  if (a->dz != nullptr) {
    ZO_CHECK(check_matrix(a->dz, a->dz_stride, a->T, dt));
    ZO_CHECK(check_matrix(a->h, a->h_stride, a->T, rt));
  }
  if (a->dh != nullptr) ZO_CHECK(check_matrix(a->dh, a->dh_stride, a->T, rt));
  if (a->dx != nullptr) {
    ZO_CHECK(check_matrix(a->dx, a->dx_stride, a->T, rt));
    if (!rows_apart(a->dx_stride, a->T, a->C)) return ZERO_EINVAL;
    if (a->dx == a->dh && a->T > 1 && a->dx_stride != a->dh_stride) return ZERO_EINVAL;
  }
  if (a->dy != nullptr) {
    ZO_CHECK(check_matrix(a->dy, a->dy_stride, a->T, dt));
    if (!rows_apart(a->dy_stride, a->T, a->C)) return ZERO_EINVAL;
  }
  if (a->dgate != nullptr && a->gate_tokens) {
    ZO_CHECK(check_matrix(a->dgate, a->dgate_stride, a->T, dt));
    if (!rows_apart(a->dgate_stride, a->T, a->C)) return ZERO_EINVAL;
  }
  const bool parts = a->dpost_w || a->dpre_w || (a->dgate && !a->gate_tokens);
  if (parts) {
    if (a->workspace == nullptr) return ZERO_EINVAL;
    if (!aligned(a->workspace, 16)) return ZERO_EALIGN;
    if (a->workspace_bytes < zo::block_norm_workspace(a->T, a->C)) return ZERO_ESIZE;
  }
  return block_apart(a, false, parts) ? ZERO_OK : ZERO_EINVAL;
}

// ------------------------------------------------------------ policy loss ---

bool policy_apart(const zero_policy_args* a, bool fwd) {
  const int eb = bytes_of(a->dtype);
  const auto numbers = [&](const void* p, int of_a_row) { return Span(p, a->N * of_a_row * 4); };
  zo::Arrays<3, 6> m;
  m.writes(Span(a->dlogits, a->N, a->dlogits_stride, a->V, eb));
  if (a->logits != a->dlogits) m.reads(Span(a->logits, a->N, a->logits_stride, a->V, eb));
  m.reads(numbers(a->action, 1));
  m.reads(numbers(a->row_weight, 1));
  if (fwd) {
    m.writes(numbers(a->loss, 1));
    m.writes(numbers(a->stats, 4));
    m.reads(numbers(a->advantage, 1));
    m.reads(numbers(a->old_logp, 1));
    m.reads(numbers(a->ref_logp, 1));
  } else {
    m.reads(numbers(a->stats, 4));
  }
  return m.apart();
}

int check_policy(const zero_policy_args* a, bool fwd) {
  if (a == nullptr || a->struct_bytes != sizeof(*a)) return ZERO_EINVAL;
  if (!known_dtype(a->dtype)) return ZERO_EINVAL;
  if (a->N < 0 || a->V < 1) return ZERO_EINVAL;
  if (a->N > kMaxRows || a->V > ZERO_POLICY_MAX_V) return ZERO_ESIZE;
  if (!(a->temperature >= 1e-30 && a->temperature <= 1e30) || !fits_f32(a->grad_scale))
    return ZERO_EINVAL;
  if (fwd && (!(a->clip_low >= 0.0 && a->clip_low <= 1.0) || !(a->clip_high >= 0.0) ||
              !fits_f32(a->clip_high) || !fits_f32(a->kl_coef)))
    return ZERO_EINVAL;
  if (a->N == 0) return ZERO_OK;
  if (!a->logits || !a->action || !a->stats) return ZERO_EINVAL;
  if (fwd ? !a->advantage || !a->loss : !a->dlogits) return ZERO_EINVAL;
  const uintptr_t eb = bytes_of(a->dtype);
  if (!aligned(a->logits, eb) || !aligned(a->dlogits, eb) || !aligned(a->action, 4) ||
      !aligned(a->stats, 4) || !aligned(a->row_weight, 4))
    return ZERO_EALIGN;
  if (fwd && (!aligned(a->advantage, 4) || !aligned(a->loss, 4) || !aligned(a->old_logp, 4) ||
              !aligned(a->ref_logp, 4)))
    return ZERO_EALIGN;
  if (a->dlogits && a->dlogits_stride < a->V && a->N > 1) return ZERO_EINVAL;
  if (a->dlogits == a->logits && a->dlogits_stride != a->logits_stride && a->N > 1)
    return ZERO_EINVAL;
  return policy_apart(a, fwd) ? ZERO_OK : ZERO_EINVAL;
}

// ------------------------------------------- norm and clipping of gradients ---

constexpr int64_t kMaxElements = int64_t(1) << 37;   // of a norm accumulator

struct Bytes {
  uintptr_t at = 0, end = 0;
  Bytes() = default;
  Bytes(const void* p, int64_t n)
      : at(reinterpret_cast<uintptr_t>(p)), end(at + static_cast<uintptr_t>(n)) {}
  // (at least one byte of both: an empty one meets none)
  bool meets(const Bytes& b) const { return std::max(at, b.at) < std::min(end, b.end); }
};

// Whether what a call writes beside the tensors (`small`, some of which may be empty) meets no tensor,
// nor the accumulators that it reads, and outputs do not meet these.
bool small_apart(const zero_grads_args* a, bool clip, const Bytes (&small)[3], const Bytes& accs) {
  Bytes around;                               // all of them: most tensors lie outside
  around.at = UINTPTR_MAX;
  const auto extend = [&](const Bytes& b) {
    if (b.at == b.end) return;
    around.at = std::min(around.at, b.at);
    around.end = std::max(around.end, b.end);
  };
  extend(accs);
  for (int i = 0; i < 3; ++i) {
    extend(small[i]);
    if (small[i].meets(accs)) return false;
    for (int j = 0; j < i; ++j)
      if (small[i].meets(small[j])) return false;
  }
  const auto meets_small = [&](const Bytes& t) {
    return t.meets(small[0]) || t.meets(small[1]) || t.meets(small[2]);
  };
  for (int64_t i = 0; i < a->count; ++i) {
    const Bytes g(a->grads[i], a->sizes[i] * bytes_of(a->dtypes[i]));
    if (g.at < around.end && around.at < g.end && meets_small(g)) return false;
    if (!clip) continue;
    const Bytes out(a->outs[i], a->sizes[i] * bytes_of(a->out_dtypes[i]));
    if (out.at < around.end && around.at < out.end && (meets_small(out) || out.meets(accs)))
      return false;
  }
  return true;
}

// Whether every output lies on no tensor but its own gradient, by their addresses in order.
bool outs_apart(const zero_grads_args* a) {
  struct Piece : Bytes {
    bool written;
  };
  std::vector<Piece> pieces;
  pieces.reserve(2 * a->count);
  for (int64_t i = 0; i < a->count; ++i) {
    if (a->sizes[i] == 0) continue;
    if (a->outs[i] != a->grads[i])
      pieces.push_back({Bytes(a->grads[i], a->sizes[i] * bytes_of(a->dtypes[i])), false});
    pieces.push_back({Bytes(a->outs[i], a->sizes[i] * bytes_of(a->out_dtypes[i])), true});
  }
  std::sort(pieces.begin(), pieces.end(),
            [](const Piece& x, const Piece& y) { return x.at < y.at; });
  uintptr_t read = 0, written = 0;            // ends of what came before
  for (const Piece& x : pieces) {
    if (x.at < written || (x.written && x.at < read)) return false;
    (x.written ? written : read) = std::max(x.written ? written : read, x.end);
  }
  return true;
}

int check_grads(const zero_grads_args* a, bool norm) {
  if (a == nullptr || a->struct_bytes != sizeof(*a)) return ZERO_EINVAL;
  if (a->count < 0 || !fits_f32(a->inv_scale)) return ZERO_EINVAL;
  if (a->count > ZERO_GRADS_MAX_COUNT) return ZERO_ESIZE;
  if (a->count > 0 && (!a->grads || !a->sizes || !a->dtypes)) return ZERO_EINVAL;
  if (!norm && a->count > 0 && (!a->outs || !a->out_dtypes)) return ZERO_EINVAL;
  int64_t total = 0;
  for (int64_t i = 0; i < a->count; ++i) {
    if (a->sizes[i] < 0 || !known_dtype(a->dtypes[i])) return ZERO_EINVAL;
    if (!norm && !known_dtype(a->out_dtypes[i])) return ZERO_EINVAL;
    if (a->sizes[i] > kMaxElements - total) return ZERO_ESIZE;
    total += a->sizes[i];
    if (a->sizes[i] == 0) continue;
    if (!a->grads[i] || (!norm && !a->outs[i])) return ZERO_EINVAL;
    if (!aligned(a->grads[i], bytes_of(a->dtypes[i])) ||
        (!norm && !aligned(a->outs[i], bytes_of(a->out_dtypes[i]))))
      return ZERO_EALIGN;
    if (!norm && a->outs[i] == a->grads[i] && a->dtypes[i] != a->out_dtypes[i])
      return ZERO_EINVAL;
  }
  if (norm) {
    if (!a->acc || !a->workspace) return ZERO_EINVAL;
    if (!aligned(a->acc, 16) || !aligned(a->workspace, 16)) return ZERO_EALIGN;
    if (a->workspace_bytes < zo::grads_workspace()) return ZERO_ESIZE;
    if (total == 0) return ZERO_OK;            // (the workspace is not used)
    return small_apart(a, false,
                       {Bytes(a->acc, sizeof(*a->acc)),
                        Bytes(a->workspace, static_cast<int64_t>(zo::grads_workspace())), Bytes()},
                       Bytes())
               ? ZERO_OK
               : ZERO_EINVAL;
  }
  if (a->n_accs < 0 || (a->n_accs > 0 && !a->accs) || !std::isfinite(a->max_norm))
    return ZERO_EINVAL;
  if (!aligned(a->accs, 16) || !aligned(a->norm_out, 4) || !aligned(a->coef_out, 4) ||
      !aligned(a->skipped_out, 4))
    return ZERO_EALIGN;
  if (!small_apart(a, true, {Bytes(a->norm_out, a->norm_out ? 4 : 0), Bytes(a->coef_out, a->coef_out ? 4 : 0),
                             Bytes(a->skipped_out, a->skipped_out ? 4 : 0)},
                   Bytes(a->accs, static_cast<int64_t>(sizeof(*a->accs)) * a->n_accs)))
    return ZERO_EINVAL;
  return a->outs_apart == 1 || outs_apart(a) ? ZERO_OK : ZERO_EINVAL;
}

}  // namespace

extern "C" {

int zero_ops_abi_version(void) { return ZERO_OPS_ABI_VERSION; }

const char* zero_ops_strerror(int status) {
  switch (status) {
    case ZERO_OK: return "ok";
    case ZERO_EINVAL:
      return "invalid argument (null pointer, struct size, dtype, head counts, scale, cap, "
             "temperature, clipping, bias map, weight or gradient without its input, rows or "
             "arrays that overlap, in place with other strides or dtypes, or missing workspace)";
    case ZERO_EALIGN:
      return "pointer or stride misaligned (rows, their weights, accumulators and workspaces need "
             "16 bytes, ranges 8, other arrays their element)";
    case ZERO_ESIZE:
      return "size not supported (head dimension, rotation, lengths, width, reach, buckets, K, V, "
             "count) or workspace too small";
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

int zero_embed_fwd(const zero_embed_args* a, void* stream) {
  try {
    ZO_CHECK(check_embed(a, true));
    if (a->N == 0) return ZERO_OK;
    return status_of(zo::launch_embed_fwd(*a, as_stream(stream)));
  } catch (...) {
    return ZERO_EHIP;
  }
}

int zero_embed_bwd(const zero_embed_args* a, void* stream) {
  try {
    ZO_CHECK(check_embed(a, false));
    return status_of(zo::launch_embed_bwd(*a, as_stream(stream)));
  } catch (...) {
    return ZERO_EHIP;
  }
}

size_t zero_embed_workspace_bytes(int64_t N, int C) {
  return N <= 0 || C < 0 || N > kMaxRows || C > ZERO_ROW_MAX_C ? 0 : zo::embed_workspace(N, C);
}

int zero_block_norm_fwd(const zero_block_norm_args* a, void* stream) {
  try {
    ZO_CHECK(check_block(a, true));
    if (a->T == 0) return ZERO_OK;
    return status_of(zo::launch_block_norm_fwd(*a, as_stream(stream)));
  } catch (...) {
    return ZERO_EHIP;
  }
}

int zero_block_norm_bwd(const zero_block_norm_args* a, void* stream) {
  try {
    ZO_CHECK(check_block(a, false));
    return status_of(zo::launch_block_norm_bwd(*a, as_stream(stream)));
  } catch (...) {
    return ZERO_EHIP;
  }
}

size_t zero_block_norm_workspace_bytes(int64_t T, int C) {
  return T <= 0 || C < 0 || C > ZERO_ROW_MAX_C ? 0 : zo::block_norm_workspace(T, C);
}

int zero_policy_fwd(const zero_policy_args* a, void* stream) {
  try {
    ZO_CHECK(check_policy(a, true));
    if (a->N == 0) return ZERO_OK;
    return status_of(zo::launch_policy(*a, true, as_stream(stream)));
  } catch (...) {
    return ZERO_EHIP;
  }
}

int zero_policy_bwd(const zero_policy_args* a, void* stream) {
  try {
    ZO_CHECK(check_policy(a, false));
    if (a->N == 0) return ZERO_OK;
    return status_of(zo::launch_policy(*a, false, as_stream(stream)));
  } catch (...) {
    return ZERO_EHIP;
  }
}

int zero_grads_norm(const zero_grads_args* a, void* stream) {
  try {
    ZO_CHECK(check_grads(a, true));
    return status_of(zo::launch_grads_norm(*a, as_stream(stream)));
  } catch (...) {
    return ZERO_EHIP;
  }
}

int zero_grads_clip(const zero_grads_args* a, void* stream) {
  try {
    ZO_CHECK(check_grads(a, false));
    return status_of(zo::launch_grads_clip(*a, as_stream(stream)));
  } catch (...) {
    return ZERO_EHIP;
  }
}

size_t zero_grads_workspace_bytes(void) { return zo::grads_workspace(); }

}  // extern "C"
