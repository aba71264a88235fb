/*
 * zero_ops.h -- C ABI of libzero_ops.so: the operators of a student model's
 * training step whose gradients the sharded optimizer step (zero_step.h)
 * reduces, for MI355X (gfx950).
 *
 *   - zero_qk_norm_rope_fwd/_bwd: the RMS norm of every query and key head
 *     with a learned weight, and the position rotation, in one pass.
 *   - zero_attn_fwd/_bwd: softmax attention whose scores may be capped by a
 *     tanh and get a learned bias by bucketed distance, where each query sees
 *     an interval of keys (documents, prefixes, causal, windows, padding);
 *     zero_attn_ranges derives the intervals from document ids.
 *   - zero_distill_fwd/_bwd: the distillation loss against a teacher's top
 *     logits, with its gradient in the same pass or from saved statistics.
 *
 * Conventions, as in zero_step.h:
 *   - Status codes are those of zero_step.h.  Every argument is checked
 *     before anything is launched; no C++ exception escapes.  Numbers that
 *     binary32 does not hold (scale, eps, grad_scale) are ZERO_EINVAL.
 *   - `stream` is a hipStream_t.  All work is enqueued on it, on the device
 *     that is current; nothing is allocated, copied to the host or
 *     synchronised, and no state outlives a call, so every call can be
 *     recorded into a HIP graph.  Scratch memory is the caller's
 *     `workspace` (16-byte aligned, any content, not shared by calls that
 *     may overlap).
 *   - Strides are in elements; the innermost dimension (the head's D values,
 *     a row's V logits) is contiguous.  Addressing is 64-bit.
 *   - Sums, softmax statistics and norms are binary32 or wider; each output
 *     element is rounded once.  Every sum has a fixed order (the only atomics
 *     set bits in shared memory), so the same call gives the same bits every
 *     time on one device.
 *   - Outputs must not overlap inputs unless stated (where the same address
 *     is allowed, other strides are ZERO_EINVAL).
 */
#ifndef ZERO_OPS_H
#define ZERO_OPS_H

#include <stddef.h>
#include <stdint.h>

#include "zero_step.h"

#ifdef __cplusplus
extern "C" {
#endif

#define ZERO_OPS_ABI_VERSION 1

/* Largest reach of the distance bias, most buckets, most teacher entries of
 * a row, and longest row of logits. */
#define ZERO_ATTN_MAX_REACH 512
#define ZERO_ATTN_MAX_BUCKETS 256
#define ZERO_DISTILL_MAX_K 1024
#define ZERO_DISTILL_MAX_V (1 << 20)

int zero_ops_abi_version(void);
const char *zero_ops_strerror(int status);

/* ---- norm of queries and keys, with the position rotation --------------
 *
 * For each token t and head h, over the head's D values:
 *   n = x * r * w,  r = 1 / sqrt(mean(x^2) + eps)   (w = 1 if NULL)
 *   y = n with the pairs (a, b) of its first rot_dim values turned by the
 *       angle pos[t] * inv_freq[i]:  (a cos - b sin, b cos + a sin).
 * Pair i is (2i, 2i+1) if `interleaved`, else (i, i + rot_dim/2).  Angles are
 * formed and reduced to one turn in binary64, so positions far beyond 2^24
 * radians keep their phase.
 *
 * Backward, with g = dy turned back, u = g * w and xhat = x * r:
 *   dx = r * (u - xhat * mean(u * xhat)),   dw = sum over tokens and heads
 *   of g * xhat.
 *
 * dtype (ZERO_BF16 or ZERO_F32) is that of x, w, y and the gradients.  D is a
 * multiple of 8 up to 256; rot_dim <= D is a multiple of 8, of 16 where the
 * pairs are half a rotation apart (ZERO_ESIZE otherwise); 0 turns nothing
 * (pos and inv_freq may be NULL).  Either of q and k may be absent (H = 0).
 * Rows start on 16 bytes: base addresses and strides (ZERO_EALIGN).  y may be
 * x itself and dq may be dyq (same strides). */
typedef struct zero_qk_norm_rope_args {
  size_t struct_bytes;          /* sizeof(zero_qk_norm_rope_args) */
  int64_t T;
  int32_t Hq, Hk, D, rot_dim;
  int32_t dtype, interleaved;
  double eps;
  const void *q, *k;            /* [T][H][D] */
  const void *wq, *wk;          /* [D] or NULL */
  const int32_t *pos;           /* [T] */
  const double *inv_freq;       /* [rot_dim / 2], radians per position */
  void *yq, *yk;                /* forward outputs */
  const void *dyq, *dyk;        /* backward inputs */
  void *dq, *dk;                /* backward outputs */
  void *dwq, *dwk;              /* [D]; NULL where the weight is NULL or its gradient unwanted */
  int64_t q_stride[2], k_stride[2];     /* token, head */
  int64_t yq_stride[2], yk_stride[2];
  int64_t dyq_stride[2], dyk_stride[2];
  int64_t dq_stride[2], dk_stride[2];
  void *workspace;              /* backward only */
  size_t workspace_bytes;
} zero_qk_norm_rope_args;

int zero_qk_norm_rope_fwd(const zero_qk_norm_rope_args *args, void *stream);
int zero_qk_norm_rope_bwd(const zero_qk_norm_rope_args *args, void *stream);
size_t zero_qk_norm_rope_workspace_bytes(int64_t T, int D);

/* ---- attention ------------------------------------------------------------
 *
 * For query i and key j of one batch row and head, with off = Tk - Tq:
 *   x = scale * q_i . k_j
 *   c = cap * tanh(x / cap)  if cap > 0, else x       (cap <= 1e30)
 *   s = c + bias_table[bias_buckets[clamp(j - i - off, -reach, reach)
 *                                   + reach]][h]   (if bias_table is given)
 * and s = -inf for keys outside the query's interval [lo, hi):
 *   ranges[b][i] = {lo, hi} if given (clipped to [0, Tk]; lo >= hi: no key),
 *   else [0, i + 1 + off) if causal, else [0, Tk).
 *   o_i = sum_j softmax_j(s) v_j,   lse_i = log sum_j exp(s_ij).
 * A query that sees no key gives o = 0, lse = -inf and gradients of 0, and takes
 * no part in any other; a key that no query sees has gradients of 0.  Both may hold
 * anything, NaN and infinities too: they are read as 0.  Masked scores are selected
 * away, not multiplied.  What a key holds that some query sees counts for the
 * queries near it, as in the formula with a weight of 0: a NaN in it may reach any
 * query whose tile (128 queries) needs the key, and backward a NaN in a query that sees
 * some key any key whose tile (128 keys) needs the query.
 *
 * Backward, from the forward's o and lse:
 *   p = exp(s - lse), dp_ij = do_i . v_j, ds = p (dp - do_i . o_i),
 *   dbias_table[bucket][h] = sum of ds over batch, queries and keys,
 *   dx = ds (1 - (c/cap)^2), dq_i = scale sum_j dx k_j,
 *   dk_j = scale sum_i dx q_i, dv_j = sum_i p do_i,
 * dk and dv summed over the Hq / Hk query heads that share a key head.  A query whose lse is
 * below -2^24 (every key that it sees has a bias of -1e9, say, or of the type's lowest value) takes
 * no part, as one that sees no key: its lse has no place for the log of the sum, and without it
 * p cannot be formed.  (Forward, its softmax is that of its scores in binary32.)
 *
 * q, k, v, o and their gradients are bf16; p and dx are rounded to bf16 for
 * the matrix products (their sums stay binary32).  Scores and lse are binary32: p is off by
 * some |lse| 2^-22 of itself.  D is 32, 64, 96 or 128;
 * Hq is a multiple of Hk.
 * Bases and strides are multiples of 16 bytes.
 *
 * bias_buckets has 2 * reach + 1 entries (entries outside [0, n_buckets) are
 * clipped); bias_table is [n_buckets][Hq], bf16 or fp32 (bias_dtype), as is
 * dbias_table.  reach <= ZERO_ATTN_MAX_REACH. */
typedef struct zero_attn_args {
  size_t struct_bytes;          /* sizeof(zero_attn_args) */
  int32_t B, Tq, Tk, Hq, Hk, D;
  int32_t causal, bias_dtype, n_buckets, reach;
  double scale, cap;
  const void *q, *k, *v;        /* [B][T][H][D] */
  const int32_t *ranges;        /* [B][Tq][2] or NULL */
  const void *bias_table;       /* or NULL */
  const int32_t *bias_buckets;
  void *o;                      /* [B][Tq][Hq][D]: forward's output, backward's input */
  float *lse;                   /* [B][Hq][Tq]: likewise */
  const void *d_o;              /* backward from here on */
  void *dq, *dk, *dv;
  void *dbias_table;            /* or NULL */
  int64_t q_stride[3], k_stride[3], v_stride[3], o_stride[3];   /* batch, token, head */
  int64_t do_stride[3], dq_stride[3], dk_stride[3], dv_stride[3];
  void *workspace;
  size_t workspace_bytes;
} zero_attn_args;

int zero_attn_fwd(const zero_attn_args *args, void *stream);
int zero_attn_bwd(const zero_attn_args *args, void *stream);
/* Bytes of workspace that the two calls take for these sizes (n_buckets 0
 * without a bias); any workspace at least as large will do. */
size_t zero_attn_workspace_bytes(int B, int Tq, int Tk, int Hq, int Hk, int D, int n_buckets,
                                 int backward);

/* The intervals of a batch of packed rows (Tq = Tk = T): doc[b][t] names the
 * document of a token, a document being a run of equal ids; a negative id is
 * padding, which sees nothing and is seen by nothing.  With `causal` a token
 * sees its document up to itself, and, where prefix[b][t] (the length of its
 * document's prefix, the same for all of the document's tokens; NULL: none)
 * reaches further, the prefix too; without, the whole document. */
int zero_attn_ranges(const int32_t *doc, const int32_t *prefix, int B, int T, int causal,
                     int32_t *ranges, void *stream);

/* ---- distillation from a teacher's top logits --------------------------
 *
 * Row n has V student logits z and K teacher entries (idx, t).  With
 * q = softmax(z / tau):
 *   p_k = softmax over the row's entries of t / tau, or, if teacher_lse is
 *   given (the log of the sum of exp(t / tau) over the teacher's whole row),
 *   p_k = exp(t_k / tau - teacher_lse), and what is left of 1 is the mass pT
 *   of a tail that is compared with the student's mass outside the entries,
 *   qT = 1 - sum_k q_k (summed over the outside entries, not by difference; pT is 0 where
 *   the entries are all of [0, V), and where qT is 0 and pT no more than the rounding of
 *   teacher_lse, (1 + |teacher_lse|) 2^-23):
 *   loss[n] = tau^2 w [ sum_k p_k (log p_k - log q_k) + pT (log pT - log qT) ]
 *   stats[n] = { log sum_j exp(z_j / tau),  c },  c = 1 - pT / qT  (1 without a tail),
 *              or, where c < -2^24, log(pT / qT) in its place (c itself is never above 1)
 *   dlogits  = grad_scale tau w (q_j - p_j) at the entries, grad_scale tau w c q_j
 *              elsewhere
 * with w = row_weight[n] (1 if NULL).  0 log 0 = 0.  Entries with idx outside
 * [0, V) are absent; a row with no entry and no tail, or with w = 0, has loss
 * 0 and gradient 0 whatever it holds (its stats are formed all the same).  The
 * entries of a row are distinct.
 *
 * zero_distill_fwd writes loss and stats, and dlogits too if given (one read
 * of the logits for all three); zero_distill_bwd writes dlogits from stats.
 * dlogits may be the logits themselves (same stride).  dtype is that of
 * logits, t and dlogits. 1e-30 <= tau <= 1e30, K <= ZERO_DISTILL_MAX_K, V <= ZERO_DISTILL_MAX_V;
 * logits and t may start at any element. */
typedef struct zero_distill_args {
  size_t struct_bytes;          /* sizeof(zero_distill_args) */
  int64_t N, V;
  int32_t K, dtype;
  double temperature, grad_scale;
  const void *logits;           /* [N][V] */
  const int32_t *teacher_idx;   /* [N][K] */
  const void *teacher_val;      /* [N][K] */
  const float *teacher_lse;     /* [N] or NULL */
  const float *row_weight;      /* [N] or NULL */
  float *loss;                  /* [N], forward */
  float *stats;                 /* [N][2]: forward's output, backward's input */
  void *dlogits;                /* [N][V] */
  int64_t logits_stride, dlogits_stride;
} zero_distill_args;

int zero_distill_fwd(const zero_distill_args *args, void *stream);
int zero_distill_bwd(const zero_distill_args *args, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* ZERO_OPS_H */
