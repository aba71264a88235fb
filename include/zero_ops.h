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
 *   - zero_embed_fwd/_bwd: the embedding lookup with a factor, and the table's
 *     gradient.
 *   - zero_block_norm_fwd/_bwd: the norm of a block's output, its gate, the
 *     residual sum and the next block's norm, in one pass.
 *   - zero_policy_fwd/_bwd: the clipped policy loss with a KL term on the
 *     student's own samples, with its gradient as the distillation loss's.
 *   - zero_grads_norm, zero_grads_clip: the exact global norm of the gradients
 *     of many tensors, and their unscaling and clipping.
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
 *   - Outputs must not overlap inputs, one another or the workspace unless
 *     stated (where the same address is allowed, other strides are
 *     ZERO_EINVAL).  From the embedding on such calls are ZERO_EINVAL; arrays
 *     whose rows lie between one another's, as columns of one buffer do, are
 *     apart.
 */
#ifndef ZERO_OPS_H
#define ZERO_OPS_H

#include <stddef.h>
#include <stdint.h>

#include "zero_step.h"

#ifdef __cplusplus
extern "C" {
#endif

#define ZERO_OPS_ABI_VERSION 2

/* Largest reach of the distance bias, most buckets, most teacher entries of
 * a row, and longest row of logits. */
#define ZERO_ATTN_MAX_REACH 512
#define ZERO_ATTN_MAX_BUCKETS 256
#define ZERO_DISTILL_MAX_K 1024
#define ZERO_DISTILL_MAX_V (1 << 20)
/* Longest row of an embedding table or a residual stream, most rows of a
 * table, longest row of logits of the policy loss, most tensors of a
 * gradient call. */
#define ZERO_ROW_MAX_C (1 << 14)
#define ZERO_EMBED_MAX_V (1 << 24)
#define ZERO_POLICY_MAX_V (1 << 20)
#define ZERO_GRADS_MAX_COUNT (1 << 16)

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

/* ---- embedding -------------------------------------------------------------
 *
 *   out[n] = scale * table[ids[n]],
 *   dtable[v] = base[v] + scale * sum of dout[n] over the n with ids[n] = v
 * (base NULL: 0).  Ids outside [0, V), such as padding, give rows of zeros and
 * have no part in the gradient.
 *
 * zero_embed_bwd writes all of dtable.  base may be dtable itself (same dtype
 * and stride): the sums are then added, and rows that no id names are left as
 * they are.  A row's sum is binary32 in a fixed order: by the order of n, in
 * pieces of at most 256 terms whose sums are then joined; base is added last, before the
 * one rounding.
 *
 * dtype (ZERO_BF16 or ZERO_F32) is that of table, out and dout, grad_dtype that
 * of dtable, base_dtype that of base.  C is a multiple of 8 up to
 * ZERO_ROW_MAX_C; rows start on 16 bytes (ZERO_EALIGN).  N <= 2^21.  Short calls need no
 * workspace (0 bytes). */
typedef struct zero_embed_args {
  size_t struct_bytes;          /* sizeof(zero_embed_args) */
  int64_t N, V;
  int32_t C, dtype, grad_dtype, base_dtype;
  double scale;
  const int32_t *ids;           /* [N] */
  const void *table;            /* [V][C], forward */
  void *out;                    /* [N][C], forward */
  const void *dout;             /* [N][C], backward from here on */
  const void *base;             /* [V][C] or NULL */
  void *dtable;                 /* [V][C] */
  int64_t table_stride, out_stride, dout_stride, base_stride, dtable_stride;
  void *workspace;              /* backward only */
  size_t workspace_bytes;
} zero_embed_args;

int zero_embed_fwd(const zero_embed_args *args, void *stream);
int zero_embed_bwd(const zero_embed_args *args, void *stream);
size_t zero_embed_workspace_bytes(int64_t N, int C);

/* ---- norms around a block --------------------------------------------------
 *
 * For each token, over its C values, with rms(v) = sqrt(mean(v^2) + eps):
 *   u = y / rms(y) * (post_w + weight_offset)   if post_norm, else y
 *   h = res_scale * x + branch_scale * gate * u         (gate 1 if NULL)
 *   z = h / rms(h) * (pre_w + weight_offset)
 * x is the residual stream, y a block's output, h the new residual stream and z
 * the next block's input.  A weight that is NULL counts as 1 (without the
 * offset).  y NULL: no block, h = res_scale * x.  h (forward) or z may be NULL:
 * not wanted; z is formed from h before its rounding.  gate is [C] for all
 * tokens (gate_tokens 0) or [T][C].
 *
 * Backward, from the forward's h, y, weights and gate, and the gradients dh (NULL:
 * 0) and dz (NULL: 0; h and pre_w are then not read) that come in:
 *   u2 = dz * (pre_w + weight_offset),  hh = h / rms(h)
 *   gh = dh + (u2 - hh * mean(u2 * hh)) / rms(h),     dx = res_scale * gh
 *   du = branch_scale * gate * gh,      dgate = branch_scale * gh * u
 *   dy = du, or with post_norm, yy = y / rms(y), u1 = du * (post_w + weight_offset),
 *   dy = (u1 - yy * mean(u1 * yy)) / rms(y)
 *   dpost_w = sum over tokens of du * yy,  dpre_w = sum of dz * hh,
 * dgate summed over the tokens too where they share the gate.  dx, dy and the
 * weights' gradients may each be NULL: not wanted.
 *
 * dtype (ZERO_BF16 or ZERO_F32) is that of y, z, the weights, the gate and
 * their gradients, res_dtype that of x, h, dh and dx: the same, or ZERO_F32.
 * C is a multiple of 8 up to ZERO_ROW_MAX_C, T <= 2^21; rows start on 16 bytes:
 * base addresses and strides (ZERO_EALIGN).  h may be x, and dx may be dh (same
 * strides).  The workspace is for backward calls that want a gradient summed over
 * the tokens. */
typedef struct zero_block_norm_args {
  size_t struct_bytes;          /* sizeof(zero_block_norm_args) */
  int64_t T;
  int32_t C, dtype, res_dtype, post_norm, gate_tokens, reserved;
  double eps, weight_offset, res_scale, branch_scale;
  const void *x;                /* [T][C], forward */
  const void *y;                /* [T][C] or NULL */
  const void *post_w;           /* [C] or NULL */
  const void *gate;             /* [C] or [T][C] or NULL */
  const void *pre_w;            /* [C] or NULL */
  void *h;                      /* [T][C]: forward's output, backward's input */
  void *z;                      /* [T][C], forward */
  const void *dh, *dz;          /* backward from here on */
  void *dx, *dy;
  void *dpost_w, *dgate, *dpre_w;
  int64_t x_stride, y_stride, gate_stride, h_stride, z_stride;
  int64_t dh_stride, dz_stride, dx_stride, dy_stride, dgate_stride;
  void *workspace;
  size_t workspace_bytes;
} zero_block_norm_args;

int zero_block_norm_fwd(const zero_block_norm_args *args, void *stream);
int zero_block_norm_bwd(const zero_block_norm_args *args, void *stream);
size_t zero_block_norm_workspace_bytes(int64_t T, int C);

/* ---- clipped policy loss --------------------------------------------------
 *
 * Row n has V student logits z and the sampled token a = action[n].  With
 * lse = log sum_j exp(z_j / tau), q_j = exp(z_j / tau - lse) and the token's log
 * probability lp = z_a / tau - lse:
 *   r = exp(lp - old_logp[n])   (old_logp NULL: lp itself, r = 1)
 *   s = min(r A, min(max(r, 1 - clip_low), 1 + clip_high) A),  A = advantage[n]
 *   e = ref_logp[n] - lp,  kl = exp(e) - e - 1     (ref_logp NULL: kl = 0)
 *   loss[n] = w (kl_coef kl - s),   w = row_weight[n] (1 if NULL)
 *   g = -A r  (0 where A > 0 and r > 1 + clip_high, and where A < 0 and
 *       r < 1 - clip_low)  + kl_coef (1 - exp(e)),  the derivative by lp
 *   stats[n] = { lse, lp, g, kl }
 *   dlogits_j = grad_scale w g / tau ([j = a] - q_j)
 * A row whose action is outside [0, V), or whose logits are all -inf, is absent:
 * loss 0, gradient 0, lp, g and kl 0 in its stats.  A row with w = 0 has loss 0 and
 * gradient 0 whatever it holds (its stats are formed all the same).  A row with
 * g = 0 has gradient 0.  g beyond binary32 counts as its largest number in the
 * gradient.
 *
 * zero_policy_fwd writes loss and stats, and dlogits too if given (one read of
 * the logits for all three); zero_policy_bwd writes dlogits from stats (lse, lp
 * and g, whatever loss they came from).  Its q_j carry lse's rounding, or, where |lse| is
 * above 32 (2048 for ZERO_BF16) and lp nearer to 0, lp's.  dlogits may be the logits themselves
 * (same stride; in place the backward gives such a row to one workgroup).  dtype is
 * that of logits and dlogits.  1e-30 <= tau <= 1e30 (and
 * z_j / tau within binary32, or the row's results are NaN), 0 <= clip_low <= 1,
 * clip_high >= 0, N <= 2^21, V <= ZERO_POLICY_MAX_V; logits and dlogits may start at any
 * element (a row of dlogits that starts elsewhere between 16 bytes than the row of
 * logits is stored element by element, in about twice the time). */
typedef struct zero_policy_args {
  size_t struct_bytes;          /* sizeof(zero_policy_args) */
  int64_t N, V;
  int32_t dtype, reserved;
  double temperature, clip_low, clip_high, kl_coef, grad_scale;
  const void *logits;           /* [N][V] */
  const int32_t *action;        /* [N] */
  const float *advantage;       /* [N], forward */
  const float *old_logp;        /* [N] or NULL, forward */
  const float *ref_logp;        /* [N] or NULL, forward */
  const float *row_weight;      /* [N] or NULL */
  float *loss;                  /* [N], forward */
  float *stats;                 /* [N][4]: forward's output, backward's input */
  void *dlogits;                /* [N][V] */
  int64_t logits_stride, dlogits_stride;
} zero_policy_args;

int zero_policy_fwd(const zero_policy_args *args, void *stream);
int zero_policy_bwd(const zero_policy_args *args, void *stream);

/* ---- the global norm of many gradients, and clipping ---------------------
 *
 * The tensors are dense vectors of sizes[i] elements at grads[i], any element
 * alignment, dtypes[i] ZERO_F32 or ZERO_BF16; the arrays of addresses, sizes and
 * dtypes are HOST memory, read during the call only.
 *
 * zero_grads_norm: the norm state of g = grads * inv_scale (binary32) of all the
 * tensors into `acc`, which is overwritten, or added to with `add`: bit for bit what
 * zero_grad_norm adds for the tensors one by one, so it may be given to zero_adamw_step,
 * and summed over ranks that each hold a part of one gradient: its shards after the
 * reduction (the sum over ranks' gradients before it is not the reduced gradient's norm).
 * At most 2^37 elements in an accumulator.
 *
 * zero_grads_clip: outs[i] = (grads[i] * inv_scale) * coef, rounded to out_dtypes[i],
 * with the skip and the coefficient that zero_step_gate derives from the n_accs
 * accumulators, max_norm and check_overflow; a skipped call writes no tensor.  outs[i]
 * may be grads[i] (same dtype), and overlaps no other tensor: looked for at each call, in
 * the order of the addresses, unless outs_apart is 1, by which the caller says that it has
 * seen to it (0.03 us a tensor on the host).  norm_out, coef_out and
 * skipped_out (each may be NULL): the global norm, infinite where a value is not finite,
 * the coefficient (0 where skipped) and 1 where skipped, else 0. */
typedef struct zero_grads_args {
  size_t struct_bytes;          /* sizeof(zero_grads_args) */
  int64_t count;
  const void *const *grads;     /* HOST [count] */
  void *const *outs;            /* HOST [count], clip */
  const int64_t *sizes;         /* HOST [count] */
  const int32_t *dtypes;        /* HOST [count] */
  const int32_t *out_dtypes;    /* HOST [count], clip */
  double inv_scale;
  zero_norm_acc *acc;           /* norm */
  int32_t add;                  /* norm */
  int32_t n_accs;               /* clip from here on */
  const zero_norm_acc *accs;
  double max_norm;
  int32_t check_overflow, outs_apart;
  float *norm_out, *coef_out;
  int32_t *skipped_out;
  void *workspace;              /* norm */
  size_t workspace_bytes;
} zero_grads_args;

int zero_grads_norm(const zero_grads_args *args, void *stream);
int zero_grads_clip(const zero_grads_args *args, void *stream);
size_t zero_grads_workspace_bytes(void);

#ifdef __cplusplus
}
#endif

#endif /* ZERO_OPS_H */
