/*
 * ts_moe_ops.h -- the operators next to the routed half, on B200 (sm_100a).
 *
 * A decoder layer's routed half (ts_moe.h) takes post-norm activations and adds
 * to a residual stream.  The calls here make those activations (ts_moe_rmsnorm),
 * multiply 8-bit rows with 8-bit matrices (ts_moe_fp8_matmul: a dense
 * projection, or the experts' products of a long prompt), apply the activation
 * between an expert's two products (ts_moe_act_quant), and tell how evenly the
 * router loads the experts (ts_moe_balance).  They need no handle.
 *
 * Conventions
 *   - All pointers inside the argument structs are device pointers on the
 *     current CUDA device, and `stream` (a cudaStream_t, NULL = legacy default
 *     stream) belongs to it.  Calls are asynchronous, allocate nothing, copy
 *     nothing to the host, and can be captured into a CUDA graph.  They keep no
 *     state between calls; calls on different streams may overlap as long as
 *     their outputs and workspaces differ.
 *   - Strides (ld_*, *_row, ...) count elements; the innermost dimension is
 *     contiguous.  Pointers are aligned to their elements, and to more where a
 *     field says so.  Outputs must not overlap inputs or each other, except where
 *     a field says so; scale strides that would put two scales in one place are
 *     refused.
 *   - 8-bit rows are E4M3 (finite range +-448, 0x7F = NaN) with one float32
 *     scale per 128 consecutive columns of a row, the last group of a row being
 *     short where the width is no multiple of 128; an element is q * scale.
 *     They are formed as scale = max(amax, 2^-100) * (1 / 448), the reciprocal and
 *     the product rounded to float32, and q = e4m3(v / scale), the quotient by that
 *     scale rounded to float32 and then to nearest even: a group of zeros has a
 *     normal scale, and a NaN or an infinity in a group makes its scale, and so
 *     its values, non-finite.
 *   - Every function returns a ts_moe_status; on failure
 *     ts_moe_last_error(NULL) gives the reason on the calling thread.  A call
 *     with no rows returns TS_MOE_OK and does nothing, except that
 *     ts_moe_balance then still writes zeros to its per-expert outputs.
 */
#ifndef TS_MOE_OPS_H
#define TS_MOE_OPS_H

#include <stdint.h>

#include "ts_moe.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Element types of 16- and 32-bit tensors. */
enum { TS_DT_BF16 = 0, TS_DT_FP16 = 1, TS_DT_FP32 = 2 };

#define TS_MOE_SCALE_BLOCK 128 /* columns of an 8-bit row, rows and columns of an 8-bit matrix, that share a scale */
#define TS_MOE_MAX_ROWS (1 << 24)

/* Root-mean-square norm, with the residual's addition before it:
 *   r = resid + delta, rounded to the residual's type (delta NULL: r = resid)
 *   v = r / sqrt(mean(r^2) + eps) * gamma        (float32 throughout)
 * resid_out <- r, y <- v rounded to y_type, q / q_scale <- v as 8-bit rows.
 * The norm reads the rounded r, so a fused call equals an addition stored to
 * the stream followed by a norm of the stream.  A row whose sum of squares
 * passes float32's largest value (|r| near 2^64 / sqrt(hidden)) gives v = 0. */
typedef struct {
  int32_t rows;        /* 0 .. TS_MOE_MAX_ROWS */
  int32_t hidden;      /* 1 .. 16384 */
  int32_t resid_type;  /* TS_DT_* of resid and resid_out */
  int32_t delta_type;  /* TS_DT_*, ignored when delta is NULL */
  int32_t gamma_type;  /* TS_DT_*, ignored when gamma is NULL */
  int32_t y_type;      /* TS_DT_*, ignored when y is NULL */
  float eps;           /* >= 0, finite */
  const void* resid;   /* [rows][hidden] */
  int64_t ld_resid;
  const void* delta;   /* [rows][hidden] or NULL */
  int64_t ld_delta;
  const void* gamma;   /* [hidden] or NULL (ones) */
  void* resid_out;     /* [rows][hidden] or NULL; may be resid itself (same ld); refused without delta */
  int64_t ld_resid_out;
  void* y;             /* [rows][hidden] or NULL */
  int64_t ld_y;
  uint8_t* q;          /* [rows][hidden] E4M3 or NULL; at least one of y, q */
  int64_t ld_q;
  float* q_scale;      /* element (row, group) at row * qs_row + group * qs_group; required iff q */
  int64_t qs_row;
  int64_t qs_group;
} ts_moe_rmsnorm_args;
ts_moe_status ts_moe_rmsnorm(const ts_moe_rmsnorm_args* args, void* stream);

/* The activation between an expert's two products, as 8-bit rows:
 *   TS_ACT_SWIGLU          v = silu(gate) * up
 *   TS_ACT_SWIGLU_CLAMPED  g = min(gate, limit), u = clamp(up, -limit, limit),
 *                          v = g * sigmoid(alpha * g) * (u + 1)
 * q / q_scale <- v.  gate and up may be the two halves of one product's rows. */
typedef struct {
  int32_t rows;     /* 0 .. TS_MOE_MAX_ROWS */
  int32_t inter;    /* 1 .. 65536 */
  int32_t act;      /* TS_ACT_* */
  int32_t in_type;  /* TS_DT_* of gate and up */
  float act_alpha;  /* finite; clamped form only */
  float act_limit;  /* > 0; clamped form only */
  const void* gate; /* [rows][inter] */
  int64_t ld_gate;
  const void* up;   /* [rows][inter] */
  int64_t ld_up;
  uint8_t* q;       /* [rows][inter] E4M3 */
  int64_t ld_q;
  float* q_scale;   /* element (row, group) at row * qs_row + group * qs_group */
  int64_t qs_row;
  int64_t qs_group;
} ts_moe_act_quant_args;
ts_moe_status ts_moe_act_quant(const ts_moe_act_quant_args* args, void* stream);

/* Product of 8-bit rows with an 8-bit matrix whose scales cover 128 x 128 blocks:
 *   out[m][n] = sum_c a_scale[m][c] * b_scale[n / 128][c] * sum_{k in block c} a[m][k] * b[n][k]  (+ add[m][n])
 * with float32 sums, rounded once to out_type.  The two scales' product is formed
 * first, in float32: it should stay in the normal range.  Grouped form (offsets given):
 * b is [num_groups][n][k], and rows offsets[g] .. offsets[g + 1] - 1 use matrix
 * g; the other rows of out are left as they were.  offsets is device memory and
 * is read on the device: the host neither knows nor waits for the group sizes.
 * Offsets are taken as min(max over the offsets up to here, rows), so that no
 * value reads or writes out of range.  a and b rows and b matrices start at
 * 16-byte boundaries (ld_a, ld_b, b_group multiples of 16, a and b 16-byte
 * aligned); k and n themselves are free.  Should a bounded wait inside the
 * kernel give up (2 s), the outputs it could not form are NaN. */
typedef struct {
  int32_t rows;       /* 0 .. TS_MOE_MAX_ROWS */
  int32_t n;          /* 1 .. 1 << 20 */
  int32_t k;          /* 1 .. 1 << 20 */
  int32_t num_groups; /* 1 .. TS_MOE_MAX_EXPERTS; 1 without offsets */
  int32_t out_type;   /* TS_DT_* of out and add */
  int32_t reserved;   /* 0 */
  const uint8_t* a;   /* [rows][k] E4M3 */
  int64_t ld_a;
  const float* a_scale; /* element (row, block) at row * as_row + block * as_block */
  int64_t as_row;
  int64_t as_block;
  const uint8_t* b;   /* [num_groups][n][k] E4M3 */
  int64_t ld_b;
  int64_t b_group;
  const float* b_scale; /* element (group, n / 128, block) at group * bs_group + (n / 128) * bs_row + block * bs_block */
  int64_t bs_group;
  int64_t bs_row;
  int64_t bs_block;
  const int32_t* offsets; /* [num_groups + 1], or NULL */
  const void* add;    /* [rows][n] or NULL; may be out itself (same ld) */
  int64_t ld_add;
  void* out;          /* [rows][n] */
  int64_t ld_out;
} ts_moe_fp8_matmul_args;
ts_moe_status ts_moe_fp8_matmul(const ts_moe_fp8_matmul_args* args, void* stream);

/* How evenly a routing loads the experts, with the loss that evens it and the
 * loss's gradient.  Over the T rows whose mask is not 0:
 *   counts[e] = entries of idx equal to e       (entries outside [0, E) count for nothing)
 *   f[e] = counts[e] * E / (K * T)
 *   p[t] = softmax(logits[t])                   (TS_SCORE_SOFTMAX_*)
 *          sigmoid(l) / sum(sigmoid(l))         (TS_SCORE_SIGMOID_RENORM)
 *   prob[e] = mean over t of p[t][e]
 *   loss = coef * sum_e f[e] * prob[e]
 *   dlogits = dloss * d loss / d logits, f held fixed; rows that the mask leaves out get 0
 * offsets[e] = counts[0] + .. + counts[e - 1] (offsets[E] the total): the group
 * bounds of ts_moe_fp8_matmul for rows sorted by expert.  With T = 0 the loss,
 * prob and the gradient are 0.  A row whose logits are all -inf has p = 0; a NaN
 * logit makes the loss and that row's gradient NaN.  logits are the ones that
 * ts_moe_route writes (add the router bias first where the weights use it), idx
 * is its idx.  Sums are formed in a fixed order: equal calls give equal bits. */
typedef struct {
  int32_t rows;     /* 0 .. TS_MOE_MAX_ROWS */
  int32_t experts;  /* E, 1 .. 256 */
  int32_t top_k;    /* K, 1 .. min(8, E) */
  int32_t score;    /* TS_SCORE_* */
  int32_t dtype;    /* TS_DT_* of logits and dlogits */
  float coef;       /* finite */
  const void* logits;   /* [rows][E] */
  int64_t ld_logits;
  const int32_t* idx;   /* [rows][K] */
  int64_t ld_idx;
  const uint8_t* mask;  /* [rows], or NULL (every row counts) */
  const float* dloss;   /* one float32, or NULL (1); read only when dlogits is given */
  float* loss;          /* one float32 */
  float* prob;          /* [E] or NULL */
  int32_t* counts;      /* [E] */
  int32_t* offsets;     /* [E + 1] or NULL */
  void* dlogits;        /* [rows][E] or NULL */
  int64_t ld_dlogits;
  void* workspace;      /* ts_moe_balance_workspace() bytes, 16-byte aligned; two calls that can overlap need two */
  uint64_t workspace_bytes;
} ts_moe_balance_args;
ts_moe_status ts_moe_balance(const ts_moe_balance_args* args, void* stream);
/* Bytes of workspace a call with these sizes needs. */
uint64_t ts_moe_balance_workspace(int32_t rows, int32_t experts);

#ifdef __cplusplus
}
#endif
#endif /* TS_MOE_OPS_H */
