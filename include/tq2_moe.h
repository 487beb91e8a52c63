/*
 * tq2_moe.h -- C ABI of libtq2's mixture-of-experts operators: the router and
 * the chosen experts' feed-forward on 4-bit or ternary weights.
 *
 * The conventions of tq2.h hold: device pointers of the caller, nothing
 * allocated or synchronised, work only enqueued on `stream`, negative
 * tq2_status values for errors and nothing enqueued with them.  Types are the
 * TQ2_TYPE_* of tq2_attn.h: F32, F16 or BF16.  Workspaces need no preparation
 * and mean nothing afterwards; calls that may run at the same time (captured
 * graphs among them) need one each.
 */
#ifndef TQ2_MOE_H
#define TQ2_MOE_H

#include "tq2_attn.h"

#ifdef __cplusplus
extern "C" {
#endif

#define TQ2_MOE_MAX_EXPERTS 1024
#define TQ2_MOE_MAX_TOP_K 16
/* Most tokens of one tq2_moe_experts call, and of one tq2_moe_route call. */
#define TQ2_MOE_MAX_TOKENS 128
#define TQ2_MOE_MAX_ROUTE_TOKENS (1 << 20)
#define TQ2_MOE_MAX_DIM 16384

/* Scores of the router. */
#define TQ2_MOE_SOFTMAX 0
#define TQ2_MOE_SIGMOID 1

/* Weight formats of the experts. */
#define TQ2_MOE_Q4 0
#define TQ2_MOE_TERNARY 1

/* All fields are 8 bytes wide. */
typedef struct tq2_moe_route_args {
  const void* x;             /* [tokens, hidden] of act_type */
  const void* weight;        /* [experts, hidden] of weight_type */
  const float* bias;         /* f32 [experts] or NULL: added to the probabilities for the choice alone */
  float* weights;            /* f32 [tokens, top_k] */
  int32_t* ids;              /* [tokens, top_k] */
  int64_t tokens;            /* 0 .. TQ2_MOE_MAX_ROUTE_TOKENS */
  int64_t hidden;            /* a multiple of 8 */
  int64_t experts;           /* top_k .. TQ2_MOE_MAX_EXPERTS */
  int64_t top_k;             /* 1 .. TQ2_MOE_MAX_TOP_K */
  int64_t act_type;
  int64_t weight_type;
  int64_t scoring;           /* TQ2_MOE_SOFTMAX (over all experts) or TQ2_MOE_SIGMOID */
  int64_t renormalize;       /* the chosen probabilities are divided by their sum */
  double scale;              /* and multiplied by this */
  void* workspace;           /* 16-byte aligned */
  int64_t workspace_bytes;
} tq2_moe_route_args;

/* Bytes of workspace that tq2_moe_route needs for these sizes, or 0 (also for
 * sizes that it refuses).  Pure host function; no pointer is looked at. */
size_t tq2_moe_route_workspace_bytes(const tq2_moe_route_args* args);

/* For each token: scores x W^T, their softmax or sigmoid p, and the top_k
 * experts of the largest score (with a bias: of the largest p + bias), largest
 * first, the lowest index first among equals; ids holds them and weights their
 * p, by `renormalize` and `scale`.
 * Accuracy: products and sums in 64 bits, so that only scores closer than
 * about 1e-14 of sum |x w| change places; weights are rounded once to f32.
 * Scores that are NaN come after all others, with a bias too, for which the
 * softmax is then that of the others (those at +infinity share it; where all
 * are -infinity, these do).  The weights of a token with a NaN score are NaN
 * where it enters their sum, and its softmax weights where the largest score is
 * infinite.  Where all chosen probabilities lie near or below the least f64
 * number their shares, which `renormalize` gives, are those of exp(score), equal
 * ones where all chosen scores are -infinity.
 * x, weight and workspace: 16-byte aligned; the others 4-byte aligned.
 * tokens == 0 is a no-op.  Errors: INVALID (null pointer, size or type out of
 * range, a scale that is not finite, a workspace that is too small), SHAPE
 * (hidden not a multiple of 8), ALIGN, ALIAS (an output overlaps another
 * operand), DEVICE, LAUNCH. */
int tq2_moe_route(const tq2_moe_route_args* args, void* stream);

typedef struct tq2_moe_experts_args {
  const void* x;             /* [tokens, hidden] of act_type */
  const void* residual;      /* the same, or NULL */
  void* out;                 /* the same; may be x or residual itself */
  const int32_t* ids;        /* [tokens, top_k] */
  const float* weights;      /* f32 [tokens, top_k] */
  const void* gate_up;       /* [experts, 2 inter, hidden]: an expert's inter gate rows, then its inter up rows */
  const void* gate_up_scales;
  const void* down;          /* [experts, hidden, inter] */
  const void* down_scales;
  int64_t tokens;            /* 0 .. TQ2_MOE_MAX_TOKENS */
  int64_t top_k;             /* 1 .. TQ2_MOE_MAX_TOP_K */
  int64_t experts;           /* 1 .. TQ2_MOE_MAX_EXPERTS */
  int64_t hidden;            /* multiples of 128 up to TQ2_MOE_MAX_DIM */
  int64_t inter;
  int64_t act_type;
  int64_t format;            /* TQ2_MOE_Q4 or TQ2_MOE_TERNARY */
  int64_t group;             /* of the 4-bit scales: 32, 64 or 128; 128 for ternary weights */
  void* workspace;
  int64_t workspace_bytes;
} tq2_moe_experts_args;

/* Bytes of workspace that tq2_moe_experts needs for these sizes, or 0 (also
 * for sizes that it refuses).  Pure host function; no pointer is looked at. */
size_t tq2_moe_experts_workspace_bytes(const tq2_moe_experts_args* args);

/* out[t] = residual[t] + sum_j weights[t, j] * (silu(x G_e^T) * (x U_e^T)) D_e^T with
 * e = ids[t, j].  A place whose id is not an expert takes no part; the same
 * expert twice counts twice; a token without any expert gets its residual, or
 * zeros.
 * TQ2_MOE_Q4: codes and scales as in tq2_q4.h, the experts' rows one after
 * another.  TQ2_MOE_TERNARY: gate_up and down are the resident weights that
 * tq2_reformat_aos_to_soa gives for n = experts * 2 * inter rows of hidden and
 * n = experts * hidden rows of inter; the scales are NULL.
 * Accuracy: weights exact; x and the rows between the projections as 31-bit
 * integers under a power of two per row and 128 columns, products and their
 * sums over a scale's columns exact, f32 beyond: each projection is within
 * 1e-5 * sum_k |x w| + 2^-30 * sum_k X_k |w|, with X_k the largest |x| of k's 128
 * columns (128 j .. 128 j + 127); the second term counts where a column far
 * above the others meets weights of almost zero.  What f32 loses below its
 * normal numbers comes on top, 2^-140 * (1 + sum |w|) at most.  A row between the
 * projections and its product with its weight have to stay below 2^127: past
 * that the output may be infinite or NaN.  The output is rounded once
 * to its type.  The order of all sums is fixed: a call repeats its results.
 * Only rows of x whose token chose an expert meet that expert's weights: a row
 * that is not finite reaches its own output alone.
 * x, residual, out, codes, scales, workspace: 16-byte aligned; ids and
 * weights: 4-byte aligned.
 * tokens == 0 is a no-op.  Errors: INVALID (null pointer, size, type, format
 * or group out of range, a workspace that is too small), SHAPE (hidden or
 * inter not a multiple of 128), ALIGN, ALIAS (out overlaps a weight, ids,
 * weights, the workspace, or x or residual other than exactly), DEVICE, LAUNCH. */
int tq2_moe_experts(const tq2_moe_experts_args* args, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* TQ2_MOE_H */
