/*
 * tq2_sample.h -- C ABI of libtq2's token choice: temperature, top-k, min-p
 * and top-p, with random numbers that the caller gives.
 *
 * The conventions of tq2.h hold: device pointers of the caller, nothing
 * allocated or synchronised, work only enqueued on `stream`, negative
 * tq2_status values for errors and nothing enqueued with them.  The workspace
 * needs no preparation and means nothing afterwards; calls that may run at the
 * same time (captured graphs among them) need one each.
 */
#ifndef TQ2_SAMPLE_H
#define TQ2_SAMPLE_H

#include "tq2_attn.h"

#ifdef __cplusplus
extern "C" {
#endif

#define TQ2_SAMPLE_MAX_ROWS 4096
#define TQ2_SAMPLE_MAX_VOCAB (1 << 20)

/* All fields are 8 bytes wide.  Where an array of settings is given it has one
 * for each row, and the number after it is not looked at. */
typedef struct tq2_sample_args {
  const void* logits;            /* [rows, vocab], rows row_stride elements apart */
  const float* u;                /* f32 [rows], in [0, 1) */
  int32_t* ids;                  /* [rows] */
  float* logprob;                /* f32 [rows] or NULL */
  const float* temperatures;     /* f32 [rows] or NULL */
  const int32_t* top_ks;         /* [rows] or NULL */
  const float* top_ps;           /* f32 [rows] or NULL */
  const float* min_ps;           /* f32 [rows] or NULL */
  int64_t rows;                  /* 0 .. TQ2_SAMPLE_MAX_ROWS */
  int64_t vocab;                 /* 1 .. TQ2_SAMPLE_MAX_VOCAB */
  int64_t row_stride;            /* 0 (one row for all) or more, if rows > 1 */
  int64_t logits_type;           /* TQ2_TYPE_F32, F16 or BF16 */
  int64_t top_k;
  double temperature;
  double top_p;
  double min_p;
  void* workspace;               /* 16-byte aligned */
  int64_t workspace_bytes;
} tq2_sample_args;

/* Bytes of workspace that tq2_sample needs for these sizes, or 0 (also for
 * sizes that it refuses).  Pure host function; no pointer is looked at. */
size_t tq2_sample_workspace_bytes(const tq2_sample_args* args);

/* The next token of each row.  With the tokens in falling order of their
 * logits l, the lowest index first among equals, and e = exp((l - max) / T):
 *   1. the first top_k are kept (all, if top_k <= 0);
 *   2. of these, those with e >= min_p;
 *   3. of these, the shortest run from the top whose sum of e reaches top_p of
 *      all of step 2's (all, if top_p >= 1; at least one);
 *   4. ids is the first whose sum of e, from the top through itself, exceeds u
 *      times that of step 3.
 * logprob is the token's log of e over step 3's sum.
 * A temperature that is not above zero takes the largest logit, the lowest
 * index among equals, with logprob 0.  Settings past their range act as the
 * nearest that is in it (temperatures below 1e-36 as 1e-36), NaN as none (u:
 * 0).  Logits that are NaN count as -infinity, which is never taken; a row of
 * nothing else gives -1 and logprob -infinity; +infinity shares all of e among
 * its equals.
 * Accuracy: e in 64 bits, held in units of 2^-43 of the largest (tokens below
 * half a unit are never taken) and summed as whole numbers: the token does
 * not hang on any order, and differs from the real numbers' only where u times
 * the sum lies within about vocab * 2^-43 of a border.
 * logits: aligned to their type; u, ids, logprob and settings: 4-byte aligned.
 * rows == 0 is a no-op.  Errors: INVALID (null pointer, size or type out of
 * range, a scalar setting that is NaN, a negative temperature, a workspace that
 * is too small), ALIGN, ALIAS (an output overlaps another operand), DEVICE,
 * LAUNCH. */
int tq2_sample(const tq2_sample_args* args, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* TQ2_SAMPLE_H */
