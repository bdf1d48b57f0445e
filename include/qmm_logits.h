/*
 * qmm_logits.h — what a program asks of a head's logits on MI355X (gfx950):
 * the log probabilities of given tokens, the entropy, and the likeliest tokens
 * with theirs.
 *
 * The logits are what qmm_mul_mat writes for an output head (one row a token),
 * or bfloat16 ones.  The conventions of qmm.h hold: the caller owns every
 * buffer, nothing is allocated, copied to the host or synchronized, work is
 * enqueued on `stream`, arguments are checked before anything is enqueued, and
 * the status codes are qmm.h's.
 */
#ifndef QMM_LOGITS_H
#define QMM_LOGITS_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* For every row l of logits, x = scale * softcap * tanh(l / softcap) (scale * l
 * without a cap) and log p(t) = x_t - log sum_i exp(x_i):
 *   logp[r][i]     = log p(tokens[r][i]); -inf for what is no token of the vocabulary
 *   entropy[r]     = - sum_t p(t) log p(t)
 *   top_ids[r][k]  = the tokens of the largest logits l in their order, equal
 *                    ones by the lowest token; top_logp[r][k] = their log p
 *   xtype    : QMM_F32 or QMM_BF16, the type of the logits
 *   logits   : device, rows of vocab values, ld values apart (at least vocab);
 *              aligned to their values
 *   rows, vocab : 1 or more, below 2^23; at most 2^28
 *   scale    : finite and positive (1 / temperature)
 *   softcap  : 0: none; else finite and positive.  Scale and scale * softcap have
 *              to be normal fp32 numbers below 2^127, 1 / softcap finite
 *   tokens, logp      : device, rows x n_tokens (at most 65536); not read where
 *                       n_tokens is 0
 *   entropy           : device, rows; NULL: not wanted
 *   top_ids, top_logp : device, rows x n_top, n_top at most 64 and at most
 *                       vocab; not read where n_top is 0
 *   work     : device, qmm_logprobs_work(...) bytes for the same sizes, 16-byte
 *              aligned; may be NULL when that is 0.  Calls that may run at the
 *              same time need one each; contents need not be kept.
 * One of the results at least has to be wanted; no output overlaps another or
 * an input.  Sums are fp32 and have terms of one sign.  A logit of -inf is a
 * token that cannot be drawn (log p = -inf, with a cap too); a row of nothing
 * else has entropy 0.  A row that holds NaN (or, without a cap, +inf) gives NaN;
 * in the order of the ids a NaN counts as -inf.  How a row is divided, and so
 * its last bits, goes by the number of rows in the call. */
int qmm_logprobs(int xtype, const void* logits, int64_t ld, int64_t rows, int64_t vocab, float scale, float softcap,
                 const int32_t* tokens, int n_tokens, float* logp, float* entropy, int n_top, int32_t* top_ids,
                 float* top_logp, void* work, size_t work_bytes, void* stream);

/* Bytes of workspace that qmm_logprobs needs; 0 also for sizes it rejects.
 * Host logic only. */
size_t qmm_logprobs_work(int xtype, int64_t rows, int64_t vocab, int n_top);

#ifdef __cplusplus
}
#endif
#endif /* QMM_LOGITS_H */
