/*
 * qmm_kv.h — a paged key-value cache on MI355X (gfx950): appending keys and
 * values with the rotation of positions applied on the way, and attention
 * over the cache for single new tokens and for prompts.
 *
 * These are the steps of a layer between its q, k and v projections
 * (qmm_mul_mat_multi) and its output projection: the cache rows are the same
 * Q8_0 blocks that qmm_quantize_act writes and qmm_dequantize reads, or
 * 16-bit floats.  The conventions of qmm.h hold for every call: the caller
 * owns every buffer, nothing is allocated, copied to the host or
 * synchronized, work is enqueued on `stream`, arguments are checked before
 * anything is enqueued, and the status codes are qmm.h's.  Arrays of 32-bit
 * values are 4-byte aligned, the angles of a rotation 8-byte; every other
 * device pointer 16-byte (QMM_ERR_ALIGN otherwise).
 *
 * What lies in device memory cannot be checked on the host.  The kernels
 * check it themselves: no read or write leaves the buffers for any contents
 * of q_start, kv_len, table, pos and prefix.  A table entry outside
 * [0, n_pages) means "no page": its keys are masked, its tokens not stored.
 */
#ifndef QMM_KV_H
#define QMM_KV_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Element types beside the block formats of qmm_type. */
enum {
    QMM_F32 = 32,  /* activations */
    QMM_F16 = 33,  /* cache rows */
    QMM_BF16 = 34  /* activations, cache rows */
};

/* How rotary pairs lie in a head: (2i, 2i+1), or (i, i + n_rot/2). */
enum { QMM_ROPE_PAIRS = 0, QMM_ROPE_HALVES = 1 };

/* The cache of one layer.  Page p holds, for head h, page_size consecutive
 * rows of head_dim values: row j of it starts at row
 * (p * n_kv + h) * page_size + j of the array, so the whole array is
 * n_pages * n_kv * page_size rows that qmm_dequantize can read. */
typedef struct {
    void* k;           /* device, qmm_kv_bytes(...) bytes, 16-byte aligned */
    void* v;           /* device, the same size                            */
    int32_t type;      /* QMM_Q8_0, QMM_F16 or QMM_BF16                    */
    int32_t n_kv;      /* key-value heads                                  */
    int32_t head_dim;  /* 64, 96, 128, 192 or 256                          */
    int32_t page_size; /* tokens of a page: a multiple of 16               */
    int64_t n_pages;
} qmm_kv_cache;

/* The new tokens of a batch and where they lie.  Sequence s has the rows
 * q_start[s] .. q_start[s+1]-1 of the inputs and outputs (none is allowed);
 * its cache holds kv_len[s] tokens, these new ones the last of them, so row
 * q_start[s] + i stands at index p = kv_len[s] - n + i, n being the number of
 * its rows.  Token j of it lies in row j % page_size of page
 * table[s * table_width + j / page_size].  Rows from q_start[n_seqs] to
 * n_tokens-1 belong to no sequence and are left as they are. */
typedef struct {
    const int32_t* q_start; /* device, n_seqs + 1, not decreasing, first 0     */
    const int32_t* kv_len;  /* device, n_seqs                                  */
    const int32_t* table;   /* device, n_seqs x table_width                    */
    int32_t n_seqs;         /* 65536 at most                                   */
    int32_t table_width;    /* pages of a sequence at most, 2^30 tokens in all */
    int64_t n_tokens;       /* rows of q, k, v and out, below 2^23             */
    int64_t max_kv;         /* largest kv_len, as far as known; 0: unknown (the
                               table's width counts).  It only decides how the
                               work is split: results hold for any value       */
} qmm_kv_batch;

/* The rotation of positions: pair i of the first n_rot values of a head turns
 * by angle a = pos * freqs[i], (x, y) -> (x cos a - y sin a, x sin a + y cos a);
 * the values behind n_rot stay.  With several axes (say time, height and
 * width) the first sections[0] pairs take their position from axis 0, the
 * next sections[1] from axis 1, and so on.  Angles and products are computed
 * in 64 bits and rounded to fp32 once, so that far positions lose nothing and
 * stored codes are defined to the bit. */
typedef struct {
    const double* freqs;   /* device, n_rot / 2 angles per position (qmm_rope_freqs) */
    const int32_t* pos;    /* device, n_axes x n_tokens; NULL: the index p of the
                              token in its sequence, on every axis                  */
    int32_t n_rot;         /* even, 2 .. head_dim                                   */
    int32_t pairing;       /* QMM_ROPE_PAIRS or QMM_ROPE_HALVES                     */
    int32_t n_axes;        /* 1 .. 4                                                */
    int32_t sections[4];   /* pairs of each axis, n_rot / 2 in all; not read for one */
} qmm_rope;

/* What the scores of attention go through, in this order:
 *   s = scale * (q . k);  s = softcap * tanh(s / softcap) if softcap > 0;
 *   s -= slopes[h] * |p - j| if slopes is given;
 * and key j is visible to the token at p if j < kv_len and
 *   (j <= p and (window == 0 or p - j < window))  or  j < prefix[s]. */
typedef struct {
    float scale;           /* finite                                             */
    float softcap;         /* 0: none; else finite and positive                  */
    int32_t window;        /* 0: none                                            */
    int32_t algo;          /* 0: chosen by the sizes (qmm_attn_choice); 1: split
                              kernels; 2: tile kernels                           */
    const float* slopes;   /* device, one a query head, or NULL                  */
    const int32_t* prefix; /* device, n_seqs, or NULL                            */
} qmm_attn_opts;

/* Bytes of the key (or value) array of a cache; 0 for a type, head_dim or
 * page_size that is not supported, or sizes that are not positive. */
size_t qmm_kv_bytes(int type, int n_kv, int head_dim, int page_size, int64_t n_pages);

/* freqs[i] = scale * base^(-2i / n_rot) / (factors ? factors[i] : 1), in 64
 * bits, for i < n_rot / 2.
 *   freqs   : device, written
 *   factors : device fp32, n_rot / 2, or NULL (a model's rope factors)
 * base and scale finite and positive. */
int qmm_rope_freqs(double* freqs, int n_rot, double base, double scale, const float* factors, void* stream);

/* Stores the new tokens' keys, rotated, and values in their cache rows, and
 * rotates the queries.
 *   rope  : NULL for no rotation
 *   xtype : QMM_F32 or QMM_BF16, the type of k, v, q and q_out
 *   k, v  : device, n_tokens rows of n_kv heads of head_dim values; rows are
 *           ldk and ldv values apart (multiples of 8, at least a row)
 *   q     : device, n_tokens rows of n_q heads, ldq values apart; NULL for none
 *   q_out : device, n_tokens x n_q x head_dim, written; may be q itself when
 *           ldq is n_q * head_dim; no other overlap is allowed.  NULL with q
 * Q8_0 rows are bit for bit what qmm_quantize_act gives for the fp32 values of
 * the rotated row; F16 and BF16 rows are these rounded to nearest even.
 * Tokens with p < 0, or whose page is missing, are not stored.  Two tokens of
 * a call must not name the same cache row. */
int qmm_kv_append(const qmm_kv_cache* cache, const qmm_kv_batch* batch, const qmm_rope* rope, int xtype, const void* k,
                  int64_t ldk, const void* v, int64_t ldv, const void* q, int64_t ldq, int n_q, void* q_out,
                  void* stream);

/* out[row][h] = sum over the visible keys j of softmax_j(s) v_j, for every
 * row of a sequence and query head h, which reads key-value head
 * h / (n_q / n_kv).  A row that sees no key gives zeros.
 *   xtype : QMM_F32 or QMM_BF16, the type of q and out
 *   q     : device, n_tokens rows of n_q heads, ldq values apart (a multiple
 *           of 8, at least a row); n_q a multiple of n_kv
 *   out   : device, n_tokens x n_q x head_dim, written; not overlapping q
 *   work  : device, qmm_attn_work(...) bytes for the same arguments, 16-byte
 *           aligned; may be NULL when that is 0.  Calls that may run at the
 *           same time need one each; contents need not be kept.
 * Fp32 results are as exact as a product in fp32, bf16 results are these
 * rounded once, whichever kernels compute them, with one reserve: over F16 and
 * Q8_0 rows the products are made of 16-bit parts, whose smallest step is 2^-38
 * of the largest query value of a head, of the largest weight of a row, and of
 * the largest key of a tile of 64 (and the largest value among 32 of any key
 * that the rows of a tile see), so that what is more than 2^16 smaller than these
 * keeps fewer bits than fp32's, and what is 2^20 smaller still 18.  What lies in the cache at
 * places that no row of the call sees has no effect, infinities and NaN
 * included; visible keys and values have to be finite.  Batches whose grids
 * would pass 2^32 work-items are refused (QMM_ERR_SHAPE).
 *
 * The kernels are chosen, and the keys divided, by what a batch's sequences have
 * on average.  Prompts beside single tokens over long caches belong in two calls
 * on parts of the batch's arrays: 2048 tokens beside one over 131072 keys (Q8_0, 32
 * heads on 8 of 128) take 9.1 ms in one, 0.15 + 0.07 in two. */
int qmm_attn(const qmm_kv_cache* cache, const qmm_kv_batch* batch, const qmm_attn_opts* opts, int xtype, const void* q,
             int64_t ldq, int n_q, void* out, void* work, size_t work_bytes, void* stream);

/* Bytes of workspace that qmm_attn needs; 0 also for arguments it rejects.
 * Host logic only: the device pointers of the structures are not read. */
size_t qmm_attn_work(const qmm_kv_cache* cache, const qmm_kv_batch* batch, const qmm_attn_opts* opts, int xtype,
                     int n_q);

/* The kernel family that algo 0 takes for these sizes: 1 = split kernels
 * (few rows a sequence; bound by reading the cache), 2 = tile kernels; 0 for
 * sizes that qmm_attn rejects.  With a window fewer keys count, and the choice
 * may be another. */
int qmm_attn_choice(const qmm_kv_cache* cache, const qmm_kv_batch* batch, int xtype, int n_q);

#ifdef __cplusplus
}
#endif
#endif /* QMM_KV_H */
