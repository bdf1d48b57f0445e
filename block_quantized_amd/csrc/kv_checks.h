// kv_checks.h — argument checks shared by the host units of the key-value cache
// and of what goes with it.
#pragma once

#include <stdint.h>

#include "kv_internal.h"

namespace qmm {
namespace {

constexpr int64_t kMaxRows = (int64_t(1) << 23) - 1;  // tokens: grids stay below 2^32 work-items
constexpr int64_t kMaxLength = int64_t(1) << 30;   // tokens of a sequence
constexpr int kMaxSeqs = 1 << 16;                  // every workgroup looks its sequence up among them
constexpr int kMaxHeads = 4096;
constexpr int kMaxWords = kTreeWords;              // of a tree's row: 64 new tokens each

inline int hip_status(hipError_t e) { return e == hipSuccess ? QMM_OK : QMM_ERR_HIP; }

inline int check_ptr(const void* p, unsigned align = 16) {
    if (!p) return QMM_ERR_NULL;
    return reinterpret_cast<uintptr_t>(p) & (align - 1) ? QMM_ERR_ALIGN : QMM_OK;
}

inline int check_type(int t) {
    if (t == QMM_Q8_0 || t == QMM_F16 || t == QMM_BF16) return QMM_OK;
    return qmm_block_size(t) || t == QMM_F32 ? QMM_ERR_UNSUPPORTED : QMM_ERR_TYPE;
}

inline int check_xtype(int t) {
    if (t == QMM_F32 || t == QMM_BF16) return QMM_OK;
    return qmm_block_size(t) || t == QMM_F16 ? QMM_ERR_UNSUPPORTED : QMM_ERR_TYPE;
}

inline int check_geometry(int type, int n_kv, int head_dim, int page_size, int64_t n_pages) {
    int rc = check_type(type);
    if (rc) return rc;
    if (n_kv <= 0 || head_dim <= 0 || page_size <= 0 || page_size % 16 || n_pages <= 0) return QMM_ERR_SHAPE;
    if (head_dim != 64 && head_dim != 96 && head_dim != 128 && head_dim != 192 && head_dim != 256)
        return QMM_ERR_UNSUPPORTED;
    if (n_kv > kMaxHeads || page_size > kMaxLength) return QMM_ERR_SHAPE;
    const int64_t page = (int64_t)n_kv * page_size * kv_row_bytes(type, head_dim);
    return n_pages > INT64_MAX / 8 / page ? QMM_ERR_SHAPE : QMM_OK;
}

inline int check_cache(const qmm_kv_cache* c) {
    if (!c) return QMM_ERR_NULL;
    int rc;
    if ((rc = check_geometry(c->type, c->n_kv, c->head_dim, c->page_size, c->n_pages))) return rc;
    if ((rc = check_ptr(c->k)) || (rc = check_ptr(c->v))) return rc;
    return QMM_OK;
}

inline int check_batch_sizes(const qmm_kv_cache* c, const qmm_kv_batch* b) {
    if (!b) return QMM_ERR_NULL;
    if (b->n_seqs <= 0 || b->table_width <= 0 || b->n_tokens <= 0 || b->max_kv < 0) return QMM_ERR_SHAPE;
    if (b->n_tokens > kMaxRows || b->n_seqs > kMaxSeqs) return QMM_ERR_SHAPE;
    if ((int64_t)b->table_width * c->page_size > kMaxLength) return QMM_ERR_SHAPE;
    return QMM_OK;
}

inline int check_batch(const qmm_kv_cache* c, const qmm_kv_batch* b) {
    int rc;
    if ((rc = check_batch_sizes(c, b))) return rc;
    if ((rc = check_ptr(b->q_start, 4)) || (rc = check_ptr(b->kv_len, 4)) || (rc = check_ptr(b->table, 4))) return rc;
    return QMM_OK;
}

inline int check_tree(const qmm_kv_tree* t) {
    if (!t) return QMM_ERR_NULL;
    if (t->words < 1 || t->words > kMaxWords) return QMM_ERR_SHAPE;
    int rc;
    if ((rc = check_ptr(t->seen)) || (rc = check_ptr(t->depth, 4))) return rc;
    return QMM_OK;
}

inline int check_rows(const void* p, int64_t ld, int64_t n, int64_t heads, int head_dim) {
    int rc;
    if ((rc = check_ptr(p))) return rc;
    if (ld < heads * head_dim || ld % 8 || ld > INT64_MAX / 8 / n) return QMM_ERR_SHAPE;
    return QMM_OK;
}

inline KvArgs kv_args(const qmm_kv_cache* c, const qmm_kv_batch* b) {
    KvArgs a = {};
    a.k = static_cast<uint8_t*>(c->k);
    a.v = static_cast<uint8_t*>(c->v);
    a.q_start = b->q_start;
    a.kv_len = b->kv_len;
    a.table = b->table;
    a.n_pages = c->n_pages;
    a.n_tokens = b->n_tokens;
    a.n_seqs = b->n_seqs;
    a.table_width = b->table_width;
    a.page_size = c->page_size;
    a.n_kv = c->n_kv;
    return a;
}

inline int64_t up_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

}  // namespace
}  // namespace qmm
