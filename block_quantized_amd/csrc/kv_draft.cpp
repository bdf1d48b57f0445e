// kv_draft.cpp — the C ABI of what checks drafted tokens beside attention
// (qmm_kv.h): trees of new tokens, and copying and compacting the rows of all
// layers.  Checks come first, as in kv.cpp.
#include "kv_checks.h"

using namespace qmm;

namespace {

// The layers' geometry is the first one's; their pools go into `l`, `count` at a time.
int check_layers(const qmm_kv_cache* caches, int count) {
    if (!caches) return QMM_ERR_NULL;
    if (count <= 0 || count > 4096) return QMM_ERR_SHAPE;
    const qmm_kv_cache& f = caches[0];
    for (int i = 0; i < count; ++i) {
        const qmm_kv_cache& c = caches[i];
        if (int rc = check_cache(&c)) return rc;
        if (c.type != f.type || c.n_kv != f.n_kv || c.head_dim != f.head_dim || c.page_size != f.page_size ||
            c.n_pages != f.n_pages)
            return QMM_ERR_SHAPE;
    }
    return QMM_OK;
}

// Whether n of the values at a lie among m at b.
bool meet(const int32_t* a, int64_t n, const int32_t* b, int64_t m) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return x < y + 4 * m && y < x + 4 * n;
}

template <typename F>
int each_layers(const qmm_kv_cache* caches, int count, F launch) {
    for (int at = 0; at < count; at += kMaxLayers) {
        const int n = count - at < kMaxLayers ? count - at : kMaxLayers;
        LayerArgs l = {};
        for (int i = 0; i < n; ++i) {
            l.pool[2 * i] = static_cast<uint8_t*>(caches[at + i].k);
            l.pool[2 * i + 1] = static_cast<uint8_t*>(caches[at + i].v);
        }
        if (int rc = hip_status(launch(at, n, l))) return rc;
    }
    return QMM_OK;
}

}  // namespace

extern "C" {

int qmm_kv_tree_build(const qmm_kv_batch* batch, const int32_t* parents, const qmm_kv_tree* tree, int32_t* pos,
                      void* stream) {
    if (!batch) return QMM_ERR_NULL;
    if (batch->n_seqs <= 0 || batch->n_seqs > kMaxSeqs || batch->n_tokens <= 0 || batch->n_tokens > kMaxRows)
        return QMM_ERR_SHAPE;
    int rc;
    if ((rc = check_ptr(batch->q_start, 4)) || (rc = check_ptr(batch->kv_len, 4)) || (rc = check_ptr(parents, 4)))
        return rc;
    if ((rc = check_tree(tree))) return rc;
    if (reinterpret_cast<uintptr_t>(pos) & 3) return QMM_ERR_ALIGN;
    TreeArgs a = {};
    a.q_start = batch->q_start;
    a.kv_len = batch->kv_len;
    a.parents = parents;
    a.seen = tree->seen;
    a.depth = tree->depth;
    a.pos = pos;
    a.n_tokens = batch->n_tokens;
    a.n_seqs = batch->n_seqs;
    a.words = tree->words;
    return hip_status(launch_kv_tree(a, static_cast<hipStream_t>(stream)));
}

int qmm_kv_copy(const qmm_kv_cache* caches, int count, const int32_t* src, const int32_t* dst, const int32_t* rows,
                int64_t n, void* stream) {
    int rc;
    if ((rc = check_layers(caches, count))) return rc;
    if (n <= 0 || n >= int64_t(1) << 31) return QMM_ERR_SHAPE;
    if ((rc = check_ptr(src, 4)) || (rc = check_ptr(dst, 4))) return rc;
    if (reinterpret_cast<uintptr_t>(rows) & 3) return QMM_ERR_ALIGN;
    const qmm_kv_cache& c = caches[0];
    CopyArgs a = {};
    a.src = src;
    a.dst = dst;
    a.rows = rows;
    a.n = n;
    a.n_pages = c.n_pages;
    a.n_kv = c.n_kv;
    a.page_size = c.page_size;
    a.row_bytes = kv_row_bytes(c.type, c.head_dim);
    a.page_bytes = (int64_t)c.n_kv * c.page_size * a.row_bytes;
    // (a workgroup takes 16 KiB of a page at most)
    if (n > (int64_t(1) << 23) / up_div(a.page_bytes, 1 << 14)) return QMM_ERR_SHAPE;
    return each_layers(caches, count, [&](int, int layers, const LayerArgs& l) {
        return launch_kv_copy(layers, l, a, static_cast<hipStream_t>(stream));
    });
}

int qmm_kv_compact(const qmm_kv_cache* caches, int count, const int32_t* table, int n_seqs, int table_width,
                   const int32_t* first, const int32_t* keep, const int32_t* n_keep, int width, int32_t* kv_len,
                   void* stream) {
    int rc;
    if ((rc = check_layers(caches, count))) return rc;
    const qmm_kv_cache& c = caches[0];
    if (n_seqs <= 0 || n_seqs > kMaxSeqs || table_width <= 0 || width < 0) return QMM_ERR_SHAPE;
    if ((int64_t)table_width * c.page_size > kMaxLength || width > kMaxLength) return QMM_ERR_SHAPE;
    if ((rc = check_ptr(table, 4)) || (rc = check_ptr(first, 4)) || (rc = check_ptr(n_keep, 4))) return rc;
    if (width && (rc = check_ptr(keep, 4))) return rc;
    if (reinterpret_cast<uintptr_t>(kv_len) & 3) return QMM_ERR_ALIGN;
    // (the inputs are read while it is written)
    if (kv_len && (meet(kv_len, n_seqs, first, n_seqs) || meet(kv_len, n_seqs, n_keep, n_seqs) ||
                   meet(kv_len, n_seqs, keep, width ? (int64_t)n_seqs * width : 0) ||
                   meet(kv_len, n_seqs, table, (int64_t)n_seqs * table_width)))
        return QMM_ERR_UNSUPPORTED;
    if ((int64_t)n_seqs * c.n_kv >= int64_t(1) << 23) return QMM_ERR_SHAPE;
    CompactArgs a = {};
    a.table = table;
    a.first = first;
    a.keep = keep;
    a.n_keep = n_keep;
    a.n_pages = c.n_pages;
    a.n_seqs = n_seqs;
    a.table_width = table_width;
    a.page_size = c.page_size;
    a.n_kv = c.n_kv;
    a.width = width;
    return each_layers(caches, count, [&](int at, int layers, const LayerArgs& l) {
        a.kv_len = at ? nullptr : kv_len;
        return launch_kv_compact(c.type, c.head_dim, layers, l, a, static_cast<hipStream_t>(stream));
    });
}

}  // extern "C"
