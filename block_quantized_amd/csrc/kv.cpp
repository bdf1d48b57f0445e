// kv.cpp — the C ABI of the key-value cache (qmm_kv.h): argument validation,
// the choice of kernels and splits, then dispatch.  As in qmm.cpp every check
// runs before anything is enqueued, and nothing allocates, copies or
// synchronizes.
#include <limits.h>
#include <math.h>
#include <stdint.h>

#include "kv_internal.h"

using namespace qmm;

namespace {

constexpr int64_t kMaxRows = (int64_t(1) << 23) - 1;  // tokens: grids stay below 2^32 work-items
constexpr int64_t kMaxLength = int64_t(1) << 30;   // tokens of a sequence
constexpr int kMaxSeqs = 1 << 16;                  // every workgroup looks its sequence up among them
constexpr int kMaxHeads = 4096;

int hip_status(hipError_t e) { return e == hipSuccess ? QMM_OK : QMM_ERR_HIP; }

int check_ptr(const void* p, unsigned align = 16) {
    if (!p) return QMM_ERR_NULL;
    return reinterpret_cast<uintptr_t>(p) & (align - 1) ? QMM_ERR_ALIGN : QMM_OK;
}

int check_type(int t) {
    if (t == QMM_Q8_0 || t == QMM_F16 || t == QMM_BF16) return QMM_OK;
    return qmm_block_size(t) || t == QMM_F32 ? QMM_ERR_UNSUPPORTED : QMM_ERR_TYPE;
}

int check_xtype(int t) {
    if (t == QMM_F32 || t == QMM_BF16) return QMM_OK;
    return qmm_block_size(t) || t == QMM_F16 ? QMM_ERR_UNSUPPORTED : QMM_ERR_TYPE;
}

int check_geometry(int type, int n_kv, int head_dim, int page_size, int64_t n_pages) {
    int rc = check_type(type);
    if (rc) return rc;
    if (n_kv <= 0 || head_dim <= 0 || page_size <= 0 || page_size % 16 || n_pages <= 0) return QMM_ERR_SHAPE;
    if (head_dim != 64 && head_dim != 96 && head_dim != 128 && head_dim != 192 && head_dim != 256)
        return QMM_ERR_UNSUPPORTED;
    if (n_kv > kMaxHeads || page_size > kMaxLength) return QMM_ERR_SHAPE;
    const int64_t page = (int64_t)n_kv * page_size * kv_row_bytes(type, head_dim);
    return n_pages > INT64_MAX / 8 / page ? QMM_ERR_SHAPE : QMM_OK;
}

int check_cache(const qmm_kv_cache* c) {
    if (!c) return QMM_ERR_NULL;
    int rc;
    if ((rc = check_geometry(c->type, c->n_kv, c->head_dim, c->page_size, c->n_pages))) return rc;
    if ((rc = check_ptr(c->k)) || (rc = check_ptr(c->v))) return rc;
    return QMM_OK;
}

int check_batch_sizes(const qmm_kv_cache* c, const qmm_kv_batch* b) {
    if (!b) return QMM_ERR_NULL;
    if (b->n_seqs <= 0 || b->table_width <= 0 || b->n_tokens <= 0 || b->max_kv < 0) return QMM_ERR_SHAPE;
    if (b->n_tokens > kMaxRows || b->n_seqs > kMaxSeqs) return QMM_ERR_SHAPE;
    if ((int64_t)b->table_width * c->page_size > kMaxLength) return QMM_ERR_SHAPE;
    return QMM_OK;
}

int check_batch(const qmm_kv_cache* c, const qmm_kv_batch* b) {
    int rc;
    if ((rc = check_batch_sizes(c, b))) return rc;
    if ((rc = check_ptr(b->q_start, 4)) || (rc = check_ptr(b->kv_len, 4)) || (rc = check_ptr(b->table, 4))) return rc;
    return QMM_OK;
}

int check_rows(const void* p, int64_t ld, int64_t n, int64_t heads, int head_dim) {
    int rc;
    if ((rc = check_ptr(p))) return rc;
    if (ld < heads * head_dim || ld % 8 || ld > INT64_MAX / 8 / n) return QMM_ERR_SHAPE;
    return QMM_OK;
}

KvArgs kv_args(const qmm_kv_cache* c, const qmm_kv_batch* b) {
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

int64_t up_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// How qmm_attn divides its work.
struct Plan {
    int algo, chunk, chunks, shift, splits, least, slots;
    int64_t items, parts;
};

// An upper bound of the keys that a row tile sees, as far as the host knows.
int64_t key_bound(const qmm_kv_cache* c, const qmm_kv_batch* b) {
    const int64_t room = (int64_t)b->table_width * c->page_size;
    return b->max_kv > 0 && b->max_kv < room ? b->max_kv : room;
}

// Tokens (log2) of a row tile of `rows` rows for `chunk` query heads: what
// fits, but no more than a sequence has.
int tile_tokens(int rows, int chunk, int64_t each) {
    int shift = 0;
    while ((2 << shift) * chunk <= rows && (1 << shift) < each) ++shift;
    return shift;
}

// Split kernels spread 16 rows' products with 32 keys over the whole chip and
// join them; tile kernels take 128 rows through tiles of 64 keys, one after
// another.  So the former's time is some 12 us (27 for heads above 128, whose
// waves' parts fill LDS; 6 less where nothing is joined) and 1 us for 1000 such
// products of 64 values, the latter's some 9 us and 3 us a step, as many steps as
// a row tile sees tiles of keys, times the rounds of 512 workgroups; or, their
// keys split (128 row tiles at most), 22 us and 9.5 for each 512 steps.  (That is an
// estimate of both: two parts for heavy steps and the types' different steps are
// not in it.)  Split against tile kernels, us: 1588 tokens, 14 heads on 2 of 64,
// fp32 over bf16: 42, 53; 3 x 1078 of the same, bf16 over Q8_0: 68, 80; 2 x 892, 32
// on 8 of 128, bf16 over Q8_0: 86, 68; 397 behind 237, 32 heads of 128 each its own,
// fp32 over fp16: 32, 40; 314, 16 on 8 of 256, the same: 35, 28; 462, 14 on 2 of 64,
// Q8_0: 19, 24; with a window of 97, 3 x 1116, bf16 over Q8_0: 33, 22; and wrong: 2 x
// 654, 32 on 8 of 64, bf16: 32 (taken), 25; 124, 16 on 8 of 256, bf16 over Q8_0: 13,
// 22 (taken).  Over 160 sizes drawn at random the choice costs 1.7% (geometric mean)
// against the better one of each.  Below 48 rows a sequence most of a tile is idle.
int choose(const qmm_kv_cache* c, const qmm_kv_batch* b, const qmm_attn_opts* o, int n_q) {
    const int G = n_q / c->n_kv;
    const int64_t each = up_div(b->n_tokens, b->n_seqs), rows = up_div(b->n_tokens * G, b->n_seqs);
    if (rows < 48) return 1;
    const int chunk = G < kTileRows ? G : kTileRows, shift = tile_tokens(kTileRows, chunk, each);
    const double keys = (double)key_bound(c, b), seen = o->window > 0 && !o->prefix ? o->window : keys;
    const double mean = fmin(fmax(keys - 0.5 * each, 1.0), seen);  // of a row
    const double most = fmin(keys, seen + (1 << shift));           // of a row tile
    const double split = (c->head_dim > 128 ? 27.0 : 12.0) - (fmin(keys, seen + each) > 128 ? 0.0 : 6.0) +
                         1e-3 * b->n_seqs * up_div(rows, 16) * c->n_kv * (mean / 32) * (c->head_dim / 64.0);
    const double groups = (double)(up_div(each, int64_t(1) << shift) * b->n_seqs) * c->n_kv * up_div(G, chunk);
    const double steps = fmax(most / 64, 1.0);
    const double tile = groups <= 128 && most > 128 ? 22.0 + 9.5 * steps * groups / 512
                                                    : 9.0 + 3.0 * steps * fmax(groups / 512, 1.0);
    return tile < split ? 2 : 1;
}

Plan plan(const qmm_kv_cache* c, const qmm_kv_batch* b, const qmm_attn_opts* o, int xtype, int n_q) {
    Plan p = {};
    const int G = n_q / c->n_kv;
    p.algo = o->algo ? o->algo : choose(c, b, o, n_q);
    const int rows = p.algo == 2 ? kTileRows : kSplitRows;
    p.chunk = G < rows ? G : rows;
    p.chunks = (int)up_div(G, p.chunk);
    p.shift = tile_tokens(rows, p.chunk, up_div(b->n_tokens, b->n_seqs));
    int64_t tiles = (b->n_tokens >> p.shift) + b->n_seqs;  // row tiles at most
    if (tiles > b->n_tokens) tiles = b->n_tokens;
    int64_t keys = key_bound(c, b);
    if (o->window > 0 && !o->prefix && o->window + b->n_tokens < keys) keys = o->window + b->n_tokens;
    // The keys are divided among up to 2048 workgroups, more than run at once, so
    // that the last of them end together (64 conversations of 8k to 16k keys: 397 us
    // with 512 workgroups, 362 with 1024, 338 with 2048, 340 with 2560); where that
    // leaves each below 2048 keys, among fewer, at least 512, two a CU (one of
    // 131k keys, 8 heads: 76 us with 512, 88 with 2048), or as many as run at once
    // (three a CU, two for heads above 128) less one a row tile, which may add a part
    // that is not full, where these are 256 to 512 (us without, with, 32 heads of 128
    // each its own over bf16, 1400 keys: 14 sequences 64, 57; 16: 68, 63; 24 of 3000, 16
    // on 8 of 256: 150, 127; but 12: 51, 55).  Below 256 the gain is small either way (18
    // of 1400: 79, 72; 72 of 8 heads: 50, 55).  A part keeps 128 keys, a tile a wave (one
    // sequence of 1940: 14 us; with 256 keys 16, with 512 22).
    // Tile kernels split only what makes four parts and more of a row tile: fewer
    // cost in writing and joining what they save (us with two, without: 309 tokens
    // twice, 32 heads, 30 and 18; 602 tokens, a window of 17: 35 and 21).  Where a
    // step is long, that is for wide heads over Q8_0 rows and with fp32 queries over
    // bf16 rows, two parts pay (16 heads on 8 of 256, us without, with: Q8_0, fp32: 1024
    // tokens 117, 86; 1500: 161, 133; 2048: 222, 165; 3000: 319, 325; bf16 rows, fp32: 96,
    // 85; 130, 125; 179, 153; 258, 297; but fp32 over fp16 rows 62, 62; 83, 85; 112, 106;
    // 166, 192).
    p.least = 4;
    const bool heavy = c->head_dim > 128 && (c->type == QMM_Q8_0 || (c->type == QMM_BF16 && xtype == QMM_F32));
    const int64_t heads = (int64_t)c->n_kv * p.chunks, most = tiles * up_div(keys, 32 * p.least);
    int64_t s = tiles * heads * up_div(keys, 64) / 32;  // (below 2^60)
    const int64_t slots = c->head_dim > 128 ? 512 : 768, rest = slots - tiles * heads;
    const int64_t low = p.algo == 2 || rest < 256 || rest > 512 ? 512 : rest;
    s = up_div(s < low || p.algo == 2 ? low : s > 2048 ? 2048 : s, heads);
    if (s > most) s = most;
    p.splits = keys > 32 * p.least && (p.algo == 1 || s >= 4 * tiles || (heavy && s > tiles)) ? (int)s : 0;
    p.items = tiles + p.splits;
    p.slots = p.chunk << p.shift;
    p.parts = p.splits ? p.items * heads * p.slots : 0;
    return p;
}

// Whether the grids of qmm_attn stay below 2^32 work-items.
bool fits(const qmm_kv_cache* c, const qmm_kv_batch* b, int n_q, const Plan& p) {
    return p.items * c->n_kv * p.chunks < int64_t(1) << (p.algo == 2 ? 23 : 24) &&
           (!p.splits || b->n_tokens * n_q < int64_t(1) << 30);
}

int check_opts(const qmm_attn_opts* o) {
    if (!o) return QMM_ERR_NULL;
    if (!isfinite(o->scale) || !isfinite(o->softcap) || o->softcap < 0 || o->window < 0) return QMM_ERR_UNSUPPORTED;
    if (o->algo < 0 || o->algo > 2) return QMM_ERR_UNSUPPORTED;
    if ((reinterpret_cast<uintptr_t>(o->slopes) | reinterpret_cast<uintptr_t>(o->prefix)) & 3) return QMM_ERR_ALIGN;
    return QMM_OK;
}

int check_attn_sizes(const qmm_kv_cache* c, const qmm_kv_batch* b, int xtype, int n_q) {
    if (!c) return QMM_ERR_NULL;
    int rc;
    if ((rc = check_xtype(xtype))) return rc;
    if ((rc = check_geometry(c->type, c->n_kv, c->head_dim, c->page_size, c->n_pages))) return rc;
    if ((rc = check_batch_sizes(c, b))) return rc;
    if (n_q <= 0 || n_q > kMaxHeads || n_q % c->n_kv) return QMM_ERR_SHAPE;
    return QMM_OK;
}

size_t work_bytes_of(const qmm_kv_cache* c, const qmm_kv_batch* b, int n_q, const Plan& p) {
    if (!p.splits) return 0;
    return up_div(p.parts * (c->head_dim + 2) * 4, 16) * 16 + (size_t)b->n_tokens * n_q * 16;
}

}  // namespace

extern "C" {

size_t qmm_kv_bytes(int type, int n_kv, int head_dim, int page_size, int64_t n_pages) {
    if (check_geometry(type, n_kv, head_dim, page_size, n_pages)) return 0;
    return (size_t)n_pages * n_kv * page_size * kv_row_bytes(type, head_dim);
}

int qmm_rope_freqs(double* freqs, int n_rot, double base, double scale, const float* factors, void* stream) {
    int rc;
    if ((rc = check_ptr(freqs, 8))) return rc;
    if (reinterpret_cast<uintptr_t>(factors) & 3) return QMM_ERR_ALIGN;
    if (n_rot <= 0 || n_rot % 2 || n_rot > 65536) return QMM_ERR_SHAPE;
    if (!isfinite(base) || base <= 0 || !isfinite(scale) || scale <= 0) return QMM_ERR_UNSUPPORTED;
    return hip_status(launch_rope_freqs(freqs, n_rot, base, scale, factors, static_cast<hipStream_t>(stream)));
}

int qmm_kv_append(const qmm_kv_cache* cache, const qmm_kv_batch* batch, const qmm_rope* rope, int xtype, const void* k,
                  int64_t ldk, const void* v, int64_t ldv, const void* q, int64_t ldq, int n_q, void* q_out,
                  void* stream) {
    int rc;
    if ((rc = check_xtype(xtype)) || (rc = check_cache(cache)) || (rc = check_batch(cache, batch))) return rc;
    const int D = cache->head_dim;
    if ((rc = check_rows(k, ldk, batch->n_tokens, cache->n_kv, D))) return rc;
    if ((rc = check_rows(v, ldv, batch->n_tokens, cache->n_kv, D))) return rc;
    AppendArgs a = {};
    a.c = kv_args(cache, batch);
    if (q || q_out) {
        if (n_q <= 0 || n_q > kMaxHeads) return QMM_ERR_SHAPE;
        if ((rc = check_rows(q, ldq, batch->n_tokens, n_q, D)) || (rc = check_ptr(q_out))) return rc;
        if (q == q_out && ldq != (int64_t)n_q * D) return QMM_ERR_SHAPE;
        a.xq = q;
        a.q_out = q_out;
        a.ldq = ldq;
        a.n_q = n_q;
    } else if (n_q) {
        return QMM_ERR_NULL;
    }
    a.xk = k;
    a.xv = v;
    a.ldk = ldk;
    a.ldv = ldv;
    if (rope) {
        if ((rc = check_ptr(rope->freqs, 8))) return rc;
        if (reinterpret_cast<uintptr_t>(rope->pos) & 3) return QMM_ERR_ALIGN;
        if (rope->n_rot <= 0 || rope->n_rot % 2 || rope->n_rot > D) return QMM_ERR_SHAPE;
        if (rope->pairing != QMM_ROPE_PAIRS && rope->pairing != QMM_ROPE_HALVES) return QMM_ERR_UNSUPPORTED;
        if (rope->n_axes < 1 || rope->n_axes > 4) return QMM_ERR_SHAPE;
        a.freqs = rope->freqs;
        a.pos = rope->pos;
        a.n_rot = rope->n_rot;
        a.pairing = rope->pairing;
        int at = 0;
        for (int i = 0; i < 3; ++i) a.bounds[i] = INT_MAX;
        if (rope->n_axes > 1) {
            for (int i = 0; i < rope->n_axes; ++i) {
                if (rope->sections[i] < 0 || rope->sections[i] > D) return QMM_ERR_SHAPE;
                at += rope->sections[i];
                if (i + 1 < rope->n_axes) a.bounds[i] = at;
            }
            if (at != rope->n_rot / 2) return QMM_ERR_SHAPE;
        }
    }
    return hip_status(launch_kv_append(cache->type, D, xtype, a, static_cast<hipStream_t>(stream)));
}

int qmm_attn_choice(const qmm_kv_cache* cache, const qmm_kv_batch* batch, int xtype, int n_q) {
    if (check_attn_sizes(cache, batch, xtype, n_q)) return 0;
    const qmm_attn_opts none = {};
    const Plan p = plan(cache, batch, &none, xtype, n_q);
    return fits(cache, batch, n_q, p) ? p.algo : 0;
}

size_t qmm_attn_work(const qmm_kv_cache* cache, const qmm_kv_batch* batch, const qmm_attn_opts* opts, int xtype,
                     int n_q) {
    if (check_attn_sizes(cache, batch, xtype, n_q) || check_opts(opts)) return 0;
    const Plan p = plan(cache, batch, opts, xtype, n_q);
    return fits(cache, batch, n_q, p) ? work_bytes_of(cache, batch, n_q, p) : 0;
}

int qmm_attn(const qmm_kv_cache* cache, const qmm_kv_batch* batch, const qmm_attn_opts* opts, int xtype, const void* q,
             int64_t ldq, int n_q, void* out, void* work, size_t work_bytes, void* stream) {
    int rc;
    if ((rc = check_xtype(xtype)) || (rc = check_cache(cache)) || (rc = check_batch(cache, batch))) return rc;
    if ((rc = check_attn_sizes(cache, batch, xtype, n_q)) || (rc = check_opts(opts))) return rc;
    if ((rc = check_rows(q, ldq, batch->n_tokens, n_q, cache->head_dim)) || (rc = check_ptr(out))) return rc;
    const Plan p = plan(cache, batch, opts, xtype, n_q);
    if (!fits(cache, batch, n_q, p)) return QMM_ERR_SHAPE;
    const size_t need = work_bytes_of(cache, batch, n_q, p);
    if (need) {
        if ((rc = check_ptr(work))) return rc;
        if (work_bytes < need) return QMM_ERR_SHAPE;
    }
    AttnArgs a = {};
    a.c = kv_args(cache, batch);
    a.q = q;
    a.out = out;
    a.work = static_cast<float*>(work);
    a.slopes = opts->slopes;
    a.prefix = opts->prefix;
    a.ldq = ldq;
    a.scale = opts->scale;
    a.softcap = opts->softcap;
    a.n_q = n_q;
    a.window = opts->window;
    a.head_dim = cache->head_dim;
    a.splits = p.splits;
    a.least = p.least;
    a.items = p.items;
    a.slots = p.slots;
    a.parts = p.parts;
    a.tile_shift = p.shift;
    a.chunk = p.chunk;
    a.chunks = p.chunks;
    return hip_status(launch_attn(p.algo, cache->type, cache->head_dim, xtype, a, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
