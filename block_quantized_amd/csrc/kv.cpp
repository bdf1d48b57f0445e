// kv.cpp — the C ABI of the key-value cache (qmm_kv.h): argument validation,
// the choice of kernels and splits, then dispatch.  As in qmm.cpp every check
// runs before anything is enqueued, and nothing allocates, copies or
// synchronizes.
#include <limits.h>
#include <math.h>
#include <stdint.h>

#include "kv_checks.h"

using namespace qmm;

namespace {

// How qmm_attn divides its work.
struct Plan {
    int algo, chunk, chunks, shift, splits, least, slots, rows;
    bool fit;  // the splits are as many items as run at once
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

// Parts that the split kernels divide the keys of a head's row tiles in.
int64_t split_parts(const qmm_kv_cache* c, int64_t tiles, int64_t heads, int64_t keys) {
    const int64_t s = tiles * heads * up_div(keys, 64) / 32;  // (below 2^60)
    const int64_t slots = c->head_dim > 128 ? 512 : 768, rest = slots - tiles * heads;
    const int64_t low = rest < 256 || rest > 512 ? 512 : rest;
    return up_div(s < low ? low : s > 2048 ? 2048 : s, heads);
}

// Row tiles of `rows` rows, over all heads, as far as the host knows.
int64_t row_tiles(const qmm_kv_batch* b, int n_kv, int G, int rows) {
    const int chunk = G < rows ? G : rows;
    const int64_t each = up_div(b->n_tokens, b->n_seqs);
    return up_div(each, int64_t(1) << tile_tokens(rows, chunk, each)) * b->n_seqs * n_kv * up_div(G, chunk);
}

// Trees of new tokens have some rows a sequence, over long caches: 2 to 100 tokens of 1 to
// 32 heads a key-value head.  Split kernels take 16 of them, the kernels of Q8_0 rows 32,
// the tile kernels 32 or 64 (heads above 128, which stage 8 keys a wave: 64).  In units of
// 1000 products of a row tile with 32 keys of 64 values, their times over 180 drawn sizes
// are some 12 us (17 for wide heads) and 0.9 us a unit, 3 us more and 0.9 a unit (of half
// as many), 1 us more and 1.7 a unit (heads of 64) or 0.6 (wider ones).  The choice by
// these costs 0.4% (Q8_0) and 3% (geometric mean) against the better one of each of 126
// other sizes.  us, split against the others: 8 drafts over 8000 keys, 32 sequences, 32
// heads on 8 of 128, Q8_0 180, 155; the same bf16 over bf16 221, 160; 13 drafts over
// 130911 keys in fp16 193, 113; 26 over 3100, 12 sequences, 16 heads on 8 of 256, bf16
// 164, 59; 12 over 2000 of 14 heads on 2 of 64, Q8_0 16.1, 17.5; 62 over 61, fp32 over
// fp16, 10.6, 15.4. Heads of 96, 192 and 256 over Q8_0 stay with the split kernels (256,
// above 4000 keys: half of the tile kernels' time), which is why those have no form for
// Q8_0 here.
Plan plan_tree(const qmm_kv_cache* c, const qmm_kv_batch* b, const qmm_attn_opts* o, int xtype, int n_q) {
    Plan p = {};
    const int G = n_q / c->n_kv;
    const bool q8 = c->type == QMM_Q8_0, only_split = q8 && c->head_dim != 64 && c->head_dim != 128;
    const int64_t each = up_div(b->n_tokens, b->n_seqs);
    const int rows = q8 || (c->head_dim <= 128 && each * G <= 32) ? 32 : 64;
    int64_t keys = key_bound(c, b);
    if (o->window > 0 && !o->prefix && o->window + each < keys) keys = o->window + each;
    const double unit = 1e-3 * (double)keys / 32 * (c->head_dim / 64.0);
    const double split = 0.9 * unit * (double)row_tiles(b, c->n_kv, G, kSplitRows);
    const double other = (q8 ? 3.0 : 1.0) + (q8 ? 0.9 : c->head_dim > 64 ? 0.6 : 1.7) * unit * (double)row_tiles(b, c->n_kv, G, rows);
    p.algo = only_split ? 1 : o->algo ? o->algo : other < split ? 2 : 1;
    p.rows = p.algo == 1 ? kSplitRows : rows;
    p.chunk = G < p.rows ? G : p.rows;
    p.chunks = (int)up_div(G, p.chunk);
    p.shift = tile_tokens(p.rows, p.chunk, each);
    int64_t tiles = (b->n_tokens >> p.shift) + b->n_seqs;  // row tiles of a head at most
    if (tiles > b->n_tokens) tiles = b->n_tokens;
    const int64_t heads = (int64_t)c->n_kv * p.chunks;
    p.least = 4;
    const int64_t most = tiles * up_div(keys, 32 * p.least);
    int64_t s;
    if (p.algo == 1) {
        s = split_parts(c, tiles, heads, keys);
    } else {
        // As many workgroups as run at once (two a CU, one of eight waves), which the kernels fit the parts into (those of
        // more than 64 sequences by their mean: a row tile's parts are some half more than the whole ones).  Twice as many would end more evenly but begin and
        // are joined as often again (Q8_0, 8 heads of 128, us with 512, 1024: 32 sequences of 6275 to 12287 keys, two row
        // tiles each, 333, 345; 8 of 11459 to 20000, one each, 89, 95; 6 of 5157 to 9000, three each, 85, 89).  By
        // the mean and an upper bound of row tiles, as the split kernels, half of the places stay empty where each sequence
        // has one (16 drafts, fp32 over bf16, 16 sequences of 8000: 182 us, 142 so).  Up to 512 keys the join would cost
        // more than it saves.
        const bool eight = p.rows == 64 && (c->head_dim > 128 || (c->type == QMM_BF16 && xtype == QMM_F32));
        const int64_t run = eight ? 256 : 512;
        const int64_t mean = up_div(each, int64_t(1) << p.shift) * b->n_seqs;  // row tiles if sequences are alike
        s = run / heads;
        if (keys <= 512) {
            s = 0;
        } else if (s > mean) {
            p.fit = b->n_seqs <= 64;
            s = p.fit ? s : s - mean / 2;
        } else {
            // Row tiles fill the places, but one sequence may be far longer than the others: parts of twice the even share
            // cut nothing else (us without, with: 64 sequences of 8 drafts, one of 131072 keys, 63 of 1024, 32 heads on 8 of
            // 128, Q8_0 2336, 170; bf16 over fp16 2364, 177).  All rows pay for the join that may follow (32 of 16 drafts, up
            // to 12287 keys: 344, 349), so not below 4096 keys of 128 values, which one workgroup walks in 75 to 120 us; and
            // every row has room in the workspace, so not from 16 times the places on, where the others' rows take
            // long, too (32 x 512 workgroups of 64 rows of 128 values: 545 MB at most).
            s = keys * c->head_dim >= 4096 * 128 && s >= 4 && mean <= 16 * s ? s / 2 : 0;
        }
    }
    if (s > most) s = most;
    p.splits = keys > 32 * p.least ? (int)s : 0;
    p.items = tiles + p.splits;
    p.slots = p.chunk << p.shift;
    p.parts = p.splits ? p.items * heads * p.slots : 0;
    return p;
}

Plan plan(const qmm_kv_cache* c, const qmm_kv_batch* b, const qmm_attn_opts* o, int xtype, int n_q, bool tree) {
    if (tree) return plan_tree(c, b, o, xtype, n_q);
    Plan p = {};
    const int G = n_q / c->n_kv;
    p.algo = o->algo ? o->algo : choose(c, b, o, n_q);
    const int rows = p.rows = p.algo == 2 ? kTileRows : kSplitRows;
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
    int64_t s = p.algo == 2 ? up_div(512, heads) : split_parts(c, tiles, heads, keys);
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

int attend(const qmm_kv_cache* cache, const qmm_kv_batch* batch, const qmm_kv_tree* tree, const qmm_attn_opts* opts,
           int xtype, const void* q, int64_t ldq, int n_q, void* out, void* work, size_t work_bytes, void* stream) {
    int rc;
    if ((rc = check_xtype(xtype)) || (rc = check_cache(cache)) || (rc = check_batch(cache, batch))) return rc;
    if ((rc = check_attn_sizes(cache, batch, xtype, n_q)) || (rc = check_opts(opts))) return rc;
    if ((rc = check_rows(q, ldq, batch->n_tokens, n_q, cache->head_dim)) || (rc = check_ptr(out))) return rc;
    const Plan p = plan(cache, batch, opts, xtype, n_q, tree != nullptr);
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
    if (tree) {
        a.tree = tree->seen;
        a.depth = tree->depth;
        a.words = tree->words;
        a.tile_rows = p.rows;
        a.fit = p.fit;
    }
    return hip_status(launch_attn(p.algo, cache->type, cache->head_dim, xtype, a, static_cast<hipStream_t>(stream)));
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
    const Plan p = plan(cache, batch, &none, xtype, n_q, false);
    return fits(cache, batch, n_q, p) ? p.algo : 0;
}

size_t qmm_attn_work(const qmm_kv_cache* cache, const qmm_kv_batch* batch, const qmm_attn_opts* opts, int xtype,
                     int n_q) {
    if (check_attn_sizes(cache, batch, xtype, n_q) || check_opts(opts)) return 0;
    const Plan p = plan(cache, batch, opts, xtype, n_q, false);
    return fits(cache, batch, n_q, p) ? work_bytes_of(cache, batch, n_q, p) : 0;
}

size_t qmm_attn_tree_work(const qmm_kv_cache* cache, const qmm_kv_batch* batch, const qmm_attn_opts* opts, int xtype,
                          int n_q) {
    if (check_attn_sizes(cache, batch, xtype, n_q) || check_opts(opts)) return 0;
    const Plan p = plan(cache, batch, opts, xtype, n_q, true);
    return fits(cache, batch, n_q, p) ? work_bytes_of(cache, batch, n_q, p) : 0;
}

int qmm_attn(const qmm_kv_cache* cache, const qmm_kv_batch* batch, const qmm_attn_opts* opts, int xtype, const void* q,
             int64_t ldq, int n_q, void* out, void* work, size_t work_bytes, void* stream) {
    return attend(cache, batch, nullptr, opts, xtype, q, ldq, n_q, out, work, work_bytes, stream);
}

int qmm_attn_tree(const qmm_kv_cache* cache, const qmm_kv_batch* batch, const qmm_kv_tree* tree, const qmm_attn_opts* opts,
                  int xtype, const void* q, int64_t ldq, int n_q, void* out, void* work, size_t work_bytes, void* stream) {
    const int rc = check_tree(tree);
    return rc ? rc : attend(cache, batch, tree, opts, xtype, q, ldq, n_q, out, work, work_bytes, stream);
}

}  // extern "C"
