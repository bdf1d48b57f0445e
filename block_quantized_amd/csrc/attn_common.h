// attn_common.h — device helpers shared by the attention kernels.
#pragma once

#include "kv_internal.h"

namespace qmm {

typedef _Float16 half2v __attribute__((ext_vector_type(2)));
typedef _Float16 half8v __attribute__((ext_vector_type(8)));
typedef __bf16 bf2v __attribute__((ext_vector_type(2)));
typedef __bf16 bf8v __attribute__((ext_vector_type(8)));
typedef float f4v __attribute__((ext_vector_type(4)));
typedef float f16v __attribute__((ext_vector_type(16)));
typedef uint32_t u4v __attribute__((ext_vector_type(4)));

constexpr float kLog2e = 1.44269504088896340736f;

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __builtin_bit_cast(float, w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __builtin_bit_cast(float, w & 0xFFFF0000u); }

// A pair of fp32 values as 16-bit parts that sum to them: two fp16 parts hold
// 22 bits, three bf16 parts 24.  fp16 callers scale their values so that the
// low part is no subnormal that matters.  (The empty asm makes the packed
// part the one value that is both used and subtracted: the compiler otherwise
// rounds x a second time for the subtraction, fused with the product that made
// it, and a pair that ties differently leaves a whole step of the high part.)
template <bool BF, int PARTS>
__device__ __forceinline__ void split_pair(float x, float y, uint32_t (&part)[PARTS]) {
#pragma unroll
    for (int i = 0; i < PARTS; ++i) {
        if constexpr (BF) {
            bf2v h;
            h.x = (__bf16)x, h.y = (__bf16)y;
            part[i] = __builtin_bit_cast(uint32_t, h);
            asm("" : "+v"(part[i]));
            x -= bf16_lo(part[i]), y -= bf16_hi(part[i]);
        } else {
            half2v h;
            h.x = (_Float16)x, h.y = (_Float16)y;
            part[i] = __builtin_bit_cast(uint32_t, h);
            asm("" : "+v"(part[i]));
            h = __builtin_bit_cast(half2v, part[i]);
            x -= (float)h.x, y -= (float)h.y;
        }
    }
}

template <bool BF>
__device__ __forceinline__ f4v mfma16(u4v a, u4v b, f4v c) {
    if constexpr (BF)
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf8v, a), __builtin_bit_cast(bf8v, b), c, 0,
                                                       0, 0);
    else
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(half8v, a), __builtin_bit_cast(half8v, b), c,
                                                      0, 0, 0);
}

// Two int8 codes, bytes I and J of w, as bf16 (exactly: they have 7 bits).  (The
// empty asm hides how w was put together, else bytes are shifted out one by one.)
template <int I, int J>
__device__ __forceinline__ uint32_t codes_bf16(uint32_t w) {
    asm("" : "+v"(w));
    const float x = (float)(int8_t)(w >> (8 * I)), y = (float)(int8_t)(w >> (8 * J));
    return __builtin_amdgcn_perm(__builtin_bit_cast(uint32_t, y), __builtin_bit_cast(uint32_t, x), 0x07060302u);
}

// Two int8 codes, bytes `sel` of x ^ 0x80808080 (so code + 128), as fp16:
// 0x6400 | u is 1024 + u, and 1152 less is the code, exactly.
__device__ __forceinline__ uint32_t codes_f16(uint32_t biased, uint32_t sel) {
    half2v h = __builtin_bit_cast(half2v, __builtin_amdgcn_perm(0x64646464u, biased, sel));
    const half2v off = {(_Float16)1152.0f, (_Float16)1152.0f};
    return __builtin_bit_cast(uint32_t, h - off);
}

// Eight int8 codes as fp16.
__device__ __forceinline__ u4v codes8_f16(uint2 w) {
    const uint32_t lo = w.x ^ 0x80808080u, hi = w.y ^ 0x80808080u;
    return u4v{codes_f16(lo, 0x04010400u), codes_f16(lo, 0x04030402u), codes_f16(hi, 0x04010400u),
               codes_f16(hi, 0x04030402u)};
}

template <int CTRL>
__device__ __forceinline__ float dpp(float x) {
    return __builtin_bit_cast(float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, x), CTRL, 0xF, 0xF, false));
}

// The sum over a wavefront's lanes, all of them active: within each 16 by DPP.
__device__ __forceinline__ int sum_lanes(int x) {
    x += __builtin_amdgcn_mov_dpp(x, 0xB1, 0xF, 0xF, false);   // lane ^ 1
    x += __builtin_amdgcn_mov_dpp(x, 0x4E, 0xF, 0xF, false);   // lane ^ 2
    x += __builtin_amdgcn_mov_dpp(x, 0x141, 0xF, 0xF, false);  // 7 - lane, of each 8
    x += __builtin_amdgcn_mov_dpp(x, 0x140, 0xF, 0xF, false);  // 15 - lane, of each 16
    return __builtin_amdgcn_readlane(x, 0) + __builtin_amdgcn_readlane(x, 16) + __builtin_amdgcn_readlane(x, 32) +
           __builtin_amdgcn_readlane(x, 48);
}

// Two fp16 parts of d c / 128 for pairs of int8 codes c and scales d: the product
// rounded, and what that leaves off, which has no more bits than fp16 holds, so
// that the parts are exact above its smallest step.  `eights`: 0x4800 | c + 128 of
// each, which is 9 + c / 128.
__device__ __forceinline__ void scaled_codes(uint32_t eights, half2v d, uint32_t (&part)[2]) {
    const half2v nine = {(_Float16)9.0f, (_Float16)9.0f};
    const half2v c = __builtin_bit_cast(half2v, eights) - nine, hi = c * d;
    part[0] = __builtin_bit_cast(uint32_t, hi);
    part[1] = __builtin_bit_cast(uint32_t, __builtin_elementwise_fma(c, d, -hi));
}

// The running maximum of a row is raised when a score (times log2 e) passes it by
// this: weights reach 2^kSlack, which spares the cross-lane maximum and the
// rescaling for almost every tile.
constexpr float kSlack = 1.0f;
// Weights carry a factor of 2^p_top: fp16 parts then reach down to 2^-39 of the
// largest weight; bf16 parts have fp32's range.
template <bool BF>
__device__ __forceinline__ constexpr float p_top() { return BF ? 0.0f : 14.0f; }

// x = cap * tanh(f x / cap) * log2 e.  Where every |f x / cap| of the wavefront is below
// 0.35, as scores mostly are, x times the polynomial in x^2 that is closest to
// tanh(x) / x there: of degree 4, 9e-10 off relative to it; elsewhere
// 1 - 2 / (e^2x + 1), which loses bits to cancellation near 0, so that small
// values keep the polynomial.
template <int N>
__device__ __forceinline__ void cap_scores(float (&x)[N], float f, float cap) {
    const float in = fminf(f / cap, 0x1p127f), out = cap * kLog2e;  // finite: a score of 0 stays 0
    float big = 0.f;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        x[i] *= in;
        big = fmaxf(big, fabsf(x[i]));
    }
    const bool large = __any(big >= 0.35f);
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const float x2 = x[i] * x[i];
        float p = fmaf(0.0193613345f, x2, -0.0537063462f);
        p = fmaf(p, x2, 0.133322014f);
        p = fmaf(p, x2, -0.333333161f);
        float t = fmaf(p * x2, x[i], x[i]);
        if (large) {
            const float e = __builtin_amdgcn_exp2f(2.0f * kLog2e * fabsf(x[i]));
            const float u = copysignf(1.0f - 2.0f * __builtin_amdgcn_rcpf(e + 1.0f), x[i]);
            t = fabsf(x[i]) < 0.35f ? t : u;
        }
        x[i] = t * out;
    }
}

// Where a row tile of a sequence stands: the tokens first .. first + tokens-1
// of it, at indexes pos .. , and the keys they may see.
struct TileAt {
    int s, first, tokens, row;  // row: of the inputs, of token `first`
    int pos, len, pre;          // index of the first token, readable keys, prefix
    int end, low;               // keys any of the tokens sees: [low, end) and [0, pre)
    int base, n, kv;            // index of the sequence's first new token, new tokens, and cached ones with them
};

// What a lane reads of its sequence (nothing of it is trusted further than
// that it is some number).
struct SeqAt {
    int q0, q1, kv, pre;
};
__device__ __forceinline__ SeqAt seq_at(const AttnArgs& a, int s) {
    const int64_t room = (int64_t)a.c.table_width * a.c.page_size;
    SeqAt q;
    const int32_t q0 = a.c.q_start[s], q1 = a.c.q_start[s + 1], kv = a.c.kv_len[s], pre = a.prefix ? a.prefix[s] : 0;
    q.q0 = clamp_row(q0, a.c.n_tokens), q.q1 = clamp_row(q1, a.c.n_tokens);
    q.kv = max(kv, 0);
    q.pre = min(max(pre, 0), (int64_t)q.kv < room ? q.kv : (int)room);
    return q;
}

// The row tile that begins with token `first` of sequence s.  In a tree any new
// token may be seen, and positions begin with the first new token's.
template <bool TREE>
__device__ __forceinline__ TileAt tile_at(const AttnArgs& a, int s, const SeqAt& q, int first) {
    TileAt t;
    t.s = s;
    t.first = first;
    t.row = q.q0 + first;
    t.tokens = min(1 << a.tile_shift, q.q1 - q.q0 - first);
    const int64_t room = (int64_t)a.c.table_width * a.c.page_size;
    t.len = (int64_t)q.kv < room ? q.kv : (int)room;
    t.pos = q.kv - (q.q1 - q.q0) + first;
    t.pre = q.pre;
    t.n = q.q1 - q.q0;
    t.kv = q.kv;
    t.base = q.kv - t.n;
    t.end = TREE ? t.len : max(0, min(t.len, t.pos + t.tokens));
    const int from = TREE ? t.base : t.pos;
    t.low = a.window > 0 && from >= a.window ? from - a.window + 1 : 0;
    return t;
}

// A row of a tree: its position, and what it sees of the new tokens.
struct TreeRow {
    const uint64_t* seen;
    const int32_t* depth;  // of the sequence's first new token
    int pos;
};
__device__ __forceinline__ TreeRow tree_row(const AttnArgs& a, const TileAt& t, int mt) {
    const int64_t row = t.row + mt;
    const int32_t d = a.depth[row];
    // (held to what a tree's can be: positions stay below kv, as the tiles' bounds take them)
    return TreeRow{a.tree + row * a.words, a.depth + (t.row - t.first), t.base + min(max(d, 0), t.n - 1)};
}
// Which of the keys kb .. kb + 63 the row sees, window and prefix apart: those
// before the new tokens, and its own of these.
__device__ __forceinline__ uint64_t tree_bits(const AttnArgs& a, const TileAt& t, const TreeRow& r, int kb) {
    const int64_t off = (int64_t)kb - t.base;
    const int64_t w = off >> 6;
    const int sh = (int)(off & 63);
    const uint64_t lo = w >= 0 && w < a.words ? r.seen[w] : 0, hi = w >= -1 && w + 1 < a.words ? r.seen[w + 1] : 0;
    const uint64_t before = off >= 0 ? 0 : off <= -64 ? ~uint64_t(0) : (uint64_t(1) << -off) - 1;
    return before | lo >> sh | (sh ? hi << (64 - sh) : 0);
}
// The position of key j.
__device__ __forceinline__ int tree_place(const TileAt& t, const TreeRow& r, int j) {
    const int i = j - t.base;  // (j is below 2^30, the base above -2^23)
    return i < 0 || i >= t.n ? j : t.base + min(max(r.depth[i], 0), t.n - 1);
}

// A work item: a row tile of a sequence, and a part of the keys it sees.
struct Work {
    TileAt at;
    int split, splits;
    int first, step;  // the row tile's first item, and from one split's to the next
};

// Work item `item`, by one wavefront; false if there are fewer.  Sequence s
// makes ceil(tokens / 2^tile_shift) row tiles, each split in as many parts as
// its keys fill chunks of equal size: the chunk is the keys of all row tiles
// over a.splits, so a.splits + (number of row tiles) items hold them all, and
// a long sequence among short ones is divided as finely as they are small
// (64 conversations of 8k to 16k keys: 382 -> 338 us against as many splits
// of each).  Without splits (0) a row tile is one item.  Items go split by
// split within a sequence; `last_first` turns the row tiles around.
template <bool TREE>
__device__ __forceinline__ bool find_work(const AttnArgs& a, int item, Work& w, bool last_first = false) {
    const int lane = threadIdx.x & 63, n = a.c.n_seqs;
    SeqAt q = {};
    unsigned tiles = 0, keys = 0;  // of the lane's sequence: row tiles, and blocks of 32 keys
    auto look = [&](int s) {
        tiles = keys = 0;
        if (s >= n) return;
        q = seq_at(a, s);
        if (q.q1 <= q.q0) return;
        tiles = ((q.q1 - q.q0 - 1) >> a.tile_shift) + 1;
        const TileAt t = tile_at<TREE>(a, s, q, 0);
        const int pre = (t.pre + 31) >> 5;
        keys = pre + max(0, ((t.len + 31) >> 5) - max(pre, t.low >> 5));
    };
    look(lane);
    unsigned chunk = 0;
    if (a.splits) {
        double all = 0.0;
        for (int s0 = 0; s0 < n; s0 += 64) {
            if (n > 64) look(s0 + lane);
            all += (double)tiles * (double)keys;
        }
#pragma unroll
        for (int k = 1; k < 64; k <<= 1) all += __shfl_xor(all, k);
        chunk = max(a.least, (int)fmin(all / (double)a.splits, 1e9) + 1);
        if constexpr (TREE) {
            // `fit` (64 sequences at most): no more items than splits, if parts of up to twice the even share make it so:
            // parts are cut to whole numbers a row tile, so equal ones of the share may be more.  Where they are too many
            // also then, as behind a long sequence among row tiles that fill the places already, twice the share stays: no
            // workgroup walks more, and the items beyond one a row tile are half of the splits at most.
            auto fits = [&](unsigned size) {
                return sum_lanes(keys ? tiles * ((keys - 1) / size + 1) : tiles) <= a.splits;
            };
            if (a.fit && !fits(chunk)) {
                unsigned low = chunk, high = 2 * chunk;
                for (int i = 0; i < 6 && high - low > 1; ++i) {  // to a 64th of the share
                    const unsigned mid = low + (high - low) / 2;
                    if (fits(mid))
                        high = mid;
                    else
                        low = mid;
                }
                chunk = high;
            }
        }
    }
    int base = 0;
    for (int s0 = 0; s0 < n; s0 += 64) {
        if (n > 64) look(s0 + lane);
        const unsigned parts = chunk && keys ? (keys - 1) / chunk + 1 : 1;
        int upto = (int)(tiles * parts);
#pragma unroll
        for (int k = 1; k < 64; k <<= 1) {
            if (k < n) {
                const int below = __shfl_up(upto, k);
                upto += lane >= k ? below : 0;
            }
        }
        const uint64_t over = __ballot(base + upto > item);
        if (over) {
            const int at = __ffsll((unsigned long long)over) - 1;
            const int t = __builtin_amdgcn_readlane((int)tiles, at), p = __builtin_amdgcn_readlane((int)parts, at);
            const int start = base + __builtin_amdgcn_readlane(upto, at) - t * p, i = item - start;
            // (not so only where q_start is no batch's)
            if (t <= 0 || i < 0 || i >= (int64_t)t * p) return false;
            w.splits = p;
            w.split = (int)((unsigned)i / (unsigned)t);
            int tile = i - w.split * t;
            w.first = start + tile;
            w.step = t;
            if (last_first) tile = t - 1 - tile;
            const SeqAt u = {__builtin_amdgcn_readlane(q.q0, at), __builtin_amdgcn_readlane(q.q1, at),
                             __builtin_amdgcn_readlane(q.kv, at), __builtin_amdgcn_readlane(q.pre, at)};
            w.at = tile_at<TREE>(a, s0 + at, u, tile << a.tile_shift);
            return true;
        }
        base += __builtin_amdgcn_readlane(upto, 63);
    }
    return false;
}

// Where the join finds the parts of a row: rows of the workspace, (first + z
// step) * (rows of an item, all heads) + slot for its splits z.  0 splits: the
// row is written already.
struct JoinOf {
    int first, splits, step, slot;
};
__device__ __forceinline__ JoinOf* join_of(const AttnArgs& a) {
    return reinterpret_cast<JoinOf*>(a.work + (a.parts * (a.head_dim + 2) + 3) / 4 * 4);
}

}  // namespace qmm
