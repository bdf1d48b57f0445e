// attn_tile.h — attention over a paged cache for many query rows a
// sequence: a workgroup takes 128 query rows (tokens x the query heads of one
// key-value head) and walks the keys in tiles of 64, which its waves stage in
// LDS together and each multiplies with its 32 (or 16) rows.
//
// With 32x32x16 MFMAs (16x16x32 in parentheses), as in the split kernels:
//   S^T = K Q^T      lane (r, h) = (lane % 32, lane / 32) gets the scores of
//                    row r with 4 keys of each 8 of the tile (of each 16);
//   O^T += V^T P^T   the keys of a step in the order the lanes hold their
//                    scores in, so P never leaves its lane.
// K lies in LDS as it is (rows 16 bytes apart from a multiple of the banks),
// V transposed, a row of 64 keys a value, in that key order: both are read as
// the MFMAs' A operands with 16-byte loads.  The larger MFMAs read half as
// much of LDS for a product; the smaller ones need half the registers a wave,
// which wide heads and three-part queries take (with eight waves of 16 rows,
// two a SIMD, instead of four of 32 and one).
//
// A wave stages the 16 (8) keys of its number in each tile, so where they lie
// in the cache is one page lookup, the same for its lanes.  The next tile's
// loads are issued before a tile is multiplied.
//
// Exactness: bf16 queries are operands as they are, and P is split into two parts
// of the cache's kind, which hold 22 bits (fp16) or 16: a bf16 result is the fp32
// one rounded, as the split kernels' is, so that it does not depend on the sizes
// that choose between them.  (With one part, 8 or 11 bits, 8191 tokens took 610 us
// instead of 790 over bf16 rows and 630 instead of 830 over fp16 rows, but the
// former's error was 0.0023 of the norm instead of 0.0017, and a tenth of the
// latter's results were neighbours of the right ones.)  fp32 queries and P are split
// into two fp16 parts (three bf16 ones for a bf16 cache), and the values of Q8_0
// rows, d times a code, into two fp16 parts, which hold them exactly: three products
// of parts instead of one, and with bf16 queries two for scores and three for P V.
// Q8_0 keys and values are staged times powers of two that keep the largest below
// 2^15: one for a tile's keys, one for each 32 values of all keys so far, so that a
// block that is small beside others loses nothing; keys and values 2^16 and more
// below the largest they share one with are held to 2^-38 of that, the parts'
// smallest step, as P is to 2^-39 of a row's largest.
//
// Bound: nothing alone; the matrix unit and the vector unit are busy for 45% of the
// time each.  A prompt of 8191 tokens (bf16 queries, 32 heads, of 128, on 8 of an
// fp16 cache; 550 GFLOP, 825 multiplied) takes 850 us, 0.97 PFLOP/s multiplied of
// the 1.33 that a large product of matrices reaches here; with three products each,
// 2048 tokens over Q8_0 (34 GFLOP, 103 multiplied) 152 us.  Of the former's time
// with P in one part (630 us) the operands' LDS reads cost 29%, the staging 20%
// (loads 12, writes 7), the masks' and maxima's pass 6, the exponentials 2 (each
// left out in turn).  Tried then and no faster: the next tile's scores multiplied
// between a tile's exponentials (647 -> 649: registers for it leave no room to read
// operands earlier), the next tile written among the products (665 -> 677), 256 rows
// a workgroup (665 -> 658, and 200 -> 215 for four prompts of 2200), 16 rows a wave
// (636 -> 933), light and heavy row tiles paired (657 -> 698), s_setprio around the
// products (no change).
//
// For trees of new tokens (some rows a sequence over long caches) a workgroup takes
// 32 or 64 rows, and two waves the same rows with half of a tile's keys each: as many
// waves share the staging, so the bound is reading again.  13 tokens over 130911 keys
// in fp16 (32 heads, of 128, on 8; bf16 queries; 537 MB): 103 us, 5.2 TB/s, and 6.6 for
// the join.  12 sequences of 26 tokens over a window of 2048 keys (16 heads, of 256, on
// 8; bf16, cap; 200 MB): 51 us and 5 for the join, 3.9 TB/s; at most 256 workgroups
// run at once, one a CU: eight sequences are cut in three a head, four in two, and the
// longest part has 1.36 times the even share of keys.  Tiles of 128 rows in this form did
// not fit the registers.
#pragma once

#include "attn_common.h"

namespace qmm {
namespace {

constexpr int kKeys = 64;  // keys of a tile

template <bool BF>
__device__ __forceinline__ f16v mfma_of(u4v a, u4v b, f16v c) {
    if constexpr (BF)
        return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf8v, a), __builtin_bit_cast(bf8v, b), c, 0,
                                                       0, 0);
    else
        return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(half8v, a), __builtin_bit_cast(half8v, b), c,
                                                      0, 0, 0);
}
template <bool BF>
__device__ __forceinline__ f4v mfma_of(u4v a, u4v b, f4v c) {
    return mfma16<BF>(a, b, c);
}

// 16-byte slot of the keys `oct` (8 in the lanes' order) in the LDS row of
// value `dim`: an order in which neither the transposing writes (four values
// apart) nor the operand reads (one apart) meet a bank more often than needed.
__device__ __forceinline__ int v_slot(int dim, int oct) {
    const int r = dim & 31;  // the same in each 32 values: reads of them differ by a constant
    return oct ^ (((r >> 1) ^ (r >> 4)) & 7);
}

// What a wave has loaded of its KEYS keys of a tile.
template <int CT, int NB, int KEYS>
struct Staged {
    static constexpr bool Q8 = CT == QMM_Q8_0;
    static constexpr int KT = ((Q8 ? 1 : 4) * KEYS * NB + 63) / 64;  // tasks of a lane: a block, or 16 bytes
    static constexpr int VT = (KEYS * NB + 63) / 64;                        // tasks of a lane: 8 keys x 4 values
    uint32_t k[KT][Q8 ? 9 : 4];
    uint32_t v[VT][Q8 ? 8 : 16];
    uint32_t vd[VT][Q8 ? 8 : 1];
};

// What the lanes of block b (from lane 8 b on) hold.
__device__ __forceinline__ float of_block(float x, int b) {
    return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, x), 8 * b));
}

// The largest group of operands, up to `most`, that n of them divide into.
constexpr int group_of(int n, int most) { return n % most ? group_of(n, most - 1) : most; }
// Parts of Q and of P, and rows of a wave.
constexpr int q_parts(int ct, bool xb) { return xb ? 1 : ct == QMM_BF16 ? 3 : 2; }
constexpr int p_parts(int ct, bool xb) { return xb ? 2 : q_parts(ct, xb); }
// With fewer rows than a tile of 128 has (trees of new tokens), two waves take the
// same rows, and half of a tile's keys each; their sums are joined at the end.
constexpr int wave_rows(int ct, int nb, bool xb, int rows = kTileRows) {
    return nb > 4 || q_parts(ct, xb) == 3 || rows == 32 ? 16 : 32;
}
constexpr int halves_of(int rows) { return rows < kTileRows ? 2 : 1; }
constexpr int waves_of(int ct, int nb, bool xb, int rows) { return rows / wave_rows(ct, nb, xb, rows) * halves_of(rows); }

template <int CT, int NB, bool XB, bool TREE, int ROWS>
__global__ __launch_bounds__(64 * waves_of(CT, NB, XB, ROWS), 2) void attn_tile_kernel(AttnArgs a) {
    constexpr int D = 32 * NB, RB = kv_row_bytes(CT, D);
    constexpr bool BF = CT == QMM_BF16, Q8 = CT == QMM_Q8_0;
    constexpr int AP = Q8 ? 2 : 1;                               // parts of K and V
    constexpr int QP = q_parts(CT, XB), PP = p_parts(CT, XB);    // of Q, of P
    constexpr int R = wave_rows(CT, NB, XB, ROWS), W = waves_of(CT, NB, XB, ROWS);  // rows of a wave, waves
    constexpr int HALVES = halves_of(ROWS), RG = W / HALVES;     // parts of a tile's keys, waves of each
    constexpr int GROUPS = 64 / R, KS = 8 * GROUPS;              // lanes of a row, values (or keys) of an MFMA's step
    constexpr int KPW = kKeys / W;                               // keys that a wave stages
    constexpr int VL = R * R / 64, NO = D / R;                   // values of an accumulator, accumulators
    typedef float accv __attribute__((ext_vector_type(VL)));
    constexpr int KROW = 2 * D + 16;                             // bytes of a row of K in LDS
    using St = Staged<CT, NB, KPW>;
    // Two buffers, and one barrier a tile, where eight waves a CU still fit.
    // (Q8_0 needs a barrier between its tile's largest scale and the staging.)
    constexpr int K_BYTES = kKeys * KROW, V_BYTES = D * kKeys * 2;
    constexpr int BUFS = !Q8 && 2 * (K_BYTES + V_BYTES) * (8 / W) <= 150 * 1024 ? 2 : 1;
    __shared__ __attribute__((aligned(16))) uint8_t s_k[BUFS * AP][K_BYTES];
    __shared__ __attribute__((aligned(16))) uint8_t s_v[BUFS * AP][V_BYTES];
    // of a tile, twice: the largest |d| of the keys that each wave staged (Q8_0), whether they have a page,
    // and the largest |d| of the values, of each 8 keys and 32 values
    __shared__ float s_big[2][W];
    __shared__ int s_page[2][W];
    __shared__ __attribute__((aligned(16))) float s_vd[Q8 ? 2 : 1][NB][8];

    // a long sequence's last tiles see the most keys: they go first.  The
    // heads of a tile are neighbours, so (with 8 of them) each XCD keeps to one
    // head's keys and values.
    const int groups = a.c.n_kv * a.chunks, item = (int)(blockIdx.x / groups), hb = blockIdx.x % groups;
    Work w;
    if (!find_work<TREE>(a, item, w, true)) return;
    const TileAt at = w.at;
    const int lane = threadIdx.x & 63, r = lane % R, h = lane / R;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int rw = HALVES > 1 ? wave % RG : wave, half = HALVES > 1 ? wave / RG : 0;  // its rows, and its keys' half
    const int kvh = hb / a.chunks, G = a.n_q / a.c.n_kv;
    const int head0 = kvh * G + (hb % a.chunks) * a.chunk;
    const int heads = min(a.chunk, kvh * G + G - head0);
    const int rows = at.tokens * heads;
    const int mr = min(R * rw + r, rows - 1), mt = mr / heads, head = head0 + mr % heads;
    TreeRow tree = {};
    if constexpr (TREE) tree = tree_row(a, at, mt);
    const int p_row = TREE ? tree.pos : at.pos + mt;
    // the positions of the wave's first and last row (in a tree, of any)
    const int p_first = TREE ? at.base : at.pos + min(R * rw, rows - 1) / heads;
    const int p_last = TREE ? at.kv - 1 : at.pos + min(R * rw + R - 1, rows - 1) / heads;
    const int all_see = TREE ? at.base : p_first + 1;  // every row of the wave sees the keys up to here
    const bool idle = R * rw >= rows;
    // the key, in its tile, of value i of the lane's scores
    auto key_of = [&](int i) {
        return (R == 32 ? 32 * (i >> 4) + 8 * ((i & 15) >> 2) + 4 * h + (i & 3)
                        : 32 * (i >> 3) + 8 * h + 4 * ((i >> 2) & 1) + (i & 3)) + 32 * half;
    };
    // LDS offset of 16 bytes of K, columns col .. of 8 values.  (With 16 rows a wave the lanes of an operand
    // read the keys 0..3 of each 8: those of the upper half turn to other columns to miss the lower ones' banks,
    // where a row is whole eights of columns.)
    auto k_at = [&](int key, int col) { return key * KROW + 16 * (R == 32 || NB % 2 ? col : col ^ ((key >> 2) & 4)); };

    // ---- the queries, as B operands: lane (r, h) holds the values 8h..8h+7 of each step
    u4v qf[D / KS][QP];
    float qs;
    {
        const int64_t base = (int64_t)(at.row + mt) * a.ldq + (int64_t)head * D + 8 * h;
        float big = 0.f;
        // twice over the row: the first for its largest value (the second comes from L1)
#pragma unroll
        for (int b = 0; b < D / KS; ++b) {
            if constexpr (XB) {
                const u4v w = *reinterpret_cast<const u4v*>(static_cast<const uint16_t*>(a.q) + base + KS * b);
#pragma unroll
                for (int i = 0; i < 4; ++i) big = fmaxf(big, fmaxf(fabsf(bf16_lo(w[i])), fabsf(bf16_hi(w[i]))));
            } else {
                const f4v* p = reinterpret_cast<const f4v*>(static_cast<const float*>(a.q) + base + KS * b);
#pragma unroll
                for (int i = 0; i < 4; ++i) big = fmaxf(big, fmaxf(fabsf(p[0][i]), fabsf(p[1][i])));
            }
        }
        if constexpr (R == 16) big = fmaxf(big, __shfl_xor(big, 16));
        big = fmaxf(big, __shfl_xor(big, 32));
        int ex = 0;
        frexpf(big, &ex);
        ex = min(max(ex, -110), 126);
        // the sign of the scale goes to the queries
        constexpr int TOP = BF ? 0 : 14;  // (bf16 parts have fp32's range)
        const float up = copysignf(ldexpf(1.0f, TOP - ex), a.scale);
        qs = ldexpf(1.0f, ex - TOP) * fabsf(a.scale);
#pragma unroll
        for (int b = 0; b < D / KS; ++b) {
            float x[8];
            if constexpr (XB) {
                const u4v w = *reinterpret_cast<const u4v*>(static_cast<const uint16_t*>(a.q) + base + KS * b);
#pragma unroll
                for (int i = 0; i < 4; ++i) x[2 * i] = bf16_lo(w[i]), x[2 * i + 1] = bf16_hi(w[i]);
            } else {
                const f4v* p = reinterpret_cast<const f4v*>(static_cast<const float*>(a.q) + base + KS * b);
                const f4v u = p[0], w = p[1];
#pragma unroll
                for (int i = 0; i < 4; ++i) x[i] = u[i], x[4 + i] = w[i];
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                uint32_t part[QP];
                split_pair<BF, QP>(x[2 * i] * up, x[2 * i + 1] * up, part);
#pragma unroll
                for (int k = 0; k < QP; ++k) qf[b][k][i] = part[k];
            }
        }
    }
    const bool capped = a.softcap > 0.f;
    if (!capped) qs *= kLog2e;
    const float slope = a.slopes ? a.slopes[head] * kLog2e : 0.f;
    const int reach = a.window > 0 ? a.window : INT32_MAX;
    // every row of the wave sees keys from low_last on, and one from low_first (no index less a window passes 32
    // bits from 0 on; rows below it see none)
    const int low_last = a.window > 0 ? max(p_last, 0) - a.window + 1 : INT32_MIN;
    const int low_first = a.window > 0 ? max(p_first, 0) - a.window + 1 : INT32_MIN;

    // ---- the tiles of this split
    const int n_pre = (at.pre + kKeys - 1) / kKeys;
    const int w0 = max(n_pre, at.low / kKeys), w1 = (at.end + kKeys - 1) / kKeys;
    const int n_tiles = n_pre + max(0, w1 - w0);
    const int per = (n_tiles + w.splits - 1) / w.splits;
    const int t0 = w.split * per, t1 = min(n_tiles, t0 + per);

    accv o[NO];
#pragma unroll
    for (int c = 0; c < NO; ++c)
#pragma unroll
        for (int i = 0; i < VL; ++i) o[c][i] = 0.f;
    float mx = -INFINITY, mref = 0.f, l = 0.f;
    int vex = -30;  // Q8_0: 2^vex is above every |d| so far of the lane's block of values, lane / 8 % NB

    int64_t my_row = -1;  // lane i: where the wave's keys of tile i from here on begin in the cache, or -1
    St st;
    // key j of the first of the wave's runs of 8 keys in the lanes' order (the second run begins RUN behind it)
    constexpr int RUN = R == 32 ? 4 : 8;
    auto nth = [](int j) { return R == 32 ? (j & 3) + 2 * (j & 4) : j; };
    // Where the wave's keys of tile t begin in the cache, or -1.
    auto row_of = [&](int t) -> int64_t {
        const int from = (t - t0) & 63;
        if (from == 0) {
            const int tt = t + lane;
            const int64_t key = (int64_t)kKeys * (tt < n_pre ? tt : tt - n_pre + w0) + KPW * wave;
            my_row = -1;
            if (tt < t1 && key < at.len) {
                const int pidx = (int)key / a.c.page_size;
                const int pg = a.c.table[(int64_t)at.s * a.c.table_width + pidx];
                if (pg >= 0 && pg < a.c.n_pages)
                    my_row = ((int64_t)pg * a.c.n_kv + kvh) * a.c.page_size + ((int)key - pidx * a.c.page_size);
            }
        }
        return (int64_t)((uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)my_row, from) |
                         (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(my_row >> 32), from) << 32);
    };
    // Whether a key of the wave's in tile t, at cache row `row`, is seen by any row of the tile: others may hold
    // anything, and count as 0.
    auto key_at = [&](int t) { return kKeys * (t < n_pre ? t : t - n_pre + w0) + KPW * wave; };
    auto all_kept = [&](int64_t row, int key0) {
        return (row >= 0) & ((key0 + KPW <= at.pre) | ((key0 >= at.low) & (key0 + KPW <= at.end)));
    };
    auto kept = [&](int64_t row, int key) {
        return (row >= 0) & (((key >= at.low) & (key < at.end)) | (key < at.pre));
    };
    // Loads the wave's keys and values of tile t, which begin at cache row `row`; the largest |d| of the Q8_0 blocks of K
    // that this lane holds.
    auto fetch = [&](int t, int64_t row) -> float {
        const int key0 = key_at(t);
        const uint8_t* kbase = a.c.k + max(row, (int64_t)0) * RB;  // uniform, with 32-bit offsets of the lanes
        const uint8_t* vbase = a.c.v + max(row, (int64_t)0) * RB;
        float big = 0.f;
#pragma unroll
        for (int i = 0; i < St::KT; ++i) {
            const uint32_t task = lane + 64 * i;
            if constexpr (Q8) {
                if (KPW * NB % 64 == 0 || task < KPW * NB) {
                    const uint8_t* p = kbase + task * kQ8_0Bytes;  // the keys' blocks lie one after another
                    st.k[i][0] = *reinterpret_cast<const uint16_t*>(p);
                    __builtin_memcpy(&st.k[i][1], p + 2, 32);
                }
            } else if (KPW * NB % 16 == 0 || task < 4 * KPW * NB) {
                __builtin_memcpy(st.k[i], reinterpret_cast<const u4v*>(kbase + 16 * task), 16);
            }
        }
#pragma unroll
        for (int i = 0; i < St::VT; ++i) {
            const uint32_t task = lane + 64 * i, oct = task / (8 * NB), c = task % (8 * NB);
            if (KPW * NB % 64 == 0 || task < KPW * NB) {
                const uint32_t off = RUN * oct * RB + (Q8 ? (c >> 3) * kQ8_0Bytes : 8 * c);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const uint8_t* p = vbase + nth(j) * RB + off;
                    if constexpr (Q8) {
                        st.vd[i][j] = *reinterpret_cast<const uint16_t*>(p);
                        __builtin_memcpy(&st.v[i][j], p + 2 + 4 * (c & 7), 4);
                    } else {
                        __builtin_memcpy(&st.v[i][2 * j], reinterpret_cast<const uint2*>(p), 8);
                    }
                }
            }
        }
        if (!all_kept(row, key0)) {
#pragma unroll
            for (int i = 0; i < St::KT; ++i) {
                const bool ok = kept(row, key0 + (lane + 64 * i) / (Q8 ? NB : 4 * NB));
#pragma unroll
                for (int j = 0; j < (Q8 ? 1 : 4); ++j) st.k[i][j] = ok ? st.k[i][j] : 0;
            }
#pragma unroll
            for (int i = 0; i < St::VT; ++i)
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const bool ok = kept(row, key0 + RUN * ((lane + 64 * i) / (8 * NB)) + nth(j));
                    if constexpr (Q8) {
                        st.vd[i][j] = ok ? st.vd[i][j] : 0;
                    } else {
                        st.v[i][2 * j] = ok ? st.v[i][2 * j] : 0, st.v[i][2 * j + 1] = ok ? st.v[i][2 * j + 1] : 0;
                    }
                }
        }
        if constexpr (Q8) {
#pragma unroll
            for (int i = 0; i < St::KT; ++i)
                if (KPW * NB % 64 == 0 || lane + 64 * i < KPW * NB) big = fmaxf(big, fabsf(h2f(st.k[i][0])));
            static_assert(St::VT == 1, "a lane stages values of one block");
            float vd = 0.f;
#pragma unroll
            for (int j = 0; j < 8; ++j) vd = fmaxf(vd, fabsf(h2f(st.vd[0][j])));
            if (lane < KPW * NB && lane % 8 == 0) s_vd[t & 1][lane / 8 % NB][KPW / 8 * wave + lane / (8 * NB)] = vd;
        }
        return big;
    };
    // Write what was fetched to buffer `to`; Q8_0 values times powers of two.
    auto store_k = [&](float k_inv, int to) {
        uint8_t(*s_kt)[K_BYTES] = s_k + AP * to;
#pragma unroll
        for (int i = 0; i < St::KT; ++i) {
            const int task = lane + 64 * i;
            if constexpr (Q8) {
                if (KPW * NB % 64 == 0 || task < KPW * NB) {
                    const int key = KPW * wave + task / NB, blk = task % NB;
                    const float d = h2f(st.k[i][0]) * k_inv;
                    uint32_t part[16][AP];
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const uint32_t w = st.k[i][1 + j];
                        split_pair<false, AP>(d * (float)(int8_t)w, d * (float)(int8_t)(w >> 8), part[2 * j]);
                        split_pair<false, AP>(d * (float)(int8_t)(w >> 16), d * (float)(int8_t)(w >> 24), part[2 * j + 1]);
                    }
#pragma unroll
                    for (int k = 0; k < AP; ++k)
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            *reinterpret_cast<u4v*>(&s_kt[k][k_at(key, 4 * blk + j)]) =
                                u4v{part[4 * j][k], part[4 * j + 1][k], part[4 * j + 2][k], part[4 * j + 3][k]};
                }
            } else if (KPW * NB % 16 == 0 || task < 4 * KPW * NB) {
                const int key = KPW * wave + task / (4 * NB), c = task % (4 * NB);
                *reinterpret_cast<u4v*>(&s_kt[0][k_at(key, c)]) = u4v{st.k[i][0], st.k[i][1], st.k[i][2], st.k[i][3]};
            }
        }
    };
    auto store_v = [&](float v_inv, int to) {
        uint8_t(*s_vt)[V_BYTES] = s_v + AP * to;
#pragma unroll
        for (int i = 0; i < St::VT; ++i) {
            const int task = lane + 64 * i;
            if (KPW * NB % 64 == 0 || task < KPW * NB) {
                const int oct = KPW / 8 * wave + task / (8 * NB), c = task % (8 * NB);
                if constexpr (Q8) {
                    float d[8];
#pragma unroll
                    for (int j = 0; j < 8; ++j) d[j] = h2f(st.vd[i][j]) * v_inv;
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        u4v w[AP];
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            uint32_t part[AP];
                            split_pair<false, AP>(d[2 * j] * (float)(int8_t)(st.v[i][2 * j] >> (8 * e)),
                                                  d[2 * j + 1] * (float)(int8_t)(st.v[i][2 * j + 1] >> (8 * e)), part);
#pragma unroll
                            for (int k = 0; k < AP; ++k) w[k][j] = part[k];
                        }
#pragma unroll
                        for (int k = 0; k < AP; ++k)
                            *reinterpret_cast<u4v*>(&s_vt[k][(4 * c + e) * (2 * kKeys) + 16 * v_slot(4 * c + e, oct)]) = w[k];
                    }
                } else {
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        u4v w;
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            w[j] = __builtin_amdgcn_perm(st.v[i][4 * j + 2 + (e >> 1)], st.v[i][4 * j + (e >> 1)],
                                                         e & 1 ? 0x07060302u : 0x05040100u);
                        *reinterpret_cast<u4v*>(&s_vt[0][(4 * c + e) * (2 * kKeys) + 16 * v_slot(4 * c + e, oct)]) = w;
                    }
                }
            }
        }
    };
    // Loads tile t, and tells the other waves about it before the barrier that all pass before it is stored.
    auto begin = [&](int t) {
        const int64_t row = row_of(t);
        float big = fetch(t, row);
        if constexpr (Q8) {
#pragma unroll
            for (int k = 1; k < 64; k <<= 1) big = fmaxf(big, __shfl_xor(big, k));
        }
        if (lane == 0) s_big[t & 1][wave] = big, s_page[t & 1][wave] = row >= 0;
    };
    // Q8_0: powers of two, the same in every wave, of tile t's K (the limit is
    // returned), and of each 32 values so far (2^vex: raised where tile t needs it,
    // o with it).  Both are staged as 2^8 d code / limit < 2^15.
    auto k_limit = [&](int t) {
        float big = 0.f;
#pragma unroll
        for (int i = 0; i < W; ++i) big = fmaxf(big, s_big[t & 1][i]);
        int ex = 0;
        frexpf(fminf(big, 65504.0f), &ex);
        return ldexpf(1.0f, ex);
    };
    auto v_limit = [&](int t) {
        float big = s_vd[t & 1][lane / 8 % NB][lane % 8];
        big = fmaxf(big, dpp<0xB1>(big));   // lane ^ 1
        big = fmaxf(big, dpp<0x4E>(big));   // lane ^ 2
        big = fmaxf(big, dpp<0x141>(big));  // 7 - lane, of each 8
        // (fp16 numbers are no subnormals in fp32)
        const int ex = max(vex, min((__builtin_bit_cast(int, big) >> 23) - 126, 16));
        if (__any(ex > vex)) {
            const float down = ldexpf(1.0f, vex - ex);
            vex = ex;
#pragma unroll
            for (int c = 0; c < NO; ++c) o[c] *= of_block(down, R * c / 32);
        }
    };

    constexpr int STEPS = D / KS, SUBS = kKeys / HALVES / R;  // of an accumulator's products, accumulators of scores
    constexpr int NK = SUBS * AP * STEPS, VSTEPS = kKeys / HALVES / KS, NV = VSTEPS * NO * AP;  // A operands of a tile: of K and of V
    constexpr int SC = R / HALVES;  // scores of a lane
    // operand i of K: (keys, part, values); of V: (step, values, part)
    auto k_operand = [&](int buf, int i) {
        const int u = i / (STEPS * AP), ap = AP - 1 - i / STEPS % AP, b = i % STEPS;
        const int key = (R == 32 ? 32 * u + r : 32 * (u >> 1) + 8 * (r >> 2) + 4 * (u & 1) + (r & 3)) + 32 * half;
        return *reinterpret_cast<const u4v*>(&s_k[AP * buf + ap][k_at(key, GROUPS * b + h)]);
    };
    auto v_operand = [&](int buf, int i) {
        const int kk = i / (NO * AP), c = i / AP % NO, ap = AP - 1 - i % AP, dim = R * c + r;
        return *reinterpret_cast<const u4v*>(&s_v[AP * buf + ap][dim * (2 * kKeys) + 16 * v_slot(dim, GROUPS * (kk + VSTEPS * half) + h)]);
    };
    float s[SC];
    // From the products of tile t to scores (f s, times log2 e), masked; raises
    // the running maximum where they pass it by kSlack.
    auto soften = [&](int t, float& f) {
        const int kb = kKeys * (t < n_pre ? t : t - n_pre + w0);
        bool page[4];  // of each 16 keys
#pragma unroll
        for (int i = 0; i < 4; ++i) page[i] = s_page[t & 1][W / 4 * i] != 0;
        if constexpr (HALVES > 1) {  // of its keys
            page[0] = half ? page[2] : page[0], page[1] = half ? page[3] : page[1];
            page[2] = page[0], page[3] = page[1];
        }
        if (capped) {
            cap_scores(s, f, a.softcap);
            f = 1.0f;
        }
        const bool whole = page[0] && page[1] && page[2] && page[3] &&
                           ((kb + kKeys <= at.pre) || (kb >= low_last && kb + kKeys <= min(at.len, all_see)));
        auto place = [&](int key) { return TREE && kb + kKeys > at.base ? tree_place(at, tree, key) : key; };
        if (a.slopes) {
#pragma unroll
            for (int i = 0; i < SC; ++i) s[i] = s[i] * f - slope * fabsf((float)(p_row - place(kb + key_of(i))));
            f = 1.0f;
        }
        if (!whole) {
            const uint64_t bits = TREE ? tree_bits(a, at, tree, kb) >> ((R == 32 ? 4 * h : 8 * h) + 32 * half) : 0;
#pragma unroll
            for (int i = 0; i < SC; ++i) {
                const int key = kb + key_of(i);
                const bool paged = R == 32 ? page[i >> 3] : (h >> 1 ? page[2 * (i >> 3) + 1] : page[2 * (i >> 3)]);
                const bool near = TREE ? (bits >> (key_of(i) - (R == 32 ? 4 * h : 8 * h) - 32 * half) & 1) &
                                             (a.window <= 0 || p_row - place(key) < reach)
                                       : (key <= p_row) & (p_row - key < reach);
                const bool seen = paged & (key < at.len) & (near | (key < at.pre));
                s[i] = seen ? s[i] : -INFINITY;
            }
        }
        float big = s[0];
#pragma unroll
        for (int i = 1; i < SC; ++i) big = fmaxf(big, s[i]);
        if (__any(big * f > mx + kSlack)) {
            if constexpr (R == 16) big = fmaxf(big, __shfl_xor(big, 16));
            big = fmaxf(big, __shfl_xor(big, 32)) * f;
            const float top = fmaxf(mx, big), ref = top == -INFINITY ? 0.f : top;
            const float down = __builtin_amdgcn_exp2f(mx - ref);
            mx = top;
            mref = ref - p_top<BF>();
            l *= down;
#pragma unroll
            for (int c = 0; c < NO; ++c) o[c] *= down;
        }
    };

    if (t0 < t1) begin(t0);
    for (int t = t0; t < t1; ++t) {
        const int buf = BUFS > 1 ? t & 1 : 0;
        float f = qs;
        if constexpr (BUFS == 1) __syncthreads();  // the tile before is multiplied, and this one's s_big told
        if constexpr (Q8) {
            const float lim = k_limit(t);
            v_limit(t);
            f *= lim * 0x1p-8f;
            store_k(0x1p8f / lim, buf);
            store_v(ldexpf(1.0f, 8 - vex), buf);
        } else {
            store_k(1.0f, buf);
            store_v(1.0f, buf);
        }
        f = fmaxf(f, 0x1p-120f);  // never 0: masked scores stay -inf times it
        __syncthreads();
        if (t + 1 < t1) begin(t + 1);

        const int kb = kKeys * (t < n_pre ? t : t - n_pre + w0);
        // nothing of this tile for any row of the wave
        if (idle || !((kb < at.pre) || (kb <= p_last && kb < at.len && kb + kKeys - 1 >= low_first))) continue;
        // Operands come from LDS some at a time, the next ones while these are
        // multiplied: left to itself the compiler waits for each before its use.
        constexpr int GK = group_of(NK, QP > 1 ? 2 : 4), GV = group_of(NO * AP, QP > 1 ? 2 : 4);
        {
            accv acc[SUBS];
#pragma unroll
            for (int u = 0; u < SUBS; ++u)
#pragma unroll
                for (int i = 0; i < VL; ++i) acc[u][i] = 0.f;
            u4v kf[2][GK];
#pragma unroll
            for (int j = 0; j < GK; ++j) kf[0][j] = k_operand(buf, j);
#pragma unroll
            for (int i = 0; i < NK; i += GK) {
                if (i + GK < NK) {
#pragma unroll
                    for (int j = 0; j < GK; ++j) kf[(i / GK + 1) & 1][j] = k_operand(buf, i + GK + j);
                }
                __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                for (int j = 0; j < GK; ++j) {
                    const int u = (i + j) / (STEPS * AP), ap = AP - 1 - (i + j) / STEPS % AP, b = (i + j) % STEPS;
#pragma unroll
                    for (int k = (ap ? 0 : QP - 1); k >= 0; --k) acc[u] = mfma_of<BF>(kf[(i / GK) & 1][j], qf[b][k], acc[u]);
                }
                __builtin_amdgcn_sched_barrier(0);
            }
#pragma unroll
            for (int i = 0; i < SC; ++i) s[i] = acc[i / VL][i % VL];
        }
        u4v vf[2][GV];
#pragma unroll
        for (int j = 0; j < GV; ++j) vf[0][j] = v_operand(buf, j);
        __builtin_amdgcn_sched_barrier(0);
        soften(t, f);
#pragma unroll
        for (int kk = 0; kk < VSTEPS; ++kk) {
            u4v pf[PP];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float x = __builtin_amdgcn_exp2f(fmaf(s[8 * kk + 2 * i], f, -mref));
                const float y = __builtin_amdgcn_exp2f(fmaf(s[8 * kk + 2 * i + 1], f, -mref));
                l += x + y;
                uint32_t part[PP];
                split_pair<BF, PP>(x, y, part);
#pragma unroll
                for (int k = 0; k < PP; ++k) pf[k][i] = part[k];
            }
            constexpr int N = NO * AP;
#pragma unroll
            for (int i = kk * N; i < kk * N + N; i += GV) {
                if (i + GV < NV) {
#pragma unroll
                    for (int j = 0; j < GV; ++j) vf[(i / GV + 1) & 1][j] = v_operand(buf, i + GV + j);
                }
                __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                for (int j = 0; j < GV; ++j) {
                    const int c = (i + j) / AP % NO, ap = AP - 1 - (i + j) % AP;
#pragma unroll
                    for (int k = (ap ? 0 : PP - 1); k >= 0; --k) o[c] = mfma_of<BF>(vf[(i / GV) & 1][j], pf[k], o[c]);
                }
                __builtin_amdgcn_sched_barrier(0);
            }
        }
    }

    if constexpr (HALVES > 1) {
        // the second half's sums go to the first's waves, through what held K
        static_assert(sizeof(s_k) >= ROWS * D * 4, "a half's sums");
        __shared__ float s_ml[2][RG][64];
        f4v(*s_o)[NO * VL / 4][64] = reinterpret_cast<f4v(*)[NO * VL / 4][64]>(&s_k[0][0]);
        __syncthreads();
        if (half) {
            s_ml[0][rw][lane] = mx, s_ml[1][rw][lane] = l;
#pragma unroll
            for (int c = 0; c < NO; ++c)
#pragma unroll
                for (int i = 0; i < VL; i += 4)
                    s_o[rw][(c * VL + i) / 4][lane] = f4v{o[c][i], o[c][i + 1], o[c][i + 2], o[c][i + 3]};
        }
        __syncthreads();
        if (half) return;
        const float other = s_ml[0][rw][lane], top = fmaxf(mx, other), ref = top == -INFINITY ? 0.f : top;
        const float f0 = __builtin_amdgcn_exp2f(mx - ref), f1 = __builtin_amdgcn_exp2f(other - ref);
        mx = top;
        l = f0 * l + f1 * s_ml[1][rw][lane];
#pragma unroll
        for (int c = 0; c < NO; ++c)
#pragma unroll
            for (int i = 0; i < VL; i += 4) {
                const f4v x = s_o[rw][(c * VL + i) / 4][lane];
#pragma unroll
                for (int j = 0; j < 4; ++j) o[c][i + j] = f0 * o[c][i + j] + f1 * x[j];
            }
    }
    if constexpr (R == 16) l += __shfl_xor(l, 16);
    l += __shfl_xor(l, 32);
    if (R * rw + r >= rows) return;
    const int64_t row = (int64_t)(at.row + mt) * a.n_q + head;
    const float lane_unit = Q8 ? ldexpf(1.0f, vex - 8) : 1.0f;
    auto unit = [&](int c) { return Q8 ? of_block(lane_unit, R * c / 32) : 1.0f; };
    if (a.splits && h == 0 && w.split == 0)
        join_of(a)[row] = JoinOf{w.first, w.splits > 1 ? w.splits : 0, w.step, hb * a.slots + R * rw + r};
    // accumulator c, value i: value R c + 8 (i / 4) + 4 h + i % 4 of the row
    if (w.splits > 1) {
        const int64_t part = ((int64_t)item * groups + hb) * a.slots + R * rw + r;
        float* ml = a.work + a.parts * D;
        if (h == 0) ml[2 * part] = mx, ml[2 * part + 1] = l;
#pragma unroll
        for (int c = 0; c < NO; ++c) {
            const float u = unit(c);
#pragma unroll
            for (int i = 0; i < VL; i += 4)
                *reinterpret_cast<f4v*>(a.work + part * D + R * c + 2 * i + 4 * h) =
                    f4v{o[c][i] * u, o[c][i + 1] * u, o[c][i + 2] * u, o[c][i + 3] * u};
        }
        return;
    }
    const float inv = l > 0.f ? 1.0f / l : l == 0.f ? 0.f : l;
#pragma unroll
    for (int c = 0; c < NO; ++c)
#pragma unroll
        for (int i = 0; i < VL; i += 4) {
            const float w = inv * unit(c);
            const float x0 = o[c][i] * w, x1 = o[c][i + 1] * w, x2 = o[c][i + 2] * w, x3 = o[c][i + 3] * w;
            const int64_t e = row * D + R * c + 2 * i + 4 * h;
            if constexpr (XB) {
                uint32_t w0[1], w1[1];
                split_pair<true, 1>(x0, x1, w0);
                split_pair<true, 1>(x2, x3, w1);
                *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + e) = make_uint2(w0[0], w1[0]);
            } else {
                *reinterpret_cast<f4v*>(static_cast<float*>(a.out) + e) = f4v{x0, x1, x2, x3};
            }
        }
}

template <int CT, int NB, bool XB, bool TREE>
hipError_t tile_typed(const AttnArgs& a, hipStream_t s) {
    const int64_t grid = a.items * a.c.n_kv * a.chunks;  // below 2^32 work-items
    hipError_t e;
    if constexpr (TREE) {
        if (NB <= 4 && a.tile_rows == 32)
            e = launch(attn_tile_kernel<CT, NB, XB, TREE, NB <= 4 ? 32 : 64>, dim3((unsigned)grid),
                       dim3(64 * waves_of(CT, NB, XB, 32)), 0, s, a);
        else
            e = launch(attn_tile_kernel<CT, NB, XB, TREE, 64>, dim3((unsigned)grid), dim3(64 * waves_of(CT, NB, XB, 64)), 0, s, a);
    } else {
        e = launch(attn_tile_kernel<CT, NB, XB, TREE, kTileRows>, dim3((unsigned)grid),
                   dim3(64 * waves_of(CT, NB, XB, kTileRows)), 0, s, a);
    }
    return e != hipSuccess || !a.splits ? e : launch_attn_join(32 * NB, XB ? QMM_BF16 : QMM_F32, a, s);
}

template <int CT, int NB, bool TREE>
hipError_t tile_x(int xtype, const AttnArgs& a, hipStream_t s) {
    return xtype == QMM_BF16 ? tile_typed<CT, NB, true, TREE>(a, s) : tile_typed<CT, NB, false, TREE>(a, s);
}

}  // namespace

// Heads of up to 128 values, and wider ones: units of their own, so that they
// compile side by side.
template <int CT, bool TREE>
hipError_t launch_attn_tile_narrow(int head_dim, int xtype, const AttnArgs& a, hipStream_t s) {
    switch (head_dim) {
    case 64: return tile_x<CT, 2, TREE>(xtype, a, s);
    case 96: return tile_x<CT, 3, TREE>(xtype, a, s);
    case 128: return tile_x<CT, 4, TREE>(xtype, a, s);
    default: return hipErrorInvalidValue;
    }
}

template <int CT, bool TREE>
hipError_t launch_attn_tile_wide(int head_dim, int xtype, const AttnArgs& a, hipStream_t s) {
    switch (head_dim) {
    case 192: return tile_x<CT, 6, TREE>(xtype, a, s);
    case 256: return tile_x<CT, 8, TREE>(xtype, a, s);
    default: return hipErrorInvalidValue;
    }
}

}  // namespace qmm
