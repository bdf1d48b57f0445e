// attn_tree_q8_0.hip — attention for trees of new tokens over Q8_0 caches: as the
// split kernels (attn_split.h), with 32 query rows a workgroup instead of 16, so
// that a sequence's cache is read and unpacked half as often.
//
// A workgroup takes the rows of one row tile (tokens x the query heads of one
// key-value head, at most 32) and one split of the keys; its four waves take the
// split's tiles of 32 keys in turn, each by itself: no barrier until the end.
// Per tile, with 32x32x16 MFMAs:
//   S^T = K Q^T   A = 32 keys, B = the rows.  Lane (r, h) = (lane % 32, lane / 32)
//                 gets the scores of row r with 4 keys of each 8;
//   O^T += V^T P^T   B = P^T: the eight keys of a step that lane (r, h) holds the
//                 scores of; A = V^T with the keys in that order, rows being 32
//                 of 64 values: lane r reads the values 2r, 2r + 1 of 64 together,
//                 one for each of two products.
// The queries lie in LDS, which all waves read.
//
// Exactness: K's codes enter as they are, their block scales applied to fp32
// block scores; values, d code, as two fp16 parts, which hold them exactly
// (scaled_codes), times a power of two for each 32 values that keeps the largest
// so far below 2^15; queries and P in 16-bit parts as in the tile kernels.
//
// Bound: two waves a SIMD, whose vector work (some 590 instructions a tile, 2400
// cycles), LDS reads and products (40, 1280 cycles) overlap in part, beside the reading.
// One sequence of 295k keys, 8 heads of 128 (642 MB; read alone 117 us): 32 fp32 rows a
// head 183 us, 64 (two row tiles) 310.  With nothing multiplied the former took 147 us,
// with nothing loaded 140 (125 now).  The tile kernels in this form (64 rows staged in
// LDS, a half of the keys each) took 290 and 345 us, the split kernels 250 and 430.
// Operands read from LDS a step ahead and converted between the products: 200 -> 187 us.
// No change (2%): loads a whole tile ahead instead of half a one, loads straight to LDS,
// non-temporal ones, every load of a tile unconditional.  More rows a wave, which would
// unpack less often, do not fit beside another wave: 253 registers of 256.
#include "attn_common.h"

namespace qmm {
namespace {

constexpr int kTreeWaves = 4, kRows = 32;

typedef uint16_t us2 __attribute__((ext_vector_type(2)));

__device__ __forceinline__ f16v mfma32(u4v a, u4v b, f16v c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(half8v, a), __builtin_bit_cast(half8v, b), c, 0, 0, 0);
}

template <int NB, bool XB>
__global__ __launch_bounds__(256, 2) void attn_tree_kernel(AttnArgs a) {
    constexpr int D = 32 * NB, RB = kv_row_bytes(QMM_Q8_0, D), STEPS = D / 16, PAIRS = D / 64;
    constexpr int QP = XB ? 1 : 2, PP = 2, AP = 2;  // parts of Q, P and V
    static_assert(NB % 2 == 0, "values come in runs of 64");
    // LDS: the queries and the waves' staging regions, then 64 values of the waves' parts at a time
    constexpr int RAW = 32 * RB, STAGE = RAW + 32 * NB * 4;
    constexpr int Q_BYTES = STEPS * QP * 64 * 16, PARTS_BYTES = kTreeWaves * kRows * 68 * 4;
    constexpr int USED_BYTES = Q_BYTES + kTreeWaves * STAGE;
    __shared__ __attribute__((aligned(16))) uint8_t smem[PARTS_BYTES > USED_BYTES ? PARTS_BYTES : USED_BYTES];
    u4v(*s_q)[QP][64] = reinterpret_cast<u4v(*)[QP][64]>(smem);
    const int groups = a.c.n_kv * a.chunks, item = (int)(blockIdx.x / groups), hb = blockIdx.x % groups;
    Work w;
    if (!find_work<true>(a, item, w)) return;
    const TileAt at = w.at;
    const int lane = threadIdx.x & 63, r = lane & 31, h = lane >> 5;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int kvh = hb / a.chunks, G = a.n_q / a.c.n_kv;
    const int head0 = kvh * G + (hb % a.chunks) * a.chunk;
    const int heads = min(a.chunk, kvh * G + G - head0);
    const int rows = min(kRows, at.tokens * heads);
    const int mr = min(r, rows - 1), mt = mr / heads, head = head0 + mr % heads;
    const TreeRow tree = tree_row(a, at, mt);

    // ---- the tiles of this split
    const int n_pre = (at.pre + 31) >> 5;
    const int w0 = max(n_pre, at.low >> 5), w1 = (at.end + 31) >> 5;
    const int n_tiles = n_pre + max(0, w1 - w0);
    const int per = (n_tiles + w.splits - 1) / w.splits;
    const int t0 = w.split * per, t1 = min(n_tiles, t0 + per);
    const int low_last = a.window > 0 ? max(at.kv, 0) - a.window : INT32_MIN;  // every row sees keys from here
    // or up to here by the prefix; new tokens are looked at one by one where slopes go by their positions
    const int pre_see = a.slopes ? min(at.pre, at.base) : at.pre;

    // ---- where the wave's tiles lie, as in the split kernels
    int64_t my_row = -1;
    struct Where {
        int64_t r0[2];
        int kb;      // first key of the tile
        bool whole;  // every row sees all of its keys, which stand at their indexes
    };
    auto place = [&](int t) {
        Where x;
        const int nth = ((t - t0 - wave) / kTreeWaves) & 31;
        if (nth == 0) {
            const int tt = t + kTreeWaves * (lane >> 1);
            const int64_t key = 32 * (int64_t)(tt < n_pre ? tt : tt - n_pre + w0) + 16 * (lane & 1);
            my_row = -1;
            if (tt < t1 && key < at.len) {
                const int pidx = (int)key / a.c.page_size;
                const int pg = a.c.table[(int64_t)at.s * a.c.table_width + pidx];
                if (pg >= 0 && pg < a.c.n_pages)
                    my_row = ((int64_t)pg * a.c.n_kv + kvh) * a.c.page_size + ((int)key - pidx * a.c.page_size);
            }
        }
#pragma unroll
        for (int u = 0; u < 2; ++u)
            x.r0[u] = (int64_t)((uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)my_row, 2 * nth + u) |
                                (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(my_row >> 32), 2 * nth + u) << 32);
        x.kb = 32 * (t < n_pre ? t : t - n_pre + w0);
        x.whole = x.r0[0] >= 0 && x.r0[1] >= 0 &&
                  ((x.kb + 32 <= pre_see) || (x.kb >= low_last && x.kb + 32 <= min(at.len, at.base)));
        return x;
    };
    int t = t0 + wave;
    Where now = {{-1, -1}, 0, false}, next = now;  // behind the last tile: row 0 of the cache
    if (t < t1) now = place(t);

    // ---- the queries, as B operands in LDS: lane (r, h) holds eight values of
    // each step, 2 further on in the blocks whose codes are read from the third on
    float qs;  // what a score is multiplied by, positive
    {
        const int64_t base = (int64_t)(at.row + mt) * a.ldq + (int64_t)head * D;
        auto shift = [](int s) { return s / 2 % 2 == 0 ? 2 : 0; };
        auto pair = [&](int s, int i) {
            const int e = 32 * (s / 2) + ((16 * (s & 1) + 8 * h + 2 * i + shift(s)) & 31);
            float2 x;
            if constexpr (XB) {
                const uint32_t w = *reinterpret_cast<const uint32_t*>(static_cast<const uint16_t*>(a.q) + base + e);
                x.x = bf16_lo(w), x.y = bf16_hi(w);
            } else {
                x = *reinterpret_cast<const float2*>(static_cast<const float*>(a.q) + base + e);
            }
            return x;
        };
        float big = 0.f;  // (twice over the row: the second time from L1)
#pragma unroll
        for (int s = 0; s < STEPS; ++s)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 x = pair(s, i);
                big = fmaxf(big, fmaxf(fabsf(x.x), fabsf(x.y)));
            }
        big = fmaxf(big, __shfl_xor(big, 32));
        int ex = 0;
        frexpf(big, &ex);
        ex = min(max(ex, -110), 126);  // an all-zero row: any finite scale does
        constexpr int TOP = 14;
        const float up = copysignf(ldexpf(1.0f, TOP - ex), a.scale);  // the sign of the scale goes to the queries
        qs = ldexpf(1.0f, ex - TOP) * fabsf(a.scale);
        // a wave writes every fourth step
        for (int s = wave; s < STEPS; s += kTreeWaves) {
            u4v q[QP];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 x = pair(s, i);
                uint32_t part[QP];
                split_pair<false, QP>(x.x * up, x.y * up, part);
#pragma unroll
                for (int k = 0; k < QP; ++k) q[k][i] = part[k];
            }
#pragma unroll
            for (int k = 0; k < QP; ++k) s_q[s][k][lane] = q[k];
        }
    }
    __syncthreads();
    const bool capped = a.softcap > 0.f;
    if (!capped) qs *= kLog2e;
    qs = fmaxf(qs, 0x1p-120f);  // never 0: masked scores stay -inf times it
    const float slope = a.slopes ? a.slopes[head] * kLog2e : 0.f;
    const int reach = a.window > 0 ? a.window : INT32_MAX;

    f16v o[PAIRS][2];
#pragma unroll
    for (int c = 0; c < PAIRS; ++c)
#pragma unroll
        for (int i = 0; i < 16; ++i) o[c][0][i] = o[c][1][i] = 0.f;
    float mx = -INFINITY, mref = 0.f, l = 0.f;

    // whether any row sees the key in half u of the tile: others may hold anything, and count as 0
    auto kept = [&](int u, int key) {
        return (key < at.len) & ((u ? now.r0[1] : now.r0[0]) >= 0) & (((key < at.end) & (key >= at.low)) | (key < at.pre));
    };
    // key i of the lane's scores, in the tile
    auto key_of = [&](int i) { return 8 * (i >> 2) + 4 * h + (i & 3); };

    float one = 1.0f;
    asm("" : "+v"(one));  // (a product with it and a difference are one instruction on mixed types, if it is no constant)
    // ---- one tile's scores to P: products in, p out; raises the running maximum where needed
    auto soften = [&](float (&sc)[16]) {
        float f = qs;
        if (!now.whole && capped) {  // the scores of masked keys may be anything
#pragma unroll
            for (int i = 0; i < 16; ++i) sc[i] = kept(i >> 3, now.kb + key_of(i)) ? sc[i] : 0.f;
        }
        if (capped) {
            cap_scores(sc, f, a.softcap);
            f = 1.0f;
        }
        auto place_of = [&](int key) { return now.whole ? key : tree_place(at, tree, key); };
        if (a.slopes) {
#pragma unroll
            for (int i = 0; i < 16; ++i) sc[i] = sc[i] * f - slope * fabsf((float)(tree.pos - place_of(now.kb + key_of(i))));
            f = 1.0f;
        }
        if (!now.whole) {
            const uint32_t bits = (uint32_t)(tree_bits(a, at, tree, now.kb) >> (4 * h));
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const int key = now.kb + key_of(i);
                const bool near = (bits >> (8 * (i >> 2) + (i & 3)) & 1) & (a.window <= 0 || tree.pos - place_of(key) < reach);
                const bool seen = (key < at.len) & (now.r0[i >> 3] >= 0) & (near | (key < at.pre));
                sc[i] = seen ? sc[i] : -INFINITY;
            }
        }
        float big = sc[0];
#pragma unroll
        for (int i = 1; i < 16; ++i) big = fmaxf(big, sc[i]);
        if (__any(big * f > mx + kSlack)) {
            big = fmaxf(big, __shfl_xor(big, 32)) * f;
            const float top = fmaxf(mx, big), ref = top == -INFINITY ? 0.f : top;
            const float down = __builtin_amdgcn_exp2f(mx - ref);  // 0 from -inf
            mx = top;
            mref = ref - p_top<false>();
            l *= down;
#pragma unroll
            for (int c = 0; c < PAIRS; ++c) o[c][0] *= down, o[c][1] *= down;
        }
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            sc[i] = __builtin_amdgcn_exp2f(fmaf(sc[i], f, -mref));
            l += sc[i];
        }
    };
    // P of step kk as B operands
    static_assert(PP == 2, "two parts of P");
    auto p_operand = [&](const float (&sc)[16], int kk, u4v (&pf)[PP]) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            // the value rounded, and what that leaves, rounded
            const float x = sc[8 * kk + 2 * i], y = sc[8 * kk + 2 * i + 1];
            half2v hi = {(_Float16)x, (_Float16)y}, lo;
            uint32_t w = __builtin_bit_cast(uint32_t, hi);
            asm("" : "+v"(w));
            hi = __builtin_bit_cast(half2v, w);
            lo.x = (_Float16)fmaf(x, one, -(float)hi.x), lo.y = (_Float16)fmaf(y, one, -(float)hi.y);
            pf[0][i] = w, pf[1][i] = __builtin_bit_cast(uint32_t, lo);
        }
    };

    // 2^vex is above every |d| so far of a block of values: lanes from 32 h on hold the blocks 2 j + h.  (An array of all
    // blocks, chosen from by h, goes to LDS by the lane's number in the workgroup, for which the compiler reads the
    // dispatch packet in host memory: 10 us a launch.)
    int vex[NB / 2];
#pragma unroll
    for (int j = 0; j < NB / 2; ++j) vex[j] = -30;

    {
        // Staged through LDS as in the split kernels, the keys of a tile and then
        // its values: raw blocks, and their scales by block and key (fp32 ones for
        // the scores; for the values times the blocks' powers of two, in fp16).
        constexpr int PIECES = 34 * NB;                // 16-byte pieces of 16 keys
        constexpr int LOADS = (2 * PIECES + 63) / 64;  // of a lane, for 32 keys
        constexpr int DL = NB / 2;                     // scales of a lane
        uint8_t* raw = smem + Q_BYTES + wave * STAGE;
        uint8_t* tab = raw + RAW;
        // Loads are under way for a whole tile's time: keys and values have registers of their own.
        u4v in_k[LOADS], in_v[LOADS];
        uint32_t din[DL];
        const int dkey = lane & 31, dblk = lane >> 5;
        const uint8_t* dsrc = raw + dkey * RB + dblk * kQ8_0Bytes;
        auto settle = [&]() {  // LDS written by the wave's lanes, read by others of them
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            __builtin_amdgcn_wave_barrier();
        };
        auto load = [&](const uint8_t* base, const Where& x, u4v (&in)[LOADS]) {
            const uint8_t* h0 = base + max(x.r0[0], (int64_t)0) * RB;
            const uint8_t* h1 = base + max(x.r0[1], (int64_t)0) * RB - 16 * PIECES;
#pragma unroll
            for (int j = 0; j < LOADS; ++j) {
                const uint32_t i = lane + 64 * j;
                if (64 * j + 63 < 2 * PIECES || i < 2 * PIECES)
                    in[j] = *reinterpret_cast<const u4v*>((i < PIECES ? h0 : h1) + 16 * i);
            }
        };
        auto stage = [&](const u4v (&in)[LOADS]) {
#pragma unroll
            for (int j = 0; j < LOADS; ++j) {
                const uint32_t i = lane + 64 * j;
                if (64 * j + 63 < 2 * PIECES || i < 2 * PIECES) *reinterpret_cast<u4v*>(raw + 16 * i) = in[j];
            }
            settle();
#pragma unroll
            for (int j = 0; j < DL; ++j) din[j] = *reinterpret_cast<const uint16_t*>(dsrc + 2 * j * kQ8_0Bytes);
        };
        const uint32_t patch = h == 1 ? 0x07060100u : 0x03020100u;
        if (t < t1) {
            load(a.c.k, now, in_k);
            load(a.c.v, now, in_v);
        }
        for (; t < t1; t += kTreeWaves) {
            stage(in_k);
            next = place(t + kTreeWaves);
            load(a.c.k, next, in_k);
#pragma unroll
            for (int j = 0; j < DL; ++j) reinterpret_cast<float*>(tab)[32 * (dblk + 2 * j) + dkey] = h2f(din[j]);
            settle();
            // ---- scores.  Operands are read from LDS a step before they are multiplied, and converted between the
            // products of the step before; a block's scales are applied between the next one's.
            float sc[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) sc[i] = 0.f;
            {
                struct Step {
                    uint2 w;
                    uint32_t first;  // of the block: its last two codes' place is taken by the first two
                    u4v q[QP];
                };
                auto read = [&](int s, Step& x) {
                    // Codes begin 2 bytes behind a multiple of 4 in every other block: there lane h takes the 8 from 2
                    // on (as its queries do), and the last one the block's first two for what lies behind its end.
                    const int b = s / 2;
                    const uint8_t* blk = raw + r * RB + b * kQ8_0Bytes;
                    const uint32_t* p = reinterpret_cast<const uint32_t*>(blk + (b % 2 ? 2 : 4) + 16 * (s & 1) + 8 * h);
                    x.w.x = p[0], x.w.y = p[1];
                    if (b % 2 == 0 && s % 2 == 1) x.first = *reinterpret_cast<const uint32_t*>(blk);
#pragma unroll
                    for (int k = 0; k < QP; ++k) x.q[k] = s_q[s][k][lane];
                };
                auto operand = [&](int s, const Step& x) {
                    uint2 w = x.w;
                    if (s / 2 % 2 == 0 && s % 2 == 1) w.y = __builtin_amdgcn_perm(x.first, w.y, patch);
                    return codes8_f16(w);
                };
                Step st[2];
                f16v acc[2];
                f4v d[4];
                u4v kf, kn;
                read(0, st[0]);
                read(1, st[1]);
                kf = operand(0, st[0]);
#pragma unroll
                for (int s = 0; s < STEPS; ++s) {
                    const int b = s / 2;
#pragma unroll
                    for (int k = QP - 1; k >= 0; --k) {
                        if (s % 2 == 0 && k == QP - 1) {
                            f16v zero;
#pragma unroll
                            for (int i = 0; i < 16; ++i) zero[i] = 0.f;
                            acc[b & 1] = mfma32(kf, st[s & 1].q[k], zero);
                        } else {
                            acc[b & 1] = mfma32(kf, st[s & 1].q[k], acc[b & 1]);
                        }
                    }
                    if (s + 1 < STEPS) kn = operand(s + 1, st[(s + 1) & 1]);
                    if (s % 2 == 0 && b > 0) {
#pragma unroll
                        for (int i = 0; i < 16; ++i) sc[i] = fmaf(acc[(b & 1) ^ 1][i], d[i / 4][i % 4], sc[i]);
                    }
                    if (s % 2 == 1) {
#pragma unroll
                        for (int i = 0; i < 4; ++i) d[i] = *reinterpret_cast<const f4v*>(tab + 128 * b + 32 * i + 16 * h);
                    }
                    if (s + 2 < STEPS) read(s + 2, st[s & 1]);
                    kf = kn;
                    __builtin_amdgcn_sched_barrier(0);
                }
#pragma unroll
                for (int i = 0; i < 16; ++i) sc[i] = fmaf(acc[(NB & 1) ^ 1][i], d[i / 4][i % 4], sc[i]);
            }
            soften(sc);
            // ---- O^T += V^T P^T
            settle();
            stage(in_v);
            {
                bool grow = false;
                float d[DL];
                int ex[DL];
#pragma unroll
                for (int j = 0; j < DL; ++j) {
                    if (!now.whole) din[j] = kept(dkey >> 4, now.kb + dkey) ? din[j] : 0;
                    d[j] = h2f(din[j]);
                    float big = fabsf(d[j]);  // of 32 lanes
                    big = fmaxf(big, dpp<0xB1>(big));   // lane ^ 1
                    big = fmaxf(big, dpp<0x4E>(big));   // lane ^ 2
                    big = fmaxf(big, dpp<0x141>(big));  // 7 - lane, of each 8
                    big = fmaxf(big, dpp<0x140>(big));  // 15 - lane, of each 16
                    big = fmaxf(big, __shfl_xor(big, 16));
                    // (fp16 numbers are no subnormals in fp32)
                    ex[j] = max(vex[j], min((__builtin_bit_cast(int, big) >> 23) - 126, 16));
                    grow |= ex[j] > vex[j];
                }
                if (__any(grow)) {
#pragma unroll
                    for (int b = 0; b < NB; ++b) {
                        const float down = ldexpf(1.0f, __builtin_amdgcn_readlane(vex[b / 2] - ex[b / 2], 32 * (b % 2)));
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            o[b / 2][0][8 * (b % 2) + i] *= down, o[b / 2][1][8 * (b % 2) + i] *= down;
                    }
                }
#pragma unroll
                for (int j = 0; j < DL; ++j) {
                    vex[j] = ex[j];
                    reinterpret_cast<_Float16*>(tab)[32 * (dblk + 2 * j) + dkey] = (_Float16)(d[j] * ldexpf(1.0f, 15 - ex[j]));
                }
            }
            settle();
            load(a.c.v, next, in_v);
            {
                // group g: the keys of a step, 64 values
                struct Group {
                    uint32_t w[4];
                    uint2 d[2];
                };
                auto read = [&](int g, Group& x) {
                    const int kk = g / PAIRS, c = g % PAIRS;
                    const uint8_t* v = raw + (16 * kk + 4 * h) * RB + (2 * c + (r >> 4)) * kQ8_0Bytes + 2 + 2 * (r & 15);
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const uint8_t* p = v + (8 * (j >> 1) + 2 * (j & 1)) * RB;
                        const us2 two = {*reinterpret_cast<const uint16_t*>(p), *reinterpret_cast<const uint16_t*>(p + RB)};
                        x.w[j] = __builtin_bit_cast(uint32_t, two);
                    }
#pragma unroll
                    for (int j = 0; j < 2; ++j)
                        x.d[j] = *reinterpret_cast<const uint2*>(tab + 64 * (2 * c + (r >> 4)) + 32 * kk + 16 * j + 8 * h);
                };
                auto operand = [&](const Group& x, u4v (&vf)[2][AP]) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const uint32_t w = x.w[j] ^ 0x80808080u;
                        const half2v d = __builtin_bit_cast(half2v, (uint32_t)(j & 1 ? x.d[j >> 1].y : x.d[j >> 1].x));
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            uint32_t part[2];
                            scaled_codes(__builtin_amdgcn_perm(0x48484848u, w, 0x04020400u + 0x00010001u * e), d, part);
                            vf[e][0][j] = part[0], vf[e][AP - 1][j] = part[1];
                        }
                    }
                };
                Group gr[2];
                u4v vf[2][2][AP], pf[2][PP];
                read(0, gr[0]);
                read(1, gr[1]);
                p_operand(sc, 0, pf[0]);
                operand(gr[0], vf[0]);
#pragma unroll
                for (int g = 0; g < 2 * PAIRS; ++g) {
                    const int kk = g / PAIRS, c = g % PAIRS;
#pragma unroll
                    for (int ap = AP - 1; ap >= 0; --ap)
#pragma unroll
                        for (int k = (ap ? 0 : PP - 1); k >= 0; --k)
#pragma unroll
                            for (int e = 0; e < 2; ++e) o[c][e] = mfma32(vf[g & 1][e][ap], pf[kk][k], o[c][e]);
                    if (g + 1 < 2 * PAIRS) operand(gr[(g + 1) & 1], vf[(g + 1) & 1]);
                    if (kk == 0 && c == PAIRS - 1) p_operand(sc, 1, pf[1]);
                    if (g + 2 < 2 * PAIRS) read(g + 2, gr[g & 1]);
#pragma unroll
                    for (int i = 0; i < 6; ++i) {
                        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);  // a product, and what fits beside it
                        __builtin_amdgcn_sched_group_barrier(0x002, 8, 0);
                    }
                    __builtin_amdgcn_sched_barrier(0);
                }
            }
            settle();
            now = next;
        }
    }

    // ---- the four waves' parts, 64 values of a row at a time
    l += __shfl_xor(l, 32);
#pragma unroll
    for (int b = 0; b < NB; ++b) {
        const float unit = ldexpf(1.0f, __builtin_amdgcn_readlane(vex[b / 2], 32 * (b % 2)) - 8);
#pragma unroll
        for (int i = 0; i < 8; ++i) o[b / 2][0][8 * (b % 2) + i] *= unit, o[b / 2][1][8 * (b % 2) + i] *= unit;
    }
    float(*s_o)[kRows][68] = reinterpret_cast<float(*)[kRows][68]>(smem);
    __shared__ float s_m[kTreeWaves][kRows], s_l[kTreeWaves][kRows];
    if (h == 0) s_m[wave][r] = mx, s_l[wave][r] = l;
#pragma unroll
    for (int c = 0; c < PAIRS; ++c) {
        __syncthreads();
        // rows 8 j + 4 h .. + 3 of both products: eight values one after another, from 2 (8 j + 4 h) on
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int i = 0; i < 2; ++i)
                *reinterpret_cast<f4v*>(&s_o[wave][r][16 * j + 8 * h + 4 * i]) =
                    f4v{o[c][0][4 * j + 2 * i], o[c][1][4 * j + 2 * i], o[c][0][4 * j + 2 * i + 1], o[c][1][4 * j + 2 * i + 1]};
        __syncthreads();
        for (int i = threadIdx.x; i < rows * 16; i += 256) {
            const int m = i / 16, e = 4 * (i % 16);
            float top = -INFINITY;
#pragma unroll
            for (int w = 0; w < kTreeWaves; ++w) top = fmaxf(top, s_m[w][m]);
            f4v sum = {0.f, 0.f, 0.f, 0.f};
            float den = 0.f;
#pragma unroll
            for (int w = 0; w < kTreeWaves; ++w) {
                const float f = top == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(s_m[w][m] - top);
                den += f * s_l[w][m];
                sum += f * *reinterpret_cast<const f4v*>(&s_o[w][m][e]);
            }
            const int64_t row = (int64_t)(at.row + m / heads) * a.n_q + head0 + m % heads;
            const int at_e = 64 * c + e;
            if (a.splits && at_e == 0 && w.split == 0)
                join_of(a)[row] = JoinOf{w.first, w.splits > 1 ? w.splits : 0, w.step, hb * a.slots + m};
            if (w.splits > 1) {
                const int64_t part = ((int64_t)item * groups + hb) * a.slots + m;
                float* ml = a.work + a.parts * D;
                if (at_e == 0) ml[2 * part] = top, ml[2 * part + 1] = den;
                *reinterpret_cast<f4v*>(a.work + part * D + at_e) = sum;
            } else {
                const float inv = den > 0.f ? 1.0f / den : den == 0.f ? 0.f : den;  // NaN stays
                sum *= inv;
                if constexpr (XB) {
                    bf2v x, y;
                    x.x = (__bf16)sum[0], x.y = (__bf16)sum[1], y.x = (__bf16)sum[2], y.y = (__bf16)sum[3];
                    uint2 w2;
                    w2.x = __builtin_bit_cast(uint32_t, x), w2.y = __builtin_bit_cast(uint32_t, y);
                    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + row * D + at_e) = w2;
                } else {
                    *reinterpret_cast<f4v*>(static_cast<float*>(a.out) + row * D + at_e) = sum;
                }
            }
        }
    }
}

template <int NB, bool XB>
hipError_t tree_typed(const AttnArgs& a, hipStream_t s) {
    const int64_t grid = a.items * a.c.n_kv * a.chunks;  // below 2^32 work-items
    hipError_t e = launch(attn_tree_kernel<NB, XB>, dim3((unsigned)grid), dim3(256), 0, s, a);
    return e != hipSuccess || !a.splits ? e : launch_attn_join(32 * NB, XB ? QMM_BF16 : QMM_F32, a, s);
}

template <int NB>
hipError_t tree_x(int xtype, const AttnArgs& a, hipStream_t s) {
    return xtype == QMM_BF16 ? tree_typed<NB, true>(a, s) : tree_typed<NB, false>(a, s);
}

}  // namespace

hipError_t launch_attn_tree_q8_0(int head_dim, int xtype, const AttnArgs& a, hipStream_t s) {
    switch (head_dim) {
    case 64: return tree_x<2>(xtype, a, s);
    case 128: return tree_x<4>(xtype, a, s);
    default: return hipErrorInvalidValue;
    }
}

}  // namespace qmm
