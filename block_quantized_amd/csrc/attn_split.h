// attn_split.h — attention over a paged cache for few query rows a
// sequence: the cache is read once, its length split over waves and
// workgroups, and the parts joined.
//
// A workgroup takes the query rows of one row tile (at most 16: tokens x the
// query heads of one key-value head) and one split of the keys; its four
// waves take the split's tiles of 32 keys in turn.  Per tile, with 16x16x32
// MFMAs:
//   S^T = K Q^T   A = 16 keys, B = the rows.  Lane (m, g) = (lane % 16,
//                 lane / 16) gets the scores of row m with the keys 4g..4g+3
//                 of both 16-key halves;
//   O^T += V^T P^T   B = P^T: row m's eight keys of lane (m, g), exactly what
//                 the lane holds, since the order of the contracted keys is
//                 free; A = V^T with the keys in that order: lane m holds the
//                 values 2m, 2m+1 of a 32-value block for these eight keys.
// So scores never leave their lane, a row's rescaling is the lane's own, and
// lane (m, g) ends with the eight consecutive values 8g..8g+7 of each block.
//
// Exactness: the cache's values enter the MFMAs as they are (fp16 and bf16
// rows; Q8_0 codes as fp16 integers for K, as bf16 ones for V, their block scales
// applied to the fp32 block scores, and to P before it is split).  Queries and P
// are split into 16-bit parts that hold 22 bits (two of fp16) or 24 (three of
// bf16).  bf16 parts have fp32's range, and so take the P d of Q8_0 rows, whose
// sizes go by the cache.  (In two fp16 parts, kept below 2^15 by one power of two a
// wave, they took 325 us instead of 340 for 64 of 8k to 16k keys, but a block whose
// d was 2^20 below another's kept 12 bits.)  Where parts are fp16, queries are
// scaled by a power of two per row so that their largest value is about 2^14, and P
// is 2^14 p: what is more than 2^16 below a row's largest is held to 2^-38 of that,
// the parts' smallest step.
//
// Bound: reading the cache.  fp32 queries, 32 heads, of 128 values, on 8 of the
// cache's: one sequence of 131k keys in Q8_0 (285 MB) 64 us, 4.5 TB/s; 64 of
// 8k to 16k (1714 MB) 314-371 us, 4.6-5.5; 13 of 750 to 1500 in bf16, each head
// with its own (244 MB) 42 us, 5.8; 32 of 2k to 4k, 256-wide in fp16 with bf16
// queries (814 MB) 153 us, 5.3.  A read of 1 GiB that computes nothing reaches
// 5.5.  In Q8_0 the vector unit is busy for 72% of the time (codes to 16 bits, P d
// split).  Slower, each against its time then: loads past the caches (172 us for
// the last), unaligned loads of whole blocks with transposing LDS reads (418 ->
// 468), all products before all scales (254 -> 277), four waves a SIMD (spills).
#pragma once

#include "attn_common.h"

namespace qmm {
namespace {

constexpr int kWaves = 4;

__device__ __forceinline__ uint32_t ld16(const uint8_t* p) { return *reinterpret_cast<const uint16_t*>(p); }

// Q8_0: LDS bytes of a wave's 32 keys or values, blocks and their scales.
template <int NB>
constexpr int kStage = 32 * 34 * NB + 64 * NB;

template <int CT, int NB, bool XB>
__global__ __launch_bounds__(256, NB <= 4 ? 3 : 2) void attn_split_kernel(AttnArgs a) {
    constexpr int D = 32 * NB, RB = kv_row_bytes(CT, D);
    // the parts of P, and those of Q, with the MFMAs that take them
    constexpr bool BF = CT != QMM_F16, Q8 = CT == QMM_Q8_0, QBF = CT == QMM_BF16;
    constexpr int PP = BF ? 3 : 2, QP = QBF ? 3 : 2;
    // LDS: the queries and the waves' staging regions, then the waves' parts
    constexpr int PARTS_BYTES = kWaves * 16 * (D + 4) * 4, Q_BYTES = NB * QP * 64 * 16;
    constexpr int USED_BYTES = Q_BYTES + (Q8 ? kWaves * kStage<NB> : 0);
    __shared__ __attribute__((aligned(16))) uint8_t smem[PARTS_BYTES > USED_BYTES ? PARTS_BYTES : USED_BYTES];
    u4v(*s_q)[QP][64] = reinterpret_cast<u4v(*)[QP][64]>(smem);
    const int groups = a.c.n_kv * a.chunks, item = (int)(blockIdx.x / groups), hb = blockIdx.x % groups;
    Work w;
    if (!find_work(a, item, w)) return;
    const TileAt at = w.at;
    const int lane = threadIdx.x & 63, m = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int kvh = hb / a.chunks, G = a.n_q / a.c.n_kv;
    const int head0 = kvh * G + (hb % a.chunks) * a.chunk;  // first query head of the tile
    const int heads = min(a.chunk, kvh * G + G - head0);
    // row m of the tile: token m / heads, head m % heads
    const int rows = min(16, at.tokens * heads);
    const int mr = min(m, rows - 1), mt = mr / heads, head = head0 + mr % heads;
    const int p_row = at.pos + mt;

    // ---- the tiles of this split
    const int n_pre = (at.pre + 31) >> 5;
    const int w0 = max(n_pre, at.low >> 5), w1 = (at.end + 31) >> 5;
    const int n_tiles = n_pre + max(0, w1 - w0);
    const int per = (n_tiles + w.splits - 1) / w.splits;
    const int t0 = w.split * per, t1 = min(n_tiles, t0 + per);
    // every row sees keys from here (no index less a window passes 32 bits from 0 on; rows below it see none)
    const int low_last = a.window > 0 ? max(at.pos + at.tokens, 0) - a.window : INT32_MIN;

    // ---- where the wave's tiles lie.  Lane i holds the cache row of 16 keys:
    // half i % 2 of the i / 2-th tile from the last lookup on; -1: no page
    int64_t my_row = -1;
    int64_t r0[2];
    int kb = 0;          // first key of the tile last placed
    bool whole = false;  // every row sees all of its keys
    auto place = [&](int t) {
        const int nth = ((t - t0 - wave) / kWaves) & 31;
        if (nth == 0) {
            const int tt = t + kWaves * (lane >> 1);
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
            r0[u] = (int64_t)((uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)my_row, 2 * nth + u) |
                              (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(my_row >> 32), 2 * nth + u) << 32);
        kb = 32 * (t < n_pre ? t : t - n_pre + w0);
        whole = r0[0] >= 0 && r0[1] >= 0 &&
                ((kb + 32 <= at.pre) || (kb >= low_last && kb + 32 <= min(at.len, at.pos + 1)));
    };
    // the first lookup is under way while the queries are prepared
    int t = t0 + wave;
    if (t < t1) place(t);

    // ---- the queries, as B operands in LDS (the waves', one quarter of the
    // blocks written by each): lane (m, g) holds the values 8g..8g+7 of each block
    float qs;  // what a score is multiplied by
    {
        float x[NB][8];
        const int64_t base = (int64_t)(at.row + mt) * a.ldq + (int64_t)head * D;
        float big = 0.f;
#pragma unroll
        for (int b = 0; b < NB; ++b) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                // pairs, since the codes of some Q8_0 blocks are taken from the third on
                const int e = 32 * b + ((8 * g + 2 * i + (Q8 && NB % 2 == 0 && b % 2 == 0 ? 2 : 0)) & 31);
                if constexpr (XB) {
                    const uint32_t w = *reinterpret_cast<const uint32_t*>(static_cast<const uint16_t*>(a.q) + base + e);
                    x[b][2 * i] = bf16_lo(w), x[b][2 * i + 1] = bf16_hi(w);
                } else {
                    const float2 w = *reinterpret_cast<const float2*>(static_cast<const float*>(a.q) + base + e);
                    x[b][2 * i] = w.x, x[b][2 * i + 1] = w.y;
                }
                big = fmaxf(big, fmaxf(fabsf(x[b][2 * i]), fabsf(x[b][2 * i + 1])));
            }
        }
        big = fmaxf(big, __shfl_xor(big, 16));
        big = fmaxf(big, __shfl_xor(big, 32));
        int ex = 0;
        frexpf(big, &ex);
        ex = min(max(ex, -110), 126);  // an all-zero row: any finite scale does
        constexpr int TOP = QBF ? 0 : 14;  // (bf16 parts have fp32's range)
        const float up = ldexpf(1.0f, TOP - ex);
        qs = ldexpf(1.0f, ex - TOP) * a.scale;
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            if ((b & 3) != wave) continue;
            u4v q[QP];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                uint32_t part[QP];
                split_pair<QBF, QP>(x[b][2 * i] * up, x[b][2 * i + 1] * up, part);
#pragma unroll
                for (int k = 0; k < QP; ++k) q[k][i] = part[k];
            }
#pragma unroll
            for (int k = 0; k < QP; ++k) s_q[b][k][lane] = q[k];
        }
    }
    __syncthreads();
    if (!(a.softcap > 0.f)) qs *= kLog2e;
    const float slope = a.slopes ? a.slopes[head] * kLog2e : 0.f;

    const int reach = a.window > 0 ? a.window : INT32_MAX;

    f4v o[NB][2];
#pragma unroll
    for (int b = 0; b < NB; ++b) o[b][0] = o[b][1] = f4v{0.f, 0.f, 0.f, 0.f};
    float mx = -INFINITY, mref = 0.f, l = 0.f;  // maximum, the same less p_top or 0, the lane's part of the sum

    // whether any row sees the key in half u of the tile: others may hold anything, and count as 0
    auto kept = [&](int u, int key) {
        return (key < at.len) & (r0[u] >= 0) & (((key < at.end) & (key >= at.low)) | (key < at.pre));
    };

    // ---- one tile's scores to P: sc in, p out; raises the running maximum where needed
    auto soften = [&](float (&sc)[8]) {
        if (!whole && a.softcap > 0.f) {  // the scores of masked keys may be anything
#pragma unroll
            for (int i = 0; i < 8; ++i) sc[i] = kept(i >> 2, kb + 16 * (i >> 2) + 4 * g + (i & 3)) ? sc[i] : 0.f;
        }
        if (a.softcap > 0.f) cap_scores(sc, 1.0f, a.softcap);
        if (a.slopes) {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                sc[i] -= slope * fabsf((float)(p_row - (kb + 16 * (i >> 2) + 4 * g + (i & 3))));
        }
        if (!whole) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int u = i >> 2, key = kb + 16 * u + 4 * g + (i & 3);
                // (without branches: ROCm 7.2's compiler keeps sc as one tuple of registers, and where the assignment
                // stood in nested branches it copied the tuple as it was before over it, with and without honoured NaNs)
                const bool seen =
                    (key < at.len) & (r0[u] >= 0) & (((key <= p_row) & (p_row - key < reach)) | (key < at.pre));
                sc[i] = seen ? sc[i] : -INFINITY;
            }
        }
        float big = fmaxf(fmaxf(fmaxf(sc[0], sc[1]), fmaxf(sc[2], sc[3])), fmaxf(fmaxf(sc[4], sc[5]), fmaxf(sc[6], sc[7])));
        if (__any(big > mx + kSlack)) {
            big = fmaxf(big, __shfl_xor(big, 16));
            big = fmaxf(big, __shfl_xor(big, 32));
            const float top = fmaxf(mx, big), ref = top == -INFINITY ? 0.f : top;
            const float down = __builtin_amdgcn_exp2f(mx - ref);  // 0 from -inf
            mx = top;
            mref = ref - p_top<BF>();
            l *= down;
#pragma unroll
            for (int b = 0; b < NB; ++b) o[b][0] *= down, o[b][1] *= down;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            sc[i] = __builtin_amdgcn_exp2f(sc[i] - mref);
            l += sc[i];
        }
    };

    if constexpr (Q8) {
        // Staged through LDS, a region of its own for each wave, the keys of a
        // tile and then its values: the raw blocks (a lane loads 16 consecutive
        // bytes at a time), and their scales once more, by block and key, so
        // that a lane finds its four keys' together.  (The scales come from LDS
        // too: a second load from memory would meet lines still under way.)
        // The values are loaded while the scores are computed, the next tile's
        // keys during V^T P^T: registers for one of the two serve both.
        constexpr int PIECES = 34 * NB;                // 16-byte pieces of 16 keys
        constexpr int LOADS = (2 * PIECES + 63) / 64;  // of a lane, for 32 keys
        constexpr int DL = (NB + 1) / 2;               // scales of a lane
        uint8_t* raw = smem + Q_BYTES + wave * kStage<NB>;
        uint8_t* tab = raw + 32 * PIECES;
        u4v in[LOADS];
        uint32_t din[DL];
        const int dkey = lane & 31, dblk = lane >> 5;
        const uint8_t* dsrc = raw + dkey * RB + dblk * kQ8_0Bytes;
        auto settle = [&]() {  // LDS written by the wave's lanes, read by others of them
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            __builtin_amdgcn_wave_barrier();
        };
        auto load = [&](const uint8_t* base) {
            const uint8_t* h0 = base + max(r0[0], (int64_t)0) * RB;
            const uint8_t* h1 = base + max(r0[1], (int64_t)0) * RB - 16 * PIECES;
#pragma unroll
            for (int j = 0; j < LOADS; ++j) {
                const uint32_t i = lane + 64 * j;
                if (64 * j + 63 < 2 * PIECES || i < 2 * PIECES)
                    in[j] = *reinterpret_cast<const u4v*>((i < PIECES ? h0 : h1) + 16 * i);
            }
        };
        auto stage = [&]() {
#pragma unroll
            for (int j = 0; j < LOADS; ++j) {
                const uint32_t i = lane + 64 * j;
                if (64 * j + 63 < 2 * PIECES || i < 2 * PIECES) *reinterpret_cast<u4v*>(raw + 16 * i) = in[j];
            }
            settle();
#pragma unroll
            for (int j = 0; j < DL; ++j)
                if (NB % 2 == 0 || dblk + 2 * j < NB) din[j] = ld16(dsrc + 2 * j * kQ8_0Bytes);
        };
        auto scales = [&]() {
#pragma unroll
            for (int j = 0; j < DL; ++j)
                if (NB % 2 == 0 || dblk + 2 * j < NB)
                    *reinterpret_cast<uint16_t*>(tab + 64 * (dblk + 2 * j) + 2 * dkey) = (uint16_t)din[j];
            settle();
        };
        const uint32_t patch = g == 3 ? 0x07060100u : 0x03020100u;
        if (t < t1) load(a.c.k);
        for (; t < t1; t += kWaves) {
            stage();
            load(a.c.v);
            scales();
            // ---- scores
            float sc[8];
            {
                f4v sum[2] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
#pragma unroll
                for (int b = 0; b < NB; ++b) {
                    u4v qf[QP];
#pragma unroll
                    for (int k = 0; k < QP; ++k) qf[k] = s_q[b][k][lane];
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        // Codes begin 2 bytes behind a multiple of 4 in every
                        // other block: there lane g takes the 8 from 8g + 2 on
                        // (as its queries do), and the last lane the block's
                        // first two for what lies behind its end.  Rows of an
                        // odd number of blocks shift by themselves.
                        const uint8_t* blk = raw + (16 * u + m) * RB + b * kQ8_0Bytes;
                        uint2 w;
                        if constexpr (NB % 2) {
                            __builtin_memcpy(&w, blk + 2 + 8 * g, 8);
                        } else {
                            const uint32_t* p = reinterpret_cast<const uint32_t*>(blk + (b % 2 ? 2 : 4) + 8 * g);
                            w.x = p[0], w.y = p[1];
                            if (b % 2 == 0) w.y = __builtin_amdgcn_perm(*reinterpret_cast<const uint32_t*>(blk), w.y, patch);
                        }
                        const u4v kf = codes8_f16(w);
                        f4v acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                        for (int k = QP - 1; k >= 0; --k) acc = mfma16<QBF>(kf, qf[k], acc);
                        const uint2 d = *reinterpret_cast<const uint2*>(tab + 64 * b + 32 * u + 8 * g);
                        sum[u][0] = fmaf(acc[0], h2f(d.x), sum[u][0]);
                        sum[u][1] = fmaf(acc[1], h2f(d.x >> 16), sum[u][1]);
                        sum[u][2] = fmaf(acc[2], h2f(d.y), sum[u][2]);
                        sum[u][3] = fmaf(acc[3], h2f(d.y >> 16), sum[u][3]);
                    }
                }
#pragma unroll
                for (int i = 0; i < 8; ++i) sc[i] = sum[i >> 2][i & 3] * qs;
            }
            soften(sc);
            // ---- O^T += V^T (P d)^T
            settle();
            stage();
            if (!whole) {
#pragma unroll
                for (int j = 0; j < DL; ++j)
                    if (NB % 2 == 0 || dblk + 2 * j < NB) din[j] = kept(dkey >> 4, kb + dkey) ? din[j] : 0;
            }
            scales();
            place(t + kWaves);  // behind the last tile, row 0 of the cache
            load(a.c.k);
#pragma unroll
            for (int b = 0; b < NB; ++b) {
                u4v pf[PP], vf[2];
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const uint2 d = *reinterpret_cast<const uint2*>(tab + 64 * b + 32 * u + 8 * g);
                    const uint8_t* v = raw + (16 * u + 4 * g) * RB + b * kQ8_0Bytes + 2 + 2 * m;
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const uint32_t dd = i ? d.y : d.x;
                        uint32_t part[PP];
                        split_pair<BF, PP>(sc[4 * u + 2 * i] * h2f(dd), sc[4 * u + 2 * i + 1] * h2f(dd >> 16), part);
#pragma unroll
                        for (int k = 0; k < PP; ++k) pf[k][2 * u + i] = part[k];
                        const uint32_t w = ld16(v + 2 * i * RB) | ld16(v + (2 * i + 1) * RB) << 16;
                        vf[0][2 * u + i] = codes_bf16<0, 2>(w);
                        vf[1][2 * u + i] = codes_bf16<1, 3>(w);
                    }
                }
#pragma unroll
                for (int j = 0; j < 2; ++j)
#pragma unroll
                    for (int k = PP - 1; k >= 0; --k) o[b][j] = mfma16<BF>(vf[j], pf[k], o[b][j]);
            }
            settle();
        }
    } else {
        // Rows of 16-bit floats are operands as they lie in memory (K), or after
        // an exchange of halves between registers (V).  Twelve waves a CU (eight
        // for wide heads) keep enough loads under way; loading a tile ahead took
        // the registers of a third of them, and was no faster.
        u4v kf[2][NB];
        uint32_t vw[2][4][NB];
        int64_t b0[2];
        const uint32_t koff = m * RB + 16 * g, voff = 4 * g * RB + 4 * m;
        auto load_k = [&]() {
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const uint8_t* kp = a.c.k + b0[u];  // uniform, and 32-bit offsets of the lanes
#pragma unroll
                for (int b = 0; b < NB; ++b) kf[u][b] = *reinterpret_cast<const u4v*>(kp + koff + 64 * b);
            }
        };
        auto load_v = [&]() {
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint8_t* vp = a.c.v + b0[u] + i * RB;
#pragma unroll
                    for (int b = 0; b < NB; ++b)
                        vw[u][i][b] = *reinterpret_cast<const uint32_t*>(vp + voff + 64 * b);
                }
        };
        for (; t < t1; t += kWaves) {
#pragma unroll
            for (int u = 0; u < 2; ++u) b0[u] = max(r0[u], (int64_t)0) * RB;
            load_k();
            load_v();
            float sc[8];
            f4v acc[2] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
#pragma unroll
            for (int k = QP - 1; k >= 0; --k)
#pragma unroll
                for (int b = 0; b < NB; ++b) {
                    const u4v qf = s_q[b][k][lane];
#pragma unroll
                    for (int u = 0; u < 2; ++u) acc[u] = mfma16<QBF>(kf[u][b], qf, acc[u]);
                }
#pragma unroll
            for (int i = 0; i < 8; ++i) sc[i] = acc[i >> 2][i & 3] * qs;
            if (!whole) {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const bool keep = kept(i >> 2, kb + 16 * (i >> 2) + 4 * g + (i & 3));
#pragma unroll
                    for (int b = 0; b < NB; ++b) vw[i >> 2][i & 3][b] = keep ? vw[i >> 2][i & 3][b] : 0;
                }
            }
            soften(sc);
            u4v pf[PP];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                uint32_t part[PP];
                split_pair<BF, PP>(sc[2 * i], sc[2 * i + 1], part);
#pragma unroll
                for (int k = 0; k < PP; ++k) pf[k][i] = part[k];
            }
#pragma unroll
            for (int b = 0; b < NB; ++b) {
                u4v vf[2];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint32_t x = vw[i >> 1][2 * (i & 1)][b], y = vw[i >> 1][2 * (i & 1) + 1][b];
                    vf[0][i] = __builtin_amdgcn_perm(y, x, 0x05040100u);
                    vf[1][i] = __builtin_amdgcn_perm(y, x, 0x07060302u);
                }
#pragma unroll
                for (int j = 0; j < 2; ++j)
#pragma unroll
                    for (int k = PP - 1; k >= 0; --k) o[b][j] = mfma16<BF>(vf[j], pf[k], o[b][j]);
            }
            place(t + kWaves);
        }
    }

    // ---- the four waves' parts: row m, values 8g..8g+7 of each block
    l += __shfl_xor(l, 16);
    l += __shfl_xor(l, 32);
    __syncthreads();
    float(*s_o)[16][D + 4] = reinterpret_cast<float(*)[16][D + 4]>(smem);
    __shared__ float s_m[kWaves][16], s_l[kWaves][16];
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 2; ++j) s_o[wave][m][32 * b + 8 * g + 2 * i + j] = o[b][j][i];
    if (g == 0) s_m[wave][m] = mx, s_l[wave][m] = l;
    __syncthreads();
    for (int i = threadIdx.x; i < rows * (D / 4); i += 256) {
        const int r = i / (D / 4), e = 4 * (i % (D / 4));
        float top = -INFINITY;
#pragma unroll
        for (int w = 0; w < kWaves; ++w) top = fmaxf(top, s_m[w][r]);
        f4v sum = {0.f, 0.f, 0.f, 0.f};
        float den = 0.f;
#pragma unroll
        for (int w = 0; w < kWaves; ++w) {
            const float f = top == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(s_m[w][r] - top);
            den += f * s_l[w][r];
            sum += f * *reinterpret_cast<const f4v*>(&s_o[w][r][e]);
        }
        const int64_t row = (int64_t)(at.row + r / heads) * a.n_q + head0 + r % heads;
        if (a.splits && e == 0 && w.split == 0)
            join_of(a)[row] = JoinOf{w.first, w.splits > 1 ? w.splits : 0, w.step, hb * a.slots + r};
        if (w.splits > 1) {
            const int64_t part = ((int64_t)item * groups + hb) * a.slots + r;
            float* ml = a.work + a.parts * D;
            if (e == 0) ml[2 * part] = top, ml[2 * part + 1] = den;
            *reinterpret_cast<f4v*>(a.work + part * D + e) = sum;
        } else {
            const float inv = den > 0.f ? 1.0f / den : den == 0.f ? 0.f : den;  // NaN stays
            sum *= inv;
            if constexpr (XB) {
                bf2v x, y;
                x.x = (__bf16)sum[0], x.y = (__bf16)sum[1], y.x = (__bf16)sum[2], y.y = (__bf16)sum[3];
                uint2 w;
                w.x = __builtin_bit_cast(uint32_t, x), w.y = __builtin_bit_cast(uint32_t, y);
                *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + row * D + e) = w;
            } else {
                *reinterpret_cast<f4v*>(static_cast<float*>(a.out) + row * D + e) = sum;
            }
        }
    }
}

template <int CT, int NB, bool XB>
hipError_t split_typed(const AttnArgs& a, hipStream_t s) {
    const int64_t grid = a.items * a.c.n_kv * a.chunks;  // below 2^32 work-items
    hipError_t e = launch(attn_split_kernel<CT, NB, XB>, dim3((unsigned)grid), dim3(256), 0, s, a);
    if (e != hipSuccess || !a.splits) return e;
    return launch_attn_join(32 * NB, XB ? QMM_BF16 : QMM_F32, a, s);
}

template <int CT, int NB>
hipError_t split_x(int xtype, const AttnArgs& a, hipStream_t s) {
    return xtype == QMM_BF16 ? split_typed<CT, NB, true>(a, s) : split_typed<CT, NB, false>(a, s);
}

}  // namespace

template <int CT>
hipError_t launch_attn_split_of(int head_dim, int xtype, const AttnArgs& a, hipStream_t s) {
    switch (head_dim) {
    case 64: return split_x<CT, 2>(xtype, a, s);
    case 96: return split_x<CT, 3>(xtype, a, s);
    case 128: return split_x<CT, 4>(xtype, a, s);
    case 192: return split_x<CT, 6>(xtype, a, s);
    case 256: return split_x<CT, 8>(xtype, a, s);
    default: return hipErrorInvalidValue;
    }
}

}  // namespace qmm
