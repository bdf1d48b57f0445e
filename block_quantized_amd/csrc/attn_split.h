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
// rows; Q8_0 codes as fp16 integers, their block scales applied to the fp32
// block scores, and to P before it is rounded).  Queries and P are split into
// 16-bit parts that hold 22 bits (two fp16) or 24 (three bf16).  Queries are
// scaled by a power of two per row so that their largest value is about 2^14,
// P is 2^8 p, and P d is kept below 2^15 by a power of two per wave: the fp16
// parts lose nothing to subnormals.
//
// The running maximum of a row is raised only when a score is above it by
// more than 2^7: p may reach 2^7, which costs fp32 sums nothing and saves the
// cross-lane maximum and the rescaling for almost every tile.
#pragma once

#include "attn_common.h"

namespace qmm {
namespace {

constexpr int kWaves = 4;

template <int CT>
__device__ __forceinline__ constexpr int parts_of() { return CT == QMM_BF16 ? 3 : 2; }

__device__ __forceinline__ uint32_t ld16(const uint8_t* p) { return *reinterpret_cast<const uint16_t*>(p); }

template <int CT, int NB, bool XB>
__global__ __launch_bounds__(256) void attn_split_kernel(AttnArgs a) {
    constexpr int D = 32 * NB, RB = kv_row_bytes(CT, D), PARTS = parts_of<CT>();
    constexpr bool BF = CT == QMM_BF16, Q8 = CT == QMM_Q8_0;
    TileAt at;
    if (!find_tile(a, blockIdx.x, at)) return;
    const int lane = threadIdx.x & 63, m = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int kvh = blockIdx.y / a.chunks, G = a.n_q / a.c.n_kv;
    const int head0 = kvh * G + (blockIdx.y % a.chunks) * a.chunk;  // first query head of the tile
    const int heads = min(a.chunk, kvh * G + G - head0);
    // row m of the tile: token m / heads, head m % heads
    const int rows = min(16, at.tokens * heads);
    const int mr = min(m, rows - 1), mt = mr / heads, head = head0 + mr % heads;
    const int p_row = at.pos + mt;

    // ---- the queries, as B operands: lane (m, g) holds the values 8g..8g+7 of each block
    u4v qf[NB][PARTS];
    float qs;  // what a score is multiplied by
    {
        float x[NB][8];
        const int64_t base = (int64_t)(at.row + mt) * a.ldq + (int64_t)head * D + 8 * g;
        float big = 0.f;
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            if constexpr (XB) {
                const u4v w = *reinterpret_cast<const u4v*>(static_cast<const uint16_t*>(a.q) + base + 32 * b);
#pragma unroll
                for (int i = 0; i < 4; ++i) x[b][2 * i] = bf16_lo(w[i]), x[b][2 * i + 1] = bf16_hi(w[i]);
            } else {
                const f4v* p = reinterpret_cast<const f4v*>(static_cast<const float*>(a.q) + base + 32 * b);
                const f4v u = p[0], w = p[1];
#pragma unroll
                for (int i = 0; i < 4; ++i) x[b][i] = u[i], x[b][4 + i] = w[i];
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) big = fmaxf(big, fabsf(x[b][i]));
        }
        big = fmaxf(big, __shfl_xor(big, 16));
        big = fmaxf(big, __shfl_xor(big, 32));
        int ex = 0;
        frexpf(big, &ex);
        ex = min(max(ex, -110), 126);  // an all-zero row: any finite scale does
        const float up = ldexpf(1.0f, 14 - ex);
        qs = ldexpf(1.0f, ex - 14) * a.scale;
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                uint32_t part[PARTS];
                split_pair<BF, PARTS>(x[b][2 * i] * up, x[b][2 * i + 1] * up, part);
#pragma unroll
                for (int k = 0; k < PARTS; ++k) qf[b][k][i] = part[k];
            }
    }
    const float inv_cap = a.softcap > 0.f ? 1.0f / a.softcap : 0.f;
    if (!(a.softcap > 0.f)) qs *= kLog2e;
    const float slope = a.slopes ? a.slopes[head] * kLog2e : 0.f;

    // ---- the tiles of this split
    const int n_pre = (at.pre + 31) >> 5;
    const int w0 = max(n_pre, at.low >> 5), w1 = (at.end + 31) >> 5;
    const int n_tiles = n_pre + max(0, w1 - w0);
    const int per = (n_tiles + a.splits - 1) / a.splits;
    const int t0 = (int)blockIdx.z * per, t1 = min(n_tiles, t0 + per);
    const int low_last = a.window > 0 ? at.pos + at.tokens - a.window : INT32_MIN;  // every row sees keys from here

    const int reach = a.window > 0 ? a.window : INT32_MAX;

    f4v o[NB][2];
#pragma unroll
    for (int b = 0; b < NB; ++b) o[b][0] = o[b][1] = f4v{0.f, 0.f, 0.f, 0.f};
    float mx = -INFINITY, mref = 0.f, l = 0.f;  // maximum, the same or 0, the lane's part of the sum
    float vlim = 0x1p-30f, vinv = 0x1p30f;      // Q8_0: a power of two that no |d| seen is above, and 1 / it

    int64_t my_row = -1;
    int have = 0;
    for (int t = t0 + wave; t < t1; t += kWaves) {
        // lane i looks up 16 keys' row in the cache: half i % 2 of the wave's tile i / 2 from here on
        if (have == 0) {
            const int tt = t + kWaves * (lane >> 1);
            const int64_t key = 32 * (int64_t)(tt < n_pre ? tt : tt - n_pre + w0) + 16 * (lane & 1);
            my_row = -1;
            if (tt < t1 && key < at.len) {
                const int pidx = (int)key / a.c.page_size;
                const int pg = a.c.table[(int64_t)at.s * a.c.table_width + pidx];
                if (pg >= 0 && pg < a.c.n_pages)
                    my_row = ((int64_t)pg * a.c.n_kv + kvh) * a.c.page_size + ((int)key - pidx * a.c.page_size);
            }
            have = 32;
        }
        const int from = 2 * (32 - have);
        --have;
        int64_t r0[2];
#pragma unroll
        for (int u = 0; u < 2; ++u)
            r0[u] = (int64_t)((uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)my_row, from + u) |
                              (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(my_row >> 32), from + u) << 32);
        const int kb = 32 * (t < n_pre ? t : t - n_pre + w0);
        const bool paged = r0[0] >= 0 && r0[1] >= 0;
        const bool whole = paged && ((kb + 32 <= at.pre) || (kb >= low_last && kb + 32 <= min(at.len, at.pos + 1)));

        // ---- loads
        u4v kf[2][NB];
        uint32_t vw[2][4][NB], kd[2][4][NB], vd[2][4][NB];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const int64_t r = max(r0[u], (int64_t)0);
            const uint8_t *kbase = a.c.k + r * RB, *vbase = a.c.v + r * RB;
            const uint8_t* kp = kbase + m * RB;
#pragma unroll
            for (int b = 0; b < NB; ++b) {
                if constexpr (Q8) {
                    uint64_t w;
                    __builtin_memcpy(&w, kp + b * kQ8_0Bytes + 2 + 8 * g, 8);
                    const uint32_t lo = (uint32_t)w ^ 0x80808080u, hi = (uint32_t)(w >> 32) ^ 0x80808080u;
                    kf[u][b][0] = codes_f16(lo, 0x04010400u), kf[u][b][1] = codes_f16(lo, 0x04030402u);
                    kf[u][b][2] = codes_f16(hi, 0x04010400u), kf[u][b][3] = codes_f16(hi, 0x04030402u);
                } else {
                    kf[u][b] = *reinterpret_cast<const u4v*>(kp + 64 * b + 16 * g);
                }
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint8_t* vp = vbase + (4 * g + i) * RB;
                const uint8_t* kq = kbase + (4 * g + i) * RB;
#pragma unroll
                for (int b = 0; b < NB; ++b) {
                    if constexpr (Q8) {
                        vw[u][i][b] = ld16(vp + b * kQ8_0Bytes + 2 + 2 * m);
                        vd[u][i][b] = ld16(vp + b * kQ8_0Bytes);
                        kd[u][i][b] = ld16(kq + b * kQ8_0Bytes);
                    } else {
                        vw[u][i][b] = *reinterpret_cast<const uint32_t*>(vp + 64 * b + 4 * m);
                    }
                }
            }
        }

        // ---- scores
        float sc[8];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            f4v acc = {0.f, 0.f, 0.f, 0.f};
            if constexpr (Q8) {
                f4v sum = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int b = 0; b < NB; ++b) {
                    acc = f4v{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int k = PARTS - 1; k >= 0; --k) acc = mfma16<BF>(kf[u][b], qf[b][k], acc);
#pragma unroll
                    for (int i = 0; i < 4; ++i) sum[i] = fmaf(acc[i], h2f(kd[u][i][b]), sum[i]);
                }
                acc = sum;
            } else {
#pragma unroll
                for (int k = PARTS - 1; k >= 0; --k)
#pragma unroll
                    for (int b = 0; b < NB; ++b) acc = mfma16<BF>(kf[u][b], qf[b][k], acc);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) sc[4 * u + i] = acc[i] * qs;
        }
        if (a.softcap > 0.f) {
#pragma unroll
            for (int i = 0; i < 8; ++i) sc[i] = a.softcap * kLog2e * tanh_fp32(sc[i] * inv_cap);
        }
        if (a.slopes) {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                sc[i] -= slope * fabsf((float)(p_row - (kb + 16 * (i >> 2) + 4 * g + (i & 3))));
        }
        if (!whole) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int u = i >> 2, key = kb + 16 * u + 4 * g + (i & 3);
                // without branches: this compiler has dropped the assignment where they were nested
                const bool ok = (key < at.len) & (r0[u] >= 0), pre = key < at.pre;
                const bool seen = ok & (((key <= p_row) & (p_row - key < reach)) | pre);
                const bool kept = ok & (((key < at.end) & (key >= at.low)) | pre);
                sc[i] = seen ? sc[i] : -INFINITY;
                // a key that no row sees may hold anything: 0 times it has to be 0
#pragma unroll
                for (int b = 0; b < NB; ++b) {
                    if constexpr (Q8) vd[u][i & 3][b] = kept ? vd[u][i & 3][b] : 0;
                    else vw[u][i & 3][b] = kept ? vw[u][i & 3][b] : 0;
                }
            }
        }

        // ---- running maximum
        float big = fmaxf(fmaxf(fmaxf(sc[0], sc[1]), fmaxf(sc[2], sc[3])), fmaxf(fmaxf(sc[4], sc[5]), fmaxf(sc[6], sc[7])));
        if (__any(big > mx + 7.0f)) {
            big = fmaxf(big, __shfl_xor(big, 16));
            big = fmaxf(big, __shfl_xor(big, 32));
            const float top = fmaxf(mx, big), ref = top == -INFINITY ? 0.f : top;
            const float down = __builtin_amdgcn_exp2f(mx - ref);  // 0 from -inf
            mx = top;
            mref = ref - 8.0f;  // p carries a factor of 2^8
            l *= down;
#pragma unroll
            for (int b = 0; b < NB; ++b) o[b][0] *= down, o[b][1] *= down;
        }
        float p[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            p[i] = __builtin_amdgcn_exp2f(sc[i] - mref);
            l += p[i];
        }

        // ---- O^T += V^T P^T
        if constexpr (Q8) {
            float dmax = 0.f;
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int b = 0; b < NB; ++b) dmax = fmaxf(dmax, fabsf(h2f(vd[u][i][b])));
            if (__any(dmax > vlim)) {
#pragma unroll
                for (int k = 1; k < 64; k <<= 1) dmax = fmaxf(dmax, __shfl_xor(dmax, k));
                int ex;
                frexpf(fminf(dmax, 65504.0f), &ex);
                const float lim = ldexpf(1.0f, ex), down = vlim / lim;
                vlim = lim, vinv = 1.0f / lim;
#pragma unroll
                for (int b = 0; b < NB; ++b) o[b][0] *= down, o[b][1] *= down;
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) p[i] *= vinv;
#pragma unroll
            for (int b = 0; b < NB; ++b) {
                u4v pf[PARTS];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    uint32_t part[PARTS];
                    const int u = i >> 1, k0 = 2 * (i & 1);
                    split_pair<BF, PARTS>(p[2 * i] * h2f(vd[u][k0][b]), p[2 * i + 1] * h2f(vd[u][k0 + 1][b]), part);
#pragma unroll
                    for (int k = 0; k < PARTS; ++k) pf[k][i] = part[k];
                }
                u4v vf[2];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int u = i >> 1, k0 = 2 * (i & 1);
                    const uint32_t w = (vw[u][k0][b] | vw[u][k0 + 1][b] << 16) ^ 0x80808080u;
                    vf[0][i] = codes_f16(w, 0x04020400u);
                    vf[1][i] = codes_f16(w, 0x04030401u);
                }
#pragma unroll
                for (int j = 0; j < 2; ++j)
#pragma unroll
                    for (int k = PARTS - 1; k >= 0; --k) o[b][j] = mfma16<BF>(vf[j], pf[k], o[b][j]);
            }
        } else {
            u4v pf[PARTS];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                uint32_t part[PARTS];
                split_pair<BF, PARTS>(p[2 * i], p[2 * i + 1], part);
#pragma unroll
                for (int k = 0; k < PARTS; ++k) pf[k][i] = part[k];
            }
#pragma unroll
            for (int b = 0; b < NB; ++b) {
                u4v vf[2];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int u = i >> 1, k0 = 2 * (i & 1);
                    const uint32_t x = vw[u][k0][b], y = vw[u][k0 + 1][b];
                    vf[0][i] = __builtin_amdgcn_perm(y, x, 0x05040100u);
                    vf[1][i] = __builtin_amdgcn_perm(y, x, 0x07060302u);
                }
#pragma unroll
                for (int j = 0; j < 2; ++j)
#pragma unroll
                    for (int k = PARTS - 1; k >= 0; --k) o[b][j] = mfma16<BF>(vf[j], pf[k], o[b][j]);
            }
        }
    }

    // ---- the four waves' parts: row m, values 8g..8g+7 of each block
    l += __shfl_xor(l, 16);
    l += __shfl_xor(l, 32);
    __shared__ float s_o[kWaves][16][D + 4];
    __shared__ float s_m[kWaves][16], s_l[kWaves][16];
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 2; ++j) s_o[wave][m][32 * b + 8 * g + 2 * i + j] = o[b][j][i] * (Q8 ? vlim : 1.0f);
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
        if (a.splits > 1) {
            const int64_t part = row * a.splits + blockIdx.z;
            float* ml = a.work + a.c.n_tokens * a.n_q * a.splits * D;
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
    const int64_t items = (a.c.n_tokens >> a.tile_shift) + a.c.n_seqs;
    const dim3 grid((unsigned)items, (unsigned)(a.c.n_kv * a.chunks), (unsigned)a.splits);
    hipError_t e = launch(attn_split_kernel<CT, NB, XB>, grid, dim3(256), 0, s, a);
    if (e != hipSuccess || a.splits == 1) return e;
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
