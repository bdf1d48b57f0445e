// kv_append.hip — the rotation of positions, and keys and values into the
// pages of a cache.
//
// Bit-exactness: what is stored is defined to the bit, as every codec result
// of this library.  Angles and rotations are computed in fp64 and rounded
// once to fp32; a Q8_0 row is then quantized by the rule of codec.hip.  This
// unit is built with -ffp-contract=off like that one.
//
// Bound: reading the rows and writing them once.  Five prompts, 6777 tokens in
// all (fp32, 32 query and 8 key-value heads of 128, Q8_0 cache; 292 MB): 61-70
// us, 4.2-4.8 TB/s, of the 5.1 that a large copy reaches.  With the sines
// computed by every head and several tokens a workgroup it took some 30 us more.
// 48 tokens take 5.1 us, one 4.0: a chain of loads (q_start, table, row).
#include "kv_internal.h"

namespace qmm {
namespace {

// sin and cos of a (radians, fp64).  Reduction by Cody and Waite: k = rint(a *
// 2/pi), r = a - k * pi/2 with pi/2 in two parts, whose products the fma takes
// exactly; then the Taylor series of sin and cos on |r| <= pi/4, whose first
// missing terms are r^17/17! < 5e-17 and r^18/18! < 3e-18.
__device__ __forceinline__ void sincos64(double a, double& sn, double& cs) {
    const double k = __builtin_rint(a * 0.63661977236758134308);
    double r = __builtin_fma(-k, 1.57079632679489655800e+00, a);
    r = __builtin_fma(-k, 6.12323399573676603587e-17, r);
    const double r2 = r * r;
    double s = -1.0 / 1307674368000.0;  // -1/15!
    s = __builtin_fma(s, r2, 1.0 / 6227020800.0);
    s = __builtin_fma(s, r2, -1.0 / 39916800.0);
    s = __builtin_fma(s, r2, 1.0 / 362880.0);
    s = __builtin_fma(s, r2, -1.0 / 5040.0);
    s = __builtin_fma(s, r2, 1.0 / 120.0);
    s = __builtin_fma(s, r2, -1.0 / 6.0);
    s = __builtin_fma(s * r2, r, r);
    double c = 1.0 / 20922789888000.0;  // 1/16!
    c = __builtin_fma(c, r2, -1.0 / 87178291200.0);
    c = __builtin_fma(c, r2, 1.0 / 479001600.0);
    c = __builtin_fma(c, r2, -1.0 / 3628800.0);
    c = __builtin_fma(c, r2, 1.0 / 40320.0);
    c = __builtin_fma(c, r2, -1.0 / 720.0);
    c = __builtin_fma(c, r2, 1.0 / 24.0);
    c = __builtin_fma(c, r2, -0.5);
    c = __builtin_fma(c, r2, 1.0);
    const int quad = (int)(k - 4.0 * __builtin_floor(k * 0.25));  // k mod 4, for any k
    const double u = (quad & 1) ? c : s, w = (quad & 1) ? s : c;
    sn = (quad & 2) ? -u : u;
    cs = (quad == 1 || quad == 2) ? -w : w;
}

__device__ __forceinline__ float bf16_f32(uint32_t bits) { return __builtin_bit_cast(float, bits << 16); }
__device__ __forceinline__ uint32_t f32_bf16(float f) {
    return (uint32_t)__builtin_bit_cast(unsigned short, (__bf16)f);
}

template <bool BF>
__device__ __forceinline__ float load1(const void* p, int64_t i) {
    if constexpr (BF) return bf16_f32(static_cast<const uint16_t*>(p)[i]);
    else return static_cast<const float*>(p)[i];
}
template <bool BF>
__device__ __forceinline__ float4 load4(const void* p, int64_t i) {  // i a multiple of 4
    if constexpr (BF) {
        const uint2 w = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(p) + i);
        return make_float4(bf16_f32(w.x & 0xFFFF), bf16_f32(w.x >> 16), bf16_f32(w.y & 0xFFFF), bf16_f32(w.y >> 16));
    } else {
        return *reinterpret_cast<const float4*>(static_cast<const float*>(p) + i);
    }
}

__global__ void rope_freqs_kernel(double* freqs, int half, double base, double scale, const float* factors) {
    const int i = blockIdx.x * 64 + threadIdx.x;
    if (i < half) freqs[i] = scale * pow(base, -(double)i / (double)half) / (factors ? (double)factors[i] : 1.0);
}

// A lane owns four consecutive values of a head, so a head is head_dim / 4
// lanes of one wavefront and a Q8_0 block 8 of them.  A wavefront takes the
// heads of one token one after another (q, then k, then v), the next head's
// loads issued before a head is worked on; the sines and cosines of the token
// come from LDS, each computed once.  A value's partner is the lane's own
// (pairs), or loaded a second time (from L1): a whole head is read before any
// of it is written, so q_out may be q.
template <int CT, int D, bool BF>
__global__ __launch_bounds__(256) void kv_append_kernel(AppendArgs a) {
    constexpr int LPH = D / 4, HPW = 64 / LPH;
    const int lane = threadIdx.x & 63, hl = lane / LPH, e = 4 * (lane % LPH);
    const int heads = a.n_q + 2 * a.c.n_kv;
    const int first = ((int)blockIdx.y * 4 + (int)(threadIdx.x >> 6)) * HPW + hl;
    const int step = (int)gridDim.y * 4 * HPW;
    // where the partners of the lane's values lie: in the lane itself; four
    // that follow one another; anywhere (halves of an odd size)
    const int half = a.n_rot / 2;
    const bool halves = a.freqs && a.pairing == QMM_ROPE_HALVES, even = half % 4 == 0;
    const bool turned = a.freqs && e < a.n_rot;
    const int across = e < half ? e + half : e - half;

    __shared__ double s_cs[128], s_sn[128];
    const int64_t t = blockIdx.x;
    const int s = __builtin_amdgcn_readfirstlane(find_seq(a.c, (int)t, a.c.n_seqs + 1));
    if (s < 0 || s >= a.c.n_seqs) return;  // a row of no sequence
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f), y = x;
    // loads the lane's values of the h-th head of the token, and their partners
    auto load = [&](int h) {
        if (hl >= HPW || h >= heads) return;
        const bool isq = h < a.n_q, isv = h >= a.n_q + a.c.n_kv;
        const void* src = isq ? a.xq : isv ? a.xv : a.xk;
        const int64_t base = t * (isq ? a.ldq : isv ? a.ldv : a.ldk) +
                             (int64_t)(isq ? h : isv ? h - a.n_q - a.c.n_kv : h - a.n_q) * D;
        x = load4<BF>(src, base + e);
        if (!halves || isv || !turned) return;
        if (even) {
            y = load4<BF>(src, base + across);
        } else {
            auto partner = [&](int i) { return i >= a.n_rot ? i : i < half ? i + half : i - half; };
            y.x = load1<BF>(src, base + partner(e)), y.y = load1<BF>(src, base + partner(e + 1));
            y.z = load1<BF>(src, base + partner(e + 2)), y.w = load1<BF>(src, base + partner(e + 3));
        }
    };
    load(first);
    // index of the token in its sequence, and its cache row (-1: none)
    const int64_t at = (int64_t)a.c.kv_len[s] - clamp_row(a.c.q_start[s + 1], a.c.n_tokens) + t;
    int64_t row = -1;
    if (at >= 0 && at < (int64_t)a.c.table_width * a.c.page_size) {  // below 2^30
        const int nth = (int)at / a.c.page_size;
        const int pg = a.c.table[(int64_t)s * a.c.table_width + nth];
        if (pg >= 0 && pg < a.c.n_pages)
            row = (int64_t)pg * a.c.n_kv * a.c.page_size + ((int)at - nth * a.c.page_size);
    }
    // a pair's sine and cosine are computed by one lane for all heads
    double cs[4], sn[4];  // 1 and 0 where a value stays
#pragma unroll
    for (int j = 0; j < 4; ++j) cs[j] = 1.0, sn[j] = 0.0;
    if (a.freqs) {
        const int pair = threadIdx.x;
        if (pair < half) {
            double p = (double)at;
            if (a.pos) {
                const int axis = (pair >= a.bounds[0]) + (pair >= a.bounds[1]) + (pair >= a.bounds[2]);
                p = (double)a.pos[axis * a.c.n_tokens + t];
            }
            sincos64(p * a.freqs[pair], s_sn[pair], s_cs[pair]);
        }
        __syncthreads();
        if (turned) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int i = e + j;
                if (i >= a.n_rot) continue;
                const int pair = !halves ? i >> 1 : i < half ? i : i - half;
                cs[j] = s_cs[pair];
                sn[j] = (halves ? i >= half : j & 1) ? s_sn[pair] : -s_sn[pair];
            }
        }
    }
    // the loop runs the same number of times in every lane: the maxima of
    // a Q8_0 block are taken across lanes
    for (int h0 = 0; h0 < heads; h0 += step) {
        const int h = h0 + first;
        const bool on = hl < HPW && h < heads;
        const bool isq = h < a.n_q, isv = h >= a.n_q + a.c.n_kv;
        const int kvh = isq ? 0 : isv ? h - a.n_q - a.c.n_kv : h - a.n_q;
        float v[4] = {x.x, x.y, x.z, x.w};
        if (on && turned && !isv) {
            const float w[4] = {halves ? y.x : x.y, halves ? y.y : x.x, halves ? y.z : x.w, halves ? y.w : x.z};
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (e + j < a.n_rot) v[j] = (float)((double)v[j] * cs[j] + (double)w[j] * sn[j]);
        }
        load(h + step);
        float d = 0.f, id = 0.f;
        if constexpr (CT == QMM_Q8_0) {
            float m = fmaxf(fmaxf(fabsf(v[0]), fabsf(v[1])), fmaxf(fabsf(v[2]), fabsf(v[3])));
            m = fmaxf(m, __shfl_xor(m, 1));
            m = fmaxf(m, __shfl_xor(m, 2));
            m = fmaxf(m, __shfl_xor(m, 4));
            rtn_scale(m, d, id);
        }
        if (!on) continue;
        if (isq) {
            const int64_t o = (t * a.n_q + h) * D + e;
            if constexpr (BF) {
                uint2 w;
                w.x = f32_bf16(v[0]) | f32_bf16(v[1]) << 16;
                w.y = f32_bf16(v[2]) | f32_bf16(v[3]) << 16;
                *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.q_out) + o) = w;
            } else {
                *reinterpret_cast<float4*>(static_cast<float*>(a.q_out) + o) = make_float4(v[0], v[1], v[2], v[3]);
            }
            continue;
        }
        if (row < 0) continue;
        uint8_t* dst = (isv ? a.c.v : a.c.k) + (row + (int64_t)kvh * a.c.page_size) * kv_row_bytes(CT, D);
        if constexpr (CT == QMM_Q8_0) {
            uint8_t* blk = dst + (e >> 5) * kQ8_0Bytes;
            uint16_t* q = reinterpret_cast<uint16_t*>(blk + 2 + (e & 31));
            const int c0 = rtn_code(v[0] * id), c1 = rtn_code(v[1] * id), c2 = rtn_code(v[2] * id),
                      c3 = rtn_code(v[3] * id);
            q[0] = (uint16_t)((c0 & 0xFF) | (c1 & 0xFF) << 8);
            q[1] = (uint16_t)((c2 & 0xFF) | (c3 & 0xFF) << 8);
            if ((e & 31) == 0) *reinterpret_cast<uint16_t*>(blk) = (uint16_t)f2h(d);
        } else {
            uint2 w;
            if constexpr (CT == QMM_F16) {
                w.x = f2h(v[0]) | f2h(v[1]) << 16;
                w.y = f2h(v[2]) | f2h(v[3]) << 16;
            } else {
                w.x = f32_bf16(v[0]) | f32_bf16(v[1]) << 16;
                w.y = f32_bf16(v[2]) | f32_bf16(v[3]) << 16;
            }
            *reinterpret_cast<uint2*>(dst + 2 * e) = w;
        }
    }
}

template <int CT, int D>
hipError_t append_typed(int xtype, const AppendArgs& a, hipStream_t s) {
    constexpr int HPW = 64 / (D / 4);
    // one token's heads are spread over workgroups while there are few tokens
    const int64_t most = (a.n_q + 2 * a.c.n_kv + 4 * HPW - 1) / (4 * HPW);
    const int64_t x = a.c.n_tokens;  // 2^23 at most
    int64_t y = (2048 + x - 1) / x;
    if (y > most) y = most;
    const dim3 grid((unsigned)x, (unsigned)y);
    return xtype == QMM_BF16 ? launch(kv_append_kernel<CT, D, true>, grid, dim3(256), 0, s, a)
                             : launch(kv_append_kernel<CT, D, false>, grid, dim3(256), 0, s, a);
}

template <int CT>
hipError_t append_dims(int head_dim, int xtype, const AppendArgs& a, hipStream_t s) {
    switch (head_dim) {
    case 64: return append_typed<CT, 64>(xtype, a, s);
    case 96: return append_typed<CT, 96>(xtype, a, s);
    case 128: return append_typed<CT, 128>(xtype, a, s);
    case 192: return append_typed<CT, 192>(xtype, a, s);
    case 256: return append_typed<CT, 256>(xtype, a, s);
    default: return hipErrorInvalidValue;
    }
}

}  // namespace

hipError_t launch_rope_freqs(double* freqs, int n_rot, double base, double scale, const float* factors,
                             hipStream_t s) {
    return launch(rope_freqs_kernel, dim3((n_rot / 2 + 63) / 64), dim3(64), 0, s, freqs, n_rot / 2, base, scale,
                  factors);
}

hipError_t launch_kv_append(int type, int head_dim, int xtype, const AppendArgs& a, hipStream_t s) {
    switch (type) {
    case QMM_Q8_0: return append_dims<QMM_Q8_0>(head_dim, xtype, a, s);
    case QMM_F16: return append_dims<QMM_F16>(head_dim, xtype, a, s);
    case QMM_BF16: return append_dims<QMM_BF16>(head_dim, xtype, a, s);
    default: return hipErrorInvalidValue;
    }
}

}  // namespace qmm
