// logprobs.hip — log probabilities of given tokens, entropy and the largest
// logits of rows of logits, which are read once.
//
// With x the logits (capped, scaled) and m their largest, p_i = exp(x_i - m):
//   R = sum of p_i without one of the largest, whose p is 1
//   E = sum of p_i (m - x_i)
//   log p(t) = x_t - m - log1p(R),   entropy = log1p(R) + E / (1 + R)
// Both sums have terms of one sign, and the largest one's 1 is never added to
// small ones: where nearly all is on one token, what the others hold keeps its
// bits.  Two parts (m, R, E) and (m', R', E') with m' <= m, f = exp(m' - m):
//   R += f (1 + R'),   E += f (E' + (m - m') (1 + R')).
//
// A wavefront takes a segment of 2048 values at a time, 32 a lane in registers,
// all loads issued together.  Its largest logits so far lie sorted in its lanes,
// a key each: the logit's bits in an order of whole numbers, then the index
// turned around, so that equal logits go by the lowest index and no two keys are
// the same.  A segment is looked through only if a lane's largest value passes
// the last of them.  Where many lanes do (always in the first segment), the
// lanes' largest keys are sorted first: the last wanted one of these is passed
// by at most 32 keys for each wanted one, in any order of the values.
//
// Rows are divided over workgroups while there are few, and the parts joined.
#include "logits_internal.h"

namespace qmm {
namespace {

typedef uint32_t u4v __attribute__((ext_vector_type(4)));
typedef unsigned long long rank_t;

constexpr float kLog2 = 0.69314718055994530942f, kInvLog2 = 1.44269504088896340736f;

// Sums of some of a row's values: m is a logit (capped, not scaled), E is in
// units of log 2.  unit: the scale, in these.
struct Sums {
    float m, rest, ent;
};
__device__ __forceinline__ Sums merge(Sums a, Sums b, float unit) {
    const bool swap = b.m > a.m;
    const Sums hi = swap ? b : a, lo = swap ? a : b;
    // (nothing but -inf: no largest one either)
    const float gap = lo.m == -INFINITY ? -INFINITY : (lo.m - hi.m) * unit;
    const float f = __builtin_amdgcn_exp2f(gap), one = 1.0f + lo.rest;
    return Sums{hi.m, hi.rest + f * one, hi.ent + f * (lo.ent - fmaxf(gap, -16384.0f) * one)};
}
__device__ __forceinline__ Sums shuffled(Sums s, int k) {
    return Sums{__shfl_xor(s.m, k), __shfl_xor(s.rest, k), __shfl_xor(s.ent, k)};
}

// A logit as a whole number of the same order; a NaN counts as -inf.
__device__ __forceinline__ uint32_t ordered(float x) {
    x = x == x ? x + 0.0f : -INFINITY;
    const uint32_t u = __builtin_bit_cast(uint32_t, x);
    return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}
__device__ __forceinline__ rank_t key_of(float x, uint32_t id) { return (rank_t)ordered(x) << 32 | (uint32_t)~id; }
__device__ __forceinline__ rank_t lane_key(rank_t k, int lane) {  // lane: the same in all lanes
    return (rank_t)(uint32_t)__builtin_amdgcn_readlane((int)(k >> 32), lane) << 32 |
           (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)k, lane);
}
__device__ __forceinline__ rank_t xor_key(rank_t k, int mask) {
    return (rank_t)(uint32_t)__shfl_xor((int)(k >> 32), mask) << 32 | (uint32_t)__shfl_xor((int)(uint32_t)k, mask);
}
// One step of a bitonic sort: the larger of two lanes' keys to the lower lane, or to the upper one.
__device__ __forceinline__ rank_t exchange(rank_t k, int mask, bool larger) {
    const rank_t o = xor_key(k, mask);
    return (k > o) == larger ? k : o;
}
__device__ __forceinline__ rank_t sorted(rank_t k, int lane) {  // descending from lane 0 on
#pragma unroll
    for (int n = 2; n <= 64; n <<= 1)
#pragma unroll
        for (int m = n / 2; m >= 1; m >>= 1) k = exchange(k, m, ((lane & m) == 0) == ((lane & n) == 0 || n == 64));
    return k;
}
// The 64 largest of two sorted lists, sorted.
__device__ __forceinline__ rank_t joined(rank_t a, rank_t b, int lane) {
    const rank_t o = xor_key(b, 63);  // b's from its last one on
    rank_t k = a > o ? a : o;
#pragma unroll
    for (int m = 32; m >= 1; m >>= 1) k = exchange(k, m, (lane & m) == 0);
    return k;
}
// A sorted list with one key more.
__device__ __forceinline__ rank_t inserted(rank_t list, rank_t k, int lane) {
    const int at = __popcll(__ballot(list > k));
    const rank_t up = (rank_t)(uint32_t)__shfl_up((int)(list >> 32), 1) << 32 | (uint32_t)__shfl_up((int)(uint32_t)list, 1);
    return lane < at ? list : lane == at ? k : up;
}

// x = cap tanh(x / cap), 2^-22 off relative to the larger of itself and 0.35 cap; -inf stays.
__device__ __forceinline__ float capped(float x, float cap, float inv) {
    const float y = x * inv, a = fabsf(y), y2 = y * y;
    float p = fmaf(0.0193613345f, y2, -0.0537063462f);
    p = fmaf(p, y2, 0.133322014f);
    p = fmaf(p, y2, -0.333333161f);
    const float small = fmaf(p * y2, y, y);
    const float e = __builtin_amdgcn_exp2f(2.0f * kInvLog2 * a);
    const float large = copysignf(1.0f - 2.0f * __builtin_amdgcn_rcpf(e + 1.0f), y);
    return x == -INFINITY ? x : cap * (a < 0.35f ? small : large);
}

__device__ __forceinline__ float bf16_f32(uint32_t u) { return __builtin_bit_cast(float, u << 16); }

template <bool BF>
__device__ __forceinline__ float logit(const LogprobArgs& a, int64_t row, int v) {
    if constexpr (BF) return bf16_f32(static_cast<const uint16_t*>(a.logits)[row * a.ld + v]);
    return static_cast<const float*>(a.logits)[row * a.ld + v];
}

// The results of a row, by one workgroup, from its sums (in every lane of every
// wavefront) and its sorted keys (wavefront 0).
template <bool BF>
__device__ void finish(const LogprobArgs& a, int64_t row, Sums s, rank_t list) {
    const int lane = threadIdx.x & 63;
    const float inv = a.softcap > 0.f ? 1.0f / a.softcap : 0.f;
    const float lse = log1pf(s.rest);
    auto logp = [&](float x) {
        if (a.softcap > 0.f) x = capped(x, a.softcap, inv);
        // the same product as the sums': the largest one's is exactly m
        const float gap = s.m == -INFINITY ? -INFINITY : (x - s.m) * a.scale;
        return gap - lse;
    };
    for (int i = threadIdx.x; i < a.given; i += blockDim.x) {
        const int t = a.tokens[row * a.given + i];
        a.logp[row * a.given + i] = t >= 0 && t < a.vocab ? logp(logit<BF>(a, row, t)) : -INFINITY;
    }
    if (threadIdx.x == 0 && a.entropy) a.entropy[row] = lse + s.ent * kLog2 / (1.0f + s.rest);
    if (threadIdx.x < 64 && lane < a.top) {
        const uint32_t id = ~(uint32_t)list;
        a.top_ids[row * a.top + lane] = (int32_t)id;
        a.top_logp[row * a.top + lane] = logp(logit<BF>(a, row, (int)id));
    }
}

template <bool BF, bool CAP>
__global__ __launch_bounds__(256) void logprobs_kernel(LogprobArgs a) {
    constexpr int N = BF ? 8 : 4, LOADS = kLaneValues / N;  // values of a load, loads of a lane
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t row = blockIdx.x / a.parts;
    const int part = blockIdx.x % a.parts;
    // Rows may begin and end anywhere: `base` is the multiple of 16 bytes at or
    // before the row, from which its whole loads are [q0, q1); the values before
    // and behind these, N - 1 at most each, are a step of their own.
    const char* base = static_cast<const char*>(a.logits) + row * a.ld * (BF ? 2 : 4);
    const int skew = (int)(reinterpret_cast<uintptr_t>(base) & 15) / (BF ? 2 : 4);
    base -= skew * (BF ? 2 : 4);
    const int q0 = skew ? 1 : 0, q1 = max((a.vocab + skew) / N, q0);
    const int from = part ? part * (a.part / N) : q0, upto = min((part + 1) * (a.part / N), q1);
    const float inv = CAP ? 1.0f / a.softcap : 0.f, unit = a.scale * kInvLog2;

    Sums sums = {-INFINITY, 0.f, 0.f};
    rank_t list = 0, least = 0;  // the largest keys, and the last wanted one of them (0: there are fewer)
    auto add = [&](rank_t k) {   // a key each
        for (uint64_t todo = __ballot(k > least); todo; todo &= todo - 1) {
            const rank_t one = lane_key(k, __ffsll((unsigned long long)todo) - 1);
            if (one <= least) continue;
            list = inserted(list, one, lane);
            const rank_t last = lane_key(list, a.top - 1);
            least = last > least ? last : least;
        }
    };
    auto few = [&](int v0, int v1) {  // the values v0 .. v1 - 1, one a lane
        const bool on = v0 + lane < v1;
        const float x = on ? logit<BF>(a, row, v0 + lane) : -INFINITY;
        if (a.top) add(on ? key_of(x, v0 + lane) : 0);
        const float y = CAP ? capped(x, a.softcap, inv) : x;
        // (a NaN or +inf: the row's sums are NaN)
        sums = merge(sums, Sums{y, y < INFINITY ? 0.f : NAN, 0.f}, unit);
    };
    const int head = min(q0 * N - skew, a.vocab), tail = max(q1 * N - skew, head);
    if (part == 0 && wave == 0) few(0, head);
    for (int at = from + wave * (kSegment / N); at < upto; at += kLogitWaves * (kSegment / N)) {
        float x[kLaneValues];
        {
            u4v w[LOADS];
            bool on[LOADS];
#pragma unroll
            for (int j = 0; j < LOADS; ++j) {
                const int q = at + 64 * j + lane;
                on[j] = q < upto;
                w[j] = *reinterpret_cast<const u4v*>(base + 16 * (int64_t)(on[j] ? q : upto - 1));
            }
#pragma unroll
            for (int j = 0; j < LOADS; ++j)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    if constexpr (BF) {
                        x[N * j + 2 * i] = on[j] ? bf16_f32(w[j][i] & 0xFFFF) : -INFINITY;
                        x[N * j + 2 * i + 1] = on[j] ? bf16_f32(w[j][i] >> 16) : -INFINITY;
                    } else {
                        // (a bit_cast of the element itself takes the vector's first one: ROCm 7.2's compiler)
                        const uint32_t u = w[j][i];
                        x[N * j + i] = on[j] ? __builtin_bit_cast(float, u) : -INFINITY;
                    }
                }
        }
        float big = x[0];
#pragma unroll
        for (int i = 1; i < kLaneValues; ++i) big = fmaxf(big, x[i]);
        // ---- the largest logits
        if (a.top) {
            // (a wavefront's indexes only rise from one segment to the next: an equal logit comes too late)
            const uint64_t pass = __ballot(ordered(big) > (uint32_t)(least >> 32));
            if (pass) {
                auto key = [&](int i) -> rank_t {
                    const int q = at + 64 * (i / N) + lane;
                    return q < upto ? key_of(x[i], (uint32_t)(q * N + i % N - skew)) : 0;
                };
                if (!least || __popcll(pass) > 12) {
                    rank_t k = 0;
#pragma unroll
                    for (int i = 0; i < kLaneValues; ++i) {
                        const rank_t o = key(i);
                        k = o > k ? o : k;
                    }
                    k = lane_key(sorted(k, lane), a.top - 1);
                    least = k > least ? k - 1 : least;  // (that key itself is wanted)
                }
#pragma unroll
                for (int i = 0; i < kLaneValues; ++i) add(key(i));
                least = lane_key(list, a.top - 1);
            }
        }
        // ---- the sums
        float y[kLaneValues], ref = big;
        if constexpr (CAP) {
            ref = -INFINITY;
#pragma unroll
            for (int i = 0; i < kLaneValues; ++i) {
                y[i] = capped(x[i], a.softcap, inv);
                ref = fmaxf(ref, y[i]);
            }
        }
        const float m = ref;
        ref = ref == -INFINITY ? 0.f : ref;
        float rest = 0.f, all = 0.f, ent = 0.f;
#pragma unroll
        for (int i = 0; i < kLaneValues; ++i) {
            const float t = ((CAP ? y[i] : x[i]) - ref) * unit, p = __builtin_amdgcn_exp2f(t);
            all += p;
            rest += t == 0.f ? 0.f : p;
            ent -= p * fmaxf(t, -16384.0f);
        }
        rest += m == -INFINITY ? 0.f : rintf(all - rest) - 1.0f;  // the equals of the largest one
        sums = merge(sums, Sums{m, rest, ent}, unit);
    }
    if (part == a.parts - 1 && wave == 0) few(tail, a.vocab);

    // ---- the lanes' sums, then the wavefronts'
#pragma unroll
    for (int k = 1; k < 64; k <<= 1) sums = merge(sums, shuffled(sums, k), unit);
    __shared__ Sums s_sums[kLogitWaves];
    __shared__ rank_t s_list[kLogitWaves][64];
    if (lane == 0) s_sums[wave] = sums;
    if (a.top) s_list[wave][lane] = list;
    __syncthreads();
    sums = s_sums[0];
#pragma unroll
    for (int w = 1; w < kLogitWaves; ++w) sums = merge(sums, s_sums[w], unit);
    if (a.top && wave == 0) {
#pragma unroll
        for (int w = 1; w < kLogitWaves; ++w) list = joined(list, s_list[w][lane], lane);
    }
    if (a.parts == 1) {
        finish<BF>(a, row, sums, list);
        return;
    }
    float* out = a.work + (row * a.parts + part) * part_words(a.top);
    if (threadIdx.x == 0) out[0] = sums.m, out[1] = sums.rest, out[2] = sums.ent;
    if (threadIdx.x < a.top) reinterpret_cast<rank_t*>(out + 4)[lane] = list;
}

// Joins the parts of a row, 256 at most: a lane takes the sums of one, a
// wavefront the keys of every fourth.
template <bool BF>
__global__ __launch_bounds__(256) void logprobs_join_kernel(LogprobArgs a) {
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t row = blockIdx.x, words = part_words(a.top);
    const float* in = a.work + row * a.parts * words;
    const float unit = a.scale * kInvLog2;
    Sums sums = {-INFINITY, 0.f, 0.f};
    if ((int)threadIdx.x < a.parts) {
        const float* p = in + threadIdx.x * words;
        sums = Sums{p[0], p[1], p[2]};
    }
    rank_t list = 0;
    if (a.top) {
        for (int p0 = wave; p0 < a.parts; p0 += 4 * kLogitWaves) {
            rank_t k[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int p = p0 + i * kLogitWaves;
                k[i] = p < a.parts && lane < a.top ? reinterpret_cast<const rank_t*>(in + p * words + 4)[lane] : 0;
            }
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (lane_key(k[i], 0) > lane_key(list, a.top - 1)) list = joined(list, k[i], lane);
        }
    }
#pragma unroll
    for (int k = 1; k < 64; k <<= 1) sums = merge(sums, shuffled(sums, k), unit);
    __shared__ Sums s_sums[kLogitWaves];
    __shared__ rank_t s_list[kLogitWaves][64];
    if (lane == 0) s_sums[wave] = sums;
    if (a.top) s_list[wave][lane] = list;
    __syncthreads();
    sums = s_sums[0];
#pragma unroll
    for (int w = 1; w < kLogitWaves; ++w) sums = merge(sums, s_sums[w], unit);
    if (a.top && wave == 0) {
#pragma unroll
        for (int w = 1; w < kLogitWaves; ++w) list = joined(list, s_list[w][lane], lane);
    }
    finish<BF>(a, row, sums, list);
}

template <bool BF>
hipError_t logprobs_typed(const LogprobArgs& a, hipStream_t s) {
    const dim3 grid((unsigned)(a.rows * a.parts)), block(64 * kLogitWaves);
    const hipError_t e = a.softcap > 0.f ? launch(logprobs_kernel<BF, true>, grid, block, 0, s, a)
                                         : launch(logprobs_kernel<BF, false>, grid, block, 0, s, a);
    if (e != hipSuccess || a.parts == 1) return e;
    return launch(logprobs_join_kernel<BF>, dim3((unsigned)a.rows), dim3(64 * kLogitWaves), 0, s, a);
}

}  // namespace

hipError_t launch_logprobs(int xtype, const LogprobArgs& a, hipStream_t s) {
    return xtype == QMM_BF16 ? logprobs_typed<true>(a, s) : logprobs_typed<false>(a, s);
}

}  // namespace qmm
