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
// lanes' largest values are sorted first: the last wanted one of these is passed
// by at most 32 values for each wanted one, in any order of the values, and of
// those that equal it the list's own last key drops the rest as it fills.
//
// Rows are divided over workgroups until there are 1024, four a CU, and the parts
// joined: few rows would leave the chip to some of its CUs.
//
// Bound: large calls by vector instructions (the vector unit is busy for 99% of the
// time), 22 to 25 issue slots a value with a cap (8 of them the cap's polynomial, 4 the
// exponential), some 15 without: 2048 rows of 151936 in bf16, cap, 8 largest, 622 MB, 211 to 216 us, 2.9 TB/s.
// 257 rows of 128256 in fp32, no cap, 4 tokens and 5 largest, 132 MB, 36 us with the
// join (31 + 5): 3.7 TB/s; 49% of the vector unit's time, two waves a SIMD.  One row
// of 128256, 20 largest: latency, 8.9 us and 4.4 for the join: loads, two sorts, the
// lists' joining; a call from Python 17.  With the sorts through LDS instead of
// registers the last two took 44 and 17.8 us, with the cap's exponential for all values
// instead of the polynomial the first 308.
#include "logits_internal.h"

namespace qmm {
namespace {

typedef uint32_t u4v __attribute__((ext_vector_type(4)));
typedef unsigned long long rank_t;

constexpr float kLog2 = 0.69314718055994530942f, kInvLog2 = 1.44269504088896340736f;

// What lane ^ M holds.
template <int CTRL, int BANKS = 0xF>
__device__ __forceinline__ uint32_t dpp(uint32_t old, uint32_t x) {
    return (uint32_t)__builtin_amdgcn_update_dpp((int)old, (int)x, CTRL, 0xF, BANKS, false);
}
template <int M>
__device__ __forceinline__ uint32_t lane_xor(uint32_t x) {
    if constexpr (M == 1) return dpp<0xB1>(x, x);
    if constexpr (M == 2) return dpp<0x4E>(x, x);
    if constexpr (M == 4) return dpp<0x114, 0xA>(dpp<0x104, 0x5>(x, x), x);  // 4 lanes up, and 4 down
    if constexpr (M == 8) return dpp<0x128>(x, x);                           // a turn by 8 of each 16
    if constexpr (M >= 16) {
        // the halves of two copies change places: one then holds the even rows (or lower half) twice, one the odd ones
        const auto r = M == 16 ? __builtin_amdgcn_permlane16_swap(x, x, false, false)
                               : __builtin_amdgcn_permlane32_swap(x, x, false, false);
        return (threadIdx.x & M) ? r[0] : r[1];
    }
}
template <int M>
__device__ __forceinline__ float lane_xor(float x) {
    return __builtin_bit_cast(float, lane_xor<M>(__builtin_bit_cast(uint32_t, x)));
}
template <int M>
__device__ __forceinline__ rank_t lane_xor(rank_t k) {
    return (rank_t)lane_xor<M>((uint32_t)(k >> 32)) << 32 | lane_xor<M>((uint32_t)k);
}

// Sums of some of a row's values: m is the largest of them, E is in units of
// log 2.  unit: what a difference of values is in these.
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
template <int M>
__device__ __forceinline__ Sums merged_lanes(Sums s, float unit) {
    if constexpr (M < 32) s = merged_lanes<M * 2>(s, unit);
    return merge(s, Sums{lane_xor<M>(s.m), lane_xor<M>(s.rest), lane_xor<M>(s.ent)}, unit);
}

// A logit as a whole number of the same order; a NaN counts as -inf.
__device__ __forceinline__ uint32_t ordered(float x) {
    x = x == x ? x + 0.0f : -INFINITY;
    const uint32_t u = __builtin_bit_cast(uint32_t, x);
    return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}
__device__ __forceinline__ float unordered(uint32_t u) {  // (no NaN's)
    return __builtin_bit_cast(float, u ^ ((uint32_t)((int32_t)~u >> 31) | 0x80000000u));
}
__device__ __forceinline__ rank_t key_of(float x, uint32_t id) { return (rank_t)ordered(x) << 32 | (uint32_t)~id; }
__device__ __forceinline__ rank_t lane_key(rank_t k, int lane) {  // lane: the same in all lanes
    return (rank_t)(uint32_t)__builtin_amdgcn_readlane((int)(k >> 32), lane) << 32 |
           (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)k, lane);
}
// One step of a bitonic sort: the larger of two lanes' keys to the lower lane, or to the upper one.
template <int M, typename T>
__device__ __forceinline__ T exchange(T k, bool larger) {
    const T o = lane_xor<M>(k);
    return (k > o) == larger ? k : o;
}
template <int N, int M, typename T>
__device__ __forceinline__ T sort_steps(T k, int lane) {
    k = exchange<M>(k, ((lane & M) == 0) == ((lane & N) == 0 || N == 64));
    if constexpr (M > 1) k = sort_steps<N, M / 2>(k, lane);
    return k;
}
template <int N, typename T>
__device__ __forceinline__ T sorted(T k, int lane) {  // descending from lane 0 on, of each N lanes
    if constexpr (N > 2) k = sorted<N / 2>(k, lane);
    return sort_steps<N, N / 2>(k, lane);
}
// The 64 largest of two sorted lists, sorted; `b` from its last one on.
__device__ __forceinline__ rank_t joined(rank_t a, rank_t b, int lane) { return sort_steps<64, 32>(a > b ? a : b, lane); }
// A sorted list with one key more.
__device__ __forceinline__ rank_t inserted(rank_t list, rank_t k, int lane) {
    const int at = __popcll(__ballot(list > k));
    const rank_t up = (rank_t)dpp<0x138>(0, (uint32_t)(list >> 32)) << 32 | dpp<0x138>(0, (uint32_t)list);  // of lane - 1
    return lane < at ? list : lane == at ? k : up;
}

// tanh y, 2^-22 off relative to the larger of itself and 0.35; -inf stays.  SMALL:
// below 0.35, where the polynomial in y^2 that is closest to tanh(y) / y does.
template <bool SMALL>
__device__ __forceinline__ float tanh_of(float y) {
    const float y2 = y * y;
    float p = fmaf(0.0193613345f, y2, -0.0537063462f);
    p = fmaf(p, y2, 0.133322014f);
    p = fmaf(p, y2, -0.333333161f);
    const float small = fmaf(p * y2, y, y);
    if constexpr (SMALL) return small;
    const float a = fabsf(y), e = __builtin_amdgcn_exp2f(2.0f * kInvLog2 * a);
    const float large = copysignf(1.0f - 2.0f * __builtin_amdgcn_rcpf(e + 1.0f), y);
    return y == -INFINITY ? y : a < 0.35f ? small : large;
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
    const bool cap = a.softcap > 0.f;
    const float inv = cap ? 1.0f / a.softcap : 0.f, unit = cap ? a.scale * a.softcap : a.scale;
    const float lse = log1pf(s.rest);
    auto logp = [&](float x) {
        if (cap) x = tanh_of<false>(x * inv);
        return (s.m == -INFINITY ? -INFINITY : (x - s.m) * unit) - lse;
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

// The wavefronts' sums and lists, joined: the sums in every lane, the list in
// the first wavefront.
__device__ __forceinline__ void join_waves(const LogprobArgs& a, float unit, int wave, int lane, Sums& sums, rank_t& list) {
    __shared__ Sums s_sums[kLogitWaves];
    __shared__ rank_t s_list[kLogitWaves][64];
    static_assert(kLogitWaves == 4, "two rounds");
    sums = merged_lanes<1>(sums, unit);
    if (lane == 0) s_sums[wave] = sums;
    if (a.top && wave >= 2) s_list[wave][lane] = list;
    __syncthreads();
    if (a.top && wave < 2) {
        list = joined(list, s_list[wave + 2][63 - lane], lane);
        if (wave == 1) s_list[1][lane] = list;
    }
    __syncthreads();
    if (a.top && wave == 0) list = joined(list, s_list[1][63 - lane], lane);
    sums = s_sums[0];
#pragma unroll
    for (int w = 1; w < kLogitWaves; ++w) sums = merge(sums, s_sums[w], unit);
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
    const float inv = CAP ? 1.0f / a.softcap : 0.f, unit = a.scale * kInvLog2 * (CAP ? a.softcap : 1.0f);

    Sums sums = {-INFINITY, 0.f, 0.f};
    rank_t list = 0, least = 0;  // the largest keys, and the last wanted one of them (0: there are fewer)
    auto add = [&](rank_t k) {   // a key each
        for (uint64_t todo = __ballot(k > least); todo; todo = __ballot(k > least) & todo & (todo - 1)) {
            list = inserted(list, lane_key(k, __ffsll((unsigned long long)todo) - 1), lane);
            const rank_t last = lane_key(list, a.top - 1);
            least = last > least ? last : least;
        }
    };
    auto few = [&](int v0, int v1) {  // the values v0 .. v1 - 1, one a lane
        const bool on = v0 + lane < v1;
        const float x = on ? logit<BF>(a, row, v0 + lane) : -INFINITY;
        if (a.top) add(on ? key_of(x, v0 + lane) : 0);
        const float y = CAP ? tanh_of<false>(x * inv) : x;
        // (a NaN or +inf: the row's sums are NaN)
        sums = merge(sums, Sums{y, y < INFINITY ? 0.f : NAN, 0.f}, unit);
    };
    const int head = min(q0 * N - skew, a.vocab), tail = max(q1 * N - skew, head);
    if (part == 0 && wave == 0) few(0, head);
    // (bf16: the next segment's loads go ahead of this one's arithmetic, 222 -> 215 us for 2048 rows of 151936 with a cap;
    // fp32 values stay in the registers they were loaded to, and the waves' number hides the loads: 36 us for 257 rows of
    // 128256, 39 with loads ahead)
    u4v w[LOADS];
    auto load = [&](int at) {
#pragma unroll
        for (int j = 0; j < LOADS; ++j)
            w[j] = *reinterpret_cast<const u4v*>(base + 16 * (int64_t)min(at + 64 * j + lane, upto - 1));
    };
    int at = from + wave * (kSegment / N);
    if (BF && at < upto) load(at);
    for (; at < upto; at += kLogitWaves * (kSegment / N)) {
        if (!BF) load(at);
        float x[kLaneValues];
        auto unpack = [&](int j, bool on) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t u = w[j][i];  // (a bit_cast of the element itself takes the vector's first one: ROCm 7.2's compiler)
                if constexpr (BF) {
                    x[N * j + 2 * i] = on ? bf16_f32(u & 0xFFFF) : -INFINITY;
                    x[N * j + 2 * i + 1] = on ? __builtin_bit_cast(float, u & 0xFFFF0000u) : -INFINITY;
                } else {
                    x[N * j + i] = on ? __builtin_bit_cast(float, u) : -INFINITY;
                }
            }
        };
        if (at + 64 * LOADS <= upto) {
#pragma unroll
            for (int j = 0; j < LOADS; ++j) unpack(j, true);
        } else {
#pragma unroll
            for (int j = 0; j < LOADS; ++j) unpack(j, at + 64 * j + lane < upto);
        }
        if (BF && at + kLogitWaves * (kSegment / N) < upto) load(at + kLogitWaves * (kSegment / N));
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
                    // as many lanes hold a value of at least the last wanted one of the lanes' largest
                    const uint32_t mine = at + lane < upto ? ordered(big) : 0;
                    const uint32_t last = (uint32_t)__builtin_amdgcn_readlane((int)sorted<64>(mine, lane), a.top - 1);
                    const rank_t below = last ? ((rank_t)last << 32) - 1 : 0;
                    least = below > least ? below : least;
                }
                const float bar = least >> 32 ? unordered((uint32_t)(least >> 32)) : -INFINITY;
#pragma unroll
                for (int i = 0; i < kLaneValues; ++i)
                    if (__any(!(x[i] < bar))) add(key(i));  // (a NaN is seen as -inf)
                least = lane_key(list, a.top - 1);
            }
        }
        // ---- the sums
        float m = big;
        if constexpr (CAP) {
            float most = 0.f;
#pragma unroll
            for (int i = 0; i < kLaneValues; ++i) x[i] *= inv;
#pragma unroll
            for (int i = 0; i < kLaneValues; ++i) most = fmaxf(most, fabsf(x[i]));
            m *= inv;
            if (__any(!(most < 0.35f))) {
                m = tanh_of<false>(m);
#pragma unroll
                for (int i = 0; i < kLaneValues; ++i) x[i] = tanh_of<false>(x[i]);
            } else {
                m = tanh_of<true>(m);
#pragma unroll
                for (int i = 0; i < kLaneValues; ++i) x[i] = tanh_of<true>(x[i]);
            }
        }
        const float ref = m == -INFINITY ? 0.f : m;
        float rest = 0.f, ent = 0.f;
        int equal = 0;  // to the largest one
#pragma unroll
        for (int i = 0; i < kLaneValues; ++i) {
            const float t = (x[i] - ref) * unit, p = __builtin_amdgcn_exp2f(t);
            rest += t == 0.f ? 0.f : p;
            equal += t == 0.f;
            ent -= p * fmaxf(t, -16384.0f);
        }
        rest += m == -INFINITY ? 0.f : (float)(equal - 1);
        sums = merge(sums, Sums{m, rest, ent}, unit);
    }
    if (part == a.parts - 1 && wave == 0) few(tail, a.vocab);

    join_waves(a, unit, wave, lane, sums, list);
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
    const float unit = a.scale * kInvLog2 * (a.softcap > 0.f ? a.softcap : 1.0f);
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
                k[i] = p < a.parts && 63 - lane < a.top ? reinterpret_cast<const rank_t*>(in + p * words + 4)[63 - lane] : 0;
            }
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (lane_key(k[i], 63) > lane_key(list, a.top - 1)) list = joined(list, k[i], lane);
        }
    }
    join_waves(a, unit, wave, lane, sums, list);
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
