// attn_join.hip — joins the splits of attention's keys, and hands an attention
// call to the kernels of its cache type.
#include "attn_common.h"

namespace qmm {
namespace {

// A row of out from its sum and denominator, lane `e / 4`'s values.
template <int D, bool XB>
__device__ __forceinline__ void put(const AttnArgs& a, int64_t row, int e, f4v sum, float den) {
    sum *= den > 0.f ? 1.0f / den : den == 0.f ? 0.f : den;
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

// Joins the splits of those rows and heads that have more than one.  A lane
// takes four values, so the lanes of a wavefront 256 / D splits at a time.  With
// few rows the four wavefronts of a workgroup share each (WHOLE); from 2048 on
// each has `each` rows of its own, whose parts it looks up together (a batch of
// thousands of short sequences has few that are split).
// Bound: latency, a chain of three loads.  32 rows of 64 splits 6.3 us, 2048 of
// 3 to 6 splits 6.4 (6.8 with a workgroup a row; 45000 of 2 took 46 us more so).
template <int D, bool XB, bool WHOLE>
__global__ __launch_bounds__(256) void attn_join_kernel(AttnArgs a, int each) {
    constexpr int LANES = D / 4, AT = (WHOLE ? 256 : 64) / LANES;  // lanes of a split, splits at a time
    const int lane = threadIdx.x & 63, thread = WHOLE ? (int)threadIdx.x : lane;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t slots = (int64_t)a.c.n_kv * a.chunks * a.slots;
    const int64_t row0 = ((int64_t)blockIdx.x * (WHOLE ? 1 : 4) + (WHOLE ? 0 : wave)) * each;
    // rows of no sequence have no parts
    const int64_t begin = (int64_t)max(a.c.q_start[0], 0) * a.n_q;
    const int64_t end = (int64_t)clamp_row(a.c.q_start[a.c.n_seqs], a.c.n_tokens) * a.n_q;
    bool split = false;
    if (lane < each && row0 + lane >= begin && row0 + lane < end) {
        const JoinOf j = join_of(a)[row0 + lane];
        // (the tests behind the first fail only for a batch that is none, whose rows nobody wrote)
        split = j.splits > 0 && j.first >= 0 && j.step > 0 && j.slot >= 0 && j.slot < slots &&
                j.first + (j.splits - 1) * (int64_t)j.step < a.items;
    }
    __shared__ f4v s_sum[WHOLE ? 256 : 1];
    __shared__ float s_den[WHOLE ? 256 : 1];
    for (uint64_t todo = __ballot(split); todo; todo &= todo - 1) {  // WHOLE: the same in every wavefront
        const int64_t row = row0 + __ffsll((unsigned long long)todo) - 1;
        const JoinOf j = join_of(a)[row];
        const float* ml = a.work + a.parts * D + 2 * (j.first * slots + j.slot);
        const float* part = a.work + (j.first * slots + j.slot) * D;
        const int64_t step = j.step * slots;
        // every wavefront for itself: the largest maximum
        float top = -INFINITY;
        for (int z = lane; z < j.splits; z += 64) top = fmaxf(top, ml[2 * step * z]);
#pragma unroll
        for (int k = 1; k < 64; k <<= 1) top = fmaxf(top, __shfl_xor(top, k));
        if (top == -INFINITY) top = 0.f;  // no part has seen a key, or one of NaN, which stays
        const int mine = thread / LANES, e = 4 * (thread % LANES);
        f4v sum = {0.f, 0.f, 0.f, 0.f};
        float den = 0.f;
        if (mine < AT) {
            for (int z = mine; z < j.splits; z += AT) {
                const float f = __builtin_amdgcn_exp2f(ml[2 * step * z] - top);
                den += f * ml[2 * step * z + 1];
                sum += f * *reinterpret_cast<const f4v*>(part + step * z * D + e);
            }
        }
        if constexpr (WHOLE) {
            s_sum[threadIdx.x] = sum, s_den[threadIdx.x] = den;
            __syncthreads();
            if (mine == 0) {
#pragma unroll
                for (int z = 1; z < AT; ++z) sum += s_sum[threadIdx.x + z * LANES], den += s_den[threadIdx.x + z * LANES];
                put<D, XB>(a, row, e, sum, den);
            }
            __syncthreads();
        } else {
#pragma unroll
            for (int z = AT / 2; z >= 1; z >>= 1) {  // AT is 1, 2 or 4; lanes behind the last split hold zeros
                den += __shfl_down(den, z * LANES);
#pragma unroll
                for (int i = 0; i < 4; ++i) sum[i] += __shfl_down(sum[i], z * LANES);
            }
            if (mine == 0) put<D, XB>(a, row, e, sum, den);
        }
    }
}

template <int D, bool XB>
hipError_t join_typed(const AttnArgs& a, hipStream_t s) {
    const int64_t rows = a.c.n_tokens * a.n_q;  // below 2^30
    if (rows < 2048) return launch(attn_join_kernel<D, XB, true>, dim3((unsigned)rows), dim3(256), 0, s, a, 1);
    // 2048 workgroups at most, until a wavefront has 64 rows
    int64_t each = (rows + 8191) / 8192;
    if (each > 64) each = 64;
    return launch(attn_join_kernel<D, XB, false>, dim3((unsigned)((rows + 4 * each - 1) / (4 * each))), dim3(256), 0, s, a,
                  (int)each);
}

template <int D>
hipError_t join_x(int xtype, const AttnArgs& a, hipStream_t s) {
    return xtype == QMM_BF16 ? join_typed<D, true>(a, s) : join_typed<D, false>(a, s);
}

}  // namespace

hipError_t launch_attn_join(int head_dim, int xtype, const AttnArgs& a, hipStream_t s) {
    switch (head_dim) {
    case 64: return join_x<64>(xtype, a, s);
    case 96: return join_x<96>(xtype, a, s);
    case 128: return join_x<128>(xtype, a, s);
    case 192: return join_x<192>(xtype, a, s);
    case 256: return join_x<256>(xtype, a, s);
    default: return hipErrorInvalidValue;
    }
}

template <int CT>
static hipError_t attn_of(int algo, int head_dim, int xtype, const AttnArgs& a, hipStream_t s) {
    if (algo != 2) return launch_attn_split_of<CT, false>(head_dim, xtype, a, s);
    return head_dim <= 128 ? launch_attn_tile_narrow<CT, false>(head_dim, xtype, a, s)
                           : launch_attn_tile_wide<CT, false>(head_dim, xtype, a, s);
}

// The same for trees of new tokens.  Q8_0 rows have kernels of their own instead of the tile kernels.
template <int CT>
static hipError_t tree_of(int algo, int head_dim, int xtype, const AttnArgs& a, hipStream_t s) {
    if (algo != 2) return launch_attn_split_of<CT, true>(head_dim, xtype, a, s);
    if constexpr (CT == QMM_Q8_0)
        return launch_attn_tree_q8_0(head_dim, xtype, a, s);
    else
        return head_dim <= 128 ? launch_attn_tile_narrow<CT, true>(head_dim, xtype, a, s)
                               : launch_attn_tile_wide<CT, true>(head_dim, xtype, a, s);
}

hipError_t launch_attn(int algo, int type, int head_dim, int xtype, const AttnArgs& a, hipStream_t s) {
    switch (type) {
    case QMM_Q8_0: return a.tree ? tree_of<QMM_Q8_0>(algo, head_dim, xtype, a, s) : attn_of<QMM_Q8_0>(algo, head_dim, xtype, a, s);
    case QMM_F16: return a.tree ? tree_of<QMM_F16>(algo, head_dim, xtype, a, s) : attn_of<QMM_F16>(algo, head_dim, xtype, a, s);
    case QMM_BF16: return a.tree ? tree_of<QMM_BF16>(algo, head_dim, xtype, a, s) : attn_of<QMM_BF16>(algo, head_dim, xtype, a, s);
    default: return hipErrorInvalidValue;
    }
}

}  // namespace qmm
