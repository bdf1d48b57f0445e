// attn_join.hip — joins the splits of attention's keys, and hands an attention
// call to the kernels of its cache type.
#include "attn_common.h"

namespace qmm {
namespace {

// Joins the splits of `each` rows and heads a workgroup, those that have more
// than one (a batch of thousands of short sequences has few).  Its four
// wavefronts take a row's splits in turn: a lane four values, so 256 / (D / 4)
// splits at a time.  A kernel of its own rather than the last workgroup's work:
// 32 rows of 64 splits take 6.2 us, most of it the launch and a chain of three
// loads; 2048 rows of 3 to 6 splits 6.8 us.
template <int D, bool XB>
__global__ __launch_bounds__(256) void attn_join_kernel(AttnArgs a, int each) {
    constexpr int LANES = D / 4, AT = 256 / LANES;  // lanes of a split, splits at a time
    const int lane = threadIdx.x & 63;
    const int64_t slots = (int64_t)a.c.n_kv * a.chunks * a.slots, row0 = (int64_t)blockIdx.x * each;
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
    __shared__ f4v s_sum[256];
    __shared__ float s_den[256];
    for (uint64_t todo = __ballot(split); todo; todo &= todo - 1) {  // the same in every wavefront
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
        const int mine = threadIdx.x / LANES, e = 4 * (threadIdx.x % LANES);
        f4v sum = {0.f, 0.f, 0.f, 0.f};
        float den = 0.f;
        if (mine < AT && top != -INFINITY) {
            for (int z = mine; z < j.splits; z += AT) {
                const float f = __builtin_amdgcn_exp2f(ml[2 * step * z] - top);
                den += f * ml[2 * step * z + 1];
                sum += f * *reinterpret_cast<const f4v*>(part + step * z * D + e);
            }
        }
        s_sum[threadIdx.x] = sum, s_den[threadIdx.x] = den;
        __syncthreads();
        if (mine == 0) {
#pragma unroll
            for (int z = 1; z < AT; ++z) sum += s_sum[threadIdx.x + z * LANES], den += s_den[threadIdx.x + z * LANES];
            const float inv = den > 0.f ? 1.0f / den : den == 0.f ? 0.f : den;
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
        __syncthreads();
    }
}

template <int D>
hipError_t join_x(int xtype, const AttnArgs& a, hipStream_t s) {
    // a row a workgroup while that makes no more than 2048 of them
    const int64_t rows = a.c.n_tokens * a.n_q;
    int64_t each = (rows + 2047) / 2048;
    if (each > 64) each = 64;
    const dim3 grid((unsigned)((rows + each - 1) / each));
    return xtype == QMM_BF16 ? launch(attn_join_kernel<D, true>, grid, dim3(256), 0, s, a, (int)each)
                             : launch(attn_join_kernel<D, false>, grid, dim3(256), 0, s, a, (int)each);
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
    if (algo != 2) return launch_attn_split_of<CT>(head_dim, xtype, a, s);
    return head_dim <= 128 ? launch_attn_tile_narrow<CT>(head_dim, xtype, a, s)
                           : launch_attn_tile_wide<CT>(head_dim, xtype, a, s);
}

hipError_t launch_attn(int algo, int type, int head_dim, int xtype, const AttnArgs& a, hipStream_t s) {
    switch (type) {
    case QMM_Q8_0: return attn_of<QMM_Q8_0>(algo, head_dim, xtype, a, s);
    case QMM_F16: return attn_of<QMM_F16>(algo, head_dim, xtype, a, s);
    case QMM_BF16: return attn_of<QMM_BF16>(algo, head_dim, xtype, a, s);
    default: return hipErrorInvalidValue;
    }
}

}  // namespace qmm
