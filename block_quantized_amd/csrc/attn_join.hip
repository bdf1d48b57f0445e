// attn_join.hip — joins the splits of attention's keys, and hands an attention
// call to the kernels of its cache type.
#include "attn_common.h"

namespace qmm {
namespace {

// Joins the splits of one row and head: D / 4 lanes.
template <int D, bool XB>
__global__ __launch_bounds__(64) void attn_join_kernel(AttnArgs a) {
    const int64_t row = blockIdx.x;
    // rows of no sequence have no parts
    const int t = (int)(row / a.n_q);
    if (t < a.c.q_start[0] || t >= clamp_row(a.c.q_start[a.c.n_seqs], a.c.n_tokens)) return;
    const float* ml = a.work + a.c.n_tokens * a.n_q * a.splits * D + 2 * row * a.splits;
    const int e = 4 * threadIdx.x;
    if (e >= D) return;
    float top = -INFINITY;
    for (int z = 0; z < a.splits; ++z) top = fmaxf(top, ml[2 * z]);
    f4v sum = {0.f, 0.f, 0.f, 0.f};
    float den = 0.f;
    for (int z = 0; z < a.splits; ++z) {
        const float f = top == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(ml[2 * z] - top);
        den += f * ml[2 * z + 1];
        sum += f * *reinterpret_cast<const f4v*>(a.work + (row * a.splits + z) * D + e);
    }
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

template <int D>
hipError_t join_x(int xtype, const AttnArgs& a, hipStream_t s) {
    const dim3 grid((unsigned)(a.c.n_tokens * a.n_q));
    return xtype == QMM_BF16 ? launch(attn_join_kernel<D, true>, grid, dim3(64), 0, s, a)
                             : launch(attn_join_kernel<D, false>, grid, dim3(64), 0, s, a);
}

}  // namespace

hipError_t launch_attn_join(int head_dim, int xtype, const AttnArgs& a, hipStream_t s) {
    if (a.c.n_tokens * a.n_q >= (int64_t(1) << 26)) return hipErrorInvalidConfiguration;  // 2^32 work-items
    switch (head_dim) {
    case 64: return join_x<64>(xtype, a, s);
    case 96: return join_x<96>(xtype, a, s);
    case 128: return join_x<128>(xtype, a, s);
    case 192: return join_x<192>(xtype, a, s);
    case 256: return join_x<256>(xtype, a, s);
    default: return hipErrorInvalidValue;
    }
}

hipError_t launch_attn(int algo, int type, int head_dim, int xtype, const AttnArgs& a, hipStream_t s) {
    switch (type) {
    case QMM_Q8_0:
        return algo == 2 ? launch_attn_tile_of<QMM_Q8_0>(head_dim, xtype, a, s)
                         : launch_attn_split_of<QMM_Q8_0>(head_dim, xtype, a, s);
    case QMM_F16:
        return algo == 2 ? launch_attn_tile_of<QMM_F16>(head_dim, xtype, a, s)
                         : launch_attn_split_of<QMM_F16>(head_dim, xtype, a, s);
    case QMM_BF16:
        return algo == 2 ? launch_attn_tile_of<QMM_BF16>(head_dim, xtype, a, s)
                         : launch_attn_split_of<QMM_BF16>(head_dim, xtype, a, s);
    default: return hipErrorInvalidValue;
    }
}

}  // namespace qmm
