// attn_common.h — device helpers shared by the attention kernels.
#pragma once

#include "kv_internal.h"

namespace qmm {

typedef _Float16 half2v __attribute__((ext_vector_type(2)));
typedef _Float16 half8v __attribute__((ext_vector_type(8)));
typedef __bf16 bf2v __attribute__((ext_vector_type(2)));
typedef __bf16 bf8v __attribute__((ext_vector_type(8)));
typedef float f4v __attribute__((ext_vector_type(4)));
typedef float f16v __attribute__((ext_vector_type(16)));
typedef uint32_t u4v __attribute__((ext_vector_type(4)));

constexpr float kLog2e = 1.44269504088896340736f;

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __builtin_bit_cast(float, w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __builtin_bit_cast(float, w & 0xFFFF0000u); }

// A pair of fp32 values as 16-bit parts that sum to them: two fp16 parts hold
// 22 bits, three bf16 parts 24.  fp16 callers scale their values so that the
// low part is no subnormal that matters.  (The empty asm makes the packed
// part the one value that is both used and subtracted: the compiler otherwise
// rounds x a second time for the subtraction, fused with the product that made
// it, and a pair that ties differently leaves a whole step of the high part.)
template <bool BF, int PARTS>
__device__ __forceinline__ void split_pair(float x, float y, uint32_t (&part)[PARTS]) {
#pragma unroll
    for (int i = 0; i < PARTS; ++i) {
        if constexpr (BF) {
            bf2v h;
            h.x = (__bf16)x, h.y = (__bf16)y;
            part[i] = __builtin_bit_cast(uint32_t, h);
            asm("" : "+v"(part[i]));
            x -= bf16_lo(part[i]), y -= bf16_hi(part[i]);
        } else {
            half2v h;
            h.x = (_Float16)x, h.y = (_Float16)y;
            part[i] = __builtin_bit_cast(uint32_t, h);
            asm("" : "+v"(part[i]));
            h = __builtin_bit_cast(half2v, part[i]);
            x -= (float)h.x, y -= (float)h.y;
        }
    }
}

template <bool BF>
__device__ __forceinline__ f4v mfma16(u4v a, u4v b, f4v c) {
    if constexpr (BF)
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf8v, a), __builtin_bit_cast(bf8v, b), c, 0,
                                                       0, 0);
    else
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(half8v, a), __builtin_bit_cast(half8v, b), c,
                                                      0, 0, 0);
}

// Two int8 codes, bytes `sel` of x ^ 0x80808080 (so code + 128), as fp16:
// 0x6400 | u is 1024 + u, and 1152 less is the code, exactly.
__device__ __forceinline__ uint32_t codes_f16(uint32_t biased, uint32_t sel) {
    half2v h = __builtin_bit_cast(half2v, __builtin_amdgcn_perm(0x64646464u, biased, sel));
    const half2v off = {(_Float16)1152.0f, (_Float16)1152.0f};
    return __builtin_bit_cast(uint32_t, h - off);
}

// tanh(x): the Taylor series (to x^11; the next term is below 4e-9 x) where
// 1 - 2 / (e^2x + 1) would lose bits to cancellation, that form elsewhere.
__device__ __forceinline__ float tanh_fp32(float x) {
    const float x2 = x * x;
    float p = -1382.0f / 155925.0f;
    p = fmaf(p, x2, 62.0f / 2835.0f);
    p = fmaf(p, x2, -17.0f / 315.0f);
    p = fmaf(p, x2, 2.0f / 15.0f);
    p = fmaf(p, x2, -1.0f / 3.0f);
    const float small = fmaf(p * x2, x, x);
    const float big = 1.0f - 2.0f / (__builtin_amdgcn_exp2f(2.0f * kLog2e * fabsf(x)) + 1.0f);
    return fabsf(x) < 0.35f ? small : copysignf(big, x);
}

// Where a row tile of a sequence stands: the tokens first .. first + tokens-1
// of it, at indexes pos .. , and the keys they may see.
struct TileAt {
    int s, first, tokens, row;  // row: of the inputs, of token `first`
    int pos, len, pre;          // index of the first token, readable keys, prefix
    int end, low;               // keys any of the tokens sees: [low, end) and [0, pre)
};

// The tile `item` of the row tiles of 2^shift tokens.  Sequence s owns the
// items from (q_start[s] >> shift) + s on: at least ceil(n / 2^shift) of them,
// and some that are empty (false).
__device__ __forceinline__ bool find_tile(const AttnArgs& a, int item, TileAt& t) {
    const int sh = a.tile_shift;
    const int s = __builtin_amdgcn_readfirstlane(find_seq(a.c, item, sh, 1, a.c.n_seqs));
    if (s < 0) return false;
    const int q0 = clamp_row(a.c.q_start[s], a.c.n_tokens), q1 = clamp_row(a.c.q_start[s + 1], a.c.n_tokens);
    const int64_t first = (int64_t)(item - ((q0 >> sh) + s)) << sh;
    if (first >= q1 - q0) return false;
    t.s = s;
    t.first = (int)first;
    t.row = q0 + t.first;
    t.tokens = min(1 << sh, q1 - q0 - t.first);
    const int kv = max(a.c.kv_len[s], 0);
    const int64_t room = (int64_t)a.c.table_width * a.c.page_size;
    t.len = (int64_t)kv < room ? kv : (int)room;
    t.pos = kv - (q1 - q0) + t.first;
    t.pre = a.prefix ? min(max(a.prefix[s], 0), t.len) : 0;
    t.end = max(0, min(t.len, t.pos + t.tokens));
    t.low = a.window > 0 && t.pos >= a.window ? t.pos - a.window + 1 : 0;
    return true;
}

}  // namespace qmm
