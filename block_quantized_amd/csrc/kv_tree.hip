// kv_tree.hip — trees of new tokens: who sees whom, depths and positions, from
// each token's parent.
#include "kv_internal.h"

namespace qmm {
namespace {

// A workgroup takes a sequence, a lane a token, whose chain of parents it walks
// in LDS.  A parent that does not stand before its token is none, so a chain
// only descends: it ends, and its words are written from the last to the first.
// Bound: latency, some 0.1 us a step of the deepest chain: 2.9 us for 5 tokens, 3.7 for
// 32 sequences of 16.
__global__ __launch_bounds__(256) void kv_tree_kernel(TreeArgs a) {
    __shared__ int16_t s_parent[64 * kTreeWords];
    const int s = blockIdx.x;
    const int q0 = clamp_row(a.q_start[s], a.n_tokens), q1 = clamp_row(a.q_start[s + 1], a.n_tokens);
    const int n = q1 - q0, most = min(n, 64 * a.words);
    if (n <= 0) return;
    for (int i = threadIdx.x; i < most; i += 256) {
        const int p = a.parents[q0 + i];
        s_parent[i] = (int16_t)(p >= 0 && p < i ? p : -1);
    }
    __syncthreads();
    const int kv = a.kv_len[s], base = max(kv, 0) - n;
    for (int i = threadIdx.x; i < n; i += 256) {
        const int64_t row = q0 + i;
        uint64_t* seen = a.seen + row * a.words;
        int word = a.words - 1, depth = 0;
        uint64_t bits = 0;
        for (int at = i < most ? i : -1; at >= 0; at = s_parent[at]) {
            for (; word > at >> 6; --word) seen[word] = bits, bits = 0;
            bits |= uint64_t(1) << (at & 63);
            ++depth;
        }
        for (; word >= 0; --word) seen[word] = bits, bits = 0;
        depth = max(depth - 1, 0);
        a.depth[row] = depth;
        if (a.pos) a.pos[row] = base + depth;
    }
}

}  // namespace

hipError_t launch_kv_tree(const TreeArgs& a, hipStream_t s) {
    return launch(kv_tree_kernel, dim3((unsigned)a.n_seqs), dim3(256), 0, s, a);
}

}  // namespace qmm
