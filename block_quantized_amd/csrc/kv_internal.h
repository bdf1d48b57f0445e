// kv_internal.h — declarations shared by the key-value cache units.
#pragma once

#include "../../include/qmm_kv.h"
#include "qmm_internal.h"

namespace qmm {

// Bytes of one cache row (one head of one token): Q8_0 blocks or 16-bit floats.
__host__ __device__ constexpr int kv_row_bytes(int type, int head_dim) {
    return type == QMM_Q8_0 ? head_dim / 32 * kQ8_0Bytes : head_dim * 2;
}

// A batch as the kernels take it (qmm_kv_batch and the cache's geometry).
struct KvArgs {
    uint8_t* k;
    uint8_t* v;
    const int32_t* q_start;
    const int32_t* kv_len;
    const int32_t* table;
    int64_t n_pages, n_tokens;
    int32_t n_seqs, table_width, page_size, n_kv;
};

struct AppendArgs {
    KvArgs c;
    const void* xk;
    const void* xv;
    const void* xq;
    void* q_out;
    int64_t ldk, ldv, ldq;
    const double* freqs;  // nullptr: no rotation
    const int32_t* pos;
    int32_t n_q, n_rot, pairing;
    int32_t bounds[3];  // first pair of the axes 1, 2, 3
};

struct AttnArgs {
    KvArgs c;
    const void* q;
    void* out;
    float* work;
    const float* slopes;
    const int32_t* prefix;
    int64_t ldq;
    float scale, softcap;
    int32_t n_q, window, head_dim;
    int32_t tile_shift;  // log2 of the tokens of a row tile
    int32_t chunk;       // query heads of a row tile
    int32_t chunks;      // row tiles of heads of a key-value head
    int32_t splits;      // parts that the keys of all row tiles are divided in (more or less); 0: not at all
    int32_t least;       // blocks of 32 keys that a part has at least
    int64_t items;       // work items of a head at most
    int32_t slots;       // rows of an item at most: tokens of a row tile x chunk
    int64_t parts;       // rows of the workspace: items x row tiles of heads x slots
    // a tree of new tokens (tree kernels only): who sees whom, and depths
    const uint64_t* tree;
    const int32_t* depth;
    int32_t words;
    int32_t tile_rows;  // of the tile kernels: 32, 64 or 128
    int32_t fit;        // splits are the items that run at once (64 sequences at most)
};

// What builds a tree from its tokens' parents.
struct TreeArgs {
    const int32_t* q_start;
    const int32_t* kv_len;
    const int32_t* parents;
    uint64_t* seen;
    int32_t* depth;
    int32_t* pos;  // nullptr: not wanted
    int64_t n_tokens;
    int32_t n_seqs, words;
};

// Words of 64 new tokens that a row of a tree has at most.
constexpr int kTreeWords = 16;

// The layers of a model, as many as a launch takes.
constexpr int kMaxLayers = 64;
struct LayerArgs {
    uint8_t* pool[2 * kMaxLayers];  // k and v of each
};

struct CopyArgs {
    const int32_t* src;
    const int32_t* dst;
    const int32_t* rows;  // nullptr: whole pages
    int64_t n, n_pages, page_bytes;
    int32_t n_kv, page_size, row_bytes;
};

struct CompactArgs {
    const int32_t* table;
    const int32_t* first;
    const int32_t* keep;
    const int32_t* n_keep;
    int32_t* kv_len;  // nullptr: not wanted
    int64_t n_pages;
    int32_t n_seqs, table_width, page_size, n_kv, width;
};

// Rows of a row tile: of the split and of the tile kernels.
constexpr int kSplitRows = 16, kTileRows = 128;

#if defined(__HIP_DEVICE_COMPILE__) || defined(__HIPCC__)
__device__ __forceinline__ int clamp_row(int32_t r, int64_t n) {
    return r < 0 ? 0 : (int64_t)r > n ? (int)n : r;
}
// The last of the `count` entries of q_start that is at most `row`, by one
// wavefront: 64 are looked at together.  -1 if there is none.
__device__ __forceinline__ int find_seq(const KvArgs& c, int row, int count) {
    const int lane = threadIdx.x & 63;
    int n = 0;
    for (int s0 = 0; s0 < count; s0 += 64) {
        const int s = s0 + lane;
        n += __popcll(__ballot(s < count && clamp_row(c.q_start[s], c.n_tokens) <= row));
    }
    return n - 1;
}
#endif

hipError_t launch_rope_freqs(double* freqs, int n_rot, double base, double scale, const float* factors, hipStream_t s);
hipError_t launch_kv_append(int type, int head_dim, int xtype, const AppendArgs& a, hipStream_t s);
// Attention by the split (1) or the tile (2) kernels, of a tree of new tokens
// where a.tree is given; each unit of a cache type instantiates its own.
hipError_t launch_attn(int algo, int type, int head_dim, int xtype, const AttnArgs& a, hipStream_t s);
template <int CT, bool TREE>
hipError_t launch_attn_split_of(int head_dim, int xtype, const AttnArgs& a, hipStream_t s);
template <int CT, bool TREE>
hipError_t launch_attn_tile_narrow(int head_dim, int xtype, const AttnArgs& a, hipStream_t s);
template <int CT, bool TREE>
hipError_t launch_attn_tile_wide(int head_dim, int xtype, const AttnArgs& a, hipStream_t s);
hipError_t launch_attn_tree_q8_0(int head_dim, int xtype, const AttnArgs& a, hipStream_t s);
hipError_t launch_kv_tree(const TreeArgs& a, hipStream_t s);
hipError_t launch_kv_copy(int layers, const LayerArgs& l, const CopyArgs& a, hipStream_t s);
hipError_t launch_kv_compact(int type, int head_dim, int layers, const LayerArgs& l, const CompactArgs& a, hipStream_t s);
hipError_t launch_attn_join(int head_dim, int xtype, const AttnArgs& a, hipStream_t s);

}  // namespace qmm
