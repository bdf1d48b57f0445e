// kv_move.hip — copying pages, and compacting the rows of sequences, over the
// layers of a model.  Rows are moved as bytes.
#include "kv_internal.h"

namespace qmm {
namespace {

typedef uint32_t u4v __attribute__((ext_vector_type(4)));

constexpr int kCopyBytes = 1 << 14;  // of a page that a workgroup takes: four 16-byte loads a lane

// blockIdx.x: a piece of a page and its pair, blockIdx.y: the keys or values of
// a layer.  PART: only the first rows of each head, so a lane looks where in its
// head it stands; the last 16 bytes of them may be cut (rows are even in size).
// Bound: reading and writing, each once.  130 pages of 32 tokens, 8 heads of 128 in
// fp16, 32 layers (545 MB): 210 us, 5.2 TB/s, a large copy's rate.  One page of 16
// layers: latency, 3.5 us.
template <bool PART>
__global__ __launch_bounds__(256) void kv_copy_kernel(LayerArgs l, CopyArgs a, int pieces) {
    const int64_t pair = blockIdx.x / pieces;
    const int64_t from = a.src[pair], to = a.dst[pair];
    if (from < 0 || from >= a.n_pages || to < 0 || to >= a.n_pages || from == to) return;
    uint8_t* pool = l.pool[blockIdx.y];
    const uint8_t* src = pool + from * a.page_bytes;
    uint8_t* dst = pool + to * a.page_bytes;
    const int64_t at = (int64_t)(blockIdx.x % pieces) * kCopyBytes + 16 * threadIdx.x;
    const int64_t head = (int64_t)a.page_size * a.row_bytes;
    const int64_t room = PART ? (int64_t)min(max(a.rows[pair], 0), a.page_size) * a.row_bytes : 0;
    u4v x[4];
    int left[4];  // bytes of the 16 that are copied
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int64_t o = at + 4096 * i;
        left[i] = o < a.page_bytes ? 16 : 0;
        if (PART && left[i]) {
            const int64_t in = room - o % head;
            left[i] = in >= 16 ? 16 : in > 0 ? (int)in : 0;
        }
        if (left[i]) x[i] = *reinterpret_cast<const u4v*>(src + o);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int64_t o = at + 4096 * i;
        if (left[i] == 16) *reinterpret_cast<u4v*>(dst + o) = x[i];
        if (PART && left[i] && left[i] < 16) {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (2 * j < left[i]) *reinterpret_cast<uint16_t*>(dst + o + 2 * j) = (uint16_t)(x[i][j / 2] >> (16 * (j & 1)));
        }
    }
}

// The largest unit that rows of RB bytes are whole numbers of (they follow one
// another without gaps).
template <int RB>
using Unit = std::conditional_t<RB % 16 == 0, u4v,
                                std::conditional_t<RB % 8 == 0, uint2, std::conditional_t<RB % 4 == 0, uint32_t, uint16_t>>>;

// A workgroup takes the keys or values of a head of a sequence in a layer, and
// moves the rows it keeps chunk by chunk.  A row's new place is at or before its
// old one, and every later row's old place behind all of a chunk's new ones: so
// a chunk is read whole before any of it is written, and chunks in their order
// read nothing that was overwritten.
// Bound: reading and writing, each once, where rows are many: 8 sequences keeping
// 1900 rows of 256 bytes of 8 heads in 16 layers (788 MB moved) in 340 us, 4.6 TB/s of
// the 5.1 of a large copy; a workgroup's next places are looked up while its rows are
// on their way (390 us without).  Eight units a lane instead of four: no change.  One
// path of 5 tokens in 32 layers: latency, 3.7 us.
template <int RB>
__global__ __launch_bounds__(256) void kv_compact_kernel(LayerArgs l, CompactArgs a) {
    using U = Unit<RB>;
    constexpr int UNITS = RB / (int)sizeof(U), PER = 4;  // units of a row, and of a lane in a chunk
    constexpr int ROWS = 256 * PER / UNITS;              // rows of a chunk
    __shared__ int64_t s_from[2][ROWS], s_to[2][ROWS];
    const int s = blockIdx.x / a.n_kv, head = blockIdx.x % a.n_kv;
    const int64_t first = a.first[s];
    const int n = min(max(a.n_keep[s], 0), a.width);
    if (a.kv_len && blockIdx.y == 0 && head == 0 && threadIdx.x == 0) a.kv_len[s] = (int32_t)(first + n);
    uint8_t* pool = l.pool[blockIdx.y];
    const int64_t room = (int64_t)a.table_width * a.page_size;
    // where the row of token j of the sequence begins, or -1
    auto row_of = [&](int64_t j) -> int64_t {
        if (j < 0 || j >= room) return -1;
        const int nth = (int)j / a.page_size;
        const int pg = a.table[(int64_t)s * a.table_width + nth];
        if (pg < 0 || pg >= a.n_pages) return -1;
        return (((int64_t)pg * a.n_kv + head) * a.page_size + ((int)j - nth * a.page_size)) * RB;
    };
    // the places of chunk c's rows, which the workgroup reads after the next barrier
    auto look_up = [&](int c) {
        for (int i = threadIdx.x; i < ROWS; i += 256) {
            int64_t from = -1, to = -1;
            if (c + i < n) {
                const int64_t j = a.keep[(int64_t)s * a.width + c + i];
                if (j != first + c + i) from = row_of(j), to = row_of(first + c + i);
            }
            s_from[c / ROWS & 1][i] = to < 0 ? -1 : from;
            s_to[c / ROWS & 1][i] = to;
        }
    };
    if (n > 0) look_up(0);
    __syncthreads();
    for (int c = 0; c < n; c += ROWS) {
        const int b = c / ROWS & 1;
        U x[PER];
        int64_t to[PER];
#pragma unroll
        for (int k = 0; k < PER; ++k) {
            const int u = 256 * k + threadIdx.x, i = u / UNITS;
            const int64_t from = i < ROWS ? s_from[b][i] : -1;
            to[k] = from < 0 ? -1 : s_to[b][i] + u % UNITS * (int)sizeof(U);
            if (from >= 0) x[k] = reinterpret_cast<const U*>(pool + from)[u % UNITS];
        }
        if (c + ROWS < n) look_up(c + ROWS);  // while the rows are on their way
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // every wave's rows have come before one is overwritten
        __syncthreads();
#pragma unroll
        for (int k = 0; k < PER; ++k)
            if (to[k] >= 0) *reinterpret_cast<U*>(pool + to[k]) = x[k];
    }
}

template <int RB>
hipError_t compact_rows(int layers, const LayerArgs& l, const CompactArgs& a, hipStream_t s) {
    return launch(kv_compact_kernel<RB>, dim3((unsigned)(a.n_seqs * a.n_kv), 2 * layers), dim3(256), 0, s, l, a);
}

}  // namespace

hipError_t launch_kv_copy(int layers, const LayerArgs& l, const CopyArgs& a, hipStream_t s) {
    const int pieces = (int)((a.page_bytes + kCopyBytes - 1) / kCopyBytes);
    const dim3 grid((unsigned)(a.n * pieces), 2 * layers);
    return a.rows ? launch(kv_copy_kernel<true>, grid, dim3(256), 0, s, l, a, pieces)
                  : launch(kv_copy_kernel<false>, grid, dim3(256), 0, s, l, a, pieces);
}

hipError_t launch_kv_compact(int type, int head_dim, int layers, const LayerArgs& l, const CompactArgs& a, hipStream_t s) {
    switch (kv_row_bytes(type, head_dim)) {
    case 68: return compact_rows<68>(layers, l, a, s);
    case 102: return compact_rows<102>(layers, l, a, s);
    case 128: return compact_rows<128>(layers, l, a, s);
    case 136: return compact_rows<136>(layers, l, a, s);
    case 192: return compact_rows<192>(layers, l, a, s);
    case 204: return compact_rows<204>(layers, l, a, s);
    case 256: return compact_rows<256>(layers, l, a, s);
    case 272: return compact_rows<272>(layers, l, a, s);
    case 384: return compact_rows<384>(layers, l, a, s);
    case 512: return compact_rows<512>(layers, l, a, s);
    default: return hipErrorInvalidValue;
    }
}

}  // namespace qmm
