// attn_tree_tile_narrow_bf16.hip — the narrow tile kernels for trees of new tokens over BF16 caches.
#include "attn_tile.h"

namespace qmm {
template hipError_t launch_attn_tile_narrow<QMM_BF16, true>(int, int, const AttnArgs&, hipStream_t);
}
