// attn_tree_tile_narrow_q8_0.hip — the narrow tile kernels for trees of new tokens over Q8_0 caches.
#include "attn_tile.h"

namespace qmm {
template hipError_t launch_attn_tile_narrow<QMM_Q8_0, true>(int, int, const AttnArgs&, hipStream_t);
}
