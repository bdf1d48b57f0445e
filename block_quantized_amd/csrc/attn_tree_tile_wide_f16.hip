// attn_tree_tile_wide_f16.hip — the wide tile kernels for trees of new tokens over F16 caches.
#include "attn_tile.h"

namespace qmm {
template hipError_t launch_attn_tile_wide<QMM_F16, true>(int, int, const AttnArgs&, hipStream_t);
}
