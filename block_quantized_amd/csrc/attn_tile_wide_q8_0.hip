// attn_tile_wide_q8_0.hip — the tile kernels for Q8_0 caches and wider heads (attn_tile.h).
#include "attn_tile.h"

namespace qmm {
template hipError_t launch_attn_tile_wide<QMM_Q8_0>(int, int, const AttnArgs&, hipStream_t);
}
