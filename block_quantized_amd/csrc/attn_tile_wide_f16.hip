// attn_tile_wide_f16.hip — the tile kernels for F16 caches and wider heads (attn_tile.h).
#include "attn_tile.h"

namespace qmm {
template hipError_t launch_attn_tile_wide<QMM_F16, false>(int, int, const AttnArgs&, hipStream_t);
}
