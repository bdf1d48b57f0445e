// attn_tile_wide_bf16.hip — the tile kernels for BF16 caches and wider heads (attn_tile.h).
#include "attn_tile.h"

namespace qmm {
template hipError_t launch_attn_tile_wide<QMM_BF16, false>(int, int, const AttnArgs&, hipStream_t);
}
