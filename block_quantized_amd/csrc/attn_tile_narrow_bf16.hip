// attn_tile_narrow_bf16.hip — the tile kernels for BF16 caches and heads of up to 128 values (attn_tile.h).
#include "attn_tile.h"

namespace qmm {
template hipError_t launch_attn_tile_narrow<QMM_BF16, false>(int, int, const AttnArgs&, hipStream_t);
}
