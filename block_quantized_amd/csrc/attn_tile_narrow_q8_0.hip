// attn_tile_narrow_q8_0.hip — the tile kernels for Q8_0 caches and heads of up to 128 values (attn_tile.h).
#include "attn_tile.h"

namespace qmm {
template hipError_t launch_attn_tile_narrow<QMM_Q8_0>(int, int, const AttnArgs&, hipStream_t);
}
