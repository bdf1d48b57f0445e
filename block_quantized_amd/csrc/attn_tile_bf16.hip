// attn_tile_bf16.hip — the tile kernels for BF16 caches (attn_tile.h), a unit of its own so
// that the cache types compile side by side.
#include "attn_tile.h"

namespace qmm {
template hipError_t launch_attn_tile_of<QMM_BF16>(int, int, const AttnArgs&, hipStream_t);
}
