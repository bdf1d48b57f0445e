// attn_tree_split_f16.hip — the split kernels for trees of new tokens over F16 caches.
#include "attn_split.h"

namespace qmm {
template hipError_t launch_attn_split_of<QMM_F16, true>(int, int, const AttnArgs&, hipStream_t);
}
