// attn_tree_split_q8_0.hip — the split kernels for trees of new tokens over Q8_0 caches.
#include "attn_split.h"

namespace qmm {
template hipError_t launch_attn_split_of<QMM_Q8_0, true>(int, int, const AttnArgs&, hipStream_t);
}
