// attn_split_f16.hip — the split kernels for F16 caches (attn_split.h), a unit of its own so
// that the cache types compile side by side.
#include "attn_split.h"

namespace qmm {
template hipError_t launch_attn_split_of<QMM_F16, false>(int, int, const AttnArgs&, hipStream_t);
}
