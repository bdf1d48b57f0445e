// Host-only stand-ins for the launchers of the key-value cache, so that its C
// ABI (kv.cpp) can be built with g++ under the sanitizers and driven without a
// GPU.  They count their calls and look at what they are given as a grid would.
#include "../../block_quantized_amd/csrc/kv_internal.h"

extern int g_launches;
long long g_items = 0, g_parts = 0;

namespace qmm {
hipError_t launch_rope_freqs(double*, int, double, double, const float*, hipStream_t) { ++g_launches; return hipSuccess; }
hipError_t launch_kv_append(int, int, int, const AppendArgs&, hipStream_t) { ++g_launches; return hipSuccess; }
hipError_t launch_attn(int, int, int, int, const AttnArgs& a, hipStream_t) {
    ++g_launches;
    g_items = a.items;
    g_parts = a.parts;
    return hipSuccess;
}
}  // namespace qmm
