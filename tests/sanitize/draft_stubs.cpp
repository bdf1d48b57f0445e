// Host-only stand-ins for the launchers behind kv_draft.cpp and logits.cpp, so
// that their checks can be built with g++ under the sanitizers and driven
// without a GPU.
#include "../../block_quantized_amd/csrc/kv_internal.h"
#include "../../block_quantized_amd/csrc/logits_internal.h"

extern int g_launches;
long long g_layers = 0, g_part_bytes = 0, g_lens = 0;

namespace qmm {
hipError_t launch_kv_tree(const TreeArgs&, hipStream_t) { ++g_launches; return hipSuccess; }
hipError_t launch_kv_copy(int layers, const LayerArgs& l, const CopyArgs&, hipStream_t) {
    ++g_launches;
    for (int i = 0; i < 2 * layers; ++i) g_layers += l.pool[i] != nullptr;
    return hipSuccess;
}
hipError_t launch_kv_compact(int, int, int layers, const LayerArgs& l, const CompactArgs& a, hipStream_t) {
    ++g_launches;
    for (int i = 0; i < 2 * layers; ++i) g_layers += l.pool[i] != nullptr;
    g_lens += a.kv_len != nullptr;
    return hipSuccess;
}
hipError_t launch_logprobs(int, const LogprobArgs& a, hipStream_t) {
    ++g_launches;
    g_part_bytes = a.parts == 1 ? 0 : a.rows * a.parts * part_words(a.top) * 4;
    return hipSuccess;
}
}  // namespace qmm
