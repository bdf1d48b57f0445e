// logits_internal.h — declarations shared by the units of qmm_logits.h.
#pragma once

#include "../../include/qmm_kv.h"
#include "../../include/qmm_logits.h"
#include "qmm_internal.h"

namespace qmm {

constexpr int kMaxTop = 64;  // alternatives of a row: a lane each

struct LogprobArgs {
    const void* logits;
    int64_t ld, rows;
    const int32_t* tokens;  // rows x given
    float* logp;
    float* entropy;    // nullptr: not wanted
    int32_t* top_ids;  // rows x top
    float* top_logp;
    float* work;  // of each part of a row: its sums, then its top keys
    float scale, softcap;
    int32_t vocab, given, top;
    int32_t parts, part;  // parts of a row, and values of one (whole segments)
};

// Values of a segment: a wavefront's 64 lanes hold so many each.
constexpr int kLaneValues = 32, kSegment = 64 * kLaneValues, kLogitWaves = 4;

// 32-bit words of a part's results: its sums, then its keys.
__host__ __device__ inline int64_t part_words(int top) { return 4 + 2 * (int64_t)top; }

hipError_t launch_logprobs(int xtype, const LogprobArgs& a, hipStream_t s);

}  // namespace qmm
