// logits.cpp — the C ABI of qmm_logits.h: argument checks and how rows are
// divided, then the launch.
#include <float.h>
#include <math.h>
#include <stdint.h>

#include "logits_internal.h"

using namespace qmm;

namespace {

constexpr int64_t kMaxLogitRows = (int64_t(1) << 23) - 1, kMaxVocab = int64_t(1) << 28;
constexpr int kMaxParts = 256;

int check_type(int t) {
    if (t == QMM_F32 || t == QMM_BF16) return QMM_OK;
    return qmm_block_size(t) || t == QMM_F16 ? QMM_ERR_UNSUPPORTED : QMM_ERR_TYPE;
}

int check_sizes(int xtype, int64_t rows, int64_t vocab, int top) {
    if (int rc = check_type(xtype)) return rc;
    if (rows <= 0 || rows > kMaxLogitRows || vocab <= 0 || vocab > kMaxVocab) return QMM_ERR_SHAPE;
    if (top < 0 || top > kMaxTop || top > vocab) return QMM_ERR_SHAPE;
    return QMM_OK;
}

bool held(double x) { return x >= FLT_MIN && 2 * x <= FLT_MAX; }  // in fp32, also times log2 e

int check_array(const void* p) {
    if (!p) return QMM_ERR_NULL;
    return reinterpret_cast<uintptr_t>(p) & 3 ? QMM_ERR_ALIGN : QMM_OK;
}

// Parts of a row and the values of one: whole turns of a workgroup's segments.
// A row is divided until there are 1024 workgroups, four a CU.
void divide(int64_t rows, int64_t vocab, int* parts, int* part) {
    const int64_t turn = (int64_t)kLogitWaves * kSegment, turns = (vocab + 7 + turn - 1) / turn;
    int64_t n = (1024 + rows - 1) / rows;
    n = n > kMaxParts ? kMaxParts : n;
    const int64_t each = (turns + n - 1) / n;
    *part = (int)(each * turn);
    *parts = (int)((turns + each - 1) / each);
}

}  // namespace

extern "C" {

size_t qmm_logprobs_work(int xtype, int64_t rows, int64_t vocab, int n_top) {
    if (check_sizes(xtype, rows, vocab, n_top)) return 0;
    int parts, part;
    divide(rows, vocab, &parts, &part);
    return parts == 1 ? 0 : (size_t)(rows * parts * part_words(n_top) * 4 + 15) / 16 * 16;
}

int qmm_logprobs(int xtype, const void* logits, int64_t ld, int64_t rows, int64_t vocab, float scale, float softcap,
                 const int32_t* tokens, int n_tokens, float* logp, float* entropy, int n_top, int32_t* top_ids,
                 float* top_logp, void* work, size_t work_bytes, void* stream) {
    int rc;
    if ((rc = check_sizes(xtype, rows, vocab, n_top))) return rc;
    if (!logits) return QMM_ERR_NULL;
    if (reinterpret_cast<uintptr_t>(logits) & (xtype == QMM_BF16 ? 1 : 3)) return QMM_ERR_ALIGN;
    if (ld < vocab || ld > INT64_MAX / 8 / rows) return QMM_ERR_SHAPE;
    if (!isfinite(scale) || scale <= 0 || !isfinite(softcap) || softcap < 0) return QMM_ERR_UNSUPPORTED;
    const double cap = softcap > 0 ? softcap : 1.0;  // what the kernels multiply by
    if (!held(scale) || !held(scale * cap) || 1.0 / cap > FLT_MAX) return QMM_ERR_UNSUPPORTED;
    if (n_tokens < 0 || n_tokens > 1 << 16) return QMM_ERR_SHAPE;
    if (n_tokens && ((rc = check_array(tokens)) || (rc = check_array(logp)))) return rc;
    if (n_top && ((rc = check_array(top_ids)) || (rc = check_array(top_logp)))) return rc;
    if (entropy && (rc = check_array(entropy))) return rc;
    if (!n_tokens && !n_top && !entropy) return QMM_ERR_NULL;
    LogprobArgs a = {};
    divide(rows, vocab, &a.parts, &a.part);
    if (const size_t need = qmm_logprobs_work(xtype, rows, vocab, n_top)) {
        if (!work) return QMM_ERR_NULL;
        if (reinterpret_cast<uintptr_t>(work) & 15) return QMM_ERR_ALIGN;
        if (work_bytes < need) return QMM_ERR_SHAPE;
    }
    a.logits = logits;
    a.ld = ld;
    a.rows = rows;
    a.tokens = tokens;
    a.logp = logp;
    a.entropy = entropy;
    a.top_ids = top_ids;
    a.top_logp = top_logp;
    a.work = static_cast<float*>(work);
    a.scale = scale;
    a.softcap = softcap;
    a.vocab = (int32_t)vocab;
    a.given = n_tokens;
    a.top = n_top;
    return launch_logprobs(xtype, a, static_cast<hipStream_t>(stream)) == hipSuccess ? QMM_OK : QMM_ERR_HIP;
}

}  // extern "C"
