// Drives the calls for drafted tokens and logits through their checks and
// planning with the launchers replaced (draft_stubs.cpp, kv_stubs.cpp,
// abi_stubs.cpp): extreme sizes among valid and invalid ones must neither
// overflow nor launch what is refused, and workspaces must hold every part.
#include <limits.h>
#include <math.h>
#include <stdint.h>
#include <stdio.h>

#include <initializer_list>
#include <vector>

#include "../../include/qmm.h"
#include "../../include/qmm_kv.h"
#include "../../include/qmm_logits.h"

extern int g_launches;
extern long long g_items, g_parts, g_layers, g_part_bytes, g_lens;

static int failures = 0;
#define EXPECT(cond)                                                    \
    do {                                                                \
        if (!(cond)) {                                                  \
            fprintf(stderr, "line %d: %s\n", __LINE__, #cond);          \
            ++failures;                                                 \
        }                                                               \
    } while (0)

alignas(16) static unsigned char buf[4096];

int main() {
    int32_t* const ints_p = reinterpret_cast<int32_t*>(buf);
    const int64_t big[] = {INT64_MIN, -1, 0, 1, 7, 4096, 1 << 23, INT32_MAX, int64_t(1) << 40, INT64_MAX};
    const int ints[] = {INT_MIN, -16, 0, 1, 16, 48, 64, 128, 1 << 20, 1 << 30, INT_MAX};
    qmm_kv_cache c = {buf, buf, QMM_Q8_0, 8, 128, 16, 100};
    qmm_kv_batch b = {ints_p, ints_p, ints_p, 1, 1, 1, 0};
    qmm_kv_tree t = {reinterpret_cast<uint64_t*>(buf), ints_p, 1};
    qmm_attn_opts o = {0.1f, 0.f, 0, 0, nullptr, nullptr};
    int valid = 0;
    for (int type : {(int)QMM_Q8_0, (int)QMM_F16, (int)QMM_BF16, (int)QMM_F32})
        for (int dim : {64, 96, 128, 256})
            for (int n_kv : {1, 8, 4096})
                for (int g : {1, 4, 7, 40, 300})
                    for (int seqs : ints)
                        for (int64_t tokens : big)
                            for (int width : ints)
                                for (int algo : {0, 1, 2}) {
                                    c.type = type, c.head_dim = dim, c.n_kv = n_kv;
                                    b.n_seqs = seqs, b.n_tokens = tokens, b.table_width = width;
                                    o.algo = algo, o.window = width & 64;
                                    const int n_q = n_kv * g, before = g_launches;
                                    const size_t need = qmm_attn_tree_work(&c, &b, &o, QMM_F32, n_q);
                                    const int rc = qmm_attn_tree(&c, &b, &t, &o, QMM_F32, buf, (int64_t)n_q * dim, n_q, buf, buf, need, nullptr);
                                    EXPECT((rc == QMM_OK) == (g_launches == before + 1));
                                    if (rc == QMM_OK) {
                                        ++valid;
                                        EXPECT(g_items > 0 && (size_t)g_parts * (dim + 2) * 4 <= need);
                                        EXPECT(g_items * n_kv < (int64_t(1) << 24));
                                    }
                                }
    EXPECT(valid > 500);
    for (int seqs : ints)
        for (int64_t tokens : big)
            for (int words : ints) {
                b.n_seqs = seqs, b.n_tokens = tokens, t.words = words;
                const int before = g_launches;
                const int rc = qmm_kv_tree_build(&b, ints_p, &t, nullptr, nullptr);
                EXPECT((rc == QMM_OK) == (g_launches == before + 1));
                EXPECT((rc == QMM_OK) == (seqs >= 1 && seqs <= 65536 && tokens >= 1 && tokens < (1 << 23) && words >= 1 && words <= 16));
            }
    c = {buf, buf, QMM_F16, 8, 128, 16, 100};
    for (int count : {1, 63, 64, 65, 200}) {
        std::vector<qmm_kv_cache> all(count, c);
        g_layers = g_lens = 0;
        EXPECT(qmm_kv_copy(all.data(), count, ints_p, ints_p, nullptr, 3, nullptr) == QMM_OK && g_layers == 2 * count);
        g_layers = 0;
        EXPECT(qmm_kv_compact(all.data(), count, ints_p, 2, 3, ints_p, ints_p, ints_p, 4, ints_p + 100, nullptr) == QMM_OK);
        EXPECT(g_layers == 2 * count && g_lens == 1);  // lengths are written once
    }
    for (int64_t n : big)
        for (int page : {16, 1 << 20, 1 << 30})
            for (int n_kv : {1, 4096}) {
                c.page_size = page, c.n_kv = n_kv;
                const int before = g_launches;
                const int rc = qmm_kv_copy(&c, 1, ints_p, ints_p, ints_p, n, nullptr);
                EXPECT((rc == QMM_OK) == (g_launches == before + 1));
            }
    c.page_size = 16, c.n_kv = 8;
    for (int seqs : ints)
        for (int tw : ints)
            for (int width : ints) {
                const int before = g_launches;
                const int rc = qmm_kv_compact(&c, 1, ints_p, seqs, tw, ints_p, ints_p, ints_p, width, nullptr, nullptr);
                EXPECT((rc == QMM_OK) == (g_launches == before + 1));
            }
    valid = 0;
    for (int xtype : {(int)QMM_F32, (int)QMM_BF16, (int)QMM_F16, -5})
        for (int64_t rows : big)
            for (int64_t vocab : {INT64_MIN, (int64_t)0, (int64_t)1, (int64_t)8185, (int64_t)8186, (int64_t)151936, int64_t(1) << 28, INT64_MAX})
                for (int64_t ld : {vocab, (int64_t)-1, INT64_MAX})
                    for (int top : ints)
                        for (float scale : {1.f, 0.f, NAN, INFINITY}) {
                            const int before = g_launches;
                            const size_t need = qmm_logprobs_work(xtype, rows, vocab, top);
                            const int rc = qmm_logprobs(xtype, buf, ld, rows, vocab, scale, 0.f, nullptr, 0, nullptr, (float*)buf, top, ints_p,
                                                        (float*)buf, buf, need, nullptr);
                            EXPECT((rc == QMM_OK) == (g_launches == before + 1));
                            valid += rc == QMM_OK;
                            if (rc == QMM_OK) EXPECT((size_t)g_part_bytes <= need);
                        }
    EXPECT(valid > 50);
    if (failures) return 1;
    printf("draft validation ok\n");
    return 0;
}
