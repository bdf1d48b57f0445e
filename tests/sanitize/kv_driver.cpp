// Drives qmm_kv.h's entry points through their validation and planning with
// the launchers replaced (kv_stubs.cpp, abi_stubs.cpp): extreme sizes among
// valid and invalid ones must neither overflow nor launch what is refused, and
// the workspace asked for must hold every part that a launch may write.
#include <limits.h>
#include <math.h>
#include <stdint.h>
#include <stdio.h>

#include <initializer_list>

#include "../../include/qmm.h"
#include "../../include/qmm_kv.h"

extern int g_launches;
extern long long g_items, g_parts;

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
    const int64_t big[] = {INT64_MIN, -1, 0, 1, 7, 4096, INT32_MAX, int64_t(1) << 40, INT64_MAX};
    const int ints[] = {INT_MIN, -16, 0, 1, 16, 48, 64, 128, 256, 1 << 20, 1 << 30, INT_MAX};
    const int types[] = {-1, 0, QMM_Q4_0, QMM_Q8_0, QMM_F32, QMM_F16, QMM_BF16, 99};
    for (int t : types)
        for (int heads : ints)
            for (int dim : ints)
                for (int page : ints)
                    for (int64_t pages : big) {
                        const size_t n = qmm_kv_bytes(t, heads, dim, page, pages);
                        EXPECT(n % 16 == 0 && n <= (size_t)INT64_MAX / 8);
                    }
    qmm_kv_cache c = {buf, buf, QMM_Q8_0, 8, 128, 16, 100};
    qmm_kv_batch b = {reinterpret_cast<int32_t*>(buf), reinterpret_cast<int32_t*>(buf), reinterpret_cast<int32_t*>(buf), 1, 1, 1, 0};
    qmm_attn_opts o = {0.1f, 0.f, 0, 0, nullptr, nullptr};
    int valid = 0;
    for (int type : types)
        for (int n_kv : {1, 8, 4096, 5000})
            for (int g : {1, 4, 7, 40, 300})
                for (int seqs : ints)
                    for (int64_t tokens : big)
                        for (int width : ints)
                            for (int64_t max_kv : big)
                                for (int algo : {0, 1, 2}) {
                                    c.type = type, c.n_kv = n_kv, b.n_seqs = seqs, b.n_tokens = tokens;
                                    b.table_width = width, b.max_kv = max_kv, o.algo = algo;
                                    o.window = width & 64;
                                    const int64_t n_q = (int64_t)n_kv * g;
                                    const int before = g_launches;
                                    const size_t need = qmm_attn_work(&c, &b, &o, QMM_F32, (int)n_q);
                                    const int choice = qmm_attn_choice(&c, &b, QMM_F32, (int)n_q);
                                    const int rc = qmm_attn(&c, &b, &o, QMM_F32, buf, n_q * 128, (int)n_q, buf, buf, need, nullptr);
                                    EXPECT((rc == QMM_OK) == (g_launches == before + 1));
                                    EXPECT((rc == QMM_OK) == (choice == 1 || choice == 2));
                                    if (rc != QMM_OK) {
                                        EXPECT(need == 0);
                                        continue;
                                    }
                                    ++valid;
                                    EXPECT(g_items > 0 && g_items <= (int64_t(1) << 24));
                                    EXPECT(need == 0 ? g_parts == 0
                                                     : need >= (size_t)g_parts * 130 * 4 + (size_t)tokens * n_q * 16);
                                    if (need) {
                                        EXPECT(qmm_attn(&c, &b, &o, QMM_F32, buf, n_q * 128, (int)n_q, buf, buf, need - 1, nullptr) ==
                                               QMM_ERR_SHAPE);
                                        EXPECT(qmm_attn(&c, &b, &o, QMM_F32, buf, n_q * 128, (int)n_q, buf, nullptr, need, nullptr) ==
                                               QMM_ERR_NULL);
                                    }
                                }
    EXPECT(valid > 1000);
    c = {buf, buf, QMM_BF16, 8, 128, 16, 100};
    b.n_seqs = 1, b.n_tokens = 3, b.table_width = 4, b.max_kv = 0;
    qmm_rope r = {reinterpret_cast<double*>(buf), nullptr, 128, QMM_ROPE_PAIRS, 1, {0, 0, 0, 0}};
    for (int n_rot : ints)
        for (int axes : ints)
            for (int sec : ints) {
                r.n_rot = n_rot, r.n_axes = axes, r.sections[0] = sec, r.sections[1] = n_rot / 2 - (sec > 0 && sec < 4096 ? sec : 0);
                const int before = g_launches;
                const int rc = qmm_kv_append(&c, &b, &r, QMM_F32, buf, 1024, buf, 1024, buf, 1024, 8, buf, nullptr);
                EXPECT((rc == QMM_OK) == (g_launches == before + 1));
                if (rc == QMM_OK) EXPECT(n_rot >= 2 && n_rot <= 128 && axes >= 1 && axes <= 4);
            }
    for (int64_t ld : big) {
        const int before = g_launches;
        const int rc = qmm_kv_append(&c, &b, nullptr, QMM_F32, buf, ld, buf, ld, nullptr, 0, 0, nullptr, nullptr);
        EXPECT((rc == QMM_OK) == (g_launches == before + 1) && (rc != QMM_OK || ld >= 1024));
    }
    for (double v : {0.0, -1.0, 1.0, 1e300, (double)INFINITY, (double)NAN})
        for (int n : ints) {
            const int rc = qmm_rope_freqs(reinterpret_cast<double*>(buf), n, v, v, nullptr, nullptr);
            if (rc == QMM_OK) EXPECT(n > 0 && n % 2 == 0 && isfinite(v) && v > 0);
        }
    if (failures) return 1;
    printf("kv validation ok\n");
    return 0;
}
