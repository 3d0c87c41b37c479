/* Refusals and workspace queries of the operators around the fast-weight
 * layer, for a build of the library's host code with AddressSanitizer and
 * UndefinedBehaviorSanitizer (tests/test_block_sanitizers.py).  No GPU is
 * needed: every case returns before any device work (valid argument sets stop
 * at the device check).  Exit status 0 when every status is the expected one. */
#include <limits.h>
#include <stdint.h>
#include <stdio.h>
#include <string.h>

#include "lact.h"

static int failures = 0, checks = 0;

#define EXPECT(call, code)                                                                     \
    do {                                                                                       \
        lact_status s_ = (call);                                                               \
        ++checks;                                                                              \
        if (s_ != (code)) {                                                                    \
            ++failures;                                                                        \
            fprintf(stderr, "line %d: %s -> %d, expected %d (%s)\n", __LINE__, #call, (int)s_, \
                    (int)(code), lact_last_error());                                           \
        }                                                                                      \
    } while (0)

/* aligned addresses that nothing dereferences */
#define F(n) ((void*)(uintptr_t)((uintptr_t)(n) << 20))

int main(void) {
    lact_attention a;
    memset(&a, 0, sizeof(a));
    a.batch = 2;
    a.heads = 4;
    a.kv_heads = 2;
    a.d = 64;
    a.io_dtype = LACT_DTYPE_BF16;
    a.scale = 0.125f;
    a.q_len = a.k_len = 64;
    a.window = 16;
    a.sinks = 4;
    const lact_strides st = {4 * 64 * 64, 64 * 64, 64}, far = {INT64_MAX, INT64_MAX, INT64_MAX};
#define FWD(p, s, ws, n) \
    lact_window_attention_forward(p, F(1), s, F(2), s, F(3), s, NULL, NULL, F(4), s, NULL, ws, n, NULL)
    EXPECT(FWD(&a, &st, NULL, 0), LACT_ERR_NO_DEVICE);
    EXPECT(FWD(NULL, &st, NULL, 0), LACT_ERR_INVALID_ARG);
    EXPECT(FWD(&a, NULL, NULL, 0), LACT_ERR_INVALID_ARG);
    EXPECT(FWD(&a, &far, NULL, 0), LACT_ERR_INVALID_ARG);
    /* the largest and smallest of every number */
    const int32_t i32[] = {INT32_MIN, -1, 0, 1, 7, INT32_MAX};
    const int64_t i64[] = {INT64_MIN, -1, 0, 1, (INT64_C(1) << 30) - 1, INT64_C(1) << 30, INT64_MAX};
    for (int i = 0; i < 6; ++i)
        for (int j = 0; j < 7; ++j)
            for (int what = 0; what < 7; ++what) {
                lact_attention b = a;
                if (what == 0) b.batch = i32[i];
                if (what == 1) b.heads = b.kv_heads = i32[i];
                if (what == 2) b.d = i32[i];
                if (what == 3) b.io_dtype = i32[i];
                b.window = i64[j];
                b.sinks = what < 4 ? 4 : i64[(j + i) % 7];
                if (what == 5) b.q_len = i64[j];
                if (what == 6) b.k_len = i64[j], b.batch = i32[i];
                (void)lact_window_attention_workspace_size(&b);
                (void)lact_window_attention_backward_workspace_size(&b);
                lact_status s = FWD(&b, &st, F(5), SIZE_MAX);
                ++checks;
                if (s == LACT_OK && b.batch != 0 && b.q_len != 0) ++failures;
            }
    size_t need = lact_window_attention_backward_workspace_size(&a);
#define BWD(n)                                                                                                  \
    lact_window_attention_backward(&a, F(1), &st, F(2), &st, F(3), &st, NULL, NULL, F(4), &st, F(5), F(6), &st, \
                                   F(7), &st, F(8), &st, F(9), &st, F(10), n, NULL)
    EXPECT(BWD(need), LACT_ERR_NO_DEVICE);
    EXPECT(BWD(need - 1), LACT_ERR_WORKSPACE_TOO_SMALL);

    lact_rotary_problem r;
    memset(&r, 0, sizeof(r));
    r.batch = 2;
    r.heads = 4;
    r.kv_heads = 2;
    r.d = 64;
    r.pairs = 32;
    r.io_dtype = LACT_DTYPE_F32;
    r.mscale = 1.f;
    r.tokens = 64;
#define ROT(s) lact_rotary(&r, F(1), s, F(2), s, F(3), NULL, F(4), s, F(5), s, NULL)
    EXPECT(ROT(&st), LACT_ERR_NO_DEVICE);
    EXPECT(ROT(&far), LACT_ERR_INVALID_ARG);
    EXPECT(lact_rotary(NULL, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0), LACT_ERR_INVALID_ARG);
    r.heads = r.kv_heads = 65536; /* the most a workgroup's items are split for */
    r.d = 8192;
    r.pairs = 2048;
    r.batch = 1;
    const lact_strides wide = {0, 8192, INT64_C(8192) * 65536};
    EXPECT(ROT(&wide), LACT_ERR_NO_DEVICE);
    double f[2048];
    float m;
    for (int sc = -1; sc < 5; ++sc)
        for (int n = -1; n <= 2049; n += 205)
            EXPECT(lact_rotary_frequencies(n, 1e4, sc, 8., 4096, 1., 32., f, &m),
                   n < 0 || n > 2048 || sc < 0 || sc > 3 ? LACT_ERR_INVALID_ARG : LACT_OK);
    EXPECT(lact_rotary_frequencies(2, 1e4, LACT_ROTARY_NTK, 8., 0, 0., 0., f, NULL), LACT_OK);
    EXPECT(lact_rotary_frequencies(2, 1e4, LACT_ROTARY_PLAIN, 1., 0, 0., 0., NULL, NULL), LACT_ERR_INVALID_ARG);

    lact_norm_problem n;
    for (int i = 0; i < 6; ++i)
        for (int j = 0; j < 7; ++j) {
            n.rows = i64[j];
            n.cols = i32[i];
            n.io_dtype = LACT_DTYPE_BF16;
            n.eps = 1e-6f;
            (void)lact_add_rmsnorm_backward_workspace_size(&n);
            for (int l = 0; l < 7; ++l) {
                lact_status s = lact_add_rmsnorm_forward(&n, F(1), i64[l], F(2), 512, F(3), F(4), i64[l], F(5), 512,
                                                         NULL, 0, NULL, NULL);
                ++checks;
                if (s == LACT_OK && n.rows != 0) ++failures;
                s = lact_add_rmsnorm_backward(&n, F(1), i64[l], F(2), F(3), 512, NULL, 0, F(4), i64[l], F(5), F(6),
                                              SIZE_MAX, NULL);
                ++checks;
                if (s == LACT_OK) ++failures;
            }
        }
    printf("%d checks, %d failures\n", checks, failures);
    return failures != 0;
}
