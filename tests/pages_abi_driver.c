/* Refusals and workspace queries of packed and paged attention, page slots and
 * page writes, for a build of the library's host code with AddressSanitizer and
 * UndefinedBehaviorSanitizer (tests/test_pages_sanitizers.py).  No GPU is
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
/* refused, or stopped where there is no device: never done */
#define NEVER_DONE(call)               \
    do {                               \
        ++checks;                      \
        if ((call) == LACT_OK) {       \
            ++failures;                \
            fprintf(stderr, "line %d: %s was done\n", __LINE__, #call); \
        }                              \
    } while (0)

/* aligned addresses that nothing dereferences */
#define F(n) ((void*)(uintptr_t)((uintptr_t)(n) << 20))

static const int32_t i32[] = {INT32_MIN, -1, 0, 1, 8, 40, 65536, (1 << 24), INT32_MAX};
static const int64_t i64[] = {INT64_MIN, -1, 0, 1, 500, (INT64_C(1) << 30) - 1, INT64_C(1) << 30, INT64_MAX};
enum { N32 = sizeof(i32) / sizeof(i32[0]), N64 = sizeof(i64) / sizeof(i64[0]) };

int main(void) {
    const lact_strides st = {1 << 20, 64, 256}, pool = {16 * 256, 64, 256}, far = {INT64_MAX, INT64_MAX, INT64_MAX},
                       one = {0, 8, 8};
    lact_packed k;
    memset(&k, 0, sizeof(k));
    k.batch = 3, k.heads = 4, k.kv_heads = 2, k.d = 64, k.io_dtype = LACT_DTYPE_BF16, k.scale = 0.125f;
    k.tokens = 200, k.longest = 100, k.window = 16, k.sinks = 4;
#define PACKED(p, s) lact_packed_attention_forward(p, F(1), s, F(2), s, F(3), s, F(4), F(5), s, F(6), NULL)
#define BACK(p, s, n)                                                                                             \
    lact_packed_attention_backward(p, F(1), s, F(2), s, F(3), s, F(4), F(5), s, F(6), F(7), s, F(8), s, F(9), s, \
                                   F(10), s, F(11), n, NULL)
    EXPECT(PACKED(&k, &st), LACT_ERR_NO_DEVICE);
    EXPECT(PACKED(NULL, &st), LACT_ERR_INVALID_ARG);
    EXPECT(PACKED(&k, NULL), LACT_ERR_INVALID_ARG);
    EXPECT(PACKED(&k, &far), LACT_ERR_INVALID_ARG);
    const size_t need = lact_packed_attention_backward_workspace_size(&k);
    EXPECT(BACK(&k, &st, need), LACT_ERR_NO_DEVICE);
    EXPECT(BACK(&k, &st, need - 1), LACT_ERR_WORKSPACE_TOO_SMALL);
    for (int i = 0; i < N32; ++i)
        for (int j = 0; j < N64; ++j)
            for (int l = 0; l < N64; ++l)
                for (int what = 0; what < 8; ++what) {
                    lact_packed b = k;
                    if (what & 1) b.batch = i32[i];
                    if (what & 2) b.heads = b.kv_heads = i32[i];
                    if (what & 4) b.d = 128, b.io_dtype = LACT_DTYPE_F32, b.flags = LACT_CLEAR_REST;
                    b.tokens = i64[j];
                    b.longest = i64[l];
                    b.window = what == 3 ? i64[l] : 16;
                    b.sinks = what == 5 ? i64[l] : 4;
                    (void)lact_packed_attention_backward_workspace_size(&b);
                    const lact_status s = PACKED(&b, &st), t = BACK(&b, &st, SIZE_MAX);
                    ++checks;
                    if (b.tokens != 0 && (t == LACT_OK || (s == LACT_OK && b.batch != 0 && b.longest != 0))) ++failures;
                }

    lact_paged g;
    memset(&g, 0, sizeof(g));
    g.batch = 3, g.heads = 4, g.kv_heads = 2, g.d = 64, g.io_dtype = LACT_DTYPE_BF16, g.scale = 0.125f;
    g.tokens = 200, g.longest = 100, g.k_len = 500, g.window = 16, g.sinks = 4, g.pages = 50, g.page = 16, g.width = 40;
#define PAGED(p, s, w, n)                                                                                              \
    lact_paged_attention(p, F(1), s, F(2), &pool, F(3), &pool, F(4), F(5), F(6), F(7), s, F(8), w, n, NULL)
    EXPECT(PAGED(&g, &st, F(9), SIZE_MAX), LACT_ERR_NO_DEVICE);
    EXPECT(PAGED(NULL, &st, F(9), SIZE_MAX), LACT_ERR_INVALID_ARG);
    EXPECT(PAGED(&g, &far, F(9), SIZE_MAX), LACT_ERR_INVALID_ARG);
    for (int i = 0; i < N32; ++i)
        for (int j = 0; j < N64; ++j)
            for (int l = 0; l < N64; ++l)
                for (int what = 0; what < 10; ++what) {
                    lact_paged b = g;
                    if (what == 0) b.batch = i32[i];
                    if (what == 1) b.heads = b.kv_heads = i32[i];
                    if (what == 2) b.page = i32[i];
                    if (what == 3) b.pages = i32[i];
                    if (what == 4) b.width = i32[i];
                    if (what == 5) b.d = 128, b.io_dtype = LACT_DTYPE_F32, b.batch = i32[i];
                    if (what == 6) b.batch = 1, b.longest = i64[l], b.tokens = INT64_MAX;
                    if (what == 7) b.batch = 1, b.window = i64[l], b.sinks = i64[j];
                    if (what >= 8) b.batch = what == 8 ? 1 : i32[i], b.width = 1 << 14, b.page = 65528, b.pages = 32768;
                    if (what != 7) b.k_len = i64[j];
                    if (what != 6) b.tokens = i64[l], b.longest = i64[l] < 0 ? 0 : i64[l] / (i + 1);
                    const size_t n = lact_paged_attention_workspace_size(&b);
                    const lact_status s = PAGED(&b, &one, F(9), n);
                    (void)PAGED(&b, &st, F(9), n);
                    ++checks;
                    if (s == LACT_OK && b.tokens != 0) ++failures;
                }

    lact_slots q;
    memset(&q, 0, sizeof(q));
    q.batch = 3, q.page = 16, q.width = 10, q.entries = 50, q.tokens = 100;
#define SLOTS(p, n) \
    lact_page_slots(p, F(1), F(2), F(3), F(4), F(5), F(6), F(7), F(8), F(9), F(10), F(11), n, NULL)
    EXPECT(SLOTS(&q, 0), LACT_ERR_NO_DEVICE);
    EXPECT(SLOTS(NULL, 0), LACT_ERR_INVALID_ARG);
    q.batch = 5000;
    EXPECT(SLOTS(&q, lact_page_slots_workspace_size(&q)), LACT_ERR_NO_DEVICE);
    EXPECT(SLOTS(&q, lact_page_slots_workspace_size(&q) - 1), LACT_ERR_WORKSPACE_TOO_SMALL);
    for (int i = 0; i < N32; ++i)
        for (int l = 0; l < N32; ++l)
            for (int j = 0; j < N64; ++j) {
                lact_slots b = {i32[i], 16, i32[l], 50, i64[j]}, c = {3, i32[i], 10, i32[l], i64[j]};
                NEVER_DONE(SLOTS(&b, lact_page_slots_workspace_size(&b)));
                NEVER_DONE(SLOTS(&c, lact_page_slots_workspace_size(&c)));
            }

    lact_write w;
    memset(&w, 0, sizeof(w));
    w.kv_heads = 4, w.d = 64, w.io_dtype = LACT_DTYPE_BF16, w.pages = 10, w.page = 16, w.tokens = 30;
#define WRITE(p, s) lact_page_write(p, F(1), s, F(2), s, F(3), F(4), &pool, F(5), &pool, NULL)
    EXPECT(WRITE(&w, &st), LACT_ERR_NO_DEVICE);
    EXPECT(WRITE(NULL, &st), LACT_ERR_INVALID_ARG);
    EXPECT(WRITE(&w, &far), LACT_ERR_INVALID_ARG);
    const lact_strides wide = {INT64_C(8192) * 65536, 8192, INT64_C(8192) * 65536};
    for (int i = 0; i < N32; ++i)
        for (int l = 0; l < N32; ++l)
            for (int j = 0; j < N64; ++j) {
                lact_write b = {i32[i], i32[l], LACT_DTYPE_F32, 10, 16, i64[j]};
                lact_write c = {4, 64, LACT_DTYPE_BF16, i32[i], i32[l], i64[j]};
                lact_status s = lact_page_write(&b, F(1), &wide, F(2), &wide, F(3), F(4), &wide, F(5), &wide, NULL);
                ++checks;
                if (s == LACT_OK && b.tokens != 0) ++failures;
                s = WRITE(&c, &st);
                ++checks;
                if (s == LACT_OK && c.tokens != 0 && c.pages != 0) ++failures;
            }
    printf("%d checks, %d failures\n", checks, failures);
    return failures != 0;
}
