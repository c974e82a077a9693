/*
 * C driver of the host side of the operators around the attention layers (norm
 * and rotation, page plan, 4-bit cache), built with AddressSanitizer and
 * UndefinedBehaviorSanitizer against a host-only build of them: refusals,
 * workspace queries and, on a host without a GPU, valid calls over sizes up to the
 * documented limits, which plan their launches and must come back as GDR_ERR_HIP
 * (or, where a launch would be too large, GDR_ERR_BAD_SHAPE).
 * Exit status: 0 pass, 1 a check failed, 77 skipped (a GPU is visible).
 */
#include <limits.h>
#include <stdint.h>
#include <stdio.h>

#include "gdr.h"

extern int hipGetDeviceCount(int* count);

static int failures = 0;
static long calls = 0;

#define EXPECT(call, want)                                                            \
    do {                                                                              \
        int got_ = (call);                                                            \
        ++calls;                                                                      \
        if (got_ != (want)) {                                                         \
            fprintf(stderr, "line %d: %s = %d, expected %d\n", __LINE__, #call, got_, \
                    (want));                                                          \
            ++failures;                                                               \
        }                                                                             \
    } while (0)
#define LAUNCHES(call)                                                                          \
    do {                                                                                        \
        int got_ = (call);                                                                      \
        ++calls;                                                                                \
        if (got_ != GDR_ERR_HIP && got_ != GDR_ERR_BAD_SHAPE) {                                 \
            fprintf(stderr, "line %d: %s = %d, expected a launch that fails\n", __LINE__, #call, got_); \
            ++failures;                                                                         \
        }                                                                                       \
    } while (0)

/* Fake, non-NULL, aligned addresses: never dereferenced on the host. */
static void* fake(int i) { return (void*)(uintptr_t)(0x100000u * (unsigned)(i + 1)); }

static void* p[16];

static void rope(int dtype, int flags, int tokens, int Hq, int Hkv, int d, int rot, long long pad) {
    const long long sq = (long long)Hq * d + pad, sk = (long long)Hkv * d + pad;
    const int norm = !(flags & GDR_ROPE_NO_NORM);
    const size_t need = gdr_attn_norm_rope_backward_workspace_bytes(dtype, tokens, Hq, Hkv, d);
    LAUNCHES(gdr_attn_norm_rope(dtype, flags, tokens, Hq, Hkv, d, rot, 1e-6f, sq, sk, p[0], p[1], norm ? (float*)p[2] : 0,
                                norm ? (float*)p[3] : 0, (int*)p[4], (float*)p[5], p[6], p[7], 0));
    if (need == 0 || need > ((size_t)1 << 20)) {
        fprintf(stderr, "workspace of %d tokens, heads %d + %d: %zu\n", tokens, Hq, Hkv, need);
        ++failures;
    }
    LAUNCHES(gdr_attn_norm_rope_backward(dtype, flags, tokens, Hq, Hkv, d, rot, 1e-6f, sq, sk, sq, sk, p[0], p[1], 0, 0,
                                         (int*)p[4], (float*)p[5], p[6], p[7], p[8], p[9], norm ? (float*)p[10] : 0, 0, p[12],
                                         need, 0));
    if (norm)
        EXPECT(gdr_attn_norm_rope_backward(dtype, flags, tokens, Hq, Hkv, d, rot, 1e-6f, sq, sk, sq, sk, p[0], p[1], 0, 0,
                                           (int*)p[4], (float*)p[5], p[6], p[7], p[8], p[9], (float*)p[10], 0, p[12], need - 1,
                                           0), GDR_ERR_WORKSPACE);
}

static void decode(int dtype, int B, int Tq, int Hq, int Hkv, int d, int page, int pages, int width, int window, int sinks) {
    const size_t need = gdr_attn_decode_mx4_workspace_bytes(dtype, B, Tq, Hq, Hkv, d, page, width, window, sinks);
    LAUNCHES(gdr_attn_decode_mx4(dtype, B, Tq, Hq, Hkv, d, page, pages, width, window, sinks, 0.1f, p[0], p[1], p[2], p[3], p[4],
                                 (int*)p[5], (int*)p[6], p[7], need ? p[8] : 0, need, 0));
    if (need)
        EXPECT(gdr_attn_decode_mx4(dtype, B, Tq, Hq, Hkv, d, page, pages, width, window, sinks, 0.1f, p[0], p[1], p[2], p[3],
                                   p[4], (int*)p[5], (int*)p[6], p[7], p[8], need - 1, 0), GDR_ERR_WORKSPACE);
}

int main(void) {
    static const int tokens[] = {1, 2, 31, 64, 1000, 8192, 1 << 20, (1 << 29) / 64};
    static const int heads[][2] = {{1, 0}, {0, 1}, {1, 1}, {4, 2}, {32, 8}, {5, 5}, {40, 1}};
    static const int totals[] = {1, 2, 33, 4096, 1 << 20, 1 << 26};
    static const int pages[] = {32, 64, 1024, 65536};
    int devices = 0, i, j, k, dtype, d;
    for (i = 0; i < 16; ++i) p[i] = fake(i);
    if (hipGetDeviceCount(&devices) == 0 && devices > 0) return 77;
    for (dtype = 0; dtype < 2; ++dtype)
        for (d = 64; d <= 128; d += 64) {
            for (i = 0; i < (int)(sizeof tokens / sizeof *tokens); ++i)
                for (j = 0; j < (int)(sizeof heads / sizeof *heads); ++j)
                    for (k = 0; k < 4; ++k)
                        if ((long long)tokens[i] * (heads[j][0] + heads[j][1]) < (1 << 29))
                            rope(dtype, k, tokens[i], heads[j][0], heads[j][1], d, k ? d : 16, 64 * k);
            rope(dtype, 0, 1, 1 << 15, 1 << 15, d, d, 0);
            rope(dtype, 1, (1 << 13) - 1, 1 << 15, 1 << 15, d, d, 0);
            for (i = 0; i < (int)(sizeof totals / sizeof *totals); ++i)
                for (j = 0; j < (int)(sizeof pages / sizeof *pages); ++j)
                    for (k = 1; k <= 65536; k *= 256) {
                        LAUNCHES(gdr_attn_append_mx4(dtype, k, totals[i], 3, d, pages[j], 100, 100, p[0], p[1], (int*)p[2],
                                                     (int*)p[3], p[4], p[5], p[6], p[7], (int*)p[8], 0));
                        LAUNCHES(gdr_attn_read_mx4(dtype, k, totals[i], 3, d, pages[j], 100, 100, p[4], p[5], p[6], p[7],
                                                   (int*)p[8], (int*)p[2], 0, p[0], p[1], 0));
                        decode(dtype, k, 1 + 21 * j, 12, 3, d, pages[j], 100, 1 + totals[i] / pages[j], 0, 0);
                        decode(dtype, k, 1 + 21 * j, 12, 3, d, pages[j], 100, 1 + totals[i] / pages[j], 1000, 70);
                    }
            decode(dtype, 1, 1, 1, 1, d, 32, 1, (INT_MAX - 4096) / 32, 0, 0);
            decode(dtype, 3, 64, 64, 1, d, 65536, 1, (INT_MAX - 4096) / 65536, INT_MAX, INT_MAX);
            decode(dtype, 100, 64, 1 << 15, 1 << 15, d, 32, 1, 5, 0, 0);
        }
    for (i = 0; i < (int)(sizeof totals / sizeof *totals); ++i)
        for (j = 1; j <= 65536; j *= 16) {
            LAUNCHES(gdr_attn_plan_pages(totals[i], j, 7, 100, INT_MAX, (int*)p[0], (int*)p[1], (int*)p[2], (int*)p[3], (int*)p[4],
                                         (int*)p[5], (int*)p[6], (int*)p[7], 0, (int*)p[8], 0));
            LAUNCHES(gdr_attn_plan_pages(INT_MAX - 1, j, 7, INT_MAX, totals[i], (int*)p[0], (int*)p[1], (int*)p[2], (int*)p[3],
                                         (int*)p[4], (int*)p[5], (int*)p[6], (int*)p[7], (int*)p[9], (int*)p[8], 0));
        }
    LAUNCHES(gdr_attn_plan_pages(0, 16, 0, 0, 0, 0, 0, 0, (int*)p[3], 0, (int*)p[5], 0, 0, 0, (int*)p[8], 0));
    if (failures) return 1;
    printf("%ld calls, all checks passed\n", calls);
    return 0;
}
