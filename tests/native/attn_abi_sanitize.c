/*
 * C driver of the attention entry points' host side, built with
 * AddressSanitizer and UndefinedBehaviorSanitizer against a host-only build of
 * them (no device code): invalid arguments, the workspace queries over a sweep
 * of sizes up to the documented limits, and, on a host without a GPU, valid
 * calls of those sizes, which plan their launches and must come back as
 * GDR_ERR_HIP (or, where a launch would be too large, GDR_ERR_BAD_SHAPE).
 * Exit status: 0 pass, 1 a check failed, 77 skipped (a GPU is visible: the
 * valid calls would launch kernels on the fake addresses used here).
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

static void* p[12];

static void backward(int dtype, int B, int Tq, int Tk, int Hq, int Hkv, int d, int window, int sinks) {
    const size_t need = gdr_attn_backward_workspace_bytes(dtype, B, Tq, Tk, Hq, Hkv, d, window, sinks);
    const float *lse = (const float*)p[4];
    const int rows = Tq > 0;
    if (rows && need < (size_t)8 * B * Tq * Hq) {
        fprintf(stderr, "workspace of B %d Tq %d Tk %d heads %d/%d: %zu\n", B, Tq, Tk, Hq, Hkv, need);
        ++failures;
    }
    if (need) {
        EXPECT(gdr_attn_backward(dtype, B, Tq, Tk, Hq, Hkv, d, window, sinks, 0.1f, p[0], p[1], p[2], p[3], lse, p[5], p[6],
                                 p[7], p[8], p[9], need - 1, 0), GDR_ERR_WORKSPACE);
        EXPECT(gdr_attn_backward(dtype, B, Tq, Tk, Hq, Hkv, d, window, sinks, 0.1f, p[0], p[1], p[2], p[3], lse, p[5], p[6],
                                 p[7], p[8], 0, need, 0), GDR_ERR_WORKSPACE);
    }
    LAUNCHES(gdr_attn_backward(dtype, B, Tq, Tk, Hq, Hkv, d, window, sinks, 0.1f, p[0], p[1], p[2], p[3], lse, p[5], p[6], p[7],
                               p[8], p[9], need, 0));
}

int main(void) {
    int ndev = 0;
    const int hip_status = hipGetDeviceCount(&ndev);
    if (hip_status == 0 && ndev > 0) {
        printf("a GPU is visible: skipped\n");
        return 77;
    }
    for (int i = 0; i < 12; ++i) p[i] = fake(i);
    float* lse = (float*)p[4];
    const int* ia = (const int*)p[10];
    const int* ib = (const int*)p[11];

    /* each kind of refusal, each integer at the ends of its type */
    const int bad[] = {-1, INT_MIN, INT_MAX};
    for (int i = 0; i < 3; ++i) {
        const int x = bad[i];
        EXPECT(gdr_attn_prefill(x, 1, 8, 8, 4, 2, 64, 0, 0, 1.f, p[0], p[1], p[2], p[3], lse, 0), GDR_ERR_BAD_ENUM);
        EXPECT(gdr_attn_prefill(1, x, 8, 8, 4, 2, 64, 0, 0, 1.f, p[0], p[1], p[2], p[3], lse, 0), GDR_ERR_BAD_SHAPE);
        EXPECT(gdr_attn_prefill(1, 1, x, 8, 4, 2, 64, 0, 0, 1.f, p[0], p[1], p[2], p[3], lse, 0), GDR_ERR_BAD_SHAPE);
        EXPECT(gdr_attn_prefill(1, 1, 8, x, 4, 2, 64, 0, 0, 1.f, p[0], p[1], p[2], p[3], lse, 0), GDR_ERR_BAD_SHAPE);
        EXPECT(gdr_attn_prefill(1, 1, 8, 8, x, 1, 64, 0, 0, 1.f, p[0], p[1], p[2], p[3], lse, 0), GDR_ERR_BAD_SHAPE);
        EXPECT(gdr_attn_prefill(1, 1, 8, 8, 4, x, 64, 0, 0, 1.f, p[0], p[1], p[2], p[3], lse, 0), GDR_ERR_BAD_SHAPE);
        EXPECT(gdr_attn_prefill(1, 1, 8, 8, 4, 2, x, 0, 0, 1.f, p[0], p[1], p[2], p[3], lse, 0), GDR_ERR_UNSUPPORTED);
        EXPECT(gdr_attn_prefill_varlen(1, x, 8, 8, 8, 4, 2, 64, 0, 0, 1.f, p[0], p[1], p[2], ia, ib, p[3], lse, 0), GDR_ERR_BAD_SHAPE);
        EXPECT(gdr_attn_prefill_varlen(1, 2, x, 8, 8, 4, 2, 64, 0, 0, 1.f, p[0], p[1], p[2], ia, ib, p[3], lse, 0), GDR_ERR_BAD_SHAPE);
        EXPECT(gdr_attn_prefill_varlen(1, 2, 8, x, 8, 4, 2, 64, 0, 0, 1.f, p[0], p[1], p[2], ia, ib, p[3], lse, 0), GDR_ERR_BAD_SHAPE);
        EXPECT(gdr_attn_decode(1, x, 4, 2, 64, 16, 8, 4, 0, 0, 1.f, p[0], p[1], p[2], p[3], p[5], ia, ib, p[6], p[9], 1u << 30, 0), GDR_ERR_BAD_SHAPE);
        EXPECT(gdr_attn_decode(1, 2, 4, 2, 64, x, 8, 4, 0, 0, 1.f, p[0], p[1], p[2], p[3], p[5], ia, ib, p[6], p[9], 1u << 30, 0), GDR_ERR_UNSUPPORTED);
        EXPECT(gdr_attn_decode(1, 2, 4, 2, 64, 16, x, 4, 0, 0, 1.f, p[0], p[1], p[2], p[3], p[5], ia, ib, p[6], p[9], 1u << 30, 0), GDR_ERR_BAD_SHAPE);
        EXPECT(gdr_attn_decode(1, 2, 4, 2, 64, 16, 8, x, 0, 0, 1.f, p[0], p[1], p[2], p[3], p[5], ia, ib, p[6], p[9], 1u << 30, 0), GDR_ERR_BAD_SHAPE);
        EXPECT(gdr_attn_append(1, 2, x, 2, 64, 16, 8, 4, p[0], p[1], ia, ib, p[2], p[3], ia, 0), GDR_ERR_BAD_SHAPE);
        EXPECT(gdr_attn_append(1, 2, 8, x, 64, 16, 8, 4, p[0], p[1], ia, ib, p[2], p[3], ia, 0), GDR_ERR_BAD_SHAPE);
        if (gdr_attn_backward_workspace_bytes(1, x, 8, 8, 4, 2, 64, 0, 0) || gdr_attn_backward_workspace_bytes(1, 1, x, 8, 4, 2, 64, 0, 0) ||
            gdr_attn_backward_workspace_bytes(1, 1, 8, x, 4, 2, 64, 0, 0) || gdr_attn_decode_workspace_bytes(1, 2, 4, 2, 64, 16, x, 0, 0) ||
            gdr_attn_decode_workspace_bytes(1, x, 4, 2, 64, 16, 1024, 0, 0) || gdr_attn_decode_workspace_bytes(1, 2, 4, 2, 64, x, 1024, 0, 0))
            ++failures;
    }
    EXPECT(gdr_attn_prefill(1, 1, 8, 8, 4, 2, 64, -1, 0, 1.f, p[0], p[1], p[2], p[3], lse, 0), GDR_ERR_BAD_SHAPE);
    EXPECT(gdr_attn_prefill(1, 1, 8, 8, 4, 2, 64, 0, INT_MIN, 1.f, p[0], p[1], p[2], p[3], lse, 0), GDR_ERR_BAD_SHAPE);
    EXPECT(gdr_attn_prefill(1, 1, 8, 8, 4, 2, 64, 0, 0, 1.f, 0, p[1], p[2], p[3], lse, 0), GDR_ERR_NULL_PTR);
    EXPECT(gdr_attn_prefill(1, 1, 8, 8, 4, 2, 64, 0, 0, 1.f, (char*)p[0] + 8, p[1], p[2], p[3], lse, 0), GDR_ERR_MISALIGNED);
    EXPECT(gdr_attn_append(0, 0, 8, 2, 64, 16, 8, 4, 0, 0, 0, 0, 0, 0, 0, 0), GDR_OK);

    /* prefill and backward: queries before, at and after the keys, masks, groups, batches, both sides of 512 key blocks */
    const int lengths[] = {0, 1, 31, 129, 2000, 65408, 65409, 200000}, windows[] = {0, 1, 64, 4096, INT_MAX}, sinks[] = {0, 4, 300, INT_MAX};
    const int heads[][2] = {{1, 1}, {3, 1}, {40, 1}, {14, 2}, {32, 8}, {16, 16}};
    for (int dtype = 0; dtype < 2; ++dtype)
        for (int i = 0; i < 8; ++i)
            for (int j = 0; j < 8; ++j)
                for (int w = 0; w < 5; ++w)
                    for (int s = 0; s < 4; ++s)
                        for (int h = 0; h < 6; ++h) {
                            const int Tq = lengths[i], Tk = lengths[j], d = (i + j + h) % 2 ? 64 : 128, B = h == 2 ? 5 : 1;
                            if (Tq == 0 && Tk == 0) continue;
                            backward(dtype, B, Tq, Tk, heads[h][0], heads[h][1], d, windows[w], sinks[s]);
                            if (Tq == 0) continue;
                            LAUNCHES(gdr_attn_prefill(dtype, B, Tq, Tk, heads[h][0], heads[h][1], d, windows[w], sinks[s], 0.1f, p[0],
                                                      p[1], p[2], p[3], lse, 0));
                            LAUNCHES(gdr_attn_prefill_varlen(dtype, B, Tq, Tk, INT_MAX, heads[h][0], heads[h][1], d, windows[w], sinks[s],
                                                             0.1f, p[0], p[1], p[2], ia, ib, p[3], lse, 0));
                        }
    /* at the limits: 2^15 heads, fewer than 2^29 rows in a sequence */
    const int most = (1 << 29) - 1;
    const int limits[][4] = {{1, 1 << 28, 1 << 15, 1}, {(1 << 14) - 1, (1 << 14) - 1, 1 << 15, 1 << 15}, {most, most, 1, 1},
                             {1, most, 1 << 15, 1}, {most, 1, 1, 1}, {1000, 1 << 24, 128, 1}, {(1 << 14) - 1, 65000, 1 << 15, 1},
                             {1 << 24, 1 << 24, 16, 16}, {1 << 24, 60000, 31, 1}};
    for (int i = 0; i < 9; ++i)
        for (int w = 0; w < 5; ++w)
            for (int s = 0; s < 4; ++s) {
                const int *l = limits[i];
                LAUNCHES(gdr_attn_prefill(1, 1, l[0], l[1], l[2], l[3], 128, windows[w], sinks[s], 0.1f, p[0], p[1], p[2], p[3], lse, 0));
                backward(i % 2, 1, l[0], l[1], l[2], l[3], 64, windows[w], sinks[s]);
            }

    /* decode and append: pages from one position up, tables from one page to 2^31 positions */
    const int batches[] = {1, 3, 256, 5000, 1 << 20};
    for (int dtype = 0; dtype < 2; ++dtype)
        for (int shift = 0; shift <= 16; shift += 4)
            for (int t = 0; t <= 30 - shift; t += 3)
                for (int b = 0; b < 5; ++b)
                    for (int w = 0; w < 5; ++w)
                        for (int h = 0; h < 6; ++h) {
                            const int page = 1 << shift, width = 1 << t, B = batches[b], Hq = heads[h][0], Hkv = heads[h][1];
                            const size_t need = gdr_attn_decode_workspace_bytes(dtype, B, Hq, Hkv, 128, page, width, windows[w], sinks[h % 4]);
                            if (need) EXPECT(gdr_attn_decode(dtype, B, Hq, Hkv, 128, page, 100, width, windows[w], sinks[h % 4], 0.1f, p[0], p[1],
                                                             p[2], p[3], p[5], ia, ib, p[6], p[9], need - 1, 0), GDR_ERR_WORKSPACE);
                            LAUNCHES(gdr_attn_decode(dtype, B, Hq, Hkv, 128, page, 100, width, windows[w], sinks[h % 4], 0.1f, p[0], p[1], p[2],
                                                     p[3], p[5], ia, ib, p[6], p[9], need, 0));
                            LAUNCHES(gdr_attn_append(dtype, B, 1 + 777 * b, Hkv, 128, page, 100, width, p[0], p[1], ia, ib, p[2], p[3], ia, 0));
                        }
    LAUNCHES(gdr_attn_append(1, 1, (1 << 29) - 1, 1, 64, 1, 1, 1, p[0], p[1], ia, ib, p[2], p[3], ia, 0));
    EXPECT(gdr_attn_append(0, 3, (1 << 14) - 1, 1 << 15, 128, 65536, 0, 1, p[0], p[1], ia, ib, p[2], p[3], ia, 0), GDR_OK);

    if (failures) {
        fprintf(stderr, "%d checks failed\n", failures);
        return 1;
    }
    printf("all checks passed (%ld calls)\n", calls);
    return 0;
}
