/*
 * Host sanitizer driver for the nvfp4_kv_* entry points at the ends of their
 * arguments' ranges (test code): strides that no count uses, tables of more
 * bytes than 64 bits hold, and the largest counts.  Built and run as
 * sanitize_kv.c is, without a GPU; device pointers are fake addresses, never
 * dereferenced on the host.
 *
 * Exit status: 0 clean, 1 a status differed from the documented one, 3 a
 * device is visible (nothing called).
 */
#include <hip/hip_runtime_api.h>
#include <stdint.h>
#include <stdio.h>

#include "nvfp4rq.h"

static int failures = 0;
static long calls = 0;

#define P(t, k) ((t *)((uintptr_t)(k) << 46))
/* the last buffer, for one of 2^62 bytes */
#define LAST(t) ((t *)((uintptr_t)1 << 62))

/* want: a status, or 100 for any that passed the checks */
static void expect(const char *what, int64_t a, int64_t b, int64_t got, int64_t want)
{
    calls++;
    if (want == 100 ? got != NVFP4_OK && got != NVFP4_ERR_HIP : got != want) {
        fprintf(stderr, "FAIL %s (%lld, %lld): %lld, expected %lld\n", what, (long long)a, (long long)b,
                (long long)got, (long long)want);
        failures++;
    }
}

static nvfp4_status plan(int64_t n, int64_t width)
{
    return nvfp4_kv_plan(P(int32_t, 1), P(int32_t, 2), n, 16, LAST(int32_t), width, P(int32_t, 4), 100,
                         P(int32_t, 5), P(int64_t, 6), 5, P(int32_t, 7), P(int32_t, 8), P(int32_t, 9),
                         P(int32_t, 10), 0);
}

int main(void)
{
    int count = -1;
    const hipError_t e = hipGetDeviceCount(&count);
    if (e == hipSuccess && count > 0) {
        fprintf(stderr, "a device is visible: this driver only runs without one\n");
        return 3;
    }
    const int64_t big[] = {(int64_t)1 << 29, ((int64_t)1 << 30) + 1, INT32_MAX - 1, INT32_MAX};
    for (int i = 0; i < 4; ++i)
        for (int j = 0; j < 4; ++j) {
            const int fits = big[i] <= ((int64_t)1 << 60) / big[j];
            expect("plan", big[i], big[j], plan(big[i], big[j]), fits ? 100 : NVFP4_ERR_SHAPE);
        }
    expect("plan of no requests", 0, INT32_MAX, plan(0, INT32_MAX), 100);
    expect("plan of no width", INT32_MAX, 0, plan(INT32_MAX, 0), 100);

    const nvfp4_kv_cache one = {P(uint8_t, 1), P(float, 2), 9, 1, 128, 16, 1};
    const nvfp4_kv_cache two = {P(uint8_t, 1), P(float, 2), 9, 2, 128, 16, 1};
    /* a stride that its count does not use */
    const int64_t top = INT64_MAX / 16 * 16;
    const int64_t far[] = {(int64_t)1 << 60, (int64_t)1 << 61, (int64_t)1 << 62, top};
    nvfp4_kv_batch b = {P(int32_t, 3), 7, P(int32_t, 4), P(int32_t, 5), 3, 4, 100, 1, 0, 0.1f};
    for (int i = 0; i < 4; ++i) {
        const int64_t f = far[i], ts[2] = {f, 128}, hs[2] = {256, f}, both[2] = {f, f}, ok[2] = {256, 128};
        expect("append", f, 0, nvfp4_kv_append(P(uint16_t, 6), P(uint16_t, 7), 1, ts, ok, P(int64_t, 8), &two, 0), 100);
        expect("append", f, 1, nvfp4_kv_append_f32(P(float, 6), P(float, 7), 1, ok, ts, P(int64_t, 8), &two, 0), 100);
        expect("append", f, 2, nvfp4_kv_append(P(uint16_t, 6), P(uint16_t, 7), 5, hs, ok, P(int64_t, 8), &one, 0), 100);
        expect("append", f, 3, nvfp4_kv_append_f32(P(float, 6), P(float, 7), 1, both, both, P(int64_t, 8), &one, 0), 100);
        expect("append", f, 4, nvfp4_kv_append(P(uint16_t, 6), P(uint16_t, 7), 0, both, both, P(int64_t, 8), &one, 0),
               NVFP4_OK);
        expect("append", f, 5, nvfp4_kv_append(P(uint16_t, 6), P(uint16_t, 7), 2, ts, ok, P(int64_t, 8), &two, 0),
               NVFP4_ERR_SHAPE);
        expect("append", f, 6, nvfp4_kv_append(P(uint16_t, 6), P(uint16_t, 7), 1, hs, ok, P(int64_t, 8), &two, 0),
               NVFP4_ERR_SHAPE);
        const int64_t qs[2] = {f, 128}, one_head[2] = {f, f};
        expect("attention", f, 0, nvfp4_kv_attention(P(uint16_t, 6), 1, 8, qs, &two, &b, P(uint16_t, 7), qs,
                                                     P(void, 8), INT64_MAX, 0), 100);
        expect("attention", f, 1, nvfp4_kv_attention_f32(P(float, 6), 1, 1, one_head, &one, &b, P(float, 7), one_head,
                                                         P(void, 8), INT64_MAX, 0), 100);
        expect("attention", f, 2, nvfp4_kv_attention(P(uint16_t, 6), 2, 8, qs, &two, &b, P(uint16_t, 7), qs,
                                                     P(void, 8), INT64_MAX, 0), NVFP4_ERR_SHAPE);
    }
    /* a stride that is too fine stays refused, used or not */
    const int64_t fine[2] = {top + 1, 128}, ok[2] = {256, 128};
    expect("append", 7, 0, nvfp4_kv_append(P(uint16_t, 6), P(uint16_t, 7), 1, fine, ok, P(int64_t, 8), &two, 0),
           NVFP4_ERR_ALIGN);

    for (int i = 0; i < 4; ++i)
        for (int j = 0; j < 4; ++j) {
            const int64_t st[2] = {1024, 128};
            b.table = LAST(int32_t);
            b.requests = big[i];
            b.table_width = big[j];
            const int fits = big[i] <= ((int64_t)1 << 60) / big[j] && big[i] < INT32_MAX;
            b.max_q = 1;  /* ranges of the rows kernel alone: any number of requests */
            expect("workspace", big[i], big[j], nvfp4_kv_attention_workspace(12, 8, &one, &b) >= 0, fits);
            expect("attention", big[i], big[j],
                   nvfp4_kv_attention(P(uint16_t, 6), 12, 8, st, &one, &b, P(uint16_t, 7), st, P(void, 8), INT64_MAX,
                                      0), fits ? 100 : NVFP4_ERR_SHAPE);
        }
    if (failures) {
        fprintf(stderr, "%d of %ld checks failed\n", failures, calls);
        return 1;
    }
    printf("K/V entry points clean at the ends of their ranges: %ld checks\n", calls);
    return 0;
}
