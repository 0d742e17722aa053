/*
 * hip_errors.c -- what a failed call leaves behind. Kernel launches are
 * checked by the runtime's record of the last error, which a successful call
 * does not clear: an error that a call has reported must not be found there by
 * the next one. This program defines the runtime's memory and error calls
 * itself (the library binds to them: it is linked with -rdynamic), makes them
 * fail in turn, and looks at the record after each refusal. Needs no GPU; no
 * kernel is launched. Prints "hip errors ok" and exits 0, or says what is wrong.
 */
#define __HIP_PLATFORM_AMD__ 1
#include <hip/hip_runtime_api.h>
#include <stdint.h>
#include <stdio.h>
#include <stdlib.h>
#include <string.h>

#include "zsp.h"

static hipError_t last = hipSuccess;
static int fail_malloc, fail_copy, fail_wait, fail_device, blocks;
static char symbol[64];

static hipError_t leave(hipError_t e) {
    if (e != hipSuccess) last = e;
    return e;
}
hipError_t hipGetLastError(void) {
    const hipError_t e = last;
    last = hipSuccess;
    return e;
}
hipError_t hipGetDevice(int* d) {
    *d = 0;
    return leave(fail_device ? hipErrorInvalidDevice : hipSuccess);
}
hipError_t hipMalloc(void** p, size_t n) {
    if (fail_malloc) return leave(hipErrorOutOfMemory);
    ++blocks;
    *p = malloc(n);
    return hipSuccess;
}
hipError_t hipFree(void* p) {
    if (p) --blocks;
    free(p);
    return hipSuccess;
}
hipError_t hipMemcpy(void* d, const void* s, size_t n, hipMemcpyKind k) {
    (void)k;
    if (fail_copy) return leave(hipErrorInvalidValue);
    memcpy(d, s, n);
    return hipSuccess;
}
hipError_t hipMemcpyAsync(void* d, const void* s, size_t n, hipMemcpyKind k, hipStream_t st) {
    (void)st;
    return hipMemcpy(d, s, n, k);
}
hipError_t hipStreamSynchronize(hipStream_t st) {
    (void)st;
    return leave(fail_wait ? hipErrorUnknown : hipSuccess);
}
hipError_t hipGetSymbolAddress(void** p, const void* s) {
    (void)s;
    *p = symbol;
    return hipSuccess;
}
const char* hipGetErrorString(hipError_t e) { return e == hipSuccess ? "no error" : "an error"; }

static int bad;

static void want(const char* what, zsp_status got, zsp_status status, int left) {
    if (got != status || last != hipSuccess || blocks != left) {
        printf("%s: status %d (not %d), error %d left, %d blocks (not %d)\n", what, (int)got,
               (int)status, (int)last, blocks, left);
        bad = 1;
        last = hipSuccess;
    }
}

int main(void) {
    void* const x[1] = {(void*)(uintptr_t)4096}; /* no call follows it */
    const int64_t numel[1] = {5000};
    const int32_t dtype[1] = {ZSP_F32};
    zsp_tensor_list* list = NULL;

    fail_malloc = 1;
    want("tensor list, no memory", zsp_tensor_list_create(x, numel, dtype, 1, NULL, &list),
         ZSP_ENOMEM, 0);
    fail_malloc = 0, fail_copy = 1;
    want("tensor list, copy", zsp_tensor_list_create(x, numel, dtype, 1, NULL, &list), ZSP_EHIP, 0);
    fail_copy = 0, fail_wait = 1;
    want("tensor list, wait", zsp_tensor_list_create(x, numel, dtype, 1, NULL, &list), ZSP_EHIP, 0);
    fail_wait = 0, fail_device = 1;
    want("tensor list, device", zsp_tensor_list_create(x, numel, dtype, 1, NULL, &list), ZSP_EHIP,
         0);
    fail_device = 0;
    if (list != NULL) {
        printf("a refused list is not NULL\n");
        bad = 1;
    }
    want("tensor list", zsp_tensor_list_create(x, numel, dtype, 1, NULL, &list), ZSP_OK, 1);
    fail_device = 1;
    want("list norm, device",
         zsp_tensor_list_norm(list, ZSP_NORM_L2, 1.0, x[0], 1 << 20, (zsp_clip*)x[0], NULL),
         ZSP_EHIP, 1);
    fail_device = 0;
    zsp_tensor_list_destroy(list);
    want("destroyed", ZSP_OK, ZSP_OK, 0);

    zsp_plan* P = NULL;
    zsp_gather_list* G = NULL;
    float* const f = (float*)x[0];
    uint16_t* const h = (uint16_t*)x[0];
    int32_t ids[65]; /* more than travel in the kernel arguments */
    void* outs[65];
    for (int i = 0; i < 65; ++i) ids[i] = 0, outs[i] = x[0];
    want("plan", zsp_partition(numel, 1, 2, &P), ZSP_OK, 0);
    fail_malloc = 1;
    want("bind, no memory", zsp_bind_state(P, ZSP_ALL_RANKS, f, f, f, h, NULL), ZSP_ENOMEM, 0);
    fail_malloc = 0, fail_copy = 1;
    want("bind, copy", zsp_bind_state(P, ZSP_ALL_RANKS, f, f, f, h, NULL), ZSP_EHIP, 0);
    fail_copy = 0;
    want("bind", zsp_bind_state(P, ZSP_ALL_RANKS, f, f, f, h, NULL), ZSP_OK, 1);
    fail_malloc = 1;
    want("gather list, no memory",
         zsp_gather_list_create(P, ids, 65, ZSP_SRC_WORK, outs, NULL, &G), ZSP_ENOMEM, 1);
    fail_malloc = 0;
    zsp_destroy(P);
    want("plan destroyed", ZSP_OK, ZSP_OK, 0);
    if (!bad) printf("hip errors ok\n");
    return bad;
}
