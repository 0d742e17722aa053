/*
 * capi_norm.c -- gradient norm, clipping and the clipped step from plain C99
 * through include/zsp.h alone. A small padded parameter list at N_d = 5: the
 * gradients reduced in two parameter ranges with a norm each, the records
 * joined, a clipped Adam step from the accumulator, the norm of the reduced
 * gradient and a clipped fused step, a step skipped for an infinite gradient;
 * and a list of tensors, one-shot and prepared. States and clipped tensors
 * are compared bit for bit with the CPU oracle (its reduced gradient times
 * the coefficient, one fp32 rounding). A total is a sum of N squares in 64
 * bits, each rounded once: within (N + 2) * 2^-53 of itself in any order; norm
 * and coefficient add one rounding to fp32.
 * Prints "capi norm ok ..." and exits 0, or says what differs and exits 1.
 * With --host-only it stops after the checks that need no GPU.
 */
#define __HIP_PLATFORM_AMD__ 1
#include <hip/hip_runtime_api.h>
#include <math.h>
#include <stddef.h>
#include <stdint.h>
#include <stdio.h>
#include <stdlib.h>
#include <string.h>

#include "oracle.h"
#include "zsp.h"

#define ND 5
#define T 5
#define CUT 2 /* parameters of the first range */

static const int64_t NUMEL[T] = {1003, 64, 3 * 4096 + 1, 5, 4096 * 4 + 7};

/* A bf16 value in (-scale, scale), by SplitMix64 on a counter. */
static uint16_t draw_bf16(uint64_t stream, uint64_t i, float scale) {
    uint64_t x = ((stream << 40) ^ i) + 0x9E3779B97F4A7C15ull;
    x = (x ^ (x >> 30)) * 0xBF58476D1CE4E5B9ull;
    x = (x ^ (x >> 27)) * 0x94D049BB133111EBull;
    x ^= x >> 31;
    const float f = (2.0f * (float)((double)(x >> 11) * (1.0 / 9007199254740992.0)) - 1.0f) * scale;
    uint32_t bits;
    memcpy(&bits, &f, 4);
    return (uint16_t)(bits >> 16);
}

static float bf16_value(uint16_t h) {
    const uint32_t bits = (uint32_t)h << 16;
    float f;
    memcpy(&f, &bits, 4);
    return f;
}

#define HIPCK(call) do { hipError_t e_ = (call); if (e_ != hipSuccess) { \
    printf("HIP error %d (%s) in %s\n", (int)e_, hipGetErrorString(e_), #call); return 1; } } while (0)
#define ZCK(call) do { zsp_status s_ = (call); if (s_ != ZSP_OK) { \
    printf("%s -> %d: %s\n", #call, (int)s_, zsp_last_error()); return 1; } } while (0)
#define WANT(call, status) do { zsp_status s_ = (call); if (s_ != (status) || !zsp_last_error()[0]) { \
    printf("%s -> %d, not %d\n", #call, (int)s_, (int)(status)); return 1; } } while (0)

static int same(const void* a, const void* b, size_t n, const char* what) {
    if (memcmp(a, b, n) == 0) return 0;
    printf("%s differs from the oracle\n", what);
    return 1;
}

/* A record against the 64-bit total of n squares. */
static int check(const zsp_clip* c, double total, double n, double max_norm, const char* what) {
    const double norm = sqrt(total), coef = norm > max_norm ? max_norm / norm : 1.0;
    const double e64 = (n + 4) / 9007199254740992.0, e = 1.0 / 16777216.0 + e64;
    if (fabs(c->total - total) <= e64 * total && fabs(c->norm - norm) <= e * norm &&
        fabs(c->coef - coef) <= e * coef)
        return 0;
    printf("%s: total %.17g norm %.9g coef %.9g, not %.17g %.9g %.9g\n", what, c->total, c->norm,
           c->coef, total, norm, coef);
    return 1;
}

static int host_checks(zsp_plan* P) {
    void* const x = (void*)(uintptr_t)4096; /* an address that no call may follow */
    void* const xs[2] = {x, x};
    const int64_t numel[2] = {8, 8};
    const int32_t dtype[2] = {ZSP_F32, ZSP_BF16};
    zsp_clip* const rec = (zsp_clip*)x;
    zsp_tensor_list* list = (zsp_tensor_list*)x;
    int64_t ws = 0;
    if (sizeof(zsp_clip) != 16 || offsetof(zsp_clip, norm) != 8 || offsetof(zsp_clip, coef) != 12) {
        printf("zsp_clip is not laid out as documented\n");
        return 1;
    }
    ZCK(zsp_norm_workspace(NULL, &ws));
    if (ws != 35856) {
        printf("workspace of a list: %lld bytes\n", (long long)ws);
        return 1;
    }
    WANT(zsp_norm_workspace(P, NULL), ZSP_EINVAL);
    WANT(zsp_grad_norm(P, ZSP_ALL_RANKS, ZSP_NORM_L2, 1.0, x, ws, rec, NULL), ZSP_ESTATE);
    WANT(zsp_adam_step_clip(P, ZSP_ALL_RANKS, NULL, 1e-3f, 0.9f, 0.999f, 1e-8f, 1, NULL),
         ZSP_EINVAL);
    WANT(zsp_norm_many((const void* const*)xs, numel, dtype, 2, ZSP_NORM_L2, -1.0, x, ws, rec,
                       NULL), ZSP_EINVAL);
    WANT(zsp_norm_many((const void* const*)xs, numel, dtype, 2, ZSP_NORM_L2, 1.0, x, ws - 1, rec,
                       NULL), ZSP_ERANGE);
    WANT(zsp_clip_many(xs, numel, dtype, 2, rec, NULL), ZSP_EINVAL); /* they overlap */
    WANT(zsp_tensor_list_create(xs, numel, NULL, 2, NULL, &list), ZSP_EINVAL);
    if (list != NULL) {
        printf("a list that was not made is not NULL\n");
        return 1;
    }
    zsp_tensor_list_destroy(NULL);
    return 0;
}

static int run(int host_only) {
    zsp_plan* P = NULL;
    ZCK(zsp_partition(NUMEL, T, ND, &P));
    if (host_checks(P)) return 1;
    if (host_only) {
        zsp_destroy(P);
        printf("capi norm host checks ok\n");
        return 0;
    }

    int64_t S = 0, padded = 0, bytes = 0, ws_bytes = 0, numel = 0;
    int64_t o_pad[T], o_sl[T], o_full[T + 1], o_shard[T + 1], o_flat[T + 1], o_S = 0;
    ZCK(zsp_plan_info(P, &S, &padded, &bytes));
    if (orc_layout(T, NUMEL, ND, o_pad, o_sl, o_full, o_shard, o_flat, &o_S) != 0 || o_S != S)
        return 1;
    numel = o_flat[T];
    const int64_t n = (int64_t)ND * S;
    float *h = malloc(4 * n), *o_master = malloc(4 * n), *o_m = malloc(4 * n),
          *o_v = malloc(4 * n), *o_g = malloc(4 * n), *scaled = malloc(4 * n);
    uint16_t *o_work = malloc(2 * n), *params = malloc(2 * numel), *hw = malloc(2 * n);
    uint16_t* grads[ND];
    for (int64_t i = 0; i < numel; ++i) params[i] = draw_bf16(1, (uint64_t)i, 0.05f);

    float *d_master, *d_m, *d_v, *d_acc;
    uint16_t *d_work, *d_params;
    void *d_grads[ND], *ws;
    zsp_clip *rec, hrec[4];
    HIPCK(hipMalloc((void**)&d_master, 4 * n));
    HIPCK(hipMalloc((void**)&d_m, 4 * n));
    HIPCK(hipMalloc((void**)&d_v, 4 * n));
    HIPCK(hipMalloc((void**)&d_acc, 4 * n));
    HIPCK(hipMalloc((void**)&d_work, 2 * n));
    HIPCK(hipMalloc((void**)&d_params, 2 * numel));
    HIPCK(hipMalloc((void**)&rec, sizeof hrec));
    HIPCK(hipMemcpy(d_params, params, 2 * numel, hipMemcpyHostToDevice));
    for (int r = 0; r < ND; ++r) {
        grads[r] = malloc(2 * padded);
        for (int64_t i = 0; i < padded; ++i) grads[r][i] = 0x7FC0; /* NaN: pads */
        for (int t = 0; t < T; ++t)
            for (int64_t k = 0; k < NUMEL[t]; ++k)
                grads[r][o_full[t] + k] =
                    draw_bf16(100 + (uint64_t)r, (uint64_t)(o_full[t] + k), 0.01f);
        HIPCK(hipMalloc(&d_grads[r], 2 * padded));
        HIPCK(hipMemcpy(d_grads[r], grads[r], 2 * padded, hipMemcpyHostToDevice));
    }
    ZCK(zsp_bind_state(P, ZSP_ALL_RANKS, d_master, d_m, d_v, d_work, d_acc));
    ZCK(zsp_load_params(P, d_params, ZSP_BF16, NULL));
    ZCK(zsp_norm_workspace(P, &ws_bytes));
    HIPCK(hipMalloc(&ws, (size_t)ws_bytes));
    if (orc_partition(T, NUMEL, ND, 0, ND, params, ORC_BF16, o_master, o_work, o_m, o_v) != 0)
        return 1;

    double part[2] = {0.0, 0.0}, largest = 0.0;
    for (int j = 0; j < ND; ++j) {
        float* g = o_g + (int64_t)j * S;
        if (orc_reduce(T, NUMEL, ND, j, (const void* const*)grads, ORC_BF16, ORC_GRADS_FULL, g))
            return 1;
        for (int64_t i = 0; i < S; ++i) {
            part[i >= o_shard[CUT]] += (double)g[i] * g[i];
            if (fabs(g[i]) > largest) largest = fabs(g[i]);
        }
    }
    const double total = part[0] + part[1], max_norm = 0.4 * sqrt(total);
    const void* const* dg = (const void* const*)d_grads;
    const float lr = 1e-3f, b1 = 0.9f, b2 = 0.999f, eps = 1e-8f;
    int bad = 0;

    /* two ranges, joined; a clipped step from the accumulator */
    ZCK(zsp_reduce_shard_norm_params(P, ZSP_ALL_RANKS, 0, CUT, dg, ZSP_BF16, ZSP_GRADS_FULL, 0,
                                     ZSP_NORM_L2, INFINITY, ws, ws_bytes, rec, NULL));
    ZCK(zsp_reduce_shard_norm_params(P, ZSP_ALL_RANKS, CUT, T - CUT, dg, ZSP_BF16,
                                     ZSP_GRADS_FULL, 0, ZSP_NORM_L2, INFINITY, ws, ws_bytes,
                                     rec + 1, NULL));
    ZCK(zsp_clip_combine(rec, 2, ZSP_NORM_L2, max_norm, rec + 2, NULL));
    ZCK(zsp_grad_norm(P, ZSP_ALL_RANKS, ZSP_NORM_MAX, INFINITY, ws, ws_bytes, rec + 3, NULL));
    ZCK(zsp_adam_step_clip(P, ZSP_ALL_RANKS, rec + 2, lr, b1, b2, eps, 1, NULL));
    HIPCK(hipDeviceSynchronize());
    HIPCK(hipMemcpy(hrec, rec, sizeof hrec, hipMemcpyDeviceToHost));
    HIPCK(hipMemcpy(h, d_acc, 4 * n, hipMemcpyDeviceToHost));
    bad += same(h, o_g, 4 * (size_t)n, "accumulator");
    bad += check(hrec, part[0], (double)n, INFINITY, "first range");
    bad += check(hrec + 1, part[1], (double)n, INFINITY, "second range");
    bad += check(hrec + 2, total, (double)n, max_norm, "joined");
    if (hrec[3].total != largest || hrec[3].coef != 1.0f) {
        printf("largest value %.9g, not %.9g\n", hrec[3].total, largest);
        ++bad;
    }
    for (int64_t i = 0; i < n; ++i) scaled[i] = o_g[i] * hrec[2].coef;
    for (int j = 0; j < ND; ++j) {
        const int64_t at = (int64_t)j * S;
        if (orc_adam(T, NUMEL, ND, j, o_master + at, o_m + at, o_v + at, o_work + at, scaled + at,
                     lr, b1, b2, eps, 1))
            return 1;
    }

    /* no accumulator: the norm of the reduced gradient, a clipped fused step */
    ZCK(zsp_reduce_norm(P, ZSP_ALL_RANKS, dg, ZSP_BF16, ZSP_GRADS_FULL, 0, ZSP_NORM_L2, max_norm,
                        ws, ws_bytes, rec, NULL));
    ZCK(zsp_reduce_adam_step_clip(P, ZSP_ALL_RANKS, dg, ZSP_BF16, ZSP_GRADS_FULL, 0, rec, lr, b1,
                                  b2, eps, 2, NULL));
    HIPCK(hipDeviceSynchronize());
    HIPCK(hipMemcpy(hrec, rec, sizeof hrec, hipMemcpyDeviceToHost));
    bad += check(hrec, total, (double)n, max_norm, "reduced gradient");
    for (int64_t i = 0; i < n; ++i) scaled[i] = o_g[i] * hrec[0].coef;
    for (int j = 0; j < ND; ++j) {
        const int64_t at = (int64_t)j * S;
        if (orc_adam(T, NUMEL, ND, j, o_master + at, o_m + at, o_v + at, o_work + at, scaled + at,
                     lr, b1, b2, eps, 2))
            return 1;
    }

    /* an infinite gradient: the step is skipped */
    const uint16_t inf = 0x7F80;
    HIPCK(hipMemcpy(d_grads[1], &inf, 2, hipMemcpyHostToDevice));
    ZCK(zsp_reduce_norm(P, ZSP_ALL_RANKS, dg, ZSP_BF16, ZSP_GRADS_FULL, 0, ZSP_NORM_L2, max_norm,
                        ws, ws_bytes, rec, NULL));
    ZCK(zsp_reduce_adam_step_clip(P, ZSP_ALL_RANKS, dg, ZSP_BF16, ZSP_GRADS_FULL, 0, rec, lr, b1,
                                  b2, eps, 3, NULL));
    HIPCK(hipDeviceSynchronize());
    HIPCK(hipMemcpy(hrec, rec, sizeof hrec, hipMemcpyDeviceToHost));
    if (!isnan(hrec[0].coef)) {
        printf("an infinite gradient left coefficient %g\n", hrec[0].coef);
        ++bad;
    }
    HIPCK(hipMemcpy(h, d_master, 4 * n, hipMemcpyDeviceToHost));
    bad += same(h, o_master, 4 * (size_t)n, "master");
    HIPCK(hipMemcpy(h, d_m, 4 * n, hipMemcpyDeviceToHost));
    bad += same(h, o_m, 4 * (size_t)n, "m");
    HIPCK(hipMemcpy(h, d_v, 4 * n, hipMemcpyDeviceToHost));
    bad += same(h, o_v, 4 * (size_t)n, "v");
    HIPCK(hipMemcpy(hw, d_work, 2 * n, hipMemcpyDeviceToHost));
    bad += same(hw, o_work, 2 * (size_t)n, "work");

    /* a list: the accumulator (fp32) and the parameters, off alignment (bf16) */
    void* xs[2] = {d_acc, d_params + 1};
    const int64_t len[2] = {n, numel - 1};
    const int32_t types[2] = {ZSP_F32, ZSP_BF16};
    double lists = total;
    for (int64_t i = 1; i < numel; ++i)
        lists += (double)bf16_value(params[i]) * bf16_value(params[i]);
    const double limit = 0.3 * sqrt(lists);
    zsp_tensor_list* L = NULL;
    ZCK(zsp_tensor_list_create(xs, len, types, 2, NULL, &L));
    ZCK(zsp_norm_many((const void* const*)xs, len, types, 2, ZSP_NORM_L2, limit, ws, ws_bytes, rec,
                      NULL));
    ZCK(zsp_tensor_list_norm(L, ZSP_NORM_L2, limit, ws, ws_bytes, rec + 1, NULL));
    ZCK(zsp_clip_many(xs, len, types, 2, rec, NULL));
    ZCK(zsp_tensor_list_clip(L, rec + 1, NULL));
    HIPCK(hipDeviceSynchronize());
    HIPCK(hipMemcpy(hrec, rec, sizeof hrec, hipMemcpyDeviceToHost));
    bad += check(hrec, lists, (double)(n + numel), limit, "list, one call");
    bad += check(hrec + 1, lists, (double)(n + numel), limit, "list, prepared");
    for (int k = 0; k < 2; ++k) {
        for (int64_t i = 0; i < n; ++i) o_g[i] = o_g[i] * hrec[k].coef;
        for (int64_t i = 1; i < numel; ++i)
            params[i] = orc_bf16_rne(bf16_value(params[i]) * hrec[k].coef);
    }
    HIPCK(hipMemcpy(h, d_acc, 4 * n, hipMemcpyDeviceToHost));
    bad += same(h, o_g, 4 * (size_t)n, "clipped fp32 tensor");
    HIPCK(hipMemcpy(hw, d_params, 2 * numel, hipMemcpyDeviceToHost));
    bad += same(hw, params, 2 * (size_t)numel, "clipped bf16 tensor");
    zsp_tensor_list_destroy(L);

    zsp_destroy(P);
    hipFree(d_master); hipFree(d_m); hipFree(d_v); hipFree(d_acc); hipFree(d_work);
    hipFree(d_params); hipFree(rec); hipFree(ws);
    for (int r = 0; r < ND; ++r) {
        hipFree(d_grads[r]);
        free(grads[r]);
    }
    free(h); free(o_master); free(o_m); free(o_v); free(o_g); free(scaled);
    free(o_work); free(params); free(hw);
    if (bad) return 1;
    printf("capi norm ok: %d parameters, N_d = %d, two clipped steps, one skipped, a list clipped "
           "twice\n", T, ND);
    return 0;
}

int main(int argc, char** argv) {
    return run(argc > 1 && strcmp(argv[1], "--host-only") == 0);
}
