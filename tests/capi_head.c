/*
 * capi_head.c -- the losses over the head from plain C99 through include/zsp.h
 * alone: cross entropy and distillation, fp32 and bf16, with both gradients,
 * some tokens left out, against the definition in 64 bits.
 * u = 2^-24, b = 2^-8 (half a step of bf16). A logit's error dl: d u sum|x w|
 * (fp32: (6 d + 4) u, three bf16 planes of each operand), 2 u |l| for 1/T. A
 * loss: T^2 (2 dl + 2^-18) and two roundings. G: (2 b + 2^-15 + dl) |c| (p + q)
 * (fp32: 2^-17 + dl). A gradient: that times the other operand, k u |G| times
 * it for the sum (fp32: 6 k u) and one rounding of the result.
 * Prints "capi head ok ..." and exits 0, or says what differs and exits 1.
 * With --host-only it stops after the checks that need no GPU.
 */
#define __HIP_PLATFORM_AMD__ 1
#include <hip/hip_runtime_api.h>
#include <math.h>
#include <stdint.h>
#include <stdio.h>
#include <stdlib.h>
#include <string.h>

#include "zsp.h"

#define N 37
#define V 301
#define D 72
#define TOP 6

/* A value in (-scale, scale) that bf16 holds, by SplitMix64 on a counter. */
static float draw(uint64_t stream, uint64_t i, float scale) {
    uint64_t x = ((stream << 40) ^ i) + 0x9E3779B97F4A7C15ull;
    x = (x ^ (x >> 30)) * 0xBF58476D1CE4E5B9ull;
    x = (x ^ (x >> 27)) * 0x94D049BB133111EBull;
    x ^= x >> 31;
    float f = (2.0f * (float)((double)(x >> 11) * (1.0 / 9007199254740992.0)) - 1.0f) * scale;
    uint32_t bits;
    memcpy(&bits, &f, 4);
    bits &= 0xffff0000u;
    memcpy(&f, &bits, 4);
    return f;
}

#define HIPCK(call) do { hipError_t e_ = (call); if (e_ != hipSuccess) { \
    printf("HIP error %d (%s) in %s\n", (int)e_, hipGetErrorString(e_), #call); return 1; } } while (0)
#define ZCK(call) do { zsp_status s_ = (call); if (s_ != ZSP_OK) { \
    printf("%s -> %d: %s\n", #call, (int)s_, zsp_last_error()); return 1; } } while (0)
#define WANT(call, status) do { zsp_status s_ = (call); if (s_ != (status) || !zsp_last_error()[0]) { \
    printf("%s -> %d, not %d\n", #call, (int)s_, (int)(status)); return 1; } } while (0)

static int host_checks(void) {
    char* const at = (char*)(uintptr_t)4096; /* addresses that no call may follow */
    float *const x = (float*)at, *const w = (float*)(at + (1 << 20)), *const loss = (float*)(at + (2 << 20));
    int64_t* const t = (int64_t*)(at + (3 << 20));
    void* const ws = at + (4 << 20);
    const int both = ZSP_HEAD_GRAD_HIDDEN | ZSP_HEAD_GRAD_HEAD;
    int64_t some = 0, all = 0;
    ZCK(zsp_head_workspace(N, V, D, ZSP_F32, 0, 0, &some));
    ZCK(zsp_head_workspace(N, V, D, ZSP_F32, TOP, both, &all));
    if (some <= 0 || all <= some) {
        printf("workspaces of %lld and %lld bytes\n", (long long)some, (long long)all);
        return 1;
    }
    WANT(zsp_head_workspace(N, V, D, ZSP_F32, 0, 8, &some), ZSP_EINVAL);
    WANT(zsp_head_workspace(N, V, D, ZSP_F32, 0, 0, NULL), ZSP_EINVAL);
    WANT(zsp_head_loss(x, w, ZSP_F32, N, V, D, t, NULL, 1.0f, loss, NULL, NULL, NULL, ws, some - 1,
                       NULL), ZSP_ERANGE);
    WANT(zsp_head_loss(x, NULL, ZSP_F32, N, V, D, t, NULL, 1.0f, loss, NULL, NULL, NULL, ws, some,
                       NULL), ZSP_EINVAL);
    WANT(zsp_head_loss(x, w, ZSP_F32, N, V, D, t, NULL, 1.0f, x, NULL, NULL, NULL, ws, some, NULL),
         ZSP_EINVAL); /* the loss overlaps hidden */
    WANT(zsp_head_distill(x, w, ZSP_F32, N, V, D, t, loss, 0, 1.0f, NULL, 1.0f, loss, NULL, NULL,
                          NULL, ws, all, NULL), ZSP_EINVAL);
    return 0;
}

static double at_type(const void* p, int64_t i, int f32) {
    if (f32) return ((const float*)p)[i];
    const uint32_t bits = (uint32_t)((const uint16_t*)p)[i] << 16;
    float f;
    memcpy(&f, &bits, 4);
    return f;
}

static int near_(double got, double want, double tol, const char* what, int64_t i) {
    if (fabs(got - want) <= tol) return 0; /* NaN is not near */
    printf("%s[%lld] = %.9g, not %.9g (tolerance %.3g)\n", what, (long long)i, got, want, tol);
    return 1;
}

static float x[N * D], w[V * D], weight[N], tlogit[N * TOP];
static int64_t idx[N * TOP];
static double G[N * V], E[N * V];

static int one_case(int f32, int top) {
    const int k = top ? top : 1;
    const double u = ldexp(1.0, -24), T = top ? 1.5 : 1.0, scale = 0.25;
    const size_t es = f32 ? 4 : 2;
    const zsp_dtype dt = f32 ? ZSP_F32 : ZSP_BF16;
    for (int i = 0; i < N * D; ++i) x[i] = draw(1, (uint64_t)i, 1.0f);
    for (int i = 0; i < V * D; ++i) w[i] = draw(2, (uint64_t)i, 0.5f);
    for (int i = 0; i < N; ++i) weight[i] = i % 11 == 3 ? 0.0f : 1.0f + draw(3, (uint64_t)i, 0.5f);
    for (int i = 0; i < N * k; ++i) {
        idx[i] = (int64_t)((uint64_t)(i + 1) * 2654435761u % V);
        tlogit[i] = draw(4, (uint64_t)i, 4.0f);
        if (i / k % 7 == 5) idx[i] = i % 2 ? -100 : V; /* tokens that do not count */
        if (k > 1 && i % k == 2) idx[i] = -1;          /* an entry left out */
        if (k > 1 && i % k == 4) idx[i] = idx[i - 1];  /* one twice */
    }
    uint16_t* hx = malloc(2 * N * D);
    uint16_t* hw = malloc(2 * V * D);
    for (int i = 0; i < N * D; ++i) { uint32_t b; memcpy(&b, &x[i], 4); hx[i] = (uint16_t)(b >> 16); }
    for (int i = 0; i < V * D; ++i) { uint32_t b; memcpy(&b, &w[i], 4); hw[i] = (uint16_t)(b >> 16); }

    void *dx, *dw, *di, *dl_, *dwt, *dloss, *dlse, *dgx, *dgw, *ws;
    int64_t bytes = 0;
    ZCK(zsp_head_workspace(N, V, D, dt, top, ZSP_HEAD_GRAD_HIDDEN | ZSP_HEAD_GRAD_HEAD, &bytes));
    HIPCK(hipMalloc(&dx, es * N * D));
    HIPCK(hipMalloc(&dw, es * V * D));
    HIPCK(hipMalloc(&di, 8 * N * k));
    HIPCK(hipMalloc(&dl_, 4 * N * k));
    HIPCK(hipMalloc(&dwt, 4 * N));
    HIPCK(hipMalloc(&dloss, 4 * N));
    HIPCK(hipMalloc(&dlse, 4 * N));
    HIPCK(hipMalloc(&dgx, es * N * D));
    HIPCK(hipMalloc(&dgw, es * V * D));
    HIPCK(hipMalloc(&ws, (size_t)bytes));
    HIPCK(hipMemcpy(dx, f32 ? (void*)x : (void*)hx, es * N * D, hipMemcpyHostToDevice));
    HIPCK(hipMemcpy(dw, f32 ? (void*)w : (void*)hw, es * V * D, hipMemcpyHostToDevice));
    HIPCK(hipMemcpy(di, idx, 8 * N * k, hipMemcpyHostToDevice));
    HIPCK(hipMemcpy(dl_, tlogit, 4 * N * k, hipMemcpyHostToDevice));
    HIPCK(hipMemcpy(dwt, weight, 4 * N, hipMemcpyHostToDevice));
    if (top)
        ZCK(zsp_head_distill(dx, dw, dt, N, V, D, di, dl_, top, (float)T, dwt, (float)scale, dloss,
                             dlse, dgx, dgw, ws, bytes, NULL));
    else
        ZCK(zsp_head_loss(dx, dw, dt, N, V, D, di, dwt, (float)scale, dloss, dlse, dgx, dgw, ws,
                          bytes, NULL));
    HIPCK(hipDeviceSynchronize());
    float loss[N], lse[N];
    void* gx = malloc(es * N * D);
    void* gw = malloc(es * V * D);
    HIPCK(hipMemcpy(loss, dloss, sizeof loss, hipMemcpyDeviceToHost));
    HIPCK(hipMemcpy(lse, dlse, sizeof lse, hipMemcpyDeviceToHost));
    HIPCK(hipMemcpy(gx, dgx, es * N * D, hipMemcpyDeviceToHost));
    HIPCK(hipMemcpy(gw, dgw, es * V * D, hipMemcpyDeviceToHost));

    int bad = 0;
    for (int i = 0; i < N; ++i) {
        double l[V], q[V], dl = 0, m = -INFINITY, s = 0, ts = 0, tm = -INFINITY, want = 0;
        memset(q, 0, sizeof q);
        for (int v = 0; v < V; ++v) {
            double sum = 0, mag = 0;
            for (int c = 0; c < D; ++c) {
                sum += (double)x[i * D + c] * w[v * D + c];
                mag += fabs((double)x[i * D + c] * w[v * D + c]);
            }
            l[v] = sum / T;
            dl = fmax(dl, (f32 ? 6 * D + 4 : D) * u * mag / T + 2 * u * fabs(l[v]));
            m = fmax(m, l[v]);
        }
        for (int v = 0; v < V; ++v) s += exp(l[v] - m);
        const double z = m + log(s);
        for (int e = i * k; e < (i + 1) * k; ++e)
            if (idx[e] >= 0 && idx[e] < V) tm = fmax(tm, top ? tlogit[e] : 0.0);
        const int on = tm > -INFINITY && weight[i] != 0.0f;
        if (on) {
            for (int e = i * k; e < (i + 1) * k; ++e)
                if (idx[e] >= 0 && idx[e] < V) ts += exp(((top ? tlogit[e] : 0.0) - tm) / T);
            for (int e = i * k; e < (i + 1) * k; ++e)
                if (idx[e] >= 0 && idx[e] < V) {
                    const double lq = ((top ? tlogit[e] : 0.0) - tm) / T - log(ts);
                    q[idx[e]] += exp(lq);
                    want += T * T * exp(lq) * (lq - (l[idx[e]] - z));
                }
        }
        bad |= near_(loss[i], want, on ? T * T * (2 * dl + ldexp(1, -18)) + 2 * u * fabs(want) : 0,
                     "loss", i);
        bad |= near_(lse[i], on ? z : 0, on ? dl + ldexp(1, -19) + u * fabs(z) : 0, "lse", i);
        const double c = on ? scale * T * weight[i] : 0;
        const double rel = (f32 ? ldexp(1, -17) : ldexp(1, -7) + ldexp(1, -15)) + dl;
        for (int v = 0; v < V; ++v) {
            const double p = exp(l[v] - z);
            G[i * V + v] = c * (p - q[v]);
            E[i * V + v] = rel * fabs(c) * (p + q[v]);
        }
    }
    const double out = f32 ? u : ldexp(1, -8), six = f32 ? 6 : 1;
    for (int i = 0; i < N && !bad; ++i)
        for (int c = 0; c < D; ++c) {
            double sum = 0, tol = 0;
            for (int v = 0; v < V; ++v) {
                sum += G[i * V + v] * w[v * D + c];
                tol += (E[i * V + v] + six * V * u * fabs(G[i * V + v])) * fabs(w[v * D + c]);
            }
            bad |= near_(at_type(gx, i * D + c, f32), sum, tol + out * fabs(sum), "grad_hidden", i * D + c);
        }
    for (int v = 0; v < V && !bad; ++v)
        for (int c = 0; c < D; ++c) {
            double sum = 0, tol = 0;
            for (int i = 0; i < N; ++i) {
                sum += G[i * V + v] * x[i * D + c];
                tol += (E[i * V + v] + six * N * u * fabs(G[i * V + v])) * fabs(x[i * D + c]);
            }
            bad |= near_(at_type(gw, v * D + c, f32), sum, tol + out * fabs(sum), "grad_head", v * D + c);
        }
    void* const dev[] = {dx, dw, di, dl_, dwt, dloss, dlse, dgx, dgw, ws};
    for (size_t i = 0; i < sizeof dev / sizeof dev[0]; ++i) HIPCK(hipFree(dev[i]));
    free(hx);
    free(hw);
    free(gx);
    free(gw);
    return bad;
}

int main(int argc, char** argv) {
    if (host_checks()) return 1;
    if (argc > 1 && strcmp(argv[1], "--host-only") == 0) {
        printf("capi head host checks ok\n");
        return 0;
    }
    for (int f32 = 0; f32 < 2; ++f32)
        for (int top = 0; top <= TOP; top += TOP) {
            printf("%s, %d entries\n", f32 ? "fp32" : "bf16", top ? top : 1);
            fflush(stdout);
            if (one_case(f32, top)) return 1;
        }
    printf("capi head ok: %d tokens x %d x %d\n", N, V, D);
    return 0;
}
