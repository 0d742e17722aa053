// zsp_head.hip -- the losses over a model's output matrix (the head) and
// their gradients, for gfx950.
//
//   l_iv = (x_i . w_v) / T          lse_i = log sum_v exp l_iv
//   p_iv = exp(l_iv - lse_i)        q_i: the target, or the teacher's softmax
//   G_iv = c_i (p_iv - q_iv)        dX = s G W      dW = s G^T X
//   c_i: the token's weight         s = scale * T
//
// The logits are never kept: the first product's tiles leave, per token and
// block of 64 columns, the block's largest logit m and the sum of
// exp(l - m), and for a call with gradients (m - l) log2(e) in 16-bit steps
// (fp32: P = exp(l - m) in fp32) for a bounded number of tokens; once the blocks
// are joined to lse, one pass turns that into G in place, and the other two
// products read G. Three products of
// 2 n v d operations each, bound by the matrix cores for long batches and by
// the reads of W and the write of dW for short ones.
//
// Tokens that do not count are left out first: the others' rows of X are
// copied together (zeros behind the last), so masked tokens cost nothing and
// whatever their rows hold reaches no sum. How many count is known to the
// device alone; tiles past it end at once.
//
// fp32 operands are held as three bf16 planes (8 bits of the value each,
// x = h + m + l exactly) and multiplied as hh + hm + mh + mm + hl + lh on the
// bf16 matrix cores: what is left out is below 2^-23 of a product.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <type_traits>

#include "zsp_head.hpp"

namespace zsp {
namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4_a2 __attribute__((ext_vector_type(4), aligned(2)));
typedef uint32_t u32x2_a2 __attribute__((ext_vector_type(2), aligned(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x4_a4 __attribute__((ext_vector_type(4), aligned(4)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

#define ZSP_LDS __attribute__((address_space(3)))

constexpr float kLog2e = 1.44269504088896340736f;

__device__ __forceinline__ float bf16_value(uint16_t u) {
    return __uint_as_float(uint32_t(u) << 16);
}
__device__ __forceinline__ uint16_t bf16_bits(float f) {
    return __builtin_bit_cast(uint16_t, static_cast<__bf16>(f));
}
__device__ __forceinline__ uint32_t bf16_pair(float lo, float hi) {
    const bf16x2 v = {static_cast<__bf16>(lo), static_cast<__bf16>(hi)};
    return __builtin_bit_cast(uint32_t, v);
}
// exp(x) by the hardware's exp2: relative error about 2^-22 for the terms of
// a softmax that matter (x > -4), a few units more for smaller ones.
__device__ __forceinline__ float fast_exp(float x) {
    return __builtin_amdgcn_exp2f(x * kLog2e);
}

// What a block of logits leaves for G of a bf16 call: (m - l) log2(e), m the
// block's largest, in steps of 64 / 65535: the two bytes that P = exp(l - m) in
// bf16 would take, without rounding p twice. Half a step moves p by 3.4e-4 of
// itself, a tenth of what the rounding of G to bf16 that follows may; rows of the
// head's gradient that are no token's target are 0.0022 to 0.0023 off (relative;
// 0.0017 of it the output's own type) in place of 0.0024 to 0.0027, in the same
// time. The last step stands for p below 2^-63.9 of the block's largest, and for
// columns past the vocabulary: 0.
constexpr float kStep = 64.0f / 65535.0f;
constexpr uint32_t kLastStep = 65535;
__device__ __forceinline__ uint32_t step_pair(float lo, float hi) {
    return __builtin_bit_cast(uint32_t,
                              __builtin_amdgcn_cvt_pknorm_u16(lo * 0.015625f, hi * 0.015625f));
}
// p from a step and (m - lse) log2(e).
__device__ __forceinline__ float step_value(uint32_t step, float at) {
    const float p = __builtin_amdgcn_exp2f(__builtin_fmaf(float(step), -kStep, at));
    return step == kLastStep ? 0.0f : p;
}

// The three planes of an fp32 value. A value that rounds to a bf16 infinity
// is cut instead; infinities and NaN stand in the first plane alone.
__device__ __forceinline__ void split3(float x, uint16_t out[3]) {
    uint32_t h = uint32_t(bf16_bits(x)) << 16;
    const uint32_t u = __float_as_uint(x);
    out[1] = out[2] = 0;
    if ((u & 0x7f800000u) == 0x7f800000u) {
        out[0] = uint16_t(h >> 16);
        return;
    }
    if ((h & 0x7f800000u) == 0x7f800000u) h = u & 0xffff0000u;
    out[0] = uint16_t(h >> 16);
    const float r = x - __uint_as_float(h);
    out[1] = bf16_bits(r);
    out[2] = bf16_bits(r - bf16_value(out[1]));
}

// ---- which tokens count, and the operands -------------------------------------------

// The teacher's entries: which tokens have one, one wave per token.
__global__ __launch_bounds__(256) void flag_kernel(const int64_t* index, const float* logit,
                                                   int64_t n, int64_t v, int32_t top,
                                                   const float* weight, uint8_t* flag) {
    const int64_t i = int64_t(blockIdx.x) * 4 + threadIdx.x / 64;
    if (i >= n) return;
    bool any = false;
    for (int32_t k = threadIdx.x % 64; k < top; k += 64) {
        const int64_t e = index[i * top + k];
        any |= e >= 0 && e < v && logit[i * top + k] != -__builtin_inff();
    }
    const bool on = __any(any) && (!weight || weight[i] != 0.0f);
    if (threadIdx.x % 64 == 0) flag[i] = on;
}

__device__ __forceinline__ bool counts(const int64_t* target, const float* weight,
                                       const uint8_t* flag, int64_t i, int64_t v) {
    if (flag) return flag[i] != 0;
    const int64_t e = target[i];
    const float w = weight ? weight[i] : 1.0f;
    return uint64_t(e) < uint64_t(v) && w != 0.0f;
}

// rows[0 .. count): the tokens that count, in order. One workgroup, kScanRun
// tokens a thread at a time; the waves' counts are joined in LDS.
constexpr int kScanThreads = 1024, kScanRun = 8;
constexpr int64_t kFlagEntries = 8192, kFlagTokens = kScanThreads * kScanRun;
__global__ __launch_bounds__(kScanThreads) void scan_kernel(const int64_t* target,
                                                            const float* logit, int32_t top,
                                                            const float* weight, uint8_t* flag,
                                                            int64_t n, int64_t v, int32_t* rows,
                                                            int32_t* count) {
    if (logit) {  // a teacher's few entries: the flags first
        __shared__ uint8_t s_flag[kFlagTokens];
        for (int64_t i = threadIdx.x; i < n; i += kScanThreads) s_flag[i] = 0;
        __syncthreads();
#pragma unroll 4
        for (int32_t k = threadIdx.x; k < int32_t(n) * top; k += kScanThreads)
            if (uint64_t(target[k]) < uint64_t(v) && logit[k] != -__builtin_inff())
                s_flag[k / top] = 1;
        __syncthreads();
        for (int64_t i = threadIdx.x; i < n; i += kScanThreads)
            flag[i] = s_flag[i] && (!weight || weight[i] != 0.0f);
        __threadfence_block();
        __syncthreads();
    }
    __shared__ int32_t s_wave[kScanThreads / 64];
    const int t = threadIdx.x, lane = t % 64, wave = t / 64;
    int32_t done = 0;
    for (int64_t base = 0; base < n; base += kScanThreads * kScanRun) {
        const int64_t first = base + wave * (64 * kScanRun) + lane;
        // all loads on their way before the first is looked at
        bool on[kScanRun];
        const int64_t last = n - 1;
        if (flag) {
            uint8_t f[kScanRun];
#pragma unroll
            for (int k = 0; k < kScanRun; ++k) f[k] = flag[min(first + k * 64, last)];
#pragma unroll
            for (int k = 0; k < kScanRun; ++k) on[k] = f[k] != 0;
        } else {
            int64_t e[kScanRun];
#pragma unroll
            for (int k = 0; k < kScanRun; ++k) e[k] = target[min(first + k * 64, last)];
#pragma unroll
            for (int k = 0; k < kScanRun; ++k) on[k] = uint64_t(e[k]) < uint64_t(v);
            if (weight) {
                float w[kScanRun];
#pragma unroll
                for (int k = 0; k < kScanRun; ++k) w[k] = weight[min(first + k * 64, last)];
#pragma unroll
                for (int k = 0; k < kScanRun; ++k) on[k] &= w[k] != 0.0f;
            }
        }
#pragma unroll
        for (int k = 0; k < kScanRun; ++k) on[k] &= first + k * 64 < n;
        int32_t mine = 0;
#pragma unroll
        for (int k = 0; k < kScanRun; ++k) mine += __popcll(__ballot(on[k]));
        if (lane == 0) s_wave[wave] = mine;
        __syncthreads();
        int32_t at = done;
        for (int w = 0; w < kScanThreads / 64; ++w) {
            if (w < wave) at += s_wave[w];
            done += s_wave[w];
        }
#pragma unroll
        for (int k = 0; k < kScanRun; ++k) {
            const uint64_t m = __ballot(on[k]);
            if (on[k]) rows[at + __popcll(m & ((1ull << lane) - 1))] = int32_t(first + k * 64);
            at += __popcll(m);
        }
        __syncthreads();
    }
    if (t == 0) *count = done;
}

// Eight elements of a row of d, from column c on; zeros past d.
template <typename T>
struct Eight {
    static constexpr bool kF32 = sizeof(T) == 4;
    u32x4 v[kF32 ? 2 : 1];

    __device__ __forceinline__ void load(const T* in, int64_t c, int64_t d) {
        if (c + 8 <= d) {
            if constexpr (kF32) {
                v[0] = *reinterpret_cast<const u32x4_a2*>(in + c);
                v[1] = *reinterpret_cast<const u32x4_a2*>(in + c + 4);
            } else {
                v[0] = *reinterpret_cast<const u32x4_a2*>(in + c);
            }
            return;
        }
        zero();
#pragma unroll
        for (int k = 0; k < 8; ++k)
            if (c + k < d) {
                if constexpr (kF32) v[k / 4][k % 4] = __float_as_uint(in[c + k]);
                else v[0][k / 2] |= uint32_t(in[c + k]) << (16 * (k % 2));
            }
    }
    __device__ __forceinline__ void zero() {
        v[0] = u32x4{0, 0, 0, 0};
        if constexpr (kF32) v[1] = v[0];
    }
    // bf16: one element in each of eight rows.
    __device__ __forceinline__ void turn(uint16_t* out, int64_t ld) const {
        if constexpr (!kF32) {
#pragma unroll
            for (int k = 0; k < 8; ++k) out[k * ld] = uint16_t(v[0][k / 2] >> (16 * (k % 2)));
        }
    }
    // As planes, `plane` elements apart.
    __device__ __forceinline__ void store(uint16_t* out, int64_t plane) const {
        if constexpr (kF32) {
            u32x4 o[3];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                uint16_t p[3], q[3];
                split3(__uint_as_float(v[k / 2][k % 2 * 2]), p);
                split3(__uint_as_float(v[k / 2][k % 2 * 2 + 1]), q);
#pragma unroll
                for (int h = 0; h < 3; ++h) o[h][k] = p[h] | uint32_t(q[h]) << 16;
            }
#pragma unroll
            for (int h = 0; h < 3; ++h) *reinterpret_cast<u32x4*>(out + h * plane) = o[h];
        } else {
            *reinterpret_cast<u32x4*>(out) = v[0];
        }
    }
};

struct SetupArgs {
    const void* hidden;
    const void* head;
    const int64_t* index;
    const float* logit;
    const float* weight;
    const uint8_t* flag;
    int32_t* rows;
    int32_t* count;
    float* coef;
    int32_t* entry;
    float* teach;
    uint16_t* start;   // [row][blocks + 1]
    uint16_t* x;
    uint16_t* xt;      // [dp][few_pad], bf16 and few tokens only, or NULL
    uint16_t* w;
    void* grad_hidden;
    float* loss;
    float* lse;
    int64_t n, v, d, dp, x_plane, w_plane;
    int32_t top, top_pad, blocks;
    int32_t row_threads, parts;               // threads a row, workgroups a row
    int32_t few_pad;
    uint32_t x_groups, entry_groups;          // workgroups of each kind; the rest copy the head
    int32_t scans;                            // each workgroup finds the tokens itself
};

constexpr int kSetupThreads = 256, kSetupRun = 2;
constexpr int kHeadRun = 4;  // rows of the head's copy a thread takes
constexpr int64_t kSelfScan = kSetupThreads * kSetupRun;

// Up to kSelfScan tokens: those that count, found by every workgroup for
// itself (a launch and its wait take 5 us; at 1400 tokens the workgroups' own
// scans took 7).
// Leaves the tokens of rows [r0, r0 + n) in s_rows.
__device__ __forceinline__ int32_t scan_here(const SetupArgs& a, int64_t r0, int n, int32_t* s_rows,
                                             int32_t* s_wave) {
    const int t = threadIdx.x, lane = t % 64, wave = t / 64;
    const int64_t first = int64_t(t) * kSetupRun;
    bool on[kSetupRun];
    int32_t mine = 0;
#pragma unroll
    for (int k = 0; k < kSetupRun; ++k) {
        const int64_t i = min(first + k, a.n - 1);
        on[k] = counts(a.index, a.weight, nullptr, i, a.v) && first + k < a.n;
        mine += on[k];
    }
    int32_t sum = mine;
    for (int o = 1; o < 64; o <<= 1) {
        const int32_t u = __shfl_up(sum, o);
        if (lane >= o) sum += u;
    }
    if (lane == 63) s_wave[wave] = sum;
    __syncthreads();
    int32_t at = sum - mine, all = 0;
    for (int w = 0; w < kSetupThreads / 64; ++w) {
        if (w < wave) at += s_wave[w];
        all += s_wave[w];
    }
#pragma unroll
    for (int k = 0; k < kSetupRun; ++k) {
        if (!on[k]) continue;
        if (at >= r0 && at < r0 + n) s_rows[at - r0] = int32_t(first + k);
        ++at;
    }
    __syncthreads();
    return all;
}

// Rows of the copied X, their coefficients and entries; the outputs of tokens
// that do not count. `row_threads` threads and `parts` workgroups a row, eight
// columns a thread.
template <typename T>
__device__ __forceinline__ void setup_rows(const SetupArgs& a, uint32_t group) {
    __shared__ int32_t s_rows[kSetupThreads], s_wave[kSetupThreads / 64];
    const int per = kSetupThreads / a.row_threads, t = threadIdx.x;
    const int64_t r0 = int64_t(group / a.parts) * per;
    const int32_t part = int32_t(group % a.parts);
    const int mine = t / a.row_threads, lane = t % a.row_threads;
    const int64_t r = r0 + mine, c = (int64_t(part) * a.row_threads + lane) * 8;
    int32_t count;
    int64_t i = 0;
    if (a.scans) {
        count = scan_here(a, r0, per, s_rows, s_wave);
        if (group == 0 && t == 0) *a.count = count;
        if (r < count) i = s_rows[mine];
        if (part == 0 && lane == 0 && r < count) a.rows[r] = int32_t(i);
    } else {
        count = *a.count;
        if (r < count) i = a.rows[r];
    }
    if (r < count) {
        if (c < a.dp) {
            Eight<T> v;
            v.load(static_cast<const T*>(a.hidden) + i * a.d, c, a.d);
            v.store(a.x + r * a.dp + c, a.x_plane);
            if (a.xt) v.turn(a.xt + c * a.few_pad + r, a.few_pad);
        }
        if (part == 0 && lane == 0) {
            a.coef[r] = a.weight ? a.weight[i] : 1.0f;
            if (a.top == 1) {
                const int64_t e = a.index[i];
                const bool out = a.logit && a.logit[i] == -__builtin_inff();
                a.entry[r] = uint64_t(e) < uint64_t(a.v) && !out ? int32_t(e) : -1;
                if (a.logit) a.teach[r] = a.logit[i];
            }
        }
    } else if (r < (int64_t(count) + kHeadDepth - 1) / kHeadDepth * kHeadDepth) {
        // zeros as far as a stage of a sum over tokens may read
        if (c < a.dp) {
            Eight<T> v;
            v.zero();
            v.store(a.x + r * a.dp + c, a.x_plane);
        }
    }
    if (a.xt && r >= count && r < a.few_pad && c < a.dp) {
        Eight<T> v;
        v.zero();
        v.turn(a.xt + c * a.few_pad + r, a.few_pad);
    }
    if (r < a.n && !counts(a.index, a.weight, a.flag, r, a.v)) {
        if (a.grad_hidden) {
            T* out = static_cast<T*>(a.grad_hidden) + r * a.d;
            for (int64_t k = int64_t(part) * a.row_threads + lane; k < a.d;
                 k += int64_t(a.parts) * a.row_threads)
                out[k] = T(0);
        }
        if (part == 0 && lane == 0) {
            a.loss[r] = 0.0f;
            if (a.lse) a.lse[r] = 0.0f;
        }
    }
}

// A token's entries in the order of their blocks of the vocabulary (equal ones
// in the teacher's), with their logits, and where each block's begin: a tile of
// the logits then looks at its own entries alone. Scanning all 64 entries of
// every token in every tile took 450 of 1330 us at 4096 x 32000 x 4096.
__device__ __forceinline__ void setup_entries(const SetupArgs& a, int64_t r) {
    __shared__ int32_t s_block[kHeadMaxTop], s_sorted[kHeadMaxTop];
    const int t = threadIdx.x;
    if (r >= *a.count) return;
    const int64_t from = int64_t(a.rows[r]) * a.top;
    for (int32_t k = t; k < a.top; k += kSetupThreads) {
        const int64_t e = a.index[from + k];
        const bool on = uint64_t(e) < uint64_t(a.v) && a.logit[from + k] != -__builtin_inff();
        s_block[k] = on ? int32_t(e) / kHeadBlock : a.blocks;
    }
    __syncthreads();
    for (int32_t k = t; k < a.top; k += kSetupThreads) {
        const int32_t b = s_block[k];
        int32_t at = 0;
        for (int32_t o = 0; o < a.top; ++o) at += s_block[o] < b || (s_block[o] == b && o < k);
        s_sorted[at] = b;
        a.entry[r * a.top_pad + at] = b < a.blocks ? int32_t(a.index[from + k]) : -1;
        a.teach[r * a.top_pad + at] = a.logit[from + k];
    }
    __syncthreads();
    uint16_t* start = a.start + r * (a.blocks + 1);
    for (int32_t k = t; k <= a.top; k += kSetupThreads) {
        const int32_t lo = k == 0 ? 0 : s_sorted[k - 1] + 1;
        const int32_t hi = k == a.top ? a.blocks : s_sorted[k];
        for (int32_t b = lo; b <= hi; ++b) start[b] = uint16_t(k);
    }
}

// What the products need, in one launch: the rows of X, the tokens' entries
// and, where it cannot be read in place, the head in planes of dp columns.
// Bound by the bytes copied (50021 x 1283 and 1777 rows of X: 268 MB in 55 us;
// 32000 x 2048 fp32 into planes 655 MB in 114), or its launch.
template <typename T>
__global__ __launch_bounds__(kSetupThreads) void setup_kernel(SetupArgs a) {
    uint32_t group = blockIdx.x;
    if (group < a.x_groups) return setup_rows<T>(a, group);
    group -= a.x_groups;
    if (group < a.entry_groups) return setup_entries(a, group);
    group -= a.entry_groups;
    const int per = kSetupThreads / a.row_threads;
    const int64_t r0 = int64_t(group / a.parts) * per * kHeadRun + threadIdx.x / a.row_threads;
    const int64_t c = (int64_t(group % a.parts) * a.row_threads + threadIdx.x % a.row_threads) * 8;
    if (c >= a.dp) return;
    const T* head = static_cast<const T*>(a.head);
    Eight<T> v[kHeadRun];  // all loads on their way before the first store
#pragma unroll
    for (int k = 0; k < kHeadRun; ++k)
        v[k].load(head + min(r0 + k * per, a.v - 1) * a.d, c, a.d);
#pragma unroll
    for (int k = 0; k < kHeadRun; ++k)
        if (r0 + k * per < a.v) v[k].store(a.w + (r0 + k * per) * a.dp + c, a.w_plane);
}

// ---- the products --------------------------------------------------------------------

// C[b, a] = sum_k A[a, k] B[b, k] in tiles of BA x BB: a runs along a row of
// the output. An operand is K-major (its k run along its rows: A[a][k]) or
// M-major (its rows are k: A[k][a]).
struct GemmArgs {
    const uint16_t* a;
    const uint16_t* b;
    int64_t lda, ldb;          // elements
    int64_t plane_a, plane_b;  // elements between planes
    int64_t a_width;           // columns of A's rows as they lie in memory
    int32_t thin;              // an fp32 head read in place
    int32_t keep;              // the head is read again, and may stay in the caches
    int64_t na;                // extent of a: further rows or columns are read as the last ones
    int64_t nb;                // extent of b; a product over tokens: bounded by *count - first
    int64_t k;                 // the sum's length, and for M-major A with na_k its real rows
    int64_t k_real;            // k's of the head that exist (later ones are read as the last)
    const int32_t* count;      // tokens that count
    int64_t first;             // the chunk's first token
    int32_t tokens_in_b, tokens_in_k;
    uint32_t slot_bits;        // log2 of the tiles the card runs at once; 0: sums are not split
    // logits
    float log2e_t;             // log2(e) / T
    float factor;              // of what goes to out
    float2* part;              // [b][na_blocks]: the largest sum, and of exp((sum - it) / T)
    int64_t nblk;
    void* p;                   // [b][ldp] steps (fp32: P), or NULL
    int64_t ldp;
    const int32_t* entry;      // [b][top_pad]
    const uint16_t* start;     // [b][blocks + 1]: a block's first entry, if top_pad > 1
    int32_t blocks;
    float* pick;               // the entries' sums
    int32_t top_pad;
    // outputs
    void* out;                 // final: [row][ldo] of the output's type, or NULL
    int64_t ldo;
    const int32_t* rows;       // row of b, or NULL: b itself
    const float* acc_in;       // fp32 [b][ldf] to add, or NULL
    float* acc_out;            // fp32 [b][ldf], instead of out
    float* split;              // fp32 [part of the sum][b][ldf], if the sums are split
    int32_t keep_parts;        // the caller joins them
    int64_t ldf;
};

enum { kLogits = 0, kOut = 1 };

// 16 bytes a lane from base + off to lds + 16 * lane. In assembly: the
// compiler would wait for every such load before each transposing LDS read.
// Nothing else here uses m0. The caller waits (wait_stage).
template <bool NT>
__device__ __forceinline__ void load_to_lds(const char* base, uint32_t off, ZSP_LDS char* lds) {
    const uint32_t at = __builtin_amdgcn_readfirstlane(uint32_t(uintptr_t(lds)));
    const uint64_t p = reinterpret_cast<uint64_t>(base);
    const uint64_t from = uint64_t(__builtin_amdgcn_readfirstlane(uint32_t(p >> 32))) << 32 |
                          uint32_t(__builtin_amdgcn_readfirstlane(uint32_t(p)));
    if constexpr (NT)
        asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2 nt" ::"s"(at),
                     "v"(off), "s"(from)
                     : "memory");
    else
        asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2" ::"s"(at),
                     "v"(off), "s"(from)
                     : "memory");
}
template <int N>
__device__ __forceinline__ void wait_stage() {
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(N) : "memory");
}
__device__ __forceinline__ void wg_barrier() {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

// Columns [col, col + 4) or [col, col + 8) of a row of `end`, which may start
// on any element. (Element by element without a loop: one that is not unrolled
// would put the vector into LDS.)
__device__ __forceinline__ void store_part(float* row, int64_t col, int64_t end, f32x4 v) {
    if (col + 4 <= end) {
        *reinterpret_cast<f32x4_a4*>(row + col) = v;
        return;
    }
    if (col < end) row[col] = v[0];
    if (col + 1 < end) row[col + 1] = v[1];
    if (col + 2 < end) row[col + 2] = v[2];
}
__device__ __forceinline__ void store_part(uint16_t* row, int64_t col, int64_t end, u32x4 v) {
    if (col + 8 <= end) {
        *reinterpret_cast<u32x4_a2*>(row + col) = v;
        return;
    }
    if (col < end) row[col] = uint16_t(v[0]);
    if (col + 1 < end) row[col + 1] = uint16_t(v[0] >> 16);
    if (col + 2 < end) row[col + 2] = uint16_t(v[1]);
    if (col + 3 < end) row[col + 3] = uint16_t(v[1] >> 16);
    if (col + 4 < end) row[col + 4] = uint16_t(v[2]);
    if (col + 5 < end) row[col + 5] = uint16_t(v[2] >> 16);
    if (col + 6 < end) row[col + 6] = uint16_t(v[3]);
}

// Two neighbouring 16 x 16 tiles of a wave as bf16 (or steps), eight columns a
// lane: the lanes of rows 1 and 3 (16 lanes each) hand their four columns of the
// first tile to rows 0 and 2 for theirs of the second, so that the four lanes of
// an output row write 64 bytes of it.
template <typename F>
__device__ __forceinline__ u32x4 pair_by(F pack, f32x4 lo, f32x4 hi) {
    const uint32_t x0 = pack(lo[0], lo[1]), y0 = pack(lo[2], lo[3]);
    const uint32_t x1 = pack(hi[0], hi[1]), y1 = pack(hi[2], hi[3]);
    const auto x = __builtin_amdgcn_permlane16_swap(x0, x1, false, false);
    const auto y = __builtin_amdgcn_permlane16_swap(y0, y1, false, false);
    return u32x4{x[0], y[0], x[1], y[1]};
}
__device__ __forceinline__ u32x4 pair_of(f32x4 lo, f32x4 hi) {
    return pair_by([](float a, float b) { return bf16_pair(a, b); }, lo, hi);
}
// The first of a lane's eight columns of the two tiles.
__device__ __forceinline__ int pair_column(int lane_row) {
    return (lane_row & 1) * 16 + (lane_row >> 1) * 8;
}

// Parts of the sums of a product of `tiles` tiles over `stages` steps of k (of
// `segs` stages each), on a card that runs 2^slot_bits tiles at once: as few
// turns as the parts, the turns' beginnings and ends (about four stages) and
// the joining of the parts (a tile's bytes there and back: 1/16 of a stage)
// allow. Where tokens do not count the device alone knows the tiles, so both
// sides ask it here. 0 slot_bits: the sums are not split.
__host__ __device__ inline uint32_t split_of(uint32_t tiles, uint32_t stages, uint32_t segs,
                                             uint32_t slot_bits) {
    if (slot_bits == 0 || tiles == 0 || tiles >> slot_bits >= 64) return 1;
    constexpr uint32_t kParts[] = {1, 2, 3, 4, 5, 6, 8, 10, 12, 16, 24, 32, 48, 64};
    uint32_t best = 1, least = ~0u;
#pragma unroll
    for (uint32_t s : kParts) {
        const uint32_t turns = (tiles * s + (1u << slot_bits) - 1) >> slot_bits;
        const uint32_t cost =
            turns * ((stages + s - 1) / s * segs + 4) * 16 + (s > 1 ? tiles * s : 0);
        if ((s == 1 || (s * 8 <= stages * segs && s <= stages && turns <= 64)) && cost < least) {
            least = cost;
            best = s;
        }
    }
    return best;
}

// One operand's share of a stage in LDS: X rows (or columns) of BK k's, in
// 16-byte groups. The wave's loads write LDS in lane order, so the order of
// the groups in a row is changed on the reading side of the load: group c of
// a row is kept at c ^ s(row), which spreads the lanes of one LDS read over
// the banks.
template <int X, int BK, int WAVES, bool MMAJ, bool CLAMP, bool NT>
struct Operand {
    static constexpr int kGroups = X * BK / 8;
    static constexpr int kLoads = kGroups / 64 / WAVES;
    static constexpr int kBytes = X * BK * 2;
    static_assert(kGroups % (64 * WAVES) == 0, "whole loads");
    static_assert(!MMAJ || X >= 128, "the M-major order wants 16 groups a row");
    static_assert(BK == 32 || BK == 64, "");

    static __device__ __forceinline__ int k_swizzle(int row) {
        return BK == 64 ? (row >> 1) & 7 : (row >> 2) & 3;
    }
    static __device__ __forceinline__ int m_swizzle(int k) {
        return ((k & 3) << 1) | (((k >> 3) & 1) << 3);
    }

    const char* base;         // of the tile's first row (M-major: column)
    int64_t ld;               // bytes
    uint32_t off[kLoads];     // bytes from base; M-major: of the first row
    int32_t krow[kLoads];     // the row, K-major: the group's first k

    __device__ __forceinline__ void init(const uint16_t* p, int64_t ld_, int64_t x0, int64_t nx,
                                         int wave, int lane) {
        ld = ld_ * 2;
        base = reinterpret_cast<const char*>(p) + x0 * (MMAJ ? 2 : ld);
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            const int q = (wave * kLoads + i) * 64 + lane;
            if constexpr (MMAJ) {
                const int k = q / (X / 8);
                int64_t x = ((q % (X / 8)) ^ m_swizzle(k)) * 8;
                x = x0 + x + 8 <= nx ? x : nx - 8 - x0;
                krow[i] = k;
                off[i] = uint32_t(x * 2 + (CLAMP ? 0 : k * ld));
            } else {
                const int r = q / (BK / 8), c = (q % (BK / 8)) ^ k_swizzle(r);
                const int64_t x = x0 + r < nx ? r : nx - 1 - x0;
                off[i] = uint32_t(x * ld + (CLAMP ? 0 : c * 16));
                krow[i] = c * 8;
            }
        }
    }
    // Load i of the stage whose first k is k0 into `lds`. CLAMP: rows (K-major:
    // groups of 8 k's) past k_last are read as that one.
    __device__ __forceinline__ void issue(int i, ZSP_LDS char* lds, int64_t plane, int64_t k0,
                                          int64_t k_last, int wave) {
        const char* src = base + 2 * plane + (MMAJ ? k0 * ld : CLAMP ? 0 : k0 * 2);
        uint32_t o = off[i];
        if constexpr (CLAMP && MMAJ) {
            const int32_t k = k_last - k0 < BK ? int32_t(k_last - k0) : BK;
            o += uint32_t(krow[i] < k ? krow[i] : k) * uint32_t(ld);
        } else if constexpr (CLAMP) {
            o += uint32_t(min(int32_t(k0) + krow[i], int32_t(k_last) - 7)) * 2;
        }
        load_to_lds<NT>(src, o, lds + (wave * kLoads + i) * 1024);
    }
    // The operand's 16 x 32 values for tile `x` (a multiple of 16, of the
    // wave's share at x_wave) and k's [32 kk, 32 kk + 32).
    static __device__ __forceinline__ bf16x8 frag(ZSP_LDS const char* lds, int x_wave, int x, int kk,
                                                  int lane) {
        if constexpr (MMAJ) {
            const int g = lane / 16, i = lane % 16;
            const int k = kk * 32 + g * 8 + i / 4;
            const int c = (x_wave + x) / 8 + (i % 4) / 2;
            const int at = k * (X * 2) + (c ^ (((i / 4) << 1) | ((g & 1) << 3))) * 16 + (i & 1) * 8;
            const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((ZSP_LDS s16x4*)(lds + at));
            const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                (ZSP_LDS s16x4*)(lds + at + 4 * X * 2));
            const s16x8 v = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
            return __builtin_bit_cast(bf16x8, v);
        } else {
            const int row = lane % 16, c = kk * 4 + lane / 16;
            const int at = (x_wave + x + row) * (BK * 2) + (c ^ k_swizzle(row)) * 16;
            return *(ZSP_LDS const bf16x8*)(lds + at);
        }
    }
};

// What a product's kernel does with a wave's sums, columns from a_wave and rows
// from b_wave on.
template <int KIND, bool F32, int TA, int TB>
__device__ __forceinline__ void finish(const GemmArgs& g, f32x4 (&acc)[TA][TB], int64_t a_wave,
                                       int64_t b_wave, int32_t nb, uint32_t part, uint32_t ns,
                                       int lane) {
    static_assert(TA * 16 == kHeadBlock, "a wave's columns are one block");
    // A lane holds, of each 16 x 16 tile, column lane % 16 (a row of the
    // output) at rows 4 (lane / 16) + 0..3 (its columns).
    const int lr = lane % 16, lg = lane / 16;
    if constexpr (KIND == kLogits) {
        // the first entry of each of this lane's tokens in this block, all
        // loads at once
        int32_t one[TB], e_from[TB], e_to[TB];
#pragma unroll
        for (int b = 0; b < TB; ++b) {
            const int64_t row = b_wave + b * 16 + lr;
            one[b] = -1;
            e_from[b] = e_to[b] = 0;
            if (row < nb && g.top_pad == 1) one[b] = g.entry[row];
            if (row < nb && g.top_pad > 1 && a_wave < g.na) {
                const uint16_t* s = g.start + row * (g.blocks + 1) + a_wave / kHeadBlock;
                e_from[b] = s[0];
                e_to[b] = s[1];
            }
        }
        if (g.top_pad > 1) {
#pragma unroll
            for (int b = 0; b < TB; ++b) {
                const int64_t row = b_wave + b * 16 + lr;
                if (e_from[b] < e_to[b]) one[b] = g.entry[row * g.top_pad + e_from[b]];
            }
        }
        // in the sums' own units: 1 / T > 0 comes to the exponent alone here, and
        // to the rest in 64 bits, when the blocks are joined
        const bool edge = a_wave + kHeadBlock > g.na;
#pragma unroll
        for (int b = 0; b < TB; ++b) {
            const int64_t row = b_wave + b * 16 + lr;
            float m = -__builtin_inff();
#pragma unroll
            for (int a = 0; a < TA; ++a)
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    if (edge && a_wave + a * 16 + lg * 4 + k >= g.na)
                        acc[a][b][k] = -__builtin_inff();
                    m = fmaxf(m, acc[a][b][k]);
                }
            m = fmaxf(m, __shfl_xor(m, 16));
            m = fmaxf(m, __shfl_xor(m, 32));
            const bool real = row < nb;
            auto take = [&](int32_t k, int32_t e) {
                const int rel = int(e - a_wave);
                if (unsigned(rel) >= unsigned(kHeadBlock) || ((rel >> 2) & 3) != lg) return;
                float l = 0.0f;
#pragma unroll
                for (int a = 0; a < TA; ++a)
#pragma unroll
                    for (int c = 0; c < 4; ++c)
                        if ((rel >> 4) == a && (rel & 3) == c) l = acc[a][b][c];
                g.pick[row * g.top_pad + k] = l;
            };
            if (real && g.top_pad == 1) take(0, one[b]);
            if (g.top_pad > 1 && e_from[b] < e_to[b]) {
                take(e_from[b], one[b]);
                const int32_t* entry = g.entry + row * g.top_pad;
                for (int32_t k = e_from[b] + 1; k < e_to[b]; k += 4) {
                    int32_t e[4];  // on their way together
#pragma unroll
                    for (int i = 0; i < 4; ++i) e[i] = entry[min(k + i, e_to[b] - 1)];
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (k + i < e_to[b]) take(k + i, e[i]);
                }
            }
            // a block without a column of the vocabulary leaves 0
            const float mm = m == -__builtin_inff() ? 0.0f : m;
            float s = 0.0f;
#pragma unroll
            for (int a = 0; a < TA; ++a)
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const float x = (acc[a][b][k] - mm) * g.log2e_t;
                    const float e = __builtin_amdgcn_exp2f(x);
                    acc[a][b][k] = F32 ? e : -x;
                    s += e;
                }
            s += __shfl_xor(s, 16);
            s += __shfl_xor(s, 32);
            if (lg == 0 && real)
                g.part[row * g.nblk + a_wave / kHeadBlock] = make_float2(m, s);
            if (g.p) {
                if constexpr (F32) {
                    float* out = static_cast<float*>(g.p) + row * g.ldp + a_wave + lg * 4;
#pragma unroll
                    for (int a = 0; a < TA; ++a)
                        *reinterpret_cast<f32x4*>(out + a * 16) = acc[a][b];
                } else {
                    uint16_t* out = static_cast<uint16_t*>(g.p) + row * g.ldp + a_wave;
#pragma unroll
                    for (int a = 0; a < TA; a += 2)
                        *reinterpret_cast<u32x4*>(out + a * 16 + pair_column(lg)) =
                            pair_by([](float x, float y) { return step_pair(x, y); }, acc[a][b],
                                    acc[a + 1][b]);
                }
            }
        }
    } else {
#pragma unroll
        for (int b = 0; b < TB; ++b) {
            const int64_t row = b_wave + b * 16 + lr;
            if (row >= nb) continue;  // the same for the lanes of a column of rows
            if (ns > 1 || g.acc_in || g.acc_out) {
                float* out = ns > 1 ? g.split + part * (int64_t(nb) * g.ldf) : g.acc_out;
#pragma unroll
                for (int a = 0; a < TA; ++a) {
                    const int64_t col = a_wave + a * 16 + lg * 4;
                    if (col >= g.na) continue;
                    const int64_t at = row * g.ldf + col;
                    if (ns == 1 && g.acc_in)
                        acc[a][b] += *reinterpret_cast<const f32x4*>(g.acc_in + at);
                    if (out) *reinterpret_cast<f32x4*>(out + at) = acc[a][b];
                }
                if (out) continue;
            }
            const int64_t at = (g.rows ? int64_t(g.rows[row]) : row) * g.ldo;
#pragma unroll
            for (int a = 0; a < TA; ++a) acc[a][b] *= g.factor;
            if constexpr (F32) {
                float* out = static_cast<float*>(g.out) + at;
#pragma unroll
                for (int a = 0; a < TA; ++a) {
                    const int64_t col = a_wave + a * 16 + lg * 4;
                    store_part(out, col, g.ldo, acc[a][b]);
                }
            } else {
                uint16_t* out = static_cast<uint16_t*>(g.out) + at;
#pragma unroll
                for (int a = 0; a < TA; a += 2) {
                    const u32x4 v = pair_of(acc[a][b], acc[a + 1][b]);
                    const int64_t col = a_wave + a * 16 + pair_column(lg);
                    store_part(out, col, g.ldo, v);
                }
            }
        }
    }
}

// The products of fp32 planes, the largest first.
__device__ __forceinline__ int plane_a_of(int seg) { return (0x201010 >> (4 * seg)) & 0xf; }
__device__ __forceinline__ int plane_b_of(int seg) { return (0x021100 >> (4 * seg)) & 0xf; }

constexpr uint32_t kThinSegs = 2;  // stages of 32 in a step of 64 k's

// The three products. WA x WB waves, each 64 columns by BB / WB rows of 16 x 16
// tiles; NST stages of 64 k's of both operands in LDS, loaded there directly.
// In tiles of 256 x 256 the matrix cores are busy 65% of the time at the 1.9 to
// 2.1 GHz that the card's power allows: 1.27 to 1.39 PFLOP/s (4096 x 32000 x
// 4096 0.78 ms a product; stages read from the caches alone 1.45, none read
// 1.52 to 1.73 at the same clocks). Where tokens are few, reading the head
// bounds it: 262 MB for 5 tokens in 42 us, 6.2 TB/s.
template <int BA, int BB, int WA, int WB, int NST, bool NT, bool AM, bool BM, bool F32, int KIND>
__global__ __launch_bounds__(64 * WA * WB) void gemm_kernel(GemmArgs g) {
    constexpr int kWaves = WA * WB, BK = kHeadDepth;
    constexpr int EA = BA / WA, EB = BB / WB, TA = EA / 16, TB = EB / 16;
    static_assert(EA == kHeadBlock && TA == 4, "a wave's columns are one block");
    using OpA = Operand<BA, BK, kWaves, AM, !BM, NT>;  // the head ends at v and d
    using OpB = Operand<BB, BK, kWaves, BM, false, false>;
    constexpr int kStage = OpA::kBytes + OpB::kBytes;
    constexpr int kPer = OpA::kLoads + OpB::kLoads;
    constexpr int kSegs = F32 ? 6 : 1;
    __shared__ __attribute__((aligned(1024))) char s_mem[NST * kStage];

    const int lane = threadIdx.x % 64;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);

    // Extents that the device alone knows, then this workgroup's tile: each
    // XCD (workgroups go to the 8 of them in turn) takes one run of the
    // tiles, four b's at a time along all a's, so that what its L2 holds of
    // both operands is used by its neighbours.
    int32_t nb = int32_t(g.nb), klen = int32_t(g.k);
    const int32_t tokens = max(*g.count - int32_t(g.first), 0);
    if (g.tokens_in_b) nb = min(nb, tokens);
    if (g.tokens_in_k) klen = min(klen, tokens);
    // a chunk behind the last token that counts adds nothing to the head's gradient
    // so far (2^20 x 256, 1 GiB there and back: such a chunk 480 -> 48 us)
    if constexpr (BM)
        if (klen == 0 && g.acc_in && g.acc_out) return;
    const uint32_t ta_n = uint32_t(g.na + BA - 1) / BA, tb_n = uint32_t(nb + BB - 1) / BB;
    const uint32_t kt_all = uint32_t(klen + BK - 1) / BK;
    const uint32_t tiles = ta_n * tb_n;
    const uint32_t ns =
        __builtin_amdgcn_readfirstlane(split_of(tiles, kt_all, kSegs, g.slot_bits));
    const uint32_t items = tiles * ns, per = (items + 7) / 8;
    const uint32_t j = blockIdx.x >> 3, item = (blockIdx.x & 7) * per + j;
    if (j >= per || item >= items) return;
    constexpr uint32_t GB = 4;
    const uint32_t part = __builtin_amdgcn_readfirstlane(item / tiles);
    const uint32_t lin = item - part * tiles;
    const uint32_t grp = lin / (GB * ta_n), b_first = grp * GB;
    const uint32_t gb = tb_n - b_first < GB ? tb_n - b_first : GB;
    const uint32_t rem = lin - grp * GB * ta_n, in_b = rem / gb;
    const int64_t a0 = int64_t(in_b) * BA, b0 = int64_t(b_first + rem - in_b * gb) * BB;

    const int wa = wave % WA, wb = wave / WA;
    f32x4 acc[TA][TB];
#pragma unroll
    for (int i = 0; i < TA; ++i)
#pragma unroll
        for (int k = 0; k < TB; ++k) acc[i][k] = f32x4{0.f, 0.f, 0.f, 0.f};

    const uint32_t kt0 = kt_all * part / ns, kt1 = kt_all * (part + 1) / ns;  // below 2^23
    const int nkt = int(kt1 - kt0), steps = nkt * kSegs;
    // Few tokens: the head's rows are read from HBM at the pace of the k's, and
    // columns of the same k of all rows lie in a few of its channels: every
    // tile starts at another k (262 MB at 4.3 -> 5.5 TB/s). Larger tiles share
    // rows through the L2 and keep in step (835 us; 850 to 910 out of step).
    constexpr bool kTurn = KIND == kLogits && NST > 2;
    const int k_turn = kTurn && nkt > 0 ? int(in_b * 3 % nkt) : 0;

    OpA oa;
    OpB ob;
    oa.init(g.a, g.lda, a0, AM ? g.a_width : g.na, wave, lane);
    ob.init(g.b, g.ldb, b0, BM ? g.ldb : (b0 + BB), wave, lane);

    int i_kt = 0, i_seg = 0, i_left = steps;  // the next stage to load
    auto issue = [&](int buf, int from, int to) {
        ZSP_LDS char* lds = (ZSP_LDS char*)s_mem + buf * kStage;
        int kt = i_kt;
        if constexpr (kTurn) kt = kt + k_turn < nkt ? kt + k_turn : kt + k_turn - nkt;
        const int64_t k0 = int64_t(int(kt0) + kt) * BK;
#pragma unroll
        for (int i = from; i < to; ++i) {
            if (i < OpA::kLoads)
                oa.issue(i, lds, F32 ? plane_a_of(i_seg) * g.plane_a : 0, k0, g.k_real - 1, wave);
            else
                ob.issue(i - OpA::kLoads, lds + OpA::kBytes,
                         F32 ? plane_b_of(i_seg) * g.plane_b : 0, k0, 0, wave);
        }
        // past the last stage it is loaded again: nothing reads it
        if (to == kPer && --i_left > 0 && ++i_seg == kSegs) {
            i_seg = 0;
            ++i_kt;
        }
    };
    // Stage s is read from buffer s % NST. Its first half of the k's is read into
    // registers while the matrix cores work on the stage before, its second
    // half while they work on the first, so that they wait for neither.
    bf16x8 fa[2][TA], fb[2][TB];
    int buf = 0;
    auto read = [&](int half, int from, int i) {
        ZSP_LDS const char* la = (ZSP_LDS const char*)s_mem + from * kStage;
        if (i < TA) fa[half][i] = OpA::frag(la, wa * EA, i * 16, half, lane);
        else fb[half][i - TA] = OpB::frag(la + OpA::kBytes, wb * EB, (i - TA) * 16, half, lane);
    };
    // Half a stage: the tiles of `half` multiplied, with the reads of the
    // other half (of buffer `from`) and, where `load`, the loads of a stage to
    // come between them, a quarter of each at a time.
    constexpr int kParts = 4, kMul = TA * TB / kParts;
    auto work = [&](auto half_c, int from, auto load_c, int into) {
        constexpr int half = decltype(half_c)::value;
#pragma unroll
        for (int q = 0; q < kParts; ++q) {
#pragma unroll
            for (int i = (TA + TB) * q / kParts; i < (TA + TB) * (q + 1) / kParts; ++i)
                read(half ^ 1, from, i);
            if constexpr (decltype(load_c)::value)
                issue(into, kPer * q / kParts, kPer * (q + 1) / kParts);
#pragma unroll
            for (int i = kMul * q; i < kMul * (q + 1); ++i)
                acc[i % TA][i / TA] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                    fa[half][i % TA], fb[half][i / TA], acc[i % TA][i / TA], 0, 0, 0);
            __builtin_amdgcn_sched_barrier(0);
        }
    };
    using std::integral_constant;
    if (steps > 0) {
#pragma unroll
        for (int i = 0; i < NST; ++i) issue(i, 0, kPer);
        wait_stage<(NST - 1) * kPer>();
        wg_barrier();
#pragma unroll
        for (int i = 0; i < TA + TB; ++i) read(0, 0, i);
    }
    for (int it = 0; it < steps; ++it) {
        __builtin_amdgcn_sched_barrier(0);
        work(integral_constant<int, 0>(), buf, integral_constant<bool, false>(), 0);
        // this wave has read all of this stage, and its part of the next has
        // landed; then that holds for every wave
        wait_stage<(NST - 2) * kPer>();
        wg_barrier();
        const int old = buf;
        buf = NST == 2 ? buf ^ 1 : buf + 1 == NST ? 0 : buf + 1;
        // behind the last stage: loaded and read, not used
        work(integral_constant<int, 1>(), buf, integral_constant<bool, true>(), old);
    }
    wait_stage<0>();  // no load into LDS outlives the workgroup

    finish<KIND, F32, TA, TB>(g, acc, a0 + wa * EA, b0 + wb * EB, nb, part, ns, lane);
}

// Few tokens and an fp32 head: the head is read in place, once for each
// product, and split into planes on its way from LDS to the matrix cores (4
// bytes an element; copied as planes first it would be 10, and 12 more for
// each product). A workgroup takes 256 rows (columns) of the head, four waves
// of 64; 16 TB tokens; stages of 32 k's. An infinity in the head comes out as
// NaN. 24 tokens x 66306 x 4224 with the gradient of hidden: 1570 us with the
// planes copied, 510 this way.
template <int TB, bool AM, int KIND>
__global__ __launch_bounds__(256) void thin_kernel(GemmArgs g) {
    constexpr int BA = 256, BB = 16 * TB, TA = 4, BK = 32, NST = TB == 4 ? 3 : 2;
    constexpr int kABytes = BA * BK * 4, kStage = kABytes + 3 * BB * BK * 2;
    constexpr int kALoads = kABytes / 1024 / 4, kBLoads = (3 * TB + 3) / 4;
    constexpr int kPer = kALoads + kBLoads;
    __shared__ __attribute__((aligned(1024))) char s_mem[NST * kStage];
    const int lane = threadIdx.x % 64, lr = lane % 16, lg = lane / 16;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);

    const int32_t nb = min(int32_t(g.nb), max(*g.count - int32_t(g.first), 0));
    const uint32_t tiles = nb > 0 ? uint32_t(g.na + BA - 1) / BA : 0;
    const uint32_t kt_all = uint32_t(g.k + kHeadDepth - 1) / kHeadDepth;
    const uint32_t ns =
        __builtin_amdgcn_readfirstlane(split_of(tiles, kt_all, kThinSegs, g.slot_bits));
    const uint32_t items = tiles * ns, per = (items + 7) / 8;
    const uint32_t j = blockIdx.x >> 3, item = (blockIdx.x & 7) * per + j;
    if (j >= per || item >= items) return;
    const uint32_t part = __builtin_amdgcn_readfirstlane(item / tiles), tile = item - part * tiles;
    const int64_t a0 = int64_t(tile) * BA;
    const uint32_t kt0 = kt_all * part / ns, kt1 = kt_all * (part + 1) / ns;
    const int nkt = int(kt1 - kt0), steps = nkt * kThinSegs;
    const int k_turn = !AM && nkt > 0 ? int(tile * 3 % nkt) : 0;  // as in gemm_kernel

    const float* head = reinterpret_cast<const float*>(g.a);
    const int32_t width = int32_t(g.a_width);
    uint32_t a_off[kALoads];
    int32_t a_k[kALoads];
#pragma unroll
    for (int i = 0; i < kALoads; ++i) {
        const int q = (wave * kALoads + i) * 64 + lane;
        if constexpr (AM) {  // rows of 256 columns, 64 groups of 4
            const int k = q / 64, c = (q % 64) ^ (((k >> 3) & 3) * 4);
            a_k[i] = k;
            a_off[i] = uint32_t(min(int32_t(a0) + c * 4, width - 4) - int32_t(a0)) * 4;
        } else {             // rows of 32 k's, 8 groups of 4
            const int r = q / 8, c = (q % 8) ^ ((r >> 1) & 7);
            a_k[i] = c * 4;
            a_off[i] = uint32_t(min(a0 + r, g.na - 1) - a0) * uint32_t(g.lda) * 4;
        }
    }
    int next = 0;  // the stage to load
    auto issue = [&](int buf) {
        ZSP_LDS char* lds = (ZSP_LDS char*)s_mem + buf * kStage;
        int kt = next / kThinSegs;
        kt = kt + k_turn < nkt ? kt + k_turn : kt + k_turn - nkt;
        const int64_t k0 = int64_t(int(kt0) + kt) * kHeadDepth + next % kThinSegs * BK;
        // half a step may lie behind the head's last row
        const int64_t k_last = g.k_real - 1, k_base = k0 < k_last ? k0 : k_last;
        const char* base = reinterpret_cast<const char*>(AM ? head + k_base * g.lda + a0
                                                            : head + a0 * g.lda);
#pragma unroll
        for (int i = 0; i < kALoads; ++i) {
            uint32_t o = a_off[i];
            if constexpr (AM)  // rows past the head's last are read as that one
                o += uint32_t(min(k0 + a_k[i], k_last) - k_base) * uint32_t(g.lda) * 4;
            else               // columns past a row's last four as those
                o += uint32_t(min(int32_t(k0) + a_k[i], width - 4)) * 4;
            load_to_lds<true>(base, o, lds + (wave * kALoads + i) * 1024);
        }
#pragma unroll
        for (int i = 0; i < kBLoads; ++i) {
            const int load = min(wave * kBLoads + i, 3 * TB - 1);
            const int r = lane / 4, c = (lane % 4) ^ ((r >> 2) & 3);
            const uint16_t* b = g.b + load / TB * g.plane_b + load % TB * 16 * g.ldb + k0;
            load_to_lds<false>(reinterpret_cast<const char*>(b),
                               uint32_t(r) * uint32_t(g.ldb) * 2 + c * 16,
                               lds + kABytes + load * 1024);
        }
        if (next + 1 < steps) ++next;  // past the last stage it is loaded again: nothing reads it
    };
    f32x4 acc[TA][TB];
#pragma unroll
    for (int i = 0; i < TA; ++i)
#pragma unroll
        for (int k = 0; k < TB; ++k) acc[i][k] = f32x4{0.f, 0.f, 0.f, 0.f};
    if (steps > 0)
        for (int i = 0; i < NST - 1; ++i) issue(i);
    int buf = 0, into = NST - 1;
    for (int it = 0; it < steps; ++it) {
        wait_stage<(NST - 2) * kPer>();
        wg_barrier();
        issue(into);
        into = into + 1 == NST ? 0 : into + 1;
        ZSP_LDS const char* la = (ZSP_LDS const char*)s_mem + buf * kStage;
        ZSP_LDS const char* lb = la + kABytes;
        buf = buf + 1 == NST ? 0 : buf + 1;
        bf16x8 fb[3][TB];
#pragma unroll
        for (int p = 0; p < 3; ++p)
#pragma unroll
            for (int b = 0; b < TB; ++b)
                fb[p][b] = *(ZSP_LDS const bf16x8*)(lb + (p * TB + b) * 1024 + lr * 64 +
                                                    (lg ^ ((lr >> 2) & 3)) * 16);
#pragma unroll
        for (int i = 0; i < TA; ++i) {
            float x[8];
            if constexpr (AM) {
                const int a = wave * 64 + i * 16 + lr;
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    x[k] = *(ZSP_LDS const float*)(la + (lg * 8 + k) * 1024 +
                                                   ((a >> 2) ^ (lg * 4)) * 16 + (a & 3) * 4);
            } else {
                const int row = wave * 64 + i * 16 + lr;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const f32x4 v = *(ZSP_LDS const f32x4*)(la + row * 128 +
                                                            ((2 * lg + h) ^ (lr >> 1)) * 16);
#pragma unroll
                    for (int k = 0; k < 4; ++k) x[h * 4 + k] = v[k];
                }
            }
            u32x4 plane[3];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                float lo = x[2 * k], hi = x[2 * k + 1];
#pragma unroll
                for (int p = 0; p < 3; ++p) {
                    const uint32_t u = bf16_pair(lo, hi);
                    plane[p][k] = u;
                    lo -= __uint_as_float(u << 16);
                    hi -= __uint_as_float(u & 0xffff0000u);
                }
            }
#pragma unroll
            for (int q = 0; q < 6; ++q)
#pragma unroll
                for (int b = 0; b < TB; ++b)
                    acc[i][b] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                        __builtin_bit_cast(bf16x8, plane[plane_a_of(q)]), fb[plane_b_of(q)][b],
                        acc[i][b], 0, 0, 0);
        }
    }
    wait_stage<0>();  // no load into LDS outlives the workgroup
    finish<KIND, true, TA, TB>(g, acc, a0 + wave * 64, 0, nb, part, ns, lane);
}

// ---- the softmax joined, the losses, G ------------------------------------------------

struct JoinArgs {
    const float2* part;
    int64_t nblk;             // between rows of part
    int32_t blocks;           // that hold columns of the vocabulary: P's others are not written
    const int32_t* count;
    int64_t first;            // the chunk's first token
    const int32_t* rows;      // of the chunk, like the next four
    const float* coef;
    const int32_t* entry;
    const float* pick;
    const float* teach;       // the teacher's logits in the entries' order, or NULL
    int32_t top, top_pad;
    float temp, log2e_t;      // T, log2(e) / T
    double inv_temp;
    float* loss;
    float* lse;
    void* p;                  // [chunk][ldp], or NULL: no gradients
    uint16_t* g;              // fp32: the planes of G; else where the steps are
    int64_t ldp, plane;
    int32_t parts;            // workgroups a token
};

// NaN wins, as in a sum
__device__ __forceinline__ float nan_max(float a, float b) { return a != a || a > b ? a : b; }

// Two largest values, and two sums, over the T threads of a workgroup, in a
// fixed order; s holds two for each wave.
template <int T>
__device__ __forceinline__ void block_max2(float& a, float& b, float* s) {
    for (int o = 32; o; o >>= 1) {
        a = nan_max(a, __shfl_xor(a, o));
        b = nan_max(b, __shfl_xor(b, o));
    }
    if constexpr (T == 64) return;
    __syncthreads();
    if (threadIdx.x % 64 == 0) {
        s[threadIdx.x / 64] = a;
        s[T / 64 + threadIdx.x / 64] = b;
    }
    __syncthreads();
    a = s[0];
    b = s[T / 64];
#pragma unroll
    for (int w = 1; w < T / 64; ++w) {
        a = nan_max(a, s[w]);
        b = nan_max(b, s[T / 64 + w]);
    }
}
template <int T>
__device__ __forceinline__ void block_sum2(double& a, double& b, double* s) {
    for (int o = 32; o; o >>= 1) {
        a += __shfl_xor(a, o);
        b += __shfl_xor(b, o);
    }
    if constexpr (T == 64) return;
    __syncthreads();
    if (threadIdx.x % 64 == 0) {
        s[threadIdx.x / 64] = a;
        s[T / 64 + threadIdx.x / 64] = b;
    }
    __syncthreads();
    a = s[0];
    b = s[T / 64];
#pragma unroll
    for (int w = 1; w < T / 64; ++w) {
        a += s[w];
        b += s[T / 64 + w];
    }
}

template <bool F32>
__device__ __forceinline__ void put_g(const JoinArgs& a, int64_t row, int64_t col, float v) {
    if constexpr (F32) {
        uint16_t h[3];
        split3(v, h);
#pragma unroll
        for (int k = 0; k < 3; ++k) a.g[k * a.plane + row * a.ldp + col] = h[k];
    } else {
        a.g[row * a.ldp + col] = bf16_bits(v);
    }
}
template <bool F32>
__device__ __forceinline__ void put_g8(const JoinArgs& a, int64_t row, int64_t col,
                                       const float v[8]) {
    if constexpr (F32) {
        Eight<float> e;
#pragma unroll
        for (int k = 0; k < 8; ++k) e.v[k / 4][k % 4] = __float_as_uint(v[k]);
        e.store(a.g + row * a.ldp + col, a.plane);
    } else {
        u32x4 o;
#pragma unroll
        for (int k = 0; k < 4; ++k) o[k] = bf16_pair(v[2 * k], v[2 * k + 1]);
        *reinterpret_cast<u32x4*>(a.g + row * a.ldp + col) = o;
    }
}

// A thread's entries of row r, read before anything waits for them: the
// teacher's softmax goes through the same joins over the workgroup as the
// model's. In 64 bits, exponentials too: the loss and p - q are small
// differences where the model agrees with its target, and with fp32
// exponentials (32 us in place of 36 for 6354 tokens x 716 x 14 entries) a
// gradient of 1.5e-6 was 4e-9 off.
template <int T, int N>
struct Entries {
    int32_t e[N];
    float t[N];

    __device__ __forceinline__ void load(const JoinArgs& a, int64_t r) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int32_t k = i * T + threadIdx.x;
            e[i] = -1;
            t[i] = 0.0f;
            if (i * T >= a.top || k >= a.top) continue;
            e[i] = a.entry[r * a.top_pad + k];
            if (a.teach) t[i] = a.teach[r * a.top_pad + k];
        }
    }
    __device__ __forceinline__ float largest(const JoinArgs& a) const {
        float m = -__builtin_inff();
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (i * T < a.top && e[i] >= 0) m = nan_max(m, t[i]);
        return m;
    }
    // Against the largest: logits may all be far below 0.
    __device__ __forceinline__ double total(const JoinArgs& a, float m) const {
        double s = 0.0;
        if (!a.teach) return s;
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (i * T < a.top && e[i] >= 0)
                s += exp((double(t[i]) - double(m)) / double(a.temp));
        return s;
    }
    // The row's loss; leaves the entries' share of the target in s_q.
    template <typename F>
    __device__ __forceinline__ double loss(const JoinArgs& a, double lse, float m, double total,
                                           float* s_q, double* s_d, F logit) const {
        if (!a.teach) {
            if (threadIdx.x == 0) s_q[0] = 1.0f;
            return threadIdx.x == 0 ? lse - logit(0, e[0]) : 0.0;
        }
        const double lq = log(total);
        double sum = 0.0, none = 0.0;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int32_t k = i * T + threadIdx.x;
            if (i * T >= a.top || k >= a.top) continue;
            double q = 0.0;
            if (e[i] >= 0) {
                const double l = (double(t[i]) - double(m)) / double(a.temp) - lq;
                q = exp(l);
                if (q != 0.0) sum += q * (l - (logit(k, e[i]) - lse));
            }
            s_q[k] = float(q);
        }
        block_sum2<T>(sum, none, s_d);
        return sum * double(a.temp) * double(a.temp);
    }
};

// The entries' own G, in columns [from, to): c (p - q) with p - q = (p - 1) +
// (1 - q) in 64 bits (in bf16 all of 1 - p would be lost where the model
// is sure of its target). Entries of one column write the same sum of their q;
// they stand in one block of the vocabulary, so beside each other.
template <bool F32, int T, typename F>
__device__ __forceinline__ void entries_gradient(const JoinArgs& a, int64_t r, int64_t from,
                                                 int64_t to, double lse, float c, const float* s_q,
                                                 F logit) {
    const int32_t* entry = a.entry + r * a.top_pad;
    for (int32_t k = threadIdx.x; k < a.top; k += T) {
        const int32_t e = entry[k];
        if (e < from || e >= to) continue;
        const int32_t block = e / kHeadBlock;
        int32_t first = k;
        while (first > 0 && entry[first - 1] / kHeadBlock == block) --first;
        double q = 0.0;
        for (int32_t o = first; o < a.top && entry[o] >= 0 && entry[o] / kHeadBlock == block; ++o)
            if (entry[o] == e) q += double(s_q[o]);
        const double x = logit(k, e) - lse;
        put_g<F32>(a, r, e, float(double(c) * (expm1(x) + (1.0 - q))));
    }
}

// A workgroup (several, where tokens are few) per token that counts: lse =
// m + log sum_b s_b exp(m_b - m) over the blocks, the loss, then the token's row
// of G = c exp(m_b - lse) P, its steps read and G written in place: bound by
// those bytes (4 an element, fp32 10; 4096 tokens x 32000 in 93 us, 5.7 TB/s)
// or, where rows are short, by the joins over the workgroup. Largest logits and
// entries come as they were summed; 1 / T is applied in 64 bits.
template <bool F32, int T>
__global__ __launch_bounds__(T) void join_kernel(JoinArgs a) {
    constexpr int kTop = T == 64 ? 64 : kHeadMaxTop;
    __shared__ double s_d[T / 32];
    __shared__ float s_f[T / 32];
    __shared__ float s_q[kTop];
    const int64_t r = blockIdx.x / a.parts, count = *a.count - a.first;
    const int32_t part_no = int32_t(blockIdx.x - r * a.parts);
    const int t = threadIdx.x;
    // this workgroup's columns
    const int64_t from = int64_t(a.blocks) * part_no / a.parts * kHeadBlock;
    const int64_t to = int64_t(a.blocks) * (part_no + 1) / a.parts * kHeadBlock;
    if (r >= count) {
        // zeros behind the last token, as far as a stage of the sum over
        // tokens may read
        if (a.p && r < (count + kHeadDepth - 1) / kHeadDepth * kHeadDepth)
            for (int64_t c = from + t * 8; c < to; c += T * 8)
                for (int k = 0; k < (F32 ? 3 : 1); ++k)
                    *reinterpret_cast<u32x4*>(a.g + k * a.plane + r * a.ldp + c) = u32x4{0, 0, 0, 0};
        return;
    }
    Entries<T, kTop / T> entries;
    entries.load(a, r);
    const int64_t token = a.rows[r];
    const float c = a.coef[r];
    const float2* part = a.part + r * a.nblk;
    float m = -__builtin_inff();
    for (int32_t b = t; b < a.blocks; b += T) m = nan_max(m, part[b].x);
    float tm = entries.largest(a);
    block_max2<T>(m, tm, s_f);
    double s = 0.0;
    for (int32_t b = t; b < a.blocks; b += T) {
        const float2 q = part[b];
        s += double(q.y) * double(q.x == m ? 1.0f : __builtin_amdgcn_exp2f((q.x - m) * a.log2e_t));
    }
    double ts = entries.total(a, tm);
    block_sum2<T>(s, ts, s_d);
    const double lse = double(m) * a.inv_temp + log(s);
    const float* pick = a.pick + r * a.top_pad;
    auto logit = [&](int32_t k, int32_t) { return double(pick[k]) * a.inv_temp; };
    const double loss = entries.loss(a, lse, tm, ts, s_q, s_d, logit);
    if (t == 0 && part_no == 0) {
        a.loss[token] = float(loss);
        if (a.lse) a.lse[token] = float(lse);
    }
    if (!a.p) return;

    // m_b / T - lse from 64 bits: rounded to fp32 first, an lse of 3000 would
    // leave every p with an error of 1e-4
    auto below = [&](float m_b) { return float(double(m_b) * a.inv_temp - lse); };
    if constexpr (F32) {
        const float* p = static_cast<const float*>(a.p) + r * a.ldp;
        for (int64_t i = from + t * 4; i < to; i += T * 4) {
            const float f = c * fast_exp(below(part[i / kHeadBlock].x));
            const f32x4 v = *reinterpret_cast<const f32x4*>(p + i);
            uint16_t h[4][3];
#pragma unroll
            for (int k = 0; k < 4; ++k) split3(f * v[k], h[k]);
#pragma unroll
            for (int k = 0; k < 3; ++k) {
                uint2 o;
                o.x = h[0][k] | uint32_t(h[1][k]) << 16;
                o.y = h[2][k] | uint32_t(h[3][k]) << 16;
                *reinterpret_cast<uint2*>(a.g + k * a.plane + r * a.ldp + i) = o;
            }
        }
    } else {
        uint16_t* p = a.g + r * a.ldp;
        for (int64_t i = from + t * 8; i < to; i += T * 8) {
            const float at = below(part[i / kHeadBlock].x) * kLog2e;
            u32x4 v = *reinterpret_cast<const u32x4*>(p + i);
#pragma unroll
            for (int k = 0; k < 4; ++k)
                v[k] = bf16_pair(c * step_value(v[k] & 0xffff, at), c * step_value(v[k] >> 16, at));
            *reinterpret_cast<u32x4*>(p + i) = v;
        }
    }
    __threadfence_block();
    __syncthreads();
    entries_gradient<F32, T>(a, r, from, to, lse, c, s_q, logit);
}

// Few tiles (a small vocabulary, or few tokens): the logits' sums over d are
// split too, their fp32 parts stand in the workspace, and a workgroup per
// token joins them in LDS and takes the softmax, the loss and G from there.
struct RawArgs {
    JoinArgs j;
    const float* raw;          // [part][row][ldp]
    int64_t v, dp;
    int64_t len;               // tokens of the chunk
    uint32_t ba, bb, segs, slot_bits;
};

template <bool F32, int T, int COLS>
__global__ __launch_bounds__(T) void raw_join_kernel(RawArgs q) {
    __shared__ float s_l[COLS];
    __shared__ double s_d[T / 32];
    __shared__ float s_f[T / 32];
    __shared__ float s_q[kHeadMaxTop];
    const JoinArgs& a = q.j;
    const int64_t r = blockIdx.x;
    const int32_t count = max(*a.count - int32_t(a.first), 0);
    const int t = threadIdx.x, cols = a.blocks * kHeadBlock, v = int32_t(q.v);
    if (r >= count) {
        if (a.p && r < (count + kHeadDepth - 1) / kHeadDepth * kHeadDepth)
            for (int c = t * 8; c < cols; c += T * 8)
                for (int k = 0; k < (F32 ? 3 : 1); ++k)
                    *reinterpret_cast<u32x4*>(a.g + k * a.plane + r * a.ldp + c) = u32x4{0, 0, 0, 0};
        return;
    }
    Entries<T, kHeadMaxTop / T> entries;
    entries.load(a, r);
    const int64_t token = a.rows[r];
    const float c = a.coef[r];
    const uint32_t tiles = (uint32_t(v) + q.ba - 1) / q.ba *
                           ((uint32_t(min(int64_t(count), q.len)) + q.bb - 1) / q.bb);
    const uint32_t ns = split_of(tiles, uint32_t(q.dp) / kHeadDepth, q.segs, q.slot_bits);
    const int64_t stride = int64_t(min(int64_t(count), q.len)) * a.ldp;
    const float* raw = q.raw + r * a.ldp;
    float m = -__builtin_inff();
    for (int c0 = t; c0 < v; c0 += 4 * T) {
        float l[4] = {0.f, 0.f, 0.f, 0.f};
        for (uint32_t s = 0; s < ns; s += 4) {
            float x[4][4];  // all on their way before the first is added
#pragma unroll
            for (uint32_t k = 0; k < 4; ++k)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    x[k][i] = raw[min(s + k, ns - 1) * stride + min(c0 + i * T, v - 1)];
#pragma unroll
            for (uint32_t k = 0; k < 4; ++k)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (s + k < ns) l[i] += x[k][i];
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (c0 + i * T >= v) break;
            s_l[c0 + i * T] = l[i];
            m = nan_max(m, l[i]);
        }
    }
    float tm = entries.largest(a);
    block_max2<T>(m, tm, s_f);
    float part = 0.0f;
    for (int i = t; i < v; i += T) part += __builtin_amdgcn_exp2f((s_l[i] - m) * a.log2e_t);
    double s = double(part), ts = entries.total(a, tm);
    block_sum2<T>(s, ts, s_d);
    const double lse = double(m) * a.inv_temp + log(s);
    auto logit = [&](int32_t, int32_t e) { return double(s_l[e]) * a.inv_temp; };
    const double loss = entries.loss(a, lse, tm, ts, s_q, s_d, logit);
    if (t == 0) {
        a.loss[token] = float(loss);
        if (a.lse) a.lse[token] = float(lse);
    }
    if (!a.p) return;
    const float shift = float(double(m) * a.inv_temp - lse) * kLog2e;  // as in join_kernel
    for (int i = t * 8; i < cols; i += T * 8) {
        float g[8];
#pragma unroll
        for (int k = 0; k < 8; ++k)
            g[k] = i + k < v ? c * __builtin_amdgcn_exp2f((s_l[i + k] - m) * a.log2e_t + shift) : 0.0f;
        put_g8<F32>(a, r, i, g);
    }
    __threadfence_block();
    __syncthreads();
    entries_gradient<F32, T>(a, r, 0, cols, lse, c, s_q, logit);
}

// The head's gradient of few tokens (bf16): rows of d for every column of the
// vocabulary, of sums over at most 32 KS tokens, so that writing them is what
// takes the time. A workgroup holds 64 columns of G (through LDS, transposed,
// in registers); its waves go along the rows of X^T, which the L2 holds, and
// write: no stage waits for another, nothing for a barrier. 32000 x 4096 of 96
// tokens: 90 us by tiles, 73 this way; of 17: 69 and 45.
struct OuterArgs {
    const uint16_t* xt;        // [dp][32 KS]
    const uint16_t* g;         // [token][ldp]
    uint16_t* out;             // [v][d]
    const int32_t* count;
    int64_t v, d, dp, ldp;
    float factor;
    int32_t parts, steps;      // workgroups for 64 columns, 64-column steps a wave
};

template <int KS>
__global__ __launch_bounds__(256) void outer_kernel(OuterArgs a) {
    __shared__ __attribute__((aligned(16))) char s_g[32 * KS * 128];
    const int lane = threadIdx.x % 64, wave = threadIdx.x / 64, lr = lane % 16, lg = lane / 16;
    const int64_t v0 = int64_t(blockIdx.x / a.parts) * 64;
    const int32_t count = *a.count;
#pragma unroll
    for (int i = 0; i < KS; ++i) {
        const int k = i * 32 + threadIdx.x / 8, c = threadIdx.x % 8;
        u32x4 q = {0, 0, 0, 0};
        if (k < count) q = *reinterpret_cast<const u32x4*>(a.g + k * a.ldp + v0 + c * 8);
        *reinterpret_cast<u32x4*>(s_g + k * 128 + c * 16) = q;
    }
    __syncthreads();
    bf16x8 fb[4][KS];
#pragma unroll
    for (int b = 0; b < 4; ++b)
#pragma unroll
        for (int k = 0; k < KS; ++k) {
            const int row = k * 32 + lg * 8 + lr / 4;
            ZSP_LDS char* at = (ZSP_LDS char*)s_g + row * 128 + b * 32 + (lr % 4) * 8;
            const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((ZSP_LDS s16x4*)at);
            const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((ZSP_LDS s16x4*)(at + 512));
            fb[b][k] = __builtin_bit_cast(
                bf16x8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
        }
    const int64_t first = (int64_t(blockIdx.x % a.parts) * 4 + wave) * a.steps * 64;
    const int64_t last = min(first + a.steps * 64, a.dp);
    // the next step's rows on their way while this one's are multiplied
    bf16x8 fa[4][KS], next[4][KS];
    auto load = [&](int64_t c0) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int k = 0; k < KS; ++k)
                next[i][k] = *reinterpret_cast<const bf16x8*>(
                    a.xt + (c0 + i * 16 + lr) * (32 * KS) + k * 32 + lg * 8);
    };
    if (first < last) load(first);
    for (int64_t c0 = first; c0 < last; c0 += 64) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int k = 0; k < KS; ++k) fa[i][k] = next[i][k];
        if (c0 + 64 < last) load(c0 + 64);
#pragma unroll
        for (int b = 0; b < 4; ++b) {
            f32x4 acc[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                acc[i] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int k = 0; k < KS; ++k)
                    acc[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fa[i][k], fb[b][k], acc[i], 0,
                                                                     0, 0);
            }
            const int64_t row = v0 + b * 16 + lr;
            uint16_t* out = a.out + row * a.d;
#pragma unroll
            for (int i = 0; i < 4; i += 2) {
                const u32x4 v = pair_of(acc[i] * a.factor, acc[i + 1] * a.factor);
                const int64_t col = c0 + i * 16 + pair_column(lg);
                if (row >= a.v) continue;
                store_part(out, col, a.d, v);
            }
        }
    }
}

hipError_t run_outer(OuterArgs a, int64_t n, hipStream_t stream) {
    const int64_t blocks = (a.v + 63) / 64, columns = a.dp / 64;
    // eight waves a CU at least, where there are columns enough
    a.parts = int32_t(std::min<int64_t>((511 + blocks) / blocks, (columns + 3) / 4));
    a.steps = int32_t((columns + a.parts * 4 - 1) / (a.parts * 4));
    const uint32_t grid = uint32_t(blocks * a.parts);
    switch ((n + 31) / 32) {
        case 1: outer_kernel<1><<<grid, 256, 0, stream>>>(a); break;
        case 2: outer_kernel<2><<<grid, 256, 0, stream>>>(a); break;
        case 3: outer_kernel<3><<<grid, 256, 0, stream>>>(a); break;
        default: outer_kernel<4><<<grid, 256, 0, stream>>>(a); break;
    }
    return hipGetLastError();
}

// A gradient's split sums joined, in order: four columns a thread, `parts`
// workgroups a row. Bound by reading the parts (3 of 2401 x 4096 in 24 us).
// Nothing to do where the product's sums were not split.
struct SplitArgs {
    GemmArgs g;
    uint32_t ba, bb, segs, parts;
};

template <bool F32>
__device__ __forceinline__ void join_split(const SplitArgs& a, int32_t nb, uint32_t ns, int64_t i) {
    const GemmArgs& g = a.g;
    const int64_t row = i / a.parts;
    const int64_t col = ((i - row * a.parts) * 256 + threadIdx.x) * 4;
    if (col >= g.ldo) return;
    const int64_t at = row * g.ldf + col;
    f32x4 v = {0.f, 0.f, 0.f, 0.f};
    if (g.acc_in) v = *reinterpret_cast<const f32x4*>(g.acc_in + at);
    const float* part = g.split + at;
    const int64_t stride = int64_t(nb) * g.ldf;
    for (uint32_t s = 0; s < ns; s += 4) {
        f32x4 q[4];  // all on their way before the first is added
#pragma unroll
        for (uint32_t k = 0; k < 4; ++k)
            q[k] = *reinterpret_cast<const f32x4*>(part + min(s + k, ns - 1) * stride);
#pragma unroll
        for (uint32_t k = 0; k < 4; ++k)
            if (s + k < ns) v += q[k];
    }
    if (g.acc_out) {
        *reinterpret_cast<f32x4*>(g.acc_out + at) = v;
        return;
    }
    v *= g.factor;
    const int64_t o = (g.rows ? int64_t(g.rows[row]) : row) * g.ldo + col;
    if constexpr (F32) {
        float* out = static_cast<float*>(g.out) + o;
        if (col + 4 <= g.ldo) {
            *reinterpret_cast<f32x4_a4*>(out) = v;
        } else {
            for (int k = 0; k < 4; ++k)
                if (col + k < g.ldo) out[k] = v[k];
        }
    } else {
        uint16_t* out = static_cast<uint16_t*>(g.out) + o;
        if (col + 4 <= g.ldo) {
            *reinterpret_cast<u32x2_a2*>(out) = u32x2_a2{bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3])};
        } else {
            for (int k = 0; k < 4; ++k)
                if (col + k < g.ldo) out[k] = bf16_bits(v[k]);
        }
    }
}

template <bool F32>
__global__ __launch_bounds__(256) void split_kernel(SplitArgs a) {
    const GemmArgs& g = a.g;
    int32_t nb = int32_t(g.nb), klen = int32_t(g.k);
    const int32_t tokens = max(*g.count - int32_t(g.first), 0);
    if (g.tokens_in_b) nb = min(nb, tokens);
    if (g.tokens_in_k) klen = min(klen, tokens);
    const uint32_t tiles = (uint32_t(g.na) + a.ba - 1) / a.ba * ((uint32_t(nb) + a.bb - 1) / a.bb);
    const uint32_t ns =
        split_of(tiles, uint32_t(klen + kHeadDepth - 1) / kHeadDepth, a.segs, g.slot_bits);
    if (ns == 1) return;
    for (int64_t i = blockIdx.x; i < int64_t(nb) * a.parts; i += gridDim.x) join_split<F32>(a, nb, ns, i);
}

// ---- launches ------------------------------------------------------------------------

// A product's tiles: columns and rows of a tile, how many the card runs at once
// (log2), and which form.
enum Form { kFormBig, kFormWide, kFormMid, kFormMidOnce, kFormLow, kFormLow2, kFormThin };
constexpr HeadTiles kBig{256, 256, 8, kFormBig}, kWide{128, 256, 8, kFormWide},
    kMid{128, 128, 9, kFormMid}, kMidOnce{128, 128, 9, kFormMidOnce},
    kLow{128, 64, 8, kFormLow}, kLow2{128, 128, 8, kFormLow2};

uint32_t tiles_along(int64_t extent, uint32_t tile) { return uint32_t((extent + tile - 1) / tile); }
uint32_t stages_of(int64_t k) { return uint32_t((k + kHeadDepth - 1) / kHeadDepth); }

// Where split_of may answer more than 1: two parts take two stages of eight at
// least, and parts save less than one turn of 16 x stages, while s of them cost
// the joining of tiles * s and the ends of the further turns: nothing is saved
// beyond eight tiles a stage. (The host's bound: on the device the test takes as
// long as what it spares, 333 tokens x 10007 x 768 fp32 138 -> 141 us.)
bool split_may_pay(uint32_t tiles, uint32_t stages, uint32_t segs, uint32_t slot_bits) {
    return slot_bits != 0 && tiles != 0 && tiles >> slot_bits < 64 && stages * segs >= 16 &&
           tiles < stages * segs * 8 + 32;
}

// The most parts that split_of makes of sums of up to `stages`, by trying all
// lengths from the longest on, until the largest number is met that a smaller
// one does not beat at every length: with costs between those of k / s stages
// and of (k + s - 1) / s, which are straight lines, at both ends of its range.
uint32_t most_parts(uint32_t tiles, uint32_t stages, uint32_t segs, uint32_t slot_bits) {
    if (!split_may_pay(tiles, stages, segs, slot_bits)) return 1;
    constexpr uint32_t kParts[] = {2, 3, 4, 5, 6, 8, 10, 12, 16, 24, 32, 48, 64};  // split_of's
    auto turns = [&](uint32_t s) { return double((tiles * s + (1u << slot_bits) - 1) >> slot_bits); };
    auto cost = [&](uint32_t s, double part) {
        return turns(s) * (part * segs + 4) * 16 + (s > 1 ? double(tiles) * s : 0.0);
    };
    uint32_t largest = 1;
    for (uint32_t s : kParts) {
        const uint32_t from = std::max(s, (s * 8 + segs - 1) / segs);  // its shortest sum
        if (from > stages || turns(s) > 64) continue;
        auto beats = [&](uint32_t o) {
            auto better = [&](double k) { return cost(o, (k + o - 1) / o) <= cost(s, k / s); };
            return better(from) && better(stages);
        };
        bool beaten = beats(1);
        for (uint32_t o : kParts)
            if (o < s) beaten |= beats(o);
        if (!beaten) largest = s;
    }
    uint32_t most = 1;
    for (uint32_t k = stages; k > 0 && most < largest; --k)
        most = std::max(most, split_of(tiles, k, segs, slot_bits));
    return most;
}

// t with the largest number of items (tiles times parts) and of partial rows
// times parts over every number of tokens up to the call's. Asked once a call,
// and within split_may_pay's and most_parts' bounds, since the host waits for it
// (2^20 tokens x 64 x 64 1000 us by trying every number of tiles, now 4).
HeadTiles bounded(const GemmArgs& g, HeadTiles t) {
    const uint32_t ta = tiles_along(g.na, t.ba), tb = tiles_along(g.nb, t.bb);
    const uint32_t kt = stages_of(g.k), slot_bits = g.slot_bits ? t.slot_bits : 0;
    auto take = [&](uint32_t b, uint32_t s) {
        t.items = std::max<uint64_t>(t.items, uint64_t(ta) * b * s);
        if (s > 1)
            t.split_rows = std::max<uint64_t>(t.split_rows,
                                              s * std::min<uint64_t>(uint64_t(b) * t.bb, g.nb));
    };
    t.items = t.split_rows = 0;
    if (g.tokens_in_k) {
        take(tb, most_parts(ta * tb, kt, t.segs, slot_bits));
        return t;
    }
    take(tb, split_of(ta * tb, kt, t.segs, slot_bits));
    for (uint32_t b = 1; g.tokens_in_b && b < tb && split_may_pay(ta * b, kt, t.segs, slot_bits); ++b)
        take(b, split_of(ta * b, kt, t.segs, slot_bits));
    return t;
}

// The parts of a split product joined, unless the caller does it.
template <bool F32, int KIND>
hipError_t join_parts(const GemmArgs& g, const HeadTiles& t, hipError_t e, hipStream_t stream) {
    if constexpr (KIND == kOut) {
        if (e == hipSuccess && t.split_rows && !g.keep_parts) {
            SplitArgs q{g, t.ba, t.bb, t.segs, uint32_t((g.ldo + 1023) / 1024)};
            const int64_t rows = g.nb * q.parts;
            split_kernel<F32><<<uint32_t(std::min<int64_t>(rows, 4096)), 256, 0, stream>>>(q);
            e = hipGetLastError();
        }
    }
    return e;
}

template <int BA, int BB, int WA, int WB, int NST, bool NT, bool AM, bool BM, bool F32, int KIND>
hipError_t run_gemm(GemmArgs g, const HeadTiles& t, hipStream_t stream) {
    static_assert(BA <= kHeadTile && BB <= kHeadTile, "");
    if (g.slot_bits) g.slot_bits = t.slot_bits;
    if (t.items == 0) return hipSuccess;
    gemm_kernel<BA, BB, WA, WB, NST, NT, AM, BM, F32, KIND>
        <<<uint32_t((t.items + 7) / 8 * 8), 64 * WA * WB, 0, stream>>>(g);
    return join_parts<F32, KIND>(g, t, hipGetLastError(), stream);
}

template <bool AM, int KIND>
hipError_t run_thin(GemmArgs g, const HeadTiles& t, hipStream_t stream) {
    if (g.slot_bits) g.slot_bits = t.slot_bits;
    if (t.items == 0) return hipSuccess;
    const uint32_t grid = uint32_t((t.items + 7) / 8 * 8);
    if (t.bb == 16) thin_kernel<1, AM, KIND><<<grid, 256, 0, stream>>>(g);
    else if (t.bb == 32) thin_kernel<2, AM, KIND><<<grid, 256, 0, stream>>>(g);
    else thin_kernel<4, AM, KIND><<<grid, 256, 0, stream>>>(g);
    return join_parts<true, KIND>(g, t, hipGetLastError(), stream);
}

// Tiles of 256 x 256 (eight waves, one workgroup on a CU) reach 1.3 PFLOP/s
// on a full card, tiles of 128 x 128 (four waves, two workgroups on a CU)
// 1.05: the smaller are taken where the larger leave more of the card idle.
// For up to 64 and 128 tokens, where reading the head is what takes the time,
// tiles of 128 x 64 and 128 x 128 with six and four stages on their way, for up
// to 256 of 128 x 256 (eight waves, three stages). They read it
// non-temporally: kept in the caches, it would only be driven out by the
// head's gradient, which they can hold instead until it is written (32000 x
// 4096 of 5 tokens 46.8 -> 42.3 us alone; 17 tokens with gradients 198 -> 175).
HeadTiles shape_of(const GemmArgs& g, uint32_t segs, bool low) {
    if (g.thin) {
        const uint32_t bb = g.nb <= 16 ? 16 : g.nb <= 32 ? 32 : 64;
        // two workgroups a CU, or one where 64 tokens leave no room for them
        return {256, bb, bb == 64 ? 8u : 9u, kFormThin, kThinSegs};
    }
    // P and X of so many tokens are not padded past 64 rows
    if (low && g.tokens_in_b && g.nb <= kHeadThin) return kLow;
    const bool few = low && g.tokens_in_b && g.nb <= 128;
    if (few && !g.slot_bits) return kLow2;
    auto cost = [&](HeadTiles t, uint64_t stage) {
        const uint32_t tiles = tiles_along(g.na, t.ba) * tiles_along(g.nb, t.bb);
        const uint32_t kt = stages_of(g.k);
        const uint32_t s = split_of(tiles, kt, segs, g.slot_bits ? t.slot_bits : 0);
        const uint64_t turns = ((uint64_t(tiles) * s - 1) >> t.slot_bits) + 1;
        return turns * ((kt + s - 1) / s * segs + 4) * stage;
    };
    // A turn's stage: 65536 outputs on a CU, 2 x 16384, or 32768 for up to 256
    // tokens, which read the head once (192 tokens x 32000 x 4096: logits 90 ->
    // 77 us, with both gradients 305 -> 282).
    const uint64_t big = cost(kBig, 2 * 105), mid = cost(kMid, 130);
    if (low && g.tokens_in_b && segs == 1 && g.nb > 128 && g.nb <= 256 &&
        cost(kWide, 107) < std::min(big, mid))
        return kWide;
    if (big <= mid) return kBig;
    // at most a workgroup a CU (half of one if the sums are split: more parts
    // serve better than more stages): more stages on their way
    const uint32_t tiles = tiles_along(g.na, 128) * tiles_along(g.nb, 128);
    const uint32_t parts = split_of(tiles, stages_of(g.k), segs, g.slot_bits ? kMid.slot_bits : 0);
    if (tiles * parts <= (g.slot_bits ? 128u : 256u)) return kLow2;
    return few ? kMidOnce : kMid;
}

HeadTiles tile_of(const GemmArgs& g, bool f32, bool low) {
    HeadTiles t = shape_of(g, f32 ? 6 : 1, low);
    if (t.form != kFormThin) t.segs = f32 ? 6 : 1;
    return t;
}

// The forms that read the head once: non-temporally (NT) or kept.
template <bool NT, bool AM, bool F32, int KIND>
hipError_t pick_once(const GemmArgs& g, const HeadTiles& t, hipStream_t stream) {
    if (t.form == kFormLow) return run_gemm<128, 64, 2, 2, 6, NT, AM, false, F32, KIND>(g, t, stream);
    if constexpr (!F32)
        if (t.form == kFormWide)
            return run_gemm<128, 256, 2, 4, 3, NT, AM, false, F32, KIND>(g, t, stream);
    if (t.form == kFormMidOnce)
        return run_gemm<128, 128, 2, 2, 2, NT, AM, false, F32, KIND>(g, t, stream);
    return run_gemm<128, 128, 2, 2, 4, NT, AM, false, F32, KIND>(g, t, stream);
}

template <bool AM, bool BM, bool F32, int KIND>
hipError_t pick_gemm(const GemmArgs& g, const HeadTiles& t, hipStream_t stream) {
    if constexpr (F32 && !BM)
        if (t.form == kFormThin) return run_thin<AM, KIND>(g, t, stream);
    if (t.form == kFormBig)
        return run_gemm<256, 256, 4, 2, 2, false, AM, BM, F32, KIND>(g, t, stream);
    if constexpr (BM) {
        if (t.form == kFormLow2)
            return run_gemm<128, 128, 2, 2, 4, false, AM, BM, F32, KIND>(g, t, stream);
    } else if (t.form != kFormMid) {
        if constexpr (!F32)  // fp32: the copied planes are read several times
            if (!g.keep) return pick_once<true, AM, F32, KIND>(g, t, stream);
        return pick_once<false, AM, F32, KIND>(g, t, stream);
    }
    return run_gemm<128, 128, 2, 2, 2, false, AM, BM, F32, KIND>(g, t, stream);
}

// The gradients' products, without their addresses: what the workspace's
// size is asked of.
GemmArgs hidden_product(const HeadShape& s, int64_t len) {
    GemmArgs h{};
    h.thin = s.thin;
    h.a_width = h.lda = s.pack_head ? s.dp : s.d;
    h.ldb = s.vp;
    h.plane_a = s.v * s.dp;
    h.plane_b = s.chunk * s.vp;
    h.na = s.dp;
    h.nb = len;
    h.k = s.v;
    h.k_real = s.v;
    h.tokens_in_b = 1;
    h.slot_bits = 1;
    h.ldo = s.d;
    h.ldf = s.dp;
    return h;
}
GemmArgs raw_product(const HeadShape& s, int64_t len) {
    GemmArgs h{};
    h.thin = s.thin;
    h.a_width = h.lda = s.pack_head ? s.dp : s.d;
    h.ldb = s.dp;
    h.plane_a = s.v * s.dp;
    h.plane_b = s.rows * s.dp;
    h.na = s.v;
    h.nb = len;
    h.k = s.dp;
    h.k_real = h.a_width;
    h.tokens_in_b = 1;
    h.slot_bits = 1;
    h.ldo = s.v;
    h.ldf = s.vp;
    return h;
}
GemmArgs head_product(const HeadShape& s, int64_t len) {
    GemmArgs h{};
    h.a_width = h.lda = s.dp;
    h.ldb = s.vp;
    h.plane_a = s.rows * s.dp;
    h.plane_b = s.chunk * s.vp;
    h.na = s.dp;
    h.nb = s.v;
    h.k = len;
    h.tokens_in_k = 1;
    h.slot_bits = 1;
    h.ldo = s.d;
    h.ldf = s.dp;
    return h;
}

// The setup's threads of a row (the most that leave at most a sixth of them
// idle), and its workgroups.
struct SetupGrid {
    int32_t row_threads = kSetupThreads, parts;
    int64_t x_groups, entry_groups, head_groups;
    int64_t all() const { return x_groups + entry_groups + head_groups; }
};
SetupGrid setup_grid(const HeadShape& s) {
    SetupGrid m;
    const int64_t eights = s.dp / 8;
    auto padded = [&] { return (eights + m.row_threads - 1) / m.row_threads * m.row_threads; };
    while (m.row_threads > 8 && (padded() - eights) * 6 > eights) m.row_threads /= 2;
    const int64_t per = kSetupThreads / m.row_threads;
    m.parts = int32_t(padded() / m.row_threads);
    const int64_t x_rows = (s.n + kHeadDepth - 1) / kHeadDepth * kHeadDepth;
    m.x_groups = (x_rows + per - 1) / per * m.parts;
    m.entry_groups = s.top > 1 ? s.n : 0;
    m.head_groups = s.pack_head ? (s.v + per * kHeadRun - 1) / (per * kHeadRun) * m.parts : 0;
    return m;
}

template <bool F32>
hipError_t run_head(const HeadShape& s, const HeadCall& c, hipStream_t stream) {
    using T = std::conditional_t<F32, float, uint16_t>;
    char* ws = c.ws;
    int32_t* count = reinterpret_cast<int32_t*>(ws + s.o_count);
    int32_t* rows = reinterpret_cast<int32_t*>(ws + s.o_rows);
    float* coef = reinterpret_cast<float*>(ws + s.o_coef);
    int32_t* entry = reinterpret_cast<int32_t*>(ws + s.o_entry);
    float* pick = reinterpret_cast<float*>(ws + s.o_pick);
    float* teach = s.teacher ? reinterpret_cast<float*>(ws + s.o_teach) : nullptr;
    uint16_t* start = s.top > 1 ? reinterpret_cast<uint16_t*>(ws + s.o_start) : nullptr;
    const int32_t blocks = int32_t((s.v + kHeadBlock - 1) / kHeadBlock);
    uint8_t* flag = s.teacher ? reinterpret_cast<uint8_t*>(ws + s.o_flag) : nullptr;
    uint16_t* x = reinterpret_cast<uint16_t*>(ws + s.o_x);
    float2* part = reinterpret_cast<float2*>(ws + s.o_part);
    const bool grads = s.grad_hidden || s.grad_head;
    hipError_t e;

    const int64_t x_plane = s.rows * s.dp, w_plane = s.v * s.dp;
    const uint16_t* w = static_cast<const uint16_t*>(c.head);
    uint16_t* packed = s.pack_head ? reinterpret_cast<uint16_t*>(ws + s.o_w) : nullptr;
    if (packed) w = packed;
    // few tokens' gradient of the head goes by its own way
    const bool few_tokens = !F32 && s.grad_head && s.n > 0 && s.n <= kHeadFew;
    const int32_t few_pad = int32_t((s.n + 31) / 32 * 32);
    uint16_t* xt = few_tokens ? reinterpret_cast<uint16_t*>(ws + s.o_xt) : nullptr;
    const bool scans = !s.teacher && s.n > 0 && s.n <= kSelfScan;
    if (!scans) {
        const bool few = s.teacher && s.n <= kFlagTokens && s.n * s.top <= kFlagEntries;
        if (flag && !few && s.n > 0) {
            flag_kernel<<<uint32_t((s.n + 3) / 4), 256, 0, stream>>>(
                c.index, c.logit, s.n, s.v, s.top, c.token_weight, flag);
            if ((e = hipGetLastError()) != hipSuccess) return e;
        }
        scan_kernel<<<1, kScanThreads, 0, stream>>>(c.index, few ? c.logit : nullptr, s.top,
                                                    c.token_weight, flag, s.n, s.v, rows, count);
        if ((e = hipGetLastError()) != hipSuccess) return e;
    }
    {
        const SetupGrid m = setup_grid(s);
        SetupArgs q{c.hidden, c.head, c.index, c.logit, c.token_weight, flag, rows, count, coef,
                    entry, teach, start, x, xt, packed, c.grad_hidden, c.loss, c.lse, s.n, s.v, s.d,
                    s.dp, x_plane, w_plane, s.top, s.top_pad, blocks, m.row_threads, m.parts, few_pad,
                    uint32_t(m.x_groups), uint32_t(m.entry_groups), scans};
        if (m.all() > 0) {
            setup_kernel<T><<<uint32_t(m.all()), kSetupThreads, 0, stream>>>(q);
            if ((e = hipGetLastError()) != hipSuccess) return e;
        }
    }

    // What all tokens have in common comes to the gradients in fp32: a factor
    // of 1/96 within G would give every target's -1 the same error in bf16.
    const float factor = c.scale * c.temperature;
    const float log2e_t = 1.0f / c.temperature * kLog2e;
    // Two reads of a head that the Infinity Cache (256 MiB) holds, and no write of
    // its gradient between: few tokens let it stay there (100 tokens x 20000 x
    // 5120: 142 -> 129 us; 131072 x 4096 of 5 tokens 406 -> 430).
    const bool keep = s.grad_hidden && !s.grad_head && s.v * s.dp * 2 <= int64_t(1) << 28;
    void* p = grads ? ws + s.o_p : nullptr;
    uint16_t* gp = reinterpret_cast<uint16_t*>(ws + (F32 ? s.o_g : s.o_p));
    const int64_t g_plane = s.chunk * s.vp;
    float* split = reinterpret_cast<float*>(ws + s.o_split);
    float* acc = reinterpret_cast<float*>(ws + s.o_acc);
    for (int64_t ch = 0; ch < s.nchunk; ++ch) {
        const int64_t first = ch * s.chunk, len = std::min(s.chunk, s.n - first);
        const bool last = ch + 1 == s.nchunk;
        GemmArgs l{};
        l.a = w;
        l.b = x + first * s.dp;
        l.thin = s.thin;
        l.keep = keep;
        l.a_width = l.lda = l.k_real = s.pack_head ? s.dp : s.d;
        l.ldb = s.dp;
        l.plane_a = w_plane;
        l.plane_b = x_plane;
        l.na = s.v;
        l.nb = len;
        l.k = s.dp;
        l.count = count;
        l.first = first;
        l.tokens_in_b = 1;
        l.log2e_t = log2e_t;
        l.part = part;
        l.nblk = s.vp / kHeadBlock;
        l.p = p;
        l.ldp = s.vp;
        l.entry = entry + first * s.top_pad;
        l.start = start ? start + first * (blocks + 1) : nullptr;
        l.blocks = blocks;
        l.pick = pick + first * s.top_pad;
        l.top_pad = s.top_pad;
        if (s.raw && len > 0) {
            GemmArgs h = raw_product(s, len);
            h.keep = keep;
            h.a = w;
            h.b = l.b;
            h.count = count;
            h.first = first;
            h.split = h.acc_out = split;
            h.keep_parts = 1;
            const HeadTiles& t = s.raw_tiles;
            if ((e = pick_gemm<false, false, F32, kOut>(h, t, stream)) != hipSuccess) return e;
            JoinArgs j{nullptr, 0, blocks, count, first, rows + first, coef + first, l.entry,
                       nullptr, teach ? teach + first * s.top_pad : nullptr, s.top, s.top_pad,
                       c.temperature, log2e_t, 1.0 / c.temperature, c.loss, c.lse, p, gp, s.vp,
                       g_plane, 1};
            RawArgs q{j, split, s.v, s.dp, len, t.ba, t.bb, t.segs, t.slot_bits};
            const int64_t pad = (len + kHeadDepth - 1) / kHeadDepth * kHeadDepth;
            const uint32_t grid = uint32_t(grads ? pad : len);
            if (s.v <= kHeadRawSmall)
                raw_join_kernel<F32, 256, kHeadRawSmall><<<grid, 256, 0, stream>>>(q);
            else
                raw_join_kernel<F32, 1024, kHeadRawColumns><<<grid, 1024, 0, stream>>>(q);
            if ((e = hipGetLastError()) != hipSuccess) return e;
        } else if (len > 0) {
            const HeadTiles t = bounded(l, tile_of(l, F32, true));
            if ((e = pick_gemm<false, false, F32, kLogits>(l, t, stream)) != hipSuccess) return e;
        }

        if (!s.raw && len > 0) {
            const int64_t pad = (len + kHeadDepth - 1) / kHeadDepth * kHeadDepth;
            // at least 2048 columns each, in up to 1024 workgroups, since each
            // reads all partials of its token (2048 workgroups: 96 tokens x
            // 32000 x 4096 take 203 us in place of 195)
            const int64_t most = std::min<int64_t>((blocks + 31) / 32, 1024 / pad);
            const int32_t parts = grads ? int32_t(std::max<int64_t>(most, 1)) : 1;
            JoinArgs j{part, l.nblk, blocks, count, first, rows + first, coef + first, l.entry,
                       l.pick, teach ? teach + first * s.top_pad : nullptr, s.top, s.top_pad,
                       c.temperature, log2e_t, 1.0 / c.temperature, c.loss, c.lse, p, gp, s.vp,
                       g_plane, parts};
            const uint32_t grid = uint32_t(grads ? pad * parts : len);
            // One wave a token, where its row is short: no barrier, and four
            // times the tokens on a CU (16384 tokens x 512 x 256 with gradients
            // 110 -> 80 us; x 4096 252 -> 241, x 8192 of 4096 tokens 156 ->
            // 158; without gradients 16384 x 4096 105 -> 81, 8192 x 32000 241
            // -> 224, 5 x 32000 x 4096 50.3 -> 51.8).
            if (s.top <= 64 && blocks <= (grads || len < 1024 ? 64 : 512))
                join_kernel<F32, 64><<<grid, 64, 0, stream>>>(j);
            else
                join_kernel<F32, 256><<<grid, 256, 0, stream>>>(j);
            if ((e = hipGetLastError()) != hipSuccess) return e;
        }

        if (s.grad_hidden && len > 0) {
            GemmArgs h = hidden_product(s, len);
            h.keep = keep;
            h.a = w;
            h.b = gp;
            h.count = count;
            h.first = first;
            h.out = c.grad_hidden;
            h.factor = factor;
            h.rows = rows + first;
            h.split = split;
            const HeadTiles& t = s.hidden_tiles[last];
            if ((e = pick_gemm<true, false, F32, kOut>(h, t, stream)) != hipSuccess) return e;
        }
        if (few_tokens) {
            const OuterArgs o{xt, gp, static_cast<uint16_t*>(c.grad_head), count, s.v, s.d, s.dp,
                              s.vp, factor, 0, 0};
            if ((e = run_outer(o, s.n, stream)) != hipSuccess) return e;
        } else if (s.grad_head) {
            GemmArgs h = head_product(s, len);
            h.a = x + first * s.dp;
            h.b = gp;
            h.k_real = s.rows - first;
            h.count = count;
            h.first = first;
            h.out = c.grad_head;
            h.factor = factor;
            h.split = split;
            h.acc_in = ch > 0 ? acc : nullptr;
            h.acc_out = ch + 1 < s.nchunk ? acc : nullptr;
            const HeadTiles& t = s.head_tiles[last];
            if ((e = pick_gemm<true, true, F32, kOut>(h, t, stream)) != hipSuccess) return e;
        }
    }
    return hipSuccess;
}

}  // namespace

// A launch holds below 2^32 threads. The others' are bounded by n, or by what
// is kept at a time.
bool head_fits_launch(const HeadShape& s) {
    return setup_grid(s).all() * kSetupThreads < int64_t(1) << 32;
}

// The logits' sums are worth splitting where a row of them fits LDS beside others
// and the whole product leaves most of the card idle. (With rows of up to 32768
// logits taken this way, 96 tokens x 32000 x 4096 with the head's gradient take
// 231 us in place of 195.) The gradients' products: of a chunk and of the last.
void head_products(HeadShape* s) {
    auto tiles = [&](const GemmArgs& g, bool low) { return bounded(g, tile_of(g, s->f32, low)); };
    int64_t bytes = 0;
    auto add = [&](const GemmArgs& g, const HeadTiles& t, int64_t rows) {
        bytes = std::max(bytes, std::max(int64_t(t.split_rows), rows) * g.ldf * 4);
    };
    s->raw = false;
    if (s->n > 0 && s->v <= kHeadRawColumns && s->nchunk == 1) {
        const GemmArgs g = raw_product(*s, s->n);
        const HeadTiles t = tile_of(g, s->f32, true);
        s->raw = split_of(tiles_along(g.na, t.ba) * tiles_along(g.nb, t.bb), stages_of(g.k), t.segs,
                          t.slot_bits) > 1;
        if (s->raw) add(g, s->raw_tiles = bounded(g, t), s->n);
    }
    for (int last = 0; last < 2; ++last) {
        const int64_t len = last ? s->n - (s->nchunk - 1) * s->chunk : s->chunk;
        if (!last && s->nchunk == 1) continue;
        if (s->grad_hidden && len > 0) {
            const GemmArgs g = hidden_product(*s, len);
            add(g, s->hidden_tiles[last] = tiles(g, true), 0);
        }
        if (s->grad_head) {
            const GemmArgs g = head_product(*s, len);
            add(g, s->head_tiles[last] = tiles(g, false), 0);
        }
    }
    s->split_bytes = bytes;
}

// By asking every number of tokens which form it takes (64 of them at a time,
// and the in-place forms 16 and 32: what the choice goes by does not change
// between), then each form for the most that it serves. Past kAsked tokens, all
// forms that those may take.
int64_t head_split_most(const HeadShape& s) {
    constexpr int64_t kAsked = 65536;
    const int64_t most = std::min(s.n, s.chunk_most);
    int64_t bytes = 0;
    auto product = [&](auto make, bool low, bool raw) {
        struct Seen {
            HeadTiles t;
            int64_t len;
            bool thin;
        } seen[12];
        int count = 0;
        auto note = [&](const HeadTiles& t, int64_t len, bool in_place) {
            int i = 0;
            while (i < count && (seen[i].t.form != t.form || seen[i].t.bb != t.bb)) ++i;
            if (i == count) seen[count++] = {t, len, in_place};
            else seen[i].len = std::max(seen[i].len, len);
        };
        HeadShape q = s;
        auto ask = [&](int64_t len, bool in_place) {
            q.thin = in_place;
            const GemmArgs g = make(q, len);
            const HeadTiles t = tile_of(g, s.f32, low);
            const uint32_t tiles = tiles_along(g.na, t.ba) * tiles_along(g.nb, t.bb);
            if (raw && split_of(tiles, stages_of(g.k), t.segs, t.slot_bits) == 1) return;
            note(t, len, in_place);
        };
        // (a head that may start anywhere may still be read in place)
        for (int64_t len : {16, 32, 64})
            if (s.f32 && s.d % 4 == 0) ask(std::min<int64_t>(len, most), true);
        if (!s.in_place || s.n > most) ask(std::min<int64_t>(64, most), false);  // or of a last chunk
        for (int64_t len = 128; len < std::min(most, kAsked); len += 64) ask(len, false);
        if (most > 64) ask(std::min(most, kAsked), false);
        if (most > kAsked)
            for (HeadTiles t : {kBig, kMid, kLow2}) {
                t.segs = s.f32 ? 6 : 1;
                q.thin = false;
                const GemmArgs g = make(q, kAsked);
                const uint32_t tiles = tiles_along(g.na, t.ba) * tiles_along(g.nb, t.bb);
                if (!raw || split_may_pay(tiles, stages_of(g.k), t.segs, t.slot_bits))
                    note(t, most, false);
            }
        for (int i = 0; i < count; ++i) {
            q.thin = seen[i].thin;
            const GemmArgs g = make(q, seen[i].len);
            const int64_t rows = int64_t(bounded(g, seen[i].t).split_rows);
            bytes = std::max(bytes, std::max(rows, raw ? seen[i].len : 0) * g.ldf * 4);
        }
    };
    if (most > 0 && s.v <= kHeadRawColumns) product(raw_product, true, true);
    if (most > 0 && s.grad_hidden) product(hidden_product, true, false);
    if (most > 0 && s.grad_head) product(head_product, false, false);
    return bytes;
}

hipError_t launch_head(const HeadShape& s, const HeadCall& c, hipStream_t stream) {
    return s.f32 ? run_head<true>(s, c, stream) : run_head<false>(s, c, stream);
}

}  // namespace zsp
