// zsp_head.hip -- the losses over a model's output matrix (the head) and
// their gradients, for gfx950.
//
//   l_iv = (x_i . w_v) / T          lse_i = log sum_v exp l_iv
//   p_iv = exp(l_iv - lse_i)        q_i: the target, or the teacher's softmax
//   G_iv = c_i (p_iv - q_iv)        dX = G W        dW = G^T X
//
// The logits are never kept: the first product's tiles leave, per token and
// block of 64 columns, the block's largest logit m and the sum of
// exp(l - m), and for a call with gradients P = exp(l - m) in bf16 for a
// bounded number of tokens; once the blocks are joined to lse, one pass turns
// P into G in place, and the other two products read G. Three products of
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
typedef float f32x4 __attribute__((ext_vector_type(4)));
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

// rows[0 .. count): the tokens that count, in order. One workgroup; each
// thread counts a run of tokens, the runs are joined by a scan.
constexpr int kScanThreads = 1024;
__global__ __launch_bounds__(kScanThreads) void scan_kernel(const int64_t* target,
                                                            const float* weight,
                                                            const uint8_t* flag, int64_t n,
                                                            int64_t v, int32_t* rows,
                                                            int32_t* count) {
    __shared__ int32_t s_wave[kScanThreads / 64];
    const int t = threadIdx.x, lane = t % 64, wave = t / 64;
    auto counts = [&](int64_t i) -> bool {
        if (flag) return flag[i] != 0;
        const int64_t e = target[i];
        return e >= 0 && e < v && (!weight || weight[i] != 0.0f);
    };
    int32_t done = 0;
    for (int64_t base = 0; base < n; base += kScanThreads) {
        const int64_t i = base + t;
        const bool on = i < n && counts(i);
        const uint64_t m = __ballot(on);
        if (lane == 0) s_wave[wave] = __popcll(m);
        __syncthreads();
        int32_t before = done, all = 0;
        for (int w = 0; w < kScanThreads / 64; ++w) {
            if (w < wave) before += s_wave[w];
            all += s_wave[w];
        }
        if (on) rows[before + __popcll(m & ((1ull << lane) - 1))] = int32_t(i);
        done += all;
        __syncthreads();
    }
    if (t == 0) *count = done;
}

struct PackArgs {
    const void* hidden;
    const int64_t* index;
    const float* logit;
    const float* weight;
    const uint8_t* flag;
    const int32_t* rows;
    const int32_t* count;
    float* coef;
    int32_t* entry;
    uint16_t* x;
    void* grad_hidden;
    float* loss;
    float* lse;
    int64_t n, v, d, dp, plane;
    int32_t top, top_pad;
    float scale;
};

// One element of a row as its planes.
template <typename T>
__device__ __forceinline__ void put(uint16_t* out, int64_t plane, const T* in, bool real) {
    if constexpr (sizeof(T) == 2) {
        *out = real ? *in : uint16_t(0);
    } else {
        uint16_t h[3] = {0, 0, 0};
        if (real) split3(*in, h);
        out[0] = h[0];
        out[plane] = h[1];
        out[2 * plane] = h[2];
    }
}

// Row r of the copied X, its coefficient and entries; the outputs of token r
// where it does not count.
template <typename T>
__global__ __launch_bounds__(256) void pack_kernel(PackArgs a) {
    const int64_t r = blockIdx.x;
    const int t = threadIdx.x;
    const int32_t count = *a.count;
    if (r < count) {
        const int64_t i = a.rows[r];
        const T* in = static_cast<const T*>(a.hidden) + i * a.d;
        uint16_t* out = a.x + r * a.dp;
        for (int64_t c = t; c < a.dp; c += 256) put(out + c, a.plane, in + c, c < a.d);
        for (int32_t k = t; k < a.top_pad; k += 256) {
            int64_t e = k < a.top ? a.index[i * a.top + k] : -1;
            if (a.logit && k < a.top && a.logit[i * a.top + k] == -__builtin_inff()) e = -1;
            a.entry[r * a.top_pad + k] = e >= 0 && e < a.v ? int32_t(e) : -1;
        }
        if (t == 0) a.coef[r] = a.weight ? a.scale * a.weight[i] : a.scale;
    } else if (r < (int64_t(count) + kHeadTile - 1) / kHeadTile * kHeadTile) {
        for (int64_t c = t; c < a.dp; c += 256)
            put<T>(a.x + r * a.dp + c, a.plane, nullptr, false);
    }
    if (r < a.n) {
        bool on;
        if (a.flag) on = a.flag[r] != 0;
        else {
            const int64_t e = a.index[r];
            on = e >= 0 && e < a.v && (!a.weight || a.weight[r] != 0.0f);
        }
        if (on) return;
        if (a.grad_hidden) {
            T* out = static_cast<T*>(a.grad_hidden) + r * a.d;
            for (int64_t c = t; c < a.d; c += 256) out[c] = T(0);
        }
        if (t == 0) {
            a.loss[r] = 0.0f;
            if (a.lse) a.lse[r] = 0.0f;
        }
    }
}

// The head's rows in planes of dp columns.
template <typename T>
__global__ __launch_bounds__(256) void pack_head_kernel(const T* head, uint16_t* out, int64_t d,
                                                        int64_t dp, int64_t plane) {
    const int64_t r = blockIdx.x;
    for (int64_t c = threadIdx.x; c < dp; c += 256)
        put(out + r * dp + c, plane, head + r * d + c, c < d);
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
    int64_t na;                // extent of a: further rows or columns are read as the last ones
    int64_t nb;                // extent of b; a product over tokens: bounded by *count - first
    int64_t k;                 // the sum's length, and for M-major A with na_k its real rows
    int64_t k_real;            // rows of an M-major A that exist (later ones read as the last)
    const int32_t* count;      // tokens that count
    int64_t first;             // the chunk's first token
    int32_t tokens_in_b, tokens_in_k;
    uint32_t nsplit;
    // logits
    float inv_temp;
    float2* part;              // [b][na_blocks]
    int64_t nblk;
    void* p;                   // [b][ldp] bf16 or fp32, or NULL
    int64_t ldp;
    const int32_t* entry;      // [b][top_pad]
    float* pick;
    int32_t top_pad;
    // outputs
    void* out;                 // final: [row][ldo] of the output's type, or NULL
    int64_t ldo;
    const int32_t* rows;       // row of b, or NULL: b itself
    int32_t aligned;           // rows of out start on 16 bytes
    const float* acc_in;       // fp32 [b][ldf] to add, or NULL
    float* acc_out;            // fp32 [split][b][ldf], instead of out
    int64_t ldf, split_stride;
};

enum { kLogits = 0, kOut = 1 };

// 16 bytes a lane from base + off to lds + 16 * lane. In assembly: the
// compiler would wait for every such load before each transposing LDS read.
// Nothing else here uses m0. The caller waits (wait_stage).
__device__ __forceinline__ void load_to_lds(const char* base, uint32_t off, ZSP_LDS char* lds) {
    const uint32_t at = __builtin_amdgcn_readfirstlane(uint32_t(uintptr_t(lds)));
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2" ::"s"(at), "v"(off),
                 "s"(base)
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

// x[a] of the four 16-lane rows g -> x[g] of row a: what row g holds of four
// tiles becomes what tile g holds in four rows.
__device__ __forceinline__ void transpose4(uint32_t x[4]) {
    auto s = __builtin_amdgcn_permlane16_swap(x[0], x[1], false, false);
    x[0] = s[0]; x[1] = s[1];
    s = __builtin_amdgcn_permlane16_swap(x[2], x[3], false, false);
    x[2] = s[0]; x[3] = s[1];
    s = __builtin_amdgcn_permlane32_swap(x[0], x[2], false, false);
    x[0] = s[0]; x[2] = s[1];
    s = __builtin_amdgcn_permlane32_swap(x[1], x[3], false, false);
    x[1] = s[0]; x[3] = s[1];
}

// One operand's share of a stage in LDS: X rows (or columns) of BK k's, in
// 16-byte groups. The wave's loads write LDS in lane order, so the order of
// the groups in a row is changed on the reading side of the load: group c of
// a row is kept at c ^ s(row), which spreads the lanes of one LDS read over
// the banks.
template <int X, int BK, int WAVES, bool MMAJ, bool CLAMP>
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
    int32_t krow[kLoads];     // M-major

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
                off[i] = uint32_t(x * ld + c * 16);
                krow[i] = 0;
            }
        }
    }
    // Load i of the stage whose first k is k0 into `lds`. CLAMP: rows past
    // k_last are read as that one.
    __device__ __forceinline__ void issue(int i, ZSP_LDS char* lds, int64_t plane, int64_t k0,
                                          int64_t k_last, int wave) {
        const char* src = base + 2 * plane + (MMAJ ? k0 * ld : k0 * 2);
        uint32_t o = off[i];
        if constexpr (CLAMP) {
            const int32_t k = k_last - k0 < BK ? int32_t(k_last - k0) : BK;
            o += uint32_t(krow[i] < k ? krow[i] : k) * uint32_t(ld);
        }
        load_to_lds(src, o, lds + (wave * kLoads + i) * 1024);
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

// The products of fp32 planes, the largest first.
__device__ __forceinline__ int plane_a_of(int seg) { return (0x201010 >> (4 * seg)) & 0xf; }
__device__ __forceinline__ int plane_b_of(int seg) { return (0x021100 >> (4 * seg)) & 0xf; }

template <int BA, int BB, int WA, int WB, bool AM, bool BM, bool F32, int KIND>
__global__ __launch_bounds__(64 * WA * WB) void gemm_kernel(GemmArgs g) {
    constexpr int kWaves = WA * WB, BK = kHeadDepth;
    constexpr int EA = BA / WA, EB = BB / WB, TA = EA / 16, TB = EB / 16;
    static_assert(EA == kHeadBlock && TA == 4, "a wave's columns are one block");
    using OpA = Operand<BA, BK, kWaves, AM, AM && !BM>;  // the head's rows end at v
    using OpB = Operand<BB, BK, kWaves, BM, false>;
    constexpr int kStage = OpA::kBytes + OpB::kBytes;
    constexpr int kPer = OpA::kLoads + OpB::kLoads;
    constexpr int kSegs = F32 ? 6 : 1;
    __shared__ __attribute__((aligned(1024))) char s_mem[2 * kStage];

    const int lane = threadIdx.x % 64;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);

    // Extents that the device alone knows, then this workgroup's tile: each
    // XCD (workgroups go to the 8 of them in turn) takes one run of the
    // tiles, four b's at a time along all a's, so that what its L2 holds of
    // both operands is used by its neighbours.
    int64_t nb = g.nb, klen = g.k;
    if (g.tokens_in_b || g.tokens_in_k) {
        int64_t c = int64_t(*g.count) - g.first;
        c = c < 0 ? 0 : c;
        if (g.tokens_in_b) nb = c < nb ? c : nb;
        else klen = c < klen ? c : klen;
    }
    const uint32_t ta_n = uint32_t((g.na + BA - 1) / BA), tb_n = uint32_t((nb + BB - 1) / BB);
    const uint32_t tiles = ta_n * tb_n, per = (tiles + 7) / 8;
    const uint32_t j = blockIdx.x >> 3, lin = (blockIdx.x & 7) * per + j;
    if (j >= per || lin >= tiles) return;
    constexpr uint32_t GB = 4;
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

    const uint32_t kt_all = uint32_t((klen + BK - 1) / BK);  // at most 2^18, 64 splits
    const uint32_t kt0 = kt_all * blockIdx.y / g.nsplit, kt1 = kt_all * (blockIdx.y + 1) / g.nsplit;
    const int nkt = int(kt1 - kt0), steps = nkt * kSegs;

    OpA oa;
    OpB ob;
    oa.init(g.a, g.lda, a0, g.na, wave, lane);
    ob.init(g.b, g.ldb, b0, BM ? g.ldb : (b0 + BB), wave, lane);

    int i_kt = 0, i_seg = 0, i_left = steps;  // the next stage to load
    auto issue = [&](int buf, int from, int to) {
        ZSP_LDS char* lds = (ZSP_LDS char*)s_mem + buf * kStage;
        const int64_t k0 = int64_t(kt0 + i_kt) * BK;
#pragma unroll
        for (int i = from; i < to; ++i) {
            if (i < OpA::kLoads)
                oa.issue(i, lds, F32 ? plane_a_of(i_seg) * g.plane_a : 0, k0, g.k_real - 1, wave);
            else
                ob.issue(i - OpA::kLoads, lds + OpA::kBytes,
                         F32 ? plane_b_of(i_seg) * g.plane_b : 0, k0, 0, wave);
        }
        // past the last stage it is loaded again: nothing reads it
        if (to == kPer && --i_left > 0 && ++i_kt == nkt) {
            i_kt = 0;
            ++i_seg;
        }
    };
    // Stage s is read from buffer s % 2. Its first half of the k's is read into
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
    // other half (of buffer `from`) and, where `load`, the loads of the stage
    // after next between them, a quarter of each at a time.
    constexpr int kParts = 4, kMul = TA * TB / kParts;
    auto work = [&](auto half_c, int from, auto load_c) {
        constexpr int half = decltype(half_c)::value;
#pragma unroll
        for (int q = 0; q < kParts; ++q) {
#pragma unroll
            for (int i = (TA + TB) * q / kParts; i < (TA + TB) * (q + 1) / kParts; ++i)
                read(half ^ 1, from, i);
            if constexpr (decltype(load_c)::value)
                issue(from ^ 1, kPer * q / kParts, kPer * (q + 1) / kParts);
#pragma unroll
            for (int i = kMul * q; i < kMul * (q + 1); ++i)
                acc[i % TA][i / TA] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                    fa[half][i % TA], fb[half][i / TA], acc[i % TA][i / TA], 0, 0, 0);
            __builtin_amdgcn_sched_barrier(0);
        }
    };
    using std::integral_constant;
    if (steps > 0) {
        issue(0, 0, kPer);
        issue(1, 0, kPer);
        wait_stage<kPer>();
        wg_barrier();
#pragma unroll
        for (int i = 0; i < TA + TB; ++i) read(0, 0, i);
    }
    for (int it = 0; it < steps; ++it) {
        __builtin_amdgcn_sched_barrier(0);
        work(integral_constant<int, 0>(), buf, integral_constant<bool, false>());
        // this wave has read all of this stage, and its part of the next has
        // landed; then that holds for every wave
        wait_stage<0>();
        wg_barrier();
        buf ^= 1;
        // behind the last stage: loaded and read, not used
        work(integral_constant<int, 1>(), buf, integral_constant<bool, true>());
    }
    wait_stage<0>();  // no load into LDS outlives the workgroup

    // A lane holds, of each 16 x 16 tile, column lane % 16 (a row of the
    // output) at rows 4 (lane / 16) + 0..3 (its columns).
    const int lr = lane % 16, lg = lane / 16;
    const int64_t a_wave = a0 + wa * EA;
    if constexpr (KIND == kLogits) {
#pragma unroll
        for (int b = 0; b < TB; ++b) {
            const int64_t row = b0 + wb * EB + b * 16 + lr;
            float m = -__builtin_inff();
#pragma unroll
            for (int a = 0; a < TA; ++a)
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    float l = acc[a][b][k] * g.inv_temp;
                    if (a_wave + a * 16 + lg * 4 + k >= g.na) l = -__builtin_inff();
                    acc[a][b][k] = l;
                    m = fmaxf(m, l);
                }
            m = fmaxf(m, __shfl_xor(m, 16));
            m = fmaxf(m, __shfl_xor(m, 32));
            const bool real = row < nb;
            if (real) {
                const int32_t* e = g.entry + row * g.top_pad;
                for (int32_t k = 0; k < g.top_pad; ++k) {
                    const int64_t rel = e[k] - a_wave;
                    if (e[k] < 0 || uint64_t(rel) >= uint64_t(EA) || ((rel >> 2) & 3) != lg) continue;
                    float l = 0.0f;
#pragma unroll
                    for (int a = 0; a < TA; ++a)
#pragma unroll
                        for (int c = 0; c < 4; ++c)
                            if ((rel >> 4) == a && (rel & 3) == c) l = acc[a][b][c];
                    g.pick[row * g.top_pad + k] = l;
                }
            }
            // a block without a column of the vocabulary leaves 0
            const float mm = m == -__builtin_inff() ? 0.0f : m;
            float s = 0.0f;
#pragma unroll
            for (int a = 0; a < TA; ++a)
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    acc[a][b][k] = fast_exp(acc[a][b][k] - mm);
                    s += acc[a][b][k];
                }
            s += __shfl_xor(s, 16);
            s += __shfl_xor(s, 32);
            if (lg == 0 && real) g.part[row * g.nblk + a_wave / kHeadBlock] = make_float2(m, s);
            if (g.p) {
                if constexpr (F32) {
                    float* out = static_cast<float*>(g.p) + row * g.ldp + a_wave + lg * 16;
                    f32x4 v[TA];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        uint32_t x[4];
#pragma unroll
                        for (int a = 0; a < 4; ++a) x[a] = __float_as_uint(acc[a][b][k]);
                        transpose4(x);
#pragma unroll
                        for (int a = 0; a < 4; ++a) v[a][k] = __uint_as_float(x[a]);
                    }
#pragma unroll
                    for (int a = 0; a < 4; ++a) *reinterpret_cast<f32x4*>(out + a * 4) = v[a];
                } else {
                    uint16_t* out = static_cast<uint16_t*>(g.p) + row * g.ldp + a_wave + lg * 16;
                    uint32_t x[4], y[4];
#pragma unroll
                    for (int a = 0; a < 4; ++a) {
                        x[a] = bf16_pair(acc[a][b][0], acc[a][b][1]);
                        y[a] = bf16_pair(acc[a][b][2], acc[a][b][3]);
                    }
                    transpose4(x);
                    transpose4(y);
                    *reinterpret_cast<u32x4*>(out) = u32x4{x[0], y[0], x[1], y[1]};
                    *reinterpret_cast<u32x4*>(out + 8) = u32x4{x[2], y[2], x[3], y[3]};
                }
            }
        }
    } else {
        const int64_t col = a_wave + lg * 16;
#pragma unroll
        for (int b = 0; b < TB; ++b) {
            const int64_t row = b0 + wb * EB + b * 16 + lr;
            f32x4 v[TA];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                uint32_t x[4];
#pragma unroll
                for (int a = 0; a < 4; ++a) x[a] = __float_as_uint(acc[a][b][k]);
                transpose4(x);
#pragma unroll
                for (int a = 0; a < 4; ++a) v[a][k] = __uint_as_float(x[a]);
            }
            if (row >= nb || col >= g.na) continue;
            if (g.acc_in) {
#pragma unroll
                for (int a = 0; a < 4; ++a)
                    v[a] += *reinterpret_cast<const f32x4*>(g.acc_in + row * g.ldf + col + a * 4);
            }
            if (g.acc_out) {
                float* out = g.acc_out + blockIdx.y * g.split_stride + row * g.ldf + col;
#pragma unroll
                for (int a = 0; a < 4; ++a) *reinterpret_cast<f32x4*>(out + a * 4) = v[a];
                continue;
            }
            const int64_t at = (g.rows ? int64_t(g.rows[row]) : row) * g.ldo + col;
            if constexpr (F32) {
                float* out = static_cast<float*>(g.out) + at;
                if (g.aligned && col + 16 <= g.ldo) {
#pragma unroll
                    for (int a = 0; a < 4; ++a) *reinterpret_cast<f32x4*>(out + a * 4) = v[a];
                } else {
#pragma unroll
                    for (int a = 0; a < 16; ++a)
                        if (col + a < g.ldo) out[a] = v[a / 4][a % 4];
                }
            } else {
                uint16_t* out = static_cast<uint16_t*>(g.out) + at;
                if (g.aligned && col + 16 <= g.ldo) {
#pragma unroll
                    for (int h = 0; h < 2; ++h)
                        *reinterpret_cast<u32x4*>(out + h * 8) =
                            u32x4{bf16_pair(v[2 * h][0], v[2 * h][1]),
                                  bf16_pair(v[2 * h][2], v[2 * h][3]),
                                  bf16_pair(v[2 * h + 1][0], v[2 * h + 1][1]),
                                  bf16_pair(v[2 * h + 1][2], v[2 * h + 1][3])};
                } else {
#pragma unroll
                    for (int a = 0; a < 16; ++a)
                        if (col + a < g.ldo) out[a] = bf16_bits(v[a / 4][a % 4]);
                }
            }
        }
    }
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
    const float* logit;       // the teacher's [n, top], or NULL
    int32_t top, top_pad;
    float temp, inv_temp;
    float* loss;
    float* lse;
    void* p;                  // [chunk][ldp], or NULL: no gradients
    uint16_t* g;              // fp32: the planes of G; else P itself
    int64_t ldp, plane;
};

__device__ __forceinline__ double block_sum(double v, double* s) {
    for (int o = 32; o; o >>= 1) v += __shfl_xor(v, o);
    __syncthreads();
    if (threadIdx.x % 64 == 0) s[threadIdx.x / 64] = v;
    __syncthreads();
    return s[0] + s[1] + s[2] + s[3];
}
// NaN wins, as in a sum
__device__ __forceinline__ float nan_max(float a, float b) { return a != a || a > b ? a : b; }
__device__ __forceinline__ float block_max(float v, float* s) {
    for (int o = 32; o; o >>= 1) v = nan_max(v, __shfl_xor(v, o));
    __syncthreads();
    if (threadIdx.x % 64 == 0) s[threadIdx.x / 64] = v;
    __syncthreads();
    return nan_max(nan_max(s[0], s[1]), nan_max(s[2], s[3]));
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

// One workgroup per token that counts: lse, the loss, then the token's row of
// G. An entry's own G is taken from its logit in 64 bits: c (p - q) from P's
// bf16 would lose all of 1 - p where the model is sure of its target.
template <bool F32>
__global__ __launch_bounds__(256) void join_kernel(JoinArgs a) {
    __shared__ double s_d[4];
    __shared__ float s_f[4];
    __shared__ float s_q[kHeadMaxTop];
    __shared__ int32_t s_e[kHeadMaxTop];
    const int64_t r = blockIdx.x, count = *a.count - a.first;
    const int64_t cols = int64_t(a.blocks) * kHeadBlock;
    const int t = threadIdx.x;
    if (r >= count) {
        // zeros behind the last token, as far as a stage of the sum over
        // tokens may read
        if (a.p && r < (count + kHeadDepth - 1) / kHeadDepth * kHeadDepth)
            for (int64_t c = t * 8; c < cols; c += 2048)
                for (int k = 0; k < (F32 ? 3 : 1); ++k)
                    *reinterpret_cast<u32x4*>(a.g + k * a.plane + r * a.ldp + c) = u32x4{0, 0, 0, 0};
        return;
    }
    const float2* part = a.part + r * a.nblk;
    float m = -__builtin_inff();
    for (int64_t b = t; b < a.blocks; b += 256) m = nan_max(m, part[b].x);
    m = block_max(m, s_f);
    double s = 0.0;
    for (int64_t b = t; b < a.blocks; b += 256) {
        const float2 q = part[b];
        s += double(q.y) * double(q.x == m ? 1.0f : fast_exp(q.x - m));
    }
    s = block_sum(s, s_d);
    const double lse = double(m) + log(s);

    // the entries' share of the target distribution, and the loss
    const int64_t token = a.rows[r];
    const int32_t* entry = a.entry + r * a.top_pad;
    const float* pick = a.pick + r * a.top_pad;
    double loss = 0.0;
    if (a.logit) {
        const float* teach = a.logit + token * a.top;
        float tm = -__builtin_inff();
        for (int32_t k = t; k < a.top; k += 256)
            if (entry[k] >= 0) tm = nan_max(tm, teach[k]);
        tm = block_max(tm, s_f);
        double ts = 0.0;
        for (int32_t k = t; k < a.top; k += 256)
            if (entry[k] >= 0) ts += exp((double(teach[k]) - double(tm)) / double(a.temp));
        ts = block_sum(ts, s_d);
        const double lq = log(ts);  // from the largest: logits may all be far below 0
        for (int32_t k = t; k < a.top; k += 256) {
            double q = 0.0;
            if (entry[k] >= 0) {
                const double l = (double(teach[k]) - double(tm)) / double(a.temp) - lq;
                q = exp(l);
                if (q != 0.0) loss += q * (l - (double(pick[k]) - lse));
            }
            s_q[k] = float(q);
            s_e[k] = entry[k];
        }
        loss = block_sum(loss, s_d) * double(a.temp) * double(a.temp);
    } else {
        loss = lse - double(pick[0]);
        if (t == 0) {
            s_q[0] = 1.0f;
            s_e[0] = entry[0];
        }
        __syncthreads();
    }
    if (t == 0) {
        a.loss[token] = float(loss);
        if (a.lse) a.lse[token] = float(lse);
    }
    if (!a.p) return;

    const float c = a.coef[r] * a.temp;
    const float l32 = float(lse);
    if constexpr (F32) {
        const float* p = static_cast<const float*>(a.p) + r * a.ldp;
        for (int64_t i = t * 4; i < cols; i += 1024) {
            const float f = c * fast_exp(part[i / kHeadBlock].x - l32);
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
        for (int64_t i = t * 8; i < cols; i += 2048) {
            const float f = c * fast_exp(part[i / kHeadBlock].x - l32);
            u32x4 v = *reinterpret_cast<const u32x4*>(p + i);
#pragma unroll
            for (int k = 0; k < 4; ++k)
                v[k] = bf16_pair(f * __uint_as_float(v[k] << 16),
                                 f * __uint_as_float(v[k] & 0xffff0000u));
            *reinterpret_cast<u32x4*>(p + i) = v;
        }
    }
    __threadfence_block();
    __syncthreads();
    // equal entries of a row write the same sum of their q
    for (int32_t k = t; k < a.top; k += 256) {
        const int32_t e = s_e[k];
        if (e < 0) continue;
        double q = 0.0;
        for (int32_t o = 0; o < a.top; ++o)
            if (s_e[o] == e) q += double(s_q[o]);
        const double x = double(pick[k]) - lse;
        // p - q = (p - 1) + (1 - q)
        put_g<F32>(a, r, e, float(double(c) * (expm1(x) + (1.0 - q))));
    }
}

// A gradient's split sums joined, in order.
struct SplitArgs {
    const float* part;
    uint32_t nsplit;
    int64_t split_stride, ldf;
    const float* acc_in;
    float* acc_out;
    void* out;
    int64_t ldo;
    const int32_t* rows;
    const int32_t* count;
    int64_t first, nrow;
    int32_t tokens;
};

template <bool F32>
__global__ __launch_bounds__(256) void split_kernel(SplitArgs a) {
    const int64_t row = blockIdx.x;
    if (a.tokens && row >= *a.count - a.first) return;
    const int64_t o = (a.rows ? int64_t(a.rows[row]) : row) * a.ldo;
    for (int64_t c = threadIdx.x; c < a.ldo; c += 256) {
        float v = a.acc_in ? a.acc_in[row * a.ldf + c] : 0.0f;
        for (uint32_t s = 0; s < a.nsplit; ++s) v += a.part[s * a.split_stride + row * a.ldf + c];
        if (a.acc_out) a.acc_out[row * a.ldf + c] = v;
        else if constexpr (F32) static_cast<float*>(a.out)[o + c] = v;
        else static_cast<uint16_t*>(a.out)[o + c] = bf16_bits(v);
    }
}

// ---- launches ------------------------------------------------------------------------

template <int BA, int BB, int WA, int WB, bool AM, bool BM, bool F32, int KIND>
hipError_t run_gemm(const GemmArgs& g, hipStream_t stream) {
    const int64_t tiles = (g.na + BA - 1) / BA * ((g.nb + BB - 1) / BB);
    if (tiles == 0) return hipSuccess;
    gemm_kernel<BA, BB, WA, WB, AM, BM, F32, KIND>
        <<<dim3(uint32_t((tiles + 7) / 8 * 8), uint32_t(g.nsplit)), 64 * WA * WB, 0, stream>>>(g);
    return hipGetLastError();
}

// Tiles of 256 x 256 (eight waves, one workgroup on a CU) reach 1.3 PFLOP/s
// on a full card, tiles of 128 x 128 (four waves, two workgroups on a CU)
// 1.05: the smaller are taken where the larger leave more of the card idle.
template <bool AM, bool BM, bool F32, int KIND>
hipError_t pick_gemm(const GemmArgs& g, hipStream_t stream) {
    auto turns = [&](int64_t tile, int64_t at_once) {
        const int64_t t = (g.na + tile - 1) / tile * ((g.nb + tile - 1) / tile) * g.nsplit;
        return (t + at_once - 1) / at_once;
    };
    // a turn is 65536 outputs on a CU at 130, or 32768 at 105
    if (turns(256, 256) * 2 * 105 <= turns(128, 512) * 130)
        return run_gemm<256, 256, 4, 2, AM, BM, F32, KIND>(g, stream);
    return run_gemm<128, 128, 2, 2, AM, BM, F32, KIND>(g, stream);
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
    uint8_t* flag = s.teacher ? reinterpret_cast<uint8_t*>(ws + s.o_flag) : nullptr;
    uint16_t* x = reinterpret_cast<uint16_t*>(ws + s.o_x);
    float2* part = reinterpret_cast<float2*>(ws + s.o_part);
    const bool grads = s.grad_hidden || s.grad_head;
    hipError_t e;

    if (flag) {
        flag_kernel<<<uint32_t((s.n + 3) / 4), 256, 0, stream>>>(
            c.index, c.logit, s.n, s.v, s.top, c.token_weight, flag);
        if ((e = hipGetLastError()) != hipSuccess) return e;
    }
    scan_kernel<<<1, kScanThreads, 0, stream>>>(c.index, c.token_weight, flag, s.n, s.v, rows,
                                                count);
    if ((e = hipGetLastError()) != hipSuccess) return e;
    const int64_t x_plane = s.rows * s.dp, w_plane = s.v * s.dp;
    if (s.rows > 0) {
        PackArgs p{c.hidden, c.index, c.logit, c.token_weight, flag, rows, count, coef, entry, x,
                   c.grad_hidden, c.loss, c.lse, s.n, s.v, s.d, s.dp, x_plane, s.top, s.top_pad,
                   c.scale};
        pack_kernel<T><<<uint32_t(s.rows), 256, 0, stream>>>(p);
        if ((e = hipGetLastError()) != hipSuccess) return e;
    }
    const uint16_t* w = static_cast<const uint16_t*>(c.head);
    if (s.pack_head) {
        uint16_t* packed = reinterpret_cast<uint16_t*>(ws + s.o_w);
        pack_head_kernel<T><<<uint32_t(s.v), 256, 0, stream>>>(static_cast<const T*>(c.head),
                                                               packed, s.d, s.dp, w_plane);
        if ((e = hipGetLastError()) != hipSuccess) return e;
        w = packed;
    }

    void* p = grads ? ws + s.o_p : nullptr;
    uint16_t* gp = reinterpret_cast<uint16_t*>(ws + (F32 ? s.o_g : s.o_p));
    const int64_t g_plane = s.chunk * s.vp;
    float* split = reinterpret_cast<float*>(ws + s.o_split);
    float* acc = reinterpret_cast<float*>(ws + s.o_acc);
    auto aligned = [](const void* q, int64_t ld, size_t size) {
        return reinterpret_cast<uintptr_t>(q) % 16 == 0 && ld * int64_t(size) % 16 == 0;
    };

    for (int64_t ch = 0; ch < s.nchunk; ++ch) {
        const int64_t first = ch * s.chunk, len = std::min(s.chunk, s.n - first);
        GemmArgs l{};
        l.a = w;
        l.b = x + first * s.dp;
        l.lda = l.ldb = s.dp;
        l.plane_a = w_plane;
        l.plane_b = x_plane;
        l.na = s.v;
        l.nb = len;
        l.k = s.dp;
        l.count = count;
        l.first = first;
        l.tokens_in_b = 1;
        l.nsplit = 1;
        l.inv_temp = 1.0f / c.temperature;
        l.part = part;
        l.nblk = s.vp / kHeadBlock;
        l.p = p;
        l.ldp = s.vp;
        l.entry = entry + first * s.top_pad;
        l.pick = pick + first * s.top_pad;
        l.top_pad = s.top_pad;
        if (len > 0 && (e = pick_gemm<false, false, F32, kLogits>(l, stream)) != hipSuccess)
            return e;

        if (len > 0) {
            JoinArgs j{part, l.nblk, int32_t((s.v + kHeadBlock - 1) / kHeadBlock), count, first, rows + first, coef + first, l.entry, l.pick,
                       c.logit, s.top, s.top_pad, c.temperature, l.inv_temp, c.loss, c.lse, p, gp,
                       s.vp, g_plane};
            const int64_t pad = (len + kHeadDepth - 1) / kHeadDepth * kHeadDepth;
            join_kernel<F32><<<uint32_t(grads ? pad : len), 256, 0, stream>>>(j);
            if ((e = hipGetLastError()) != hipSuccess) return e;
        }

        if (s.grad_hidden && len > 0) {
            GemmArgs h{};
            h.a = w;
            h.b = gp;
            h.lda = s.dp;
            h.ldb = s.vp;
            h.plane_a = w_plane;
            h.plane_b = g_plane;
            h.na = s.dp;
            h.nb = len;
            h.k = s.v;
            h.k_real = s.v;
            h.count = count;
            h.first = first;
            h.tokens_in_b = 1;
            h.nsplit = s.split_hidden;
            h.out = c.grad_hidden;
            h.ldo = s.d;
            h.rows = rows + first;
            h.aligned = aligned(c.grad_hidden, s.d, sizeof(T));
            h.ldf = s.dp;
            h.split_stride = s.chunk * s.dp;
            if (h.nsplit > 1) h.acc_out = split;
            if ((e = pick_gemm<true, false, F32, kOut>(h, stream)) != hipSuccess) return e;
            if (h.nsplit > 1) {
                SplitArgs q{split, h.nsplit, h.split_stride, s.dp, nullptr, nullptr, h.out, s.d,
                            h.rows, count, first, len, 1};
                split_kernel<F32><<<uint32_t(len), 256, 0, stream>>>(q);
                if ((e = hipGetLastError()) != hipSuccess) return e;
            }
        }
        if (s.grad_head) {
            GemmArgs h{};
            h.a = x + first * s.dp;
            h.b = gp;
            h.lda = s.dp;
            h.ldb = s.vp;
            h.plane_a = x_plane;
            h.plane_b = g_plane;
            h.na = s.dp;
            h.nb = s.v;
            h.k = len;
            h.k_real = s.rows - first;
            h.count = count;
            h.first = first;
            h.tokens_in_k = 1;
            h.nsplit = s.split_head;
            h.out = c.grad_head;
            h.ldo = s.d;
            h.aligned = aligned(c.grad_head, s.d, sizeof(T));
            h.ldf = s.dp;
            h.split_stride = s.v * s.dp;
            const float* acc_in = ch > 0 ? acc : nullptr;
            float* acc_out = ch + 1 < s.nchunk ? acc : nullptr;
            if (h.nsplit > 1) {
                h.acc_out = split;
            } else {
                h.acc_in = acc_in;
                h.acc_out = acc_out;
            }
            if ((e = pick_gemm<true, true, F32, kOut>(h, stream)) != hipSuccess) return e;
            if (h.nsplit > 1) {
                SplitArgs q{split, h.nsplit, h.split_stride, s.dp, acc_in, acc_out, h.out, s.d,
                            nullptr, count, first, s.v, 0};
                split_kernel<F32><<<uint32_t(s.v), 256, 0, stream>>>(q);
                if ((e = hipGetLastError()) != hipSuccess) return e;
            }
        }
    }
    return hipSuccess;
}

}  // namespace

hipError_t launch_head(const HeadShape& s, const HeadCall& c, hipStream_t stream) {
    return s.f32 ? run_head<true>(s, c, stream) : run_head<false>(s, c, stream);
}

}  // namespace zsp
