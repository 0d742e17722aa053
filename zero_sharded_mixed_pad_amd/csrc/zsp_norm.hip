// zsp_norm.hip -- the global gradient norm and the clipping of lists of
// tensors, for gfx950. (The norms that ride on a reduce, and the clipped
// updates, are ops of the shard kernels in zsp_kernels.hip.)
//
//   L2:  total = sum of g*g over every element, norm = sqrt(total)
//   MAX: total = largest |g|, norm = total
//   coef = 1 if norm <= max_norm, else max_norm / norm
//
// Every kernel here reads its data once: bound by memory. The squares are
// summed in 64 bits (no square of a finite fp32 value overflows or
// underflows there); a 64-bit multiply-add and a conversion per element
// stay under the time of the element's bytes. A largest absolute value is
// kept as a bit pattern: the integer order of non-negative floats, with
// every NaN above infinity, so a NaN anywhere comes out as NaN. Partials go
// to the caller's workspace and are joined in an order fixed by the sizes
// alone, without atomics: equal inputs give equal bits.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "zsp_internal.hpp"

namespace zsp {
namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4_a2 __attribute__((ext_vector_type(4), aligned(2)));
typedef uint32_t u32x4_a4 __attribute__((ext_vector_type(4), aligned(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

constexpr int kThreads = 256;  // a norm or clip workgroup: four waves
constexpr int kWaves = kThreads / kWaveLanes;

__device__ __forceinline__ float lo16(uint32_t u) { return __uint_as_float(u << 16); }
__device__ __forceinline__ float hi16(uint32_t u) { return __uint_as_float(u & 0xffff0000u); }

template <int KIND>
struct Acc {
    double s = 0.0;
    uint32_t m = 0u;
    __device__ __forceinline__ void add(float g) {
        if constexpr (KIND == ZSP_NORM_MAX) m = max(m, __float_as_uint(g) & 0x7fffffffu);
        else s = __builtin_fma(double(g), double(g), s);
    }
    __device__ __forceinline__ double value() const {
        if constexpr (KIND == ZSP_NORM_MAX) return double(__uint_as_float(m));
        else return s;
    }
};

// Joins two partials (non-negative, or NaN with a clear sign).
template <int KIND>
__device__ __forceinline__ double join(double a, double b) {
    if constexpr (KIND == ZSP_NORM_MAX) {
        const uint64_t x = __double_as_longlong(a), y = __double_as_longlong(b);
        return __longlong_as_double(x > y ? x : y);
    } else {
        return a + b;
    }
}

// The workgroup's partial, valid in thread 0.
template <int KIND, int THREADS>
__device__ __forceinline__ double block_join(double v) {
    __shared__ double s_part[THREADS / kWaveLanes];
#pragma unroll
    for (int d = kWaveLanes / 2; d > 0; d /= 2) v = join<KIND>(v, __shfl_xor(v, d));
    const int wave = threadIdx.x / kWaveLanes;
    if (threadIdx.x % kWaveLanes == 0) s_part[wave] = v;
    __syncthreads();
    if (threadIdx.x == 0)
        for (int w = 1; w < THREADS / kWaveLanes; ++w) v = join<KIND>(v, s_part[w]);
    return v;
}

// ---- The accumulator's norm ----------------------------------------------------

struct AccNormArgs {
    const int64_t* e0;
    const PieceInfo* info;
    const int32_t* tile;
    const float* acc;
    int64_t e_begin, e_len, stride;
    double* part;
};

// One quad (4-aligned E) of a tile at a piece, pad or range boundary.
template <int KIND, bool PADS>
__device__ __forceinline__ void acc_quad(const AccNormArgs& a, int64_t E, int64_t b, int64_t e,
                                         int lo, int hi, Acc<KIND>& t) {
    if (E >= e || E + 4 <= b) return;
    PieceInfo pi{};
    int p = lo;
    if constexpr (PADS) {
        const int64_t first = E > b ? E : b;
        int h = hi;
        while (p < h) {
            const int mid = (p + h + 1) >> 1;
            if (a.e0[mid] <= first) p = mid;
            else h = mid - 1;
        }
        pi = a.info[p];
    }
    for (int k = 0; k < 4; ++k) {
        const int64_t i = E + k;
        if (i < b || i >= e) continue;
        if constexpr (PADS) {
            while (i >= pi.end) pi = a.info[++p];
            if (i >= pi.vend) continue;
        }
        t.add(a.acc[i]);
    }
}

// Workgroup x of rank y takes every gridDim.x-th group of four tiles of the
// rank's span, one tile per wave.
template <int KIND, bool PADS>
__global__ __launch_bounds__(kThreads) void acc_norm_kernel(const AccNormArgs a) {
    const int lane = threadIdx.x % kWaveLanes, wave = threadIdx.x / kWaveLanes;
    const int64_t b = a.e_begin + int64_t(blockIdx.y) * a.stride, e = b + a.e_len;
    Acc<KIND> t;
    for (int64_t tile = b / kTile + int64_t(blockIdx.x) * kWaves + wave; tile * kTile < e;
         tile += int64_t(gridDim.x) * kWaves) {
        const int64_t T0 = tile * kTile;
        int lo = 0, hi = 0;
        bool whole = T0 >= b && T0 + kTile <= e;
        if constexpr (PADS) {
            lo = a.tile[tile];
            hi = a.tile[tile + 1];
            whole = whole && lo == hi && T0 + kTile <= a.info[lo].vend;
        }
        if (whole) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const f32x4 v = *reinterpret_cast<const f32x4*>(a.acc + T0 + h * 256 + lane * 4);
                t.add(v.x);
                t.add(v.y);
                t.add(v.z);
                t.add(v.w);
            }
        } else {
            acc_quad<KIND, PADS>(a, T0 + lane * 4, b, e, lo, hi, t);
            acc_quad<KIND, PADS>(a, T0 + 256 + lane * 4, b, e, lo, hi, t);
        }
    }
    const double v = block_join<KIND, kThreads>(t.value());
    if (threadIdx.x == 0) a.part[int64_t(blockIdx.y) * gridDim.x + blockIdx.x] = v;
}

// ---- Lists of tensors -------------------------------------------------------------

struct TableArgs {
    const ListChunk* chunks;
    int64_t nchunk;
    double* part;
    const zsp_clip* clip;
    int32_t add_to;  // partials already there that a list norm joins
};

struct TensorArgs {
    int64_t nchunk;
    double* part;
    const zsp_clip* clip;
    int32_t n;
    int32_t add_to;
    ArgTensor t[kTensorArgMax];
    int32_t chunk0[kTensorArgMax + 1];
};

// Chunk c of a list in the kernel arguments, read from the argument segment
// (the struct is the kernel's only explicit argument, so it starts at 0).
__device__ __forceinline__ ListChunk arg_chunk(int64_t c, int n) {
    const char* seg = (const char*)__builtin_amdgcn_kernarg_segment_ptr();
    const int32_t* c0 = reinterpret_cast<const int32_t*>(seg + offsetof(TensorArgs, chunk0));
    const ArgTensor* ts = reinterpret_cast<const ArgTensor*>(seg + offsetof(TensorArgs, t));
    int lo = 0, hi = n - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (c0[mid] <= c) lo = mid;
        else hi = mid - 1;
    }
    const ArgTensor t = ts[lo];
    const int64_t at = (c - c0[lo]) * kListChunk, numel = t.numel_type >> 1;
    const int32_t type = int32_t(t.numel_type & 1);
    const int64_t left = numel - at;
    ListChunk r;
    r.p = static_cast<char*>(t.p) + at * (type == ZSP_BF16 ? 2 : 4);
    r.n = int32_t(left < kListChunk ? left : kListChunk);
    r.dtype = type;
    return r;
}

template <int KIND>
__device__ __forceinline__ void chunk_norm(const ListChunk& c, int lane, Acc<KIND>& t) {
    if (c.dtype == ZSP_BF16) {
        const uint16_t* p = static_cast<const uint16_t*>(c.p);
        const int groups = c.n / 8;
        for (int i = lane; i < groups; i += kWaveLanes) {
            const u32x4 v = *reinterpret_cast<const u32x4_a2*>(p + i * 8);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                t.add(lo16(v[k]));
                t.add(hi16(v[k]));
            }
        }
        const int i = groups * 8 + lane;
        if (i < c.n) t.add(__uint_as_float(uint32_t(p[i]) << 16));
    } else {
        const float* p = static_cast<const float*>(c.p);
        const int groups = c.n / 4;
        for (int i = lane; i < groups; i += kWaveLanes) {
            const u32x4 v = *reinterpret_cast<const u32x4_a4*>(p + i * 4);
#pragma unroll
            for (int k = 0; k < 4; ++k) t.add(__uint_as_float(v[k]));
        }
        const int i = groups * 4 + lane;
        if (i < c.n) t.add(p[i]);
    }
}

template <int KIND, bool TABLE, typename Args>
__global__ __launch_bounds__(kThreads) void list_norm_kernel(const Args a) {
    const int lane = threadIdx.x % kWaveLanes;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWaveLanes);
    Acc<KIND> t;
    for (int64_t c = int64_t(blockIdx.x) * kWaves + wave; c < a.nchunk;
         c += int64_t(gridDim.x) * kWaves) {
        if constexpr (TABLE) chunk_norm(a.chunks[c], lane, t);
        else chunk_norm(arg_chunk(c, a.n), lane, t);
    }
    double v = block_join<KIND, kThreads>(t.value());
    if (threadIdx.x == 0) {
        if (int(blockIdx.x) < a.add_to) v = join<KIND>(a.part[blockIdx.x], v);
        a.part[blockIdx.x] = v;
    }
}

__device__ __forceinline__ uint32_t scale2(uint32_t u, float s) {
    bf16x2 r;
    r.x = static_cast<__bf16>(lo16(u) * s);
    r.y = static_cast<__bf16>(hi16(u) * s);
    return __builtin_bit_cast(uint32_t, r);
}

// x * coef in fp32, rounded once more to a bf16 tensor's type.
__device__ __forceinline__ void chunk_scale(const ListChunk& c, int lane, float s) {
    if (c.dtype == ZSP_BF16) {
        uint16_t* p = static_cast<uint16_t*>(c.p);
        const int groups = c.n / 8;
        for (int i = lane; i < groups; i += kWaveLanes) {
            u32x4_a2* q = reinterpret_cast<u32x4_a2*>(p + i * 8);
            const u32x4 v = *q;
            *q = u32x4{scale2(v.x, s), scale2(v.y, s), scale2(v.z, s), scale2(v.w, s)};
        }
        const int i = groups * 8 + lane;
        if (i < c.n)
            p[i] = __builtin_bit_cast(
                uint16_t, static_cast<__bf16>(__uint_as_float(uint32_t(p[i]) << 16) * s));
    } else {
        float* p = static_cast<float*>(c.p);
        const int groups = c.n / 4;
        for (int i = lane; i < groups; i += kWaveLanes) {
            u32x4_a4* q = reinterpret_cast<u32x4_a4*>(p + i * 4);
            const u32x4 v = *q;
            u32x4 o;
#pragma unroll
            for (int k = 0; k < 4; ++k) o[k] = __float_as_uint(__uint_as_float(v[k]) * s);
            *q = o;
        }
        const int i = groups * 4 + lane;
        if (i < c.n) p[i] *= s;
    }
}

template <bool TABLE, typename Args>
__global__ __launch_bounds__(kThreads) void list_clip_kernel(const Args a) {
    const float s = a.clip->coef;
    // 1: nothing to change. NaN: the norm was not finite, nothing is changed.
    if (s == 1.0f || s != s) return;
    const int lane = threadIdx.x % kWaveLanes;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWaveLanes);
    for (int64_t c = int64_t(blockIdx.x) * kWaves + wave; c < a.nchunk;
         c += int64_t(gridDim.x) * kWaves) {
        if constexpr (TABLE) chunk_scale(a.chunks[c], lane, s);
        else chunk_scale(arg_chunk(c, a.n), lane, s);
    }
}

// ---- Joining partials -------------------------------------------------------------

constexpr int kFinishThreads = 1024;
// Partials that one workgroup joins by itself; more are folded to
// kFoldBlocks values first.
constexpr int64_t kFinishMax = 8192;

__device__ __forceinline__ void write_record(double total, int kind, float max_norm,
                                             zsp_clip* out) {
    const double norm = kind == ZSP_NORM_MAX ? total : __builtin_sqrt(total);
    float coef = 1.0f;
    if (!(norm <= 1.7976931348623157e308)) coef = __builtin_nanf("");
    else if (norm > double(max_norm)) coef = float(double(max_norm) / norm);
    out->total = total;
    out->norm = float(norm);
    out->coef = coef;
}

// Workgroup b joins the b-th run of ceil(n / gridDim.x) partials.
template <int KIND>
__global__ __launch_bounds__(kThreads) void fold_kernel(const double* part, int64_t n,
                                                        double* out) {
    const int64_t per = (n + gridDim.x - 1) / gridDim.x;
    const int64_t b = per * blockIdx.x, e = b + per < n ? b + per : n;
    double v = 0.0;
    for (int64_t i = b + threadIdx.x; i < e; i += kThreads) v = join<KIND>(v, part[i]);
    v = block_join<KIND, kThreads>(v);
    if (threadIdx.x == 0) out[blockIdx.x] = v;
}

template <int KIND>
__global__ __launch_bounds__(kFinishThreads) void finish_kernel(const double* part, int64_t n,
                                                                float max_norm, zsp_clip* out) {
    double v = 0.0;
    for (int64_t i = threadIdx.x; i < n; i += kFinishThreads) v = join<KIND>(v, part[i]);
    v = block_join<KIND, kFinishThreads>(v);
    if (threadIdx.x == 0) write_record(v, KIND, max_norm, out);
}

// The records' totals are all read before *out, which may be one of them, is
// written. A total that is no norm's (negative) gives a NaN.
template <int KIND>
__global__ __launch_bounds__(kThreads) void combine_kernel(const zsp_clip* parts, int32_t n,
                                                           float max_norm, zsp_clip* out) {
    double v = 0.0;
    for (int64_t i = threadIdx.x; i < n; i += kThreads) {
        double t = parts[i].total;
        if constexpr (KIND == ZSP_NORM_MAX) t = __builtin_fabs(t);
        v = join<KIND>(v, t);
    }
    v = block_join<KIND, kThreads>(v);
    if (threadIdx.x == 0) write_record(v, KIND, max_norm, out);
}

int list_blocks(int64_t nchunk) {
    return int(std::min<int64_t>((nchunk + kWaves - 1) / kWaves, kNormBlocks));
}

void tensor_args(const TensorsLaunch& L, TensorArgs& a) {
    a.nchunk = L.nchunk;
    a.n = L.n_args;
    for (int i = 0; i < L.n_args; ++i) a.t[i] = L.args[i];
    for (int i = 0; i <= L.n_args; ++i) a.chunk0[i] = L.chunk0[i];
}

template <int KIND>
hipError_t list_norm_t(const TensorsLaunch& L, double* part, int64_t blocks, int32_t add_to,
                       hipStream_t stream) {
    const dim3 grid(static_cast<uint32_t>(blocks)), block(kThreads);
    if (L.n_args > 0) {
        TensorArgs a{};
        tensor_args(L, a);
        a.part = part;
        a.add_to = add_to;
        hipLaunchKernelGGL((list_norm_kernel<KIND, false, TensorArgs>), grid, block, 0, stream, a);
    } else {
        TableArgs a{};
        a.chunks = L.chunks;
        a.nchunk = L.nchunk;
        a.part = part;
        a.add_to = add_to;
        hipLaunchKernelGGL((list_norm_kernel<KIND, true, TableArgs>), grid, block, 0, stream, a);
    }
    return hipGetLastError();
}

template <int KIND>
hipError_t finish_t(double* part, int64_t n, int64_t parts_cap, float max_norm, zsp_clip* out,
                    hipStream_t stream) {
    if (n > kFinishMax) {
        double* fold = part + parts_cap;
        hipLaunchKernelGGL(fold_kernel<KIND>, dim3(kFoldBlocks), dim3(kThreads), 0, stream, part,
                           n, fold);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
        part = fold;
        n = kFoldBlocks;
    }
    hipLaunchKernelGGL(finish_kernel<KIND>, dim3(1), dim3(kFinishThreads), 0, stream, part, n,
                       max_norm, out);
    return hipGetLastError();
}

template <int KIND>
hipError_t acc_norm_t(const AccNormArgs& a, bool pads, dim3 grid, hipStream_t stream) {
    if (pads)
        hipLaunchKernelGGL((acc_norm_kernel<KIND, true>), grid, dim3(kThreads), 0, stream, a);
    else
        hipLaunchKernelGGL((acc_norm_kernel<KIND, false>), grid, dim3(kThreads), 0, stream, a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_acc_norm(const AccNormLaunch& L, int64_t* nparts, hipStream_t stream) {
    *nparts = 0;
    if (L.e_len <= 0 || L.spans <= 0) return hipSuccess;
    if (L.spans > ZSP_MAX_RANKS) return hipErrorInvalidValue;
    AccNormArgs a{};
    a.e0 = L.tab.e0;
    a.info = L.tab.info;
    a.tile = L.tab.tile;
    a.acc = L.acc;
    a.e_begin = L.e_begin;
    a.e_len = L.e_len;
    a.stride = L.stride;
    a.part = L.part;
    // workgroups per span: at most kNormBlocks (+ one per span) in all
    const int64_t tiles = L.e_len / kTile + 2;
    const int64_t most = kNormBlocks / L.spans + 1;
    const int64_t x = std::max<int64_t>(1, std::min((tiles + kWaves - 1) / kWaves, most));
    *nparts = x * L.spans;
    const dim3 grid(static_cast<uint32_t>(x), static_cast<uint32_t>(L.spans));
    return L.kind == ZSP_NORM_MAX ? acc_norm_t<ZSP_NORM_MAX>(a, L.pads, grid, stream)
                                  : acc_norm_t<ZSP_NORM_L2>(a, L.pads, grid, stream);
}

hipError_t launch_finish(double* part, int64_t n, int64_t parts_cap, zsp_norm_kind kind,
                         float max_norm, zsp_clip* out, hipStream_t stream) {
    return kind == ZSP_NORM_MAX
               ? finish_t<ZSP_NORM_MAX>(part, n, parts_cap, max_norm, out, stream)
               : finish_t<ZSP_NORM_L2>(part, n, parts_cap, max_norm, out, stream);
}

hipError_t launch_combine(const zsp_clip* parts, int32_t n, zsp_norm_kind kind, float max_norm,
                          zsp_clip* out, hipStream_t stream) {
    if (kind == ZSP_NORM_MAX)
        hipLaunchKernelGGL(combine_kernel<ZSP_NORM_MAX>, dim3(1), dim3(kThreads), 0, stream, parts,
                           n, max_norm, out);
    else
        hipLaunchKernelGGL(combine_kernel<ZSP_NORM_L2>, dim3(1), dim3(kThreads), 0, stream, parts,
                           n, max_norm, out);
    return hipGetLastError();
}

hipError_t launch_list_norm(const TensorsLaunch& L, zsp_norm_kind kind, double* part,
                            int64_t* nparts, bool add, hipStream_t stream) {
    if (L.nchunk <= 0) return hipSuccess;
    const int64_t blocks = list_blocks(L.nchunk);
    const int32_t add_to = add ? static_cast<int32_t>(*nparts) : 0;
    *nparts = std::max(*nparts, blocks);
    return kind == ZSP_NORM_MAX ? list_norm_t<ZSP_NORM_MAX>(L, part, blocks, add_to, stream)
                                : list_norm_t<ZSP_NORM_L2>(L, part, blocks, add_to, stream);
}

hipError_t launch_list_clip(const TensorsLaunch& L, const zsp_clip* clip, hipStream_t stream) {
    if (L.nchunk <= 0) return hipSuccess;
    const dim3 grid(static_cast<uint32_t>(list_blocks(L.nchunk))), block(kThreads);
    if (L.n_args > 0) {
        TensorArgs a{};
        tensor_args(L, a);
        a.clip = clip;
        hipLaunchKernelGGL((list_clip_kernel<false, TensorArgs>), grid, block, 0, stream, a);
    } else {
        TableArgs a{};
        a.chunks = L.chunks;
        a.nchunk = L.nchunk;
        a.clip = clip;
        hipLaunchKernelGGL((list_clip_kernel<true, TableArgs>), grid, block, 0, stream, a);
    }
    return hipGetLastError();
}

}  // namespace zsp
