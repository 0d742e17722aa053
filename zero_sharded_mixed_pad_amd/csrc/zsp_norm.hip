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
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

// A norm's wave reads 16-byte groups, one per lane and load, in batches of
// kBatch loads (8 KiB) that all go out before the first is used.
constexpr int kBatch = 8;
static_assert(kListChunkBytes == kBatch * kWaveLanes * 16, "a chunk is one batch");

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
    __device__ __forceinline__ void add4(u32x4 v) {
#pragma unroll
        for (int k = 0; k < 4; ++k) add(__uint_as_float(v[k]));
    }
    __device__ __forceinline__ void add8(u32x4 v) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            add(lo16(v[k]));
            add(hi16(v[k]));
        }
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

// A wave's partial, the same in every lane.
template <int KIND>
__device__ __forceinline__ double wave_join(double v) {
#pragma unroll
    for (int d = kWaveLanes / 2; d > 0; d /= 2) v = join<KIND>(v, __shfl_xor(v, d));
    return v;
}

// The workgroup's partial, valid in thread 0.
template <int KIND, int THREADS>
__device__ __forceinline__ double block_join(double v) {
    __shared__ double s_part[THREADS / kWaveLanes];
    v = wave_join<KIND>(v);
    const int wave = threadIdx.x / kWaveLanes;
    if (threadIdx.x % kWaveLanes == 0) s_part[wave] = v;
    __syncthreads();
    if (threadIdx.x == 0)
        for (int w = 1; w < THREADS / kWaveLanes; ++w) v = join<KIND>(v, s_part[w]);
    return v;
}

// Lists: 16 bytes at any 2-byte offset. Every byte is read once here, and
// the non-temporal hint raised the read rate of a 0.8 GB norm from 6.3 to
// 6.9 TB/s.
__device__ __forceinline__ u32x4 ld16(const char* p) {
    return __builtin_nontemporal_load(reinterpret_cast<const u32x4_a2*>(p));
}

// ---- The accumulator's norm ----------------------------------------------------
// One wave per workgroup; a wave takes groups of kGroup elements (one batch
// of loads), every gridDim.x-th one of its rank's span. No load of the
// accumulator waits for a table: a group inside one piece needs the table
// only to know that, and one that meets pad slots marks them in a bitmap in
// LDS, a lane per piece, and zeroes what it loaded there.
constexpr int kGroup = kBatch * kWaveLanes * 4;
constexpr int kGroupTiles = kGroup / kTile;

struct AccNormArgs {
    const int64_t* e0;
    const PieceInfo* info;
    const int32_t* tile;
    const float* acc;
    int64_t ntile;
    int64_t e_begin, e_len, stride;
    double* part;
};

// Marks the pad slots of the group at G0, which meets pieces lo .. hi: bit
// i % 32 of word i / 32 for element G0 + i. No wave reads another's bits.
__device__ __forceinline__ void mark_pads(const AccNormArgs& a, int64_t G0, int lo, int hi,
                                          int lane, uint32_t* bits) {
    static_assert(kGroup / 32 == kWaveLanes, "a word per lane");
    bits[lane] = 0u;
    __syncthreads();
    for (int p = lo + lane; p <= hi; p += kWaveLanes) {
        const PieceInfo pi = a.info[p];
        int64_t b = pi.vend - G0, e = pi.end - G0;
        b = b < 0 ? 0 : b;
        e = e > kGroup ? kGroup : e;
        while (b < e) {
            const int w = int(b) / 32, at = int(b) % 32;
            const int n = int(e - b) < 32 - at ? int(e - b) : 32 - at;
            atomicOr(&bits[w], (n == 32 ? ~0u : ((1u << n) - 1u)) << at);
            b += n;
        }
    }
    __syncthreads();
}

template <int KIND, bool PADS>
__global__ __launch_bounds__(kWaveLanes) void acc_norm_kernel(const AccNormArgs a) {
    __shared__ uint32_t s_bits[kGroup / 32];
    const int lane = threadIdx.x;
    const int64_t b = a.e_begin + int64_t(blockIdx.y) * a.stride, e = b + a.e_len;
    Acc<KIND> t;
    for (int64_t g = b / kGroup + blockIdx.x; g * kGroup < e; g += gridDim.x) {
        const int64_t G0 = g * kGroup;
        const bool inside = G0 >= b && G0 + kGroup <= e;
        u32x4 v[kBatch];
        if (inside) {
            const f32x4* p = reinterpret_cast<const f32x4*>(a.acc + G0) + lane;
#pragma unroll
            for (int r = 0; r < kBatch; ++r)
                v[r] = __builtin_bit_cast(u32x4, __builtin_nontemporal_load(p + r * kWaveLanes));
        } else {
            // elements outside the span: one of its ends again, unused
            float x[kBatch][4];
#pragma unroll
            for (int r = 0; r < kBatch; ++r)
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int64_t E = G0 + (r * kWaveLanes + lane) * 4 + k;
                    x[r][k] = a.acc[E < b ? b : E < e ? E : e - 1];
                }
#pragma unroll
            for (int r = 0; r < kBatch; ++r)
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int64_t E = G0 + (r * kWaveLanes + lane) * 4 + k;
                    v[r][k] = E >= b && E < e ? __float_as_uint(x[r][k]) : 0u;
                }
        }
        if constexpr (PADS) {
            const int64_t t1 = (g + 1) * kGroupTiles;
            const int lo = a.tile[g * kGroupTiles];
            const int hi = a.tile[t1 < a.ntile ? t1 : a.ntile];
            if (lo != hi || G0 + kGroup > a.info[lo].vend) {
                mark_pads(a, G0, lo, hi, lane, s_bits);
#pragma unroll
                for (int r = 0; r < kBatch; ++r) {
                    const uint32_t m = s_bits[8 * r + lane / 8] >> (lane % 8 * 4);
#pragma unroll
                    for (int k = 0; k < 4; ++k) v[r][k] = (m >> k) & 1u ? 0u : v[r][k];
                }
            }
        }
#pragma unroll
        for (int r = 0; r < kBatch; ++r) t.add4(v[r]);
    }
    const double v = wave_join<KIND>(t.value());
    if (lane == 0) a.part[int64_t(blockIdx.y) * gridDim.x + blockIdx.x] = v;
}

// ---- Lists of tensors -------------------------------------------------------------
// A chunk is kListChunkBytes of one tensor: 512 groups of 16 bytes (8 bf16
// or 4 fp32 values), then what is left of its last group. A norm's wave
// takes a whole chunk per batch of loads; a clip's wave, which also writes,
// takes one group per lane (1 KiB): short waves, each reading then writing
// one run, measured 6.7 TB/s on 0.8 GB, and waves of 4 KiB 6.1.

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

// Chunk c of a list in device memory, or in the kernel arguments (read from
// the argument segment: the struct is the kernel's only explicit argument,
// so it starts at 0). c is wave-uniform.
__device__ __forceinline__ ListChunk get_chunk(const TableArgs& a, int64_t c) {
    return a.chunks[c];
}

__device__ __forceinline__ ListChunk get_chunk(const TensorArgs& a, int64_t c) {
    const char* seg = (const char*)__builtin_amdgcn_kernarg_segment_ptr();
    const int32_t* c0 = reinterpret_cast<const int32_t*>(seg + offsetof(TensorArgs, chunk0));
    const ArgTensor* ts = reinterpret_cast<const ArgTensor*>(seg + offsetof(TensorArgs, t));
    int lo = 0, hi = a.n - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (c0[mid] <= c) lo = mid;
        else hi = mid - 1;
    }
    const ArgTensor t = ts[lo];
    const int32_t type = int32_t(t.numel_type & 1);
    const int64_t most = chunk_elems(type);
    const int64_t at = (c - c0[lo]) * most, left = (t.numel_type >> 1) - at;
    ListChunk r;
    r.p = static_cast<char*>(t.p) + at * (kListChunkBytes / most);
    r.n = int32_t(left < most ? left : most);
    r.dtype = type;
    return r;
}

template <int KIND>
__device__ __forceinline__ void chunk_norm(const ListChunk& c, int lane, Acc<KIND>& t) {
    const char* p = static_cast<const char*>(c.p);
    const bool bf = c.dtype == ZSP_BF16;
    const int groups = bf ? c.n / 8 : c.n / 4;
    if (groups > 0) {
        u32x4 v[kBatch];
#pragma unroll
        for (int r = 0; r < kBatch; ++r) {
            const int i = r * kWaveLanes + lane;  // past the last group: the last again, unused
            v[r] = ld16(p + 16 * (i < groups ? i : groups - 1));
        }
        if (groups < kBatch * kWaveLanes) {
#pragma unroll
            for (int r = 0; r < kBatch; ++r)
                if (r * kWaveLanes + lane >= groups) v[r] = u32x4{0u, 0u, 0u, 0u};
        }
        if (bf) {
#pragma unroll
            for (int r = 0; r < kBatch; ++r) t.add8(v[r]);
        } else {
#pragma unroll
            for (int r = 0; r < kBatch; ++r) t.add4(v[r]);
        }
    }
    const int i = groups * (bf ? 8 : 4) + lane;
    if (i < c.n)
        t.add(bf ? __uint_as_float(uint32_t(reinterpret_cast<const uint16_t*>(p)[i]) << 16)
                 : reinterpret_cast<const float*>(p)[i]);
}

template <int KIND, typename Args>
__global__ __launch_bounds__(kWaveLanes) void list_norm_kernel(const Args a) {
    const int lane = threadIdx.x;
    Acc<KIND> t;
    for (int64_t c = blockIdx.x; c < a.nchunk; c += gridDim.x) chunk_norm(get_chunk(a, c), lane, t);
    double v = wave_join<KIND>(t.value());
    if (lane == 0) {
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

// Run `part` of a chunk: x * coef in fp32, rounded once more to a bf16
// tensor's type.
__device__ __forceinline__ void chunk_scale(const ListChunk& c, int part, int lane, float s) {
    const bool bf = c.dtype == ZSP_BF16;
    const int groups = bf ? c.n / 8 : c.n / 4;
    const int i = part * kWaveLanes + lane;
    char* p = static_cast<char*>(c.p);
    if (i < groups) {
        const u32x4 v = ld16(p + 16 * i);
        u32x4 o;
        if (bf) {
            o = u32x4{scale2(v.x, s), scale2(v.y, s), scale2(v.z, s), scale2(v.w, s)};
        } else {
#pragma unroll
            for (int k = 0; k < 4; ++k) o[k] = __float_as_uint(__uint_as_float(v[k]) * s);
        }
        __builtin_nontemporal_store(o, reinterpret_cast<u32x4_a2*>(p + 16 * i));
    } else if (i == groups) {
        // the lane behind the last group: the elements that fill no group
        if (bf) {
            uint16_t* q = static_cast<uint16_t*>(c.p);
            for (int k = groups * 8; k < c.n; ++k)
                q[k] = __builtin_bit_cast(
                    uint16_t, static_cast<__bf16>(__uint_as_float(uint32_t(q[k]) << 16) * s));
        } else {
            float* q = static_cast<float*>(c.p);
            for (int k = groups * 4; k < c.n; ++k) q[k] *= s;
        }
    }
}

template <typename Args>
__global__ __launch_bounds__(kWaveLanes) void list_clip_kernel(const Args a) {
    const float s = a.clip->coef;
    // 1: nothing to change. NaN: the norm was not finite, nothing is changed.
    if (s == 1.0f || s != s) return;
    for (int64_t w = blockIdx.x; w < a.nchunk * kBatch; w += gridDim.x)
        chunk_scale(get_chunk(a, w / kBatch), int(w % kBatch), threadIdx.x, s);
}

// ---- Joining partials -------------------------------------------------------------

constexpr int kFinishThreads = 1024;
constexpr int kThreads = 256;
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

void tensor_args(const TensorsLaunch& L, TensorArgs& a) {
    a.nchunk = L.nchunk;
    a.n = L.n_args;
    for (int i = 0; i < L.n_args; ++i) a.t[i] = L.args[i];
    for (int i = 0; i <= L.n_args; ++i) a.chunk0[i] = L.chunk0[i];
}

template <int KIND>
hipError_t list_norm_t(const TensorsLaunch& L, double* part, int64_t blocks, int32_t add_to,
                       hipStream_t stream) {
    const dim3 grid(static_cast<uint32_t>(blocks)), block(kWaveLanes);
    if (L.n_args > 0) {
        TensorArgs a{};
        tensor_args(L, a);
        a.part = part;
        a.add_to = add_to;
        hipLaunchKernelGGL((list_norm_kernel<KIND, TensorArgs>), grid, block, 0, stream, a);
    } else {
        TableArgs a{};
        a.chunks = L.chunks;
        a.nchunk = L.nchunk;
        a.part = part;
        a.add_to = add_to;
        hipLaunchKernelGGL((list_norm_kernel<KIND, TableArgs>), grid, block, 0, stream, a);
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
        hipLaunchKernelGGL((acc_norm_kernel<KIND, true>), grid, dim3(kWaveLanes), 0, stream, a);
    else
        hipLaunchKernelGGL((acc_norm_kernel<KIND, false>), grid, dim3(kWaveLanes), 0, stream, a);
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
    a.ntile = L.tab.ntile;
    a.part = L.part;
    // workgroups per span: at most kNormBlocks (+ one per span) in all
    const int64_t groups = L.e_len / kGroup + 2;
    const int64_t x = std::min<int64_t>(groups, kNormBlocks / L.spans + 1);
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
    const int64_t blocks = std::min<int64_t>(L.nchunk, kNormBlocks);
    const int32_t add_to = add ? static_cast<int32_t>(*nparts) : 0;
    *nparts = std::max(*nparts, blocks);
    return kind == ZSP_NORM_MAX ? list_norm_t<ZSP_NORM_MAX>(L, part, blocks, add_to, stream)
                                : list_norm_t<ZSP_NORM_L2>(L, part, blocks, add_to, stream);
}

hipError_t launch_list_clip(const TensorsLaunch& L, const zsp_clip* clip, hipStream_t stream) {
    if (L.nchunk <= 0) return hipSuccess;
    // a wave per run; its work-items must fit in 32 bits
    const int64_t waves = std::min<int64_t>(L.nchunk * kBatch, int64_t(1) << 25);
    const dim3 grid(static_cast<uint32_t>(waves)), block(kWaveLanes);
    if (L.n_args > 0) {
        TensorArgs a{};
        tensor_args(L, a);
        a.clip = clip;
        hipLaunchKernelGGL((list_clip_kernel<TensorArgs>), grid, block, 0, stream, a);
    } else {
        TableArgs a{};
        a.chunks = L.chunks;
        a.nchunk = L.nchunk;
        a.clip = clip;
        hipLaunchKernelGGL((list_clip_kernel<TableArgs>), grid, block, 0, stream, a);
    }
    return hipGetLastError();
}

}  // namespace zsp
