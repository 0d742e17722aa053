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
// alone: equal inputs give equal bits.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "zsp_internal.hpp"
#include "zsp_wave.hpp"

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

template <int KIND>
__device__ __forceinline__ double join(double a, double b) {
    if constexpr (KIND == ZSP_NORM_MAX) return JoinMax()(a, b);
    else return JoinSum()(a, b);
}

// A wave's partial, the same in every lane.
template <int KIND>
__device__ __forceinline__ double wave_value(double v) {
    return wave_join(v, [](double a, double b) { return join<KIND>(a, b); });
}

// The workgroup's partial, valid in thread 0.
template <int KIND, int THREADS>
__device__ __forceinline__ double block_join(double v) {
    __shared__ double s_part[THREADS / kWaveLanes];
    v = wave_value<KIND>(v);
    const int wave = threadIdx.x / kWaveLanes;
    if (threadIdx.x % kWaveLanes == 0) s_part[wave] = v;
    __syncthreads();
    if (threadIdx.x == 0)
        for (int w = 1; w < THREADS / kWaveLanes; ++w) v = join<KIND>(v, s_part[w]);
    return v;
}

__device__ __forceinline__ void write_record(double total, int kind, double max_norm,
                                             zsp_clip* out) {
    const double norm = kind == ZSP_NORM_MAX ? total : __builtin_sqrt(total);
    float coef = 1.0f;
    if (!(norm <= 1.7976931348623157e308)) coef = __builtin_nanf("");
    else if (norm > max_norm) coef = float(max_norm / norm);
    out->total = total;
    out->norm = float(norm);
    out->coef = coef;
}

// The form of a small norm: one workgroup, one batch of loads per wave at
// most, and no second launch to join partials (nine small tensors: 4.0 us,
// and 3.4 + 1.9 in two launches, each of which costs the host 3 us more).
constexpr int kOneThreads = 1024;
constexpr int kOneWaves = kOneThreads / kWaveLanes;

// Lists: 16 bytes at any 2-byte offset. Every byte is read once here, and
// the non-temporal hint raised the read rate of a 0.8 GB norm from 6.3 to
// 6.9 TB/s.
__device__ __forceinline__ u32x4 ld16(const char* p) {
    return __builtin_nontemporal_load(reinterpret_cast<const u32x4_a2*>(p));
}

// ---- The accumulator's norm ----------------------------------------------------
// Bound by HBM's reads: 0.81 GB (202 M elements over 8 ranks) in 118 us, 6.9
// TB/s, and with pad slots at every slice's end 119. Two 1 KiB loads per
// wave and step, and a tile's table ahead of its data, took 138 and 178.
// A wave takes groups of kGroup elements (one batch of loads), every n-th one
// of its rank's span, n the waves of the span. One wave per workgroup; a norm
// of at most kOneWaves groups is one workgroup, which writes the record
// itself. No load of the accumulator waits for a table: a group inside one
// piece needs the table only to know that, and one that meets pad slots
// marks them in a bitmap in LDS, a lane per piece, and zeroes what it loaded
// there.
constexpr int kGroup = kBatch * kWaveLanes * 4;
constexpr int kGroupTiles = kGroup / kTile;

struct AccNormArgs {
    const PieceInfo* info;
    const int32_t* tile;
    const float* acc;
    int64_t ntile;
    int64_t e_begin, e_len, stride;
    double* part;
    double max_norm;  // of the form that writes the record
    zsp_clip* out;
};

// Marks the pad slots of the group at G0, which meets pieces lo .. hi: bit
// i % 32 of word i / 32 for element G0 + i. The words are the wave's own, and
// a wave's LDS operations run in order: the fences hold the compiler to that.
__device__ __forceinline__ void wave_sync() {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

__device__ __forceinline__ void mark_pads(const AccNormArgs& a, int64_t G0, int lo, int hi,
                                          int lane, uint32_t* bits) {
    static_assert(kGroup / 32 == kWaveLanes, "a word per lane");
    wave_sync();
    bits[lane] = 0u;
    wave_sync();
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
    wave_sync();
}

// Workgroups go to the 8 XCDs in turn. A norm's workgroup takes the place
// that puts runs of 8 neighbours on one XCD: a line of the table they read
// (chunk records, pieces of tiles) is then fetched into one L2 (10,000
// tensors 37.7 us, in plain order 38.9).
__device__ __forceinline__ int norm_place(int b, int n) {
    return b < n / 64 * 64 ? b / 64 * 64 + b % 8 * 8 + b / 8 % 8 : b;
}

template <int KIND, bool PADS, bool ONE>
__global__ __launch_bounds__(ONE ? kOneThreads : kWaveLanes) void acc_norm_kernel(
    const AccNormArgs a) {
    __shared__ uint32_t s_all[PADS ? (ONE ? kOneWaves : 1) * (kGroup / 32) : 1];
    const int lane = threadIdx.x % kWaveLanes;
    const int wave = ONE ? __builtin_amdgcn_readfirstlane(threadIdx.x / kWaveLanes) : 0;
    uint32_t* const s_bits = s_all + (PADS ? wave * (kGroup / 32) : 0);
    const int64_t b = a.e_begin + int64_t(blockIdx.y) * a.stride, e = b + a.e_len;
    Acc<KIND> t;
    for (int64_t g = b / kGroup + (ONE ? wave : norm_place(blockIdx.x, gridDim.x)); g * kGroup < e;
         g += ONE ? kOneWaves : int(gridDim.x)) {
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
    if constexpr (ONE) {
        const double v = block_join<KIND, kOneThreads>(t.value());
        if (threadIdx.x == 0) write_record(v, KIND, a.max_norm, a.out);
    } else {
        const double v = wave_value<KIND>(t.value());
        if (lane == 0) a.part[int64_t(blockIdx.y) * gridDim.x + blockIdx.x] = v;
    }
}

// ---- Lists of tensors -------------------------------------------------------------
// A chunk is kListChunkBytes of one tensor: 512 groups of 16 bytes (8 bf16
// or 4 fp32 values), then what is left of its last group. A norm's wave
// takes a whole chunk per batch of loads: 0.40 GB of bf16 in nine tensors in
// 62 us (6.6 TB/s; the 64-bit arithmetic of twice the elements per byte is
// half of that), 0.24 GB in 10,000 tensors in 38. A clip's wave, which also
// writes, takes one group per lane (1 KiB): short waves, each reading then
// writing one run, took 242 us for 0.81 GB of fp32 (6.7 TB/s read and
// written), and waves of 4 KiB 267 (of 16 KiB in a loop, 330).

struct TableArgs {
    const ListChunk* chunks;
    int64_t nchunk;
    double* part;
    const zsp_clip* clip;
    zsp_clip* out;    // of the one-workgroup form
    double max_norm;  // likewise
    int32_t add_to;   // partials already there that a list norm joins
};

struct TensorArgs {
    int64_t nchunk;
    int64_t chunk_first;  // of the launch
    double* part;
    const zsp_clip* clip;
    zsp_clip* out;
    double max_norm;
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
    c += a.chunk_first;
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

template <int KIND, bool ONE, typename Args>
__global__ __launch_bounds__(ONE ? kOneThreads : kWaveLanes) void list_norm_kernel(const Args a) {
    const int lane = threadIdx.x % kWaveLanes;
    const int first = ONE ? __builtin_amdgcn_readfirstlane(threadIdx.x / kWaveLanes)
                          : norm_place(blockIdx.x, gridDim.x);
    Acc<KIND> t;
    for (int64_t c = first; c < a.nchunk; c += ONE ? kOneWaves : int(gridDim.x))
        chunk_norm(get_chunk(a, c), lane, t);
    if constexpr (ONE) {
        const double v = block_join<KIND, kOneThreads>(t.value());
        if (threadIdx.x == 0) write_record(v, KIND, a.max_norm, a.out);
    } else {
        double v = wave_value<KIND>(t.value());
        if (lane == 0) {
            if (int(blockIdx.x) < a.add_to) v = join<KIND>(a.part[blockIdx.x], v);
            a.part[blockIdx.x] = v;
        }
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

// Workgroups go to the 8 XCDs in turn; each XCD takes runs of kClipRun
// consecutive waves (64 KiB of a tensor), so that a cache line which two
// waves share -- a tensor starts at any element -- is written in one L2.
// 10,000 tensors, every seventh off alignment: 78 us, and 103 with the waves
// in plain order; 0.8 GB in nine aligned tensors: 242 and 258.
constexpr int kClipRun = 64;

template <typename Args>
__global__ __launch_bounds__(kWaveLanes) void list_clip_kernel(const Args a) {
    const int64_t x = blockIdx.x % 8, i = blockIdx.x / 8;
    const int64_t w = (i / kClipRun * 8 + x) * kClipRun + i % kClipRun;
    if (w >= a.nchunk * kBatch) return;  // the grid is rounded up to 8 runs
    const ListChunk c = get_chunk(a, w / kBatch);
    const float s = a.clip->coef;
    // 1: nothing to change. NaN: the norm was not finite, nothing is changed.
    if (s == 1.0f || s != s) return;
    chunk_scale(c, int(w % kBatch), threadIdx.x, s);
}

// ---- Joining partials -------------------------------------------------------------

constexpr int kFinishThreads = 1024;
constexpr int kThreads = 256;
static_assert(kNormBlocks + ZSP_MAX_RANKS <= kFinishMax, "these norms set no ticket");

// Joins part[first], part[first + step], ... below n, eight loads in flight
// (past the end the last again, unused).
template <int KIND>
__device__ __forceinline__ double join_strided(const double* part, int64_t first, int64_t step,
                                               int64_t n) {
    double v = 0.0;
    for (int64_t i = first; i < n; i += step * 8) {
        double x[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const int64_t j = i + k * step;
            x[k] = part[j < n ? j : n - 1];
        }
#pragma unroll
        for (int k = 0; k < 8; ++k)
            if (i + k * step < n) v = join<KIND>(v, x[k]);
    }
    return v;
}

// A long list of partials in one launch: workgroup b joins the b-th run of
// ceil(n / gridDim.x), and the workgroup that takes the last ticket (0 when
// the launch begins) joins the runs, in their order whichever it is. No
// workgroup waits for another. 46,000 partials 4.8 us and 790,000 7.4, where
// a fold and a finish took 4.6 each and the gap between two launches; with
// 256 runs 8.7 and 9.5 (tickets are taken one after another, 17 ns each).
template <int KIND>
__global__ __launch_bounds__(kThreads) void fold_kernel(const double* part, int64_t n, double* runs,
                                                        uint32_t* ticket, double max_norm,
                                                        zsp_clip* out) {
    __shared__ uint32_t s_last;
    const int64_t per = (n + gridDim.x - 1) / gridDim.x;
    const int64_t b = per * blockIdx.x, e = b + per < n ? b + per : n;
    double v = block_join<KIND, kThreads>(join_strided<KIND>(part, b + threadIdx.x, kThreads, e));
    if (threadIdx.x == 0) {
        __hip_atomic_store(runs + blockIdx.x, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        s_last = __hip_atomic_fetch_add(ticket, 1u, __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_AGENT) ==
                 gridDim.x - 1;
    }
    __syncthreads();
    if (!s_last) return;
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "agent");
    static_assert(kFoldBlocks <= kThreads, "a run per thread");
    v = threadIdx.x < gridDim.x ? __hip_atomic_load(runs + threadIdx.x, __ATOMIC_RELAXED,
                                                    __HIP_MEMORY_SCOPE_AGENT)
                                : 0.0;
    v = block_join<KIND, kThreads>(v);
    if (threadIdx.x == 0) write_record(v, KIND, max_norm, out);
}

template <int KIND>
__global__ __launch_bounds__(kFinishThreads) void finish_kernel(const double* part, int64_t n,
                                                                double max_norm, zsp_clip* out) {
    double v = join_strided<KIND>(part, threadIdx.x, kFinishThreads, n);
    v = block_join<KIND, kFinishThreads>(v);
    if (threadIdx.x == 0) write_record(v, KIND, max_norm, out);
}

// The records' totals are all read before *out, which may be one of them, is
// written. A total that is no norm's (negative) gives a NaN.
template <int KIND>
__global__ __launch_bounds__(kThreads) void combine_kernel(const zsp_clip* parts, int32_t n,
                                                           double max_norm, zsp_clip* out) {
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

template <int KIND, bool ONE>
hipError_t list_norm_t(const TensorsLaunch& L, double* part, int64_t blocks, int32_t add_to,
                       double max_norm, zsp_clip* out, hipStream_t stream) {
    const dim3 grid(static_cast<uint32_t>(blocks)), block(ONE ? kOneThreads : kWaveLanes);
    if (L.n_args > 0) {
        TensorArgs a{};
        tensor_args(L, a);
        a.part = part;
        a.add_to = add_to;
        a.max_norm = max_norm;
        a.out = out;
        hipLaunchKernelGGL((list_norm_kernel<KIND, ONE, TensorArgs>), grid, block, 0, stream, a);
    } else {
        TableArgs a{};
        a.chunks = L.chunks;
        a.nchunk = L.nchunk;
        a.part = part;
        a.add_to = add_to;
        a.max_norm = max_norm;
        a.out = out;
        hipLaunchKernelGGL((list_norm_kernel<KIND, ONE, TableArgs>), grid, block, 0, stream, a);
    }
    return hipGetLastError();
}

template <int KIND>
hipError_t finish_t(double* part, int64_t n, int64_t parts_cap, double max_norm, zsp_clip* out,
                    hipStream_t stream) {
    if (n > kFinishMax) {
        const int64_t per = kThreads * 8;  // a round of loads
        const int64_t runs = std::min<int64_t>(kFoldBlocks, (n + per - 1) / per);
        hipLaunchKernelGGL(fold_kernel<KIND>, dim3(static_cast<uint32_t>(runs)), dim3(kThreads), 0,
                           stream, part, n, part + parts_cap, norm_ticket(part, parts_cap),
                           max_norm, out);
        return hipGetLastError();
    }
    hipLaunchKernelGGL(finish_kernel<KIND>, dim3(1), dim3(kFinishThreads), 0, stream, part, n,
                       max_norm, out);
    return hipGetLastError();
}

template <int KIND>
hipError_t acc_norm_t(const AccNormArgs& a, bool pads, bool one, dim3 grid, hipStream_t stream) {
    const dim3 block(one ? kOneThreads : kWaveLanes);
    if (pads && one)
        hipLaunchKernelGGL((acc_norm_kernel<KIND, true, true>), grid, block, 0, stream, a);
    else if (pads)
        hipLaunchKernelGGL((acc_norm_kernel<KIND, true, false>), grid, block, 0, stream, a);
    else if (one)
        hipLaunchKernelGGL((acc_norm_kernel<KIND, false, true>), grid, block, 0, stream, a);
    else
        hipLaunchKernelGGL((acc_norm_kernel<KIND, false, false>), grid, block, 0, stream, a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_acc_norm(const AccNormLaunch& L, double max_norm, zsp_clip* out,
                           int64_t* nparts, bool* done, hipStream_t stream) {
    *nparts = 0;
    *done = false;
    if (L.e_len <= 0 || L.spans <= 0) return hipSuccess;
    if (L.spans > ZSP_MAX_RANKS) return hipErrorInvalidValue;
    AccNormArgs a{};
    a.info = L.tab.info;
    a.tile = L.tab.tile;
    a.ntile = L.tab.ntile;
    a.acc = L.acc;
    a.e_begin = L.e_begin;
    a.e_len = L.e_len;
    a.stride = L.stride;
    a.part = L.part;
    a.max_norm = max_norm;
    a.out = out;
    // workgroups per span: at most kNormBlocks (+ one per span) in all
    const int64_t groups = L.e_len / kGroup + 2;
    const int64_t x = std::min<int64_t>(groups, kNormBlocks / L.spans + 1);
    *done = L.spans == 1 && groups <= kOneWaves;
    *nparts = *done ? 0 : x * L.spans;
    const dim3 grid(*done ? 1u : static_cast<uint32_t>(x), static_cast<uint32_t>(L.spans));
    return L.kind == ZSP_NORM_MAX ? acc_norm_t<ZSP_NORM_MAX>(a, L.pads, *done, grid, stream)
                                  : acc_norm_t<ZSP_NORM_L2>(a, L.pads, *done, grid, stream);
}

hipError_t launch_finish(double* part, int64_t n, int64_t parts_cap, zsp_norm_kind kind,
                         double max_norm, zsp_clip* out, hipStream_t stream) {
    return kind == ZSP_NORM_MAX
               ? finish_t<ZSP_NORM_MAX>(part, n, parts_cap, max_norm, out, stream)
               : finish_t<ZSP_NORM_L2>(part, n, parts_cap, max_norm, out, stream);
}

hipError_t launch_combine(const zsp_clip* parts, int32_t n, zsp_norm_kind kind, double max_norm,
                          zsp_clip* out, hipStream_t stream) {
    if (kind == ZSP_NORM_MAX)
        hipLaunchKernelGGL(combine_kernel<ZSP_NORM_MAX>, dim3(1), dim3(kThreads), 0, stream, parts,
                           n, max_norm, out);
    else
        hipLaunchKernelGGL(combine_kernel<ZSP_NORM_L2>, dim3(1), dim3(kThreads), 0, stream, parts,
                           n, max_norm, out);
    return hipGetLastError();
}

bool list_norm_is_small(int64_t nchunk) { return nchunk <= kOneWaves; }

hipError_t launch_list_norm_one(const TensorsLaunch& L, zsp_norm_kind kind, double max_norm,
                                zsp_clip* out, hipStream_t stream) {
    return kind == ZSP_NORM_MAX
               ? list_norm_t<ZSP_NORM_MAX, true>(L, nullptr, 1, 0, max_norm, out, stream)
               : list_norm_t<ZSP_NORM_L2, true>(L, nullptr, 1, 0, max_norm, out, stream);
}

hipError_t launch_list_norm(const TensorsLaunch& L, zsp_norm_kind kind, double* part,
                            int64_t* nparts, hipStream_t stream) {
    if (L.nchunk <= 0) return hipSuccess;
    const int64_t blocks = std::min<int64_t>(L.nchunk, kNormBlocks);
    const int32_t there = static_cast<int32_t>(*nparts);
    *nparts = std::max(*nparts, blocks);
    return kind == ZSP_NORM_MAX
               ? list_norm_t<ZSP_NORM_MAX, false>(L, part, blocks, there, 0, nullptr, stream)
               : list_norm_t<ZSP_NORM_L2, false>(L, part, blocks, there, 0, nullptr, stream);
}

hipError_t launch_list_clip(const TensorsLaunch& L, const zsp_clip* clip, hipStream_t stream) {
    // work-items of a launch must fit in 32 bits: a long list takes several
    constexpr int64_t kMost = int64_t(1) << 22;
    for (int64_t at = 0; at < L.nchunk; at += kMost) {
        const int64_t n = std::min(L.nchunk - at, kMost);
        const int64_t round = 8 * kClipRun;
        const int64_t blocks = (n * kBatch + round - 1) / round * round;
        const dim3 grid(static_cast<uint32_t>(blocks)), block(kWaveLanes);
        if (L.n_args > 0) {
            TensorArgs a{};
            tensor_args(L, a);
            a.chunk_first = at;
            a.nchunk = n;
            a.clip = clip;
            hipLaunchKernelGGL((list_clip_kernel<TensorArgs>), grid, block, 0, stream, a);
        } else {
            TableArgs a{};
            a.chunks = L.chunks + at;
            a.nchunk = n;
            a.clip = clip;
            hipLaunchKernelGGL((list_clip_kernel<TableArgs>), grid, block, 0, stream, a);
        }
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

}  // namespace zsp
