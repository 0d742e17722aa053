// zsp_tensors.cpp -- the norm and the clipping of lists of tensors
// (zsp_norm_many, zsp_clip_many and the prepared zsp_tensor_list): argument
// checks, chunk tables, launches.
//
// A list is cut into chunks of kListChunkBytes, each inside one tensor. A
// one-shot list travels in the kernel arguments, kTensorArgMax tensors with
// elements per launch: nothing is staged, so any list can be captured into a
// HIP graph. Later launches of a long list join their partials to the first
// one's. A prepared list keeps one record per chunk in device memory and is
// one launch whatever its length.
#include <algorithm>
#include <climits>
#include <new>
#include <utility>
#include <vector>

#include "zsp_entry.hpp"
#include "zsp_internal.hpp"

struct zsp_tensor_list {
    int device = -1;
    int64_t nchunk = 0;
    zsp::ListChunk* dev = nullptr;
    bool overlap = false;  // some tensors share memory: no clipping
};

namespace zsp {
namespace {

int64_t chunks_of(int64_t numel, int32_t dtype) {
    const int64_t c = chunk_elems(dtype);
    return numel / c + (numel % c != 0);
}
int64_t size_of(int32_t dtype) { return dtype == ZSP_BF16 ? 2 : 4; }

// Checks as zsp_norm_many documents them; the number of chunks.
zsp_status check_tensors(const void* const* x, const int64_t* numel, const int32_t* dtype,
                         int32_t n, int64_t* nchunk) {
    if (n < 0) return set_error(ZSP_EINVAL, "n = %d is negative", n);
    if (n > 0 && (!x || !numel || !dtype))
        return set_error(ZSP_EINVAL, "x, numel or dtype is NULL");
    int64_t c = 0;
    for (int32_t i = 0; i < n; ++i) {
        if (dtype[i] != ZSP_F32 && dtype[i] != ZSP_BF16)
            return set_error(ZSP_EINVAL, "bad dtype[%d] = %d", i, dtype[i]);
        if (numel[i] < 0)
            return set_error(ZSP_EINVAL, "numel[%d] = %lld is negative", i, (long long)numel[i]);
        if (numel[i] == 0) continue;
        if (!x[i]) return set_error(ZSP_EINVAL, "x[%d] is NULL", i);
        if (reinterpret_cast<uintptr_t>(x[i]) % uintptr_t(size_of(dtype[i])))
            return set_error(ZSP_EINVAL, "x[%d] is not aligned to its element type", i);
        // each count is at most 2^52, so the sum cannot wrap before the check
        c += chunks_of(numel[i], dtype[i]);
        if (c > INT32_MAX)
            return set_error(ZSP_ERANGE, "list of 2^31 chunks of %d bytes or more",
                             kListChunkBytes);
    }
    *nchunk = c;
    return ZSP_OK;
}

// Whether two of the tensors share memory. Lists in order of address (views
// into one buffer) are seen to be apart in one pass.
zsp_status find_overlap(const void* const* x, const int64_t* numel, const int32_t* dtype,
                        int32_t n, bool* overlap) {
    *overlap = false;
    uintptr_t end = 0;
    bool in_order = true;
    for (int32_t i = 0; i < n && in_order; ++i) {
        if (numel[i] == 0) continue;
        const uintptr_t b = reinterpret_cast<uintptr_t>(x[i]);
        in_order = b >= end;
        end = b + uintptr_t(numel[i]) * uintptr_t(size_of(dtype[i]));
    }
    if (in_order) return ZSP_OK;
    try {
        std::vector<std::pair<uintptr_t, uintptr_t>> r;
        r.reserve(size_t(n));
        for (int32_t i = 0; i < n; ++i) {
            if (numel[i] == 0) continue;
            const uintptr_t b = reinterpret_cast<uintptr_t>(x[i]);
            r.emplace_back(b, b + uintptr_t(numel[i]) * uintptr_t(size_of(dtype[i])));
        }
        std::sort(r.begin(), r.end());
        for (size_t i = 1; i < r.size() && !*overlap; ++i) *overlap = r[i].first < r[i - 1].second;
    } catch (const std::bad_alloc&) {
        return set_error(ZSP_ENOMEM, "out of host memory");
    }
    return ZSP_OK;
}

// Calls f(launch) for runs of at most kTensorArgMax tensors with elements.
template <typename F>
zsp_status for_each_launch(const void* const* x, const int64_t* numel, const int32_t* dtype,
                           int32_t n, F f) {
    TensorsLaunch L;
    L.chunk0[0] = 0;
    for (int32_t i = 0; i < n; ++i) {
        if (numel[i] > 0) {
            L.args[L.n_args] = ArgTensor{const_cast<void*>(x[i]), numel[i] * 2 + dtype[i]};
            L.nchunk += chunks_of(numel[i], dtype[i]);
            L.chunk0[++L.n_args] = static_cast<int32_t>(L.nchunk);
        }
        if (L.n_args > 0 && (L.n_args == kTensorArgMax || i == n - 1)) {
            const hipError_t e = f(L);
            if (e != hipSuccess) return set_hip_error(e, "tensor list launch");
            L.n_args = 0;
            L.nchunk = 0;
        }
    }
    return ZSP_OK;
}

zsp_status check_device(const zsp_tensor_list* L) {
    if (!L) return set_error(ZSP_EINVAL, "list is NULL");
    int dev = -1;
    const hipError_t e = hipGetDevice(&dev);
    if (e != hipSuccess) return set_hip_error(e, "hipGetDevice");
    if (dev != L->device)
        return set_error(ZSP_ESTATE, "list made on device %d but device %d is current", L->device,
                         dev);
    return ZSP_OK;
}

zsp_status finish(const NormCall& nc, int64_t nparts, hipStream_t stream) {
    const hipError_t e = launch_finish(static_cast<double*>(nc.ws), nparts, norm_parts(0, 0),
                                       nc.kind, nc.max_norm, nc.out, stream);
    if (e != hipSuccess) return set_hip_error(e, "norm launch");
    return ZSP_OK;
}

}  // namespace
}  // namespace zsp

extern "C" {

zsp_status zsp_norm_many(const void* const* x, const int64_t* numel, const int32_t* dtype,
                         int32_t n, zsp_norm_kind kind, double max_norm, void* ws,
                         int64_t ws_bytes, zsp_clip* out, void* stream) {
    using namespace zsp;
    const NormCall nc{kind, max_norm, ws, ws_bytes, out};
    int64_t nchunk = 0;
    zsp_status st = check_tensors(x, numel, dtype, n, &nchunk);
    if (st == ZSP_OK) st = check_norm(nc, norm_parts(0, 0));
    if (st != ZSP_OK) return st;
    const hipStream_t hs = static_cast<hipStream_t>(stream);
    int64_t nparts = 0;
    bool done = false;
    st = for_each_launch(x, numel, dtype, n, [&](const TensorsLaunch& L) {
        done = L.nchunk == nchunk && list_norm_is_small(nchunk);
        return done ? launch_list_norm_one(L, kind, max_norm, out, hs)
                    : launch_list_norm(L, kind, static_cast<double*>(ws), &nparts, hs);
    });
    return st != ZSP_OK || done ? st : finish(nc, nparts, hs);
}

zsp_status zsp_clip_many(void* const* x, const int64_t* numel, const int32_t* dtype, int32_t n,
                         const zsp_clip* clip, void* stream) {
    using namespace zsp;
    int64_t nchunk = 0;
    zsp_status st = check_tensors(x, numel, dtype, n, &nchunk);
    if (st == ZSP_OK) st = check_clip(clip, "clip");
    bool overlap = false;
    if (st == ZSP_OK) st = find_overlap(x, numel, dtype, n, &overlap);
    if (st != ZSP_OK) return st;
    if (overlap) return set_error(ZSP_EINVAL, "tensors to clip overlap");
    return for_each_launch(x, numel, dtype, n, [&](const TensorsLaunch& L) {
        return launch_list_clip(L, clip, static_cast<hipStream_t>(stream));
    });
}

zsp_status zsp_tensor_list_create(void* const* x, const int64_t* numel, const int32_t* dtype,
                                  int32_t n, void* stream, zsp_tensor_list** out) {
    using namespace zsp;
    if (!out) return set_error(ZSP_EINVAL, "list is NULL");
    *out = nullptr;
    int64_t nchunk = 0;
    bool overlap = false;
    zsp_status st = check_tensors(x, numel, dtype, n, &nchunk);
    if (st == ZSP_OK) st = find_overlap(x, numel, dtype, n, &overlap);
    if (st != ZSP_OK) return st;
    std::vector<ListChunk> host;
    try {
        host.reserve(size_t(nchunk));
    } catch (const std::bad_alloc&) {
        return set_error(ZSP_ENOMEM, "out of host memory (%lld chunks)", (long long)nchunk);
    }
    for (int32_t i = 0; i < n; ++i)
        for (int64_t at = 0; at < numel[i]; at += chunk_elems(dtype[i]))
            host.push_back(ListChunk{static_cast<char*>(x[i]) + at * size_of(dtype[i]),
                                     int32_t(std::min(chunk_elems(dtype[i]), numel[i] - at)),
                                     dtype[i]});
    zsp_tensor_list* L = new (std::nothrow) zsp_tensor_list();
    if (!L) return set_error(ZSP_ENOMEM, "out of host memory");
    L->nchunk = nchunk;
    L->overlap = overlap;
    hipError_t e = hipGetDevice(&L->device);
    if (e != hipSuccess) {
        delete L;
        return set_hip_error(e, "hipGetDevice");
    }
    if (nchunk > 0) {
        const size_t bytes = size_t(nchunk) * sizeof(ListChunk);
        void* dev = nullptr;
        if ((e = hipMalloc(&dev, bytes)) != hipSuccess) {
            delete L;
            return set_error(ZSP_ENOMEM, "device list of %zu bytes: %s", bytes,
                             hip_error_text(e));
        }
        const hipStream_t hs = static_cast<hipStream_t>(stream);
        e = hipMemcpyAsync(dev, host.data(), bytes, hipMemcpyHostToDevice, hs);
        // the host table, and calls on any stream, wait for the copy
        const hipError_t e2 = hipStreamSynchronize(hs);
        if (e == hipSuccess) e = e2;
        if (e != hipSuccess) {
            (void)hipFree(dev);
            delete L;
            return set_hip_error(e, "list copy");
        }
        L->dev = static_cast<ListChunk*>(dev);
    }
    *out = L;
    return ZSP_OK;
}

zsp_status zsp_tensor_list_norm(const zsp_tensor_list* list, zsp_norm_kind kind, double max_norm,
                                void* ws, int64_t ws_bytes, zsp_clip* out, void* stream) {
    using namespace zsp;
    const NormCall nc{kind, max_norm, ws, ws_bytes, out};
    zsp_status st = check_device(list);
    if (st == ZSP_OK) st = check_norm(nc, norm_parts(0, 0));
    if (st != ZSP_OK) return st;
    const hipStream_t hs = static_cast<hipStream_t>(stream);
    TensorsLaunch L;
    L.chunks = list->dev;
    L.nchunk = list->nchunk;
    int64_t nparts = 0;
    const bool one = list_norm_is_small(L.nchunk);
    const hipError_t e =
        one ? launch_list_norm_one(L, kind, max_norm, out, hs)
            : launch_list_norm(L, kind, static_cast<double*>(ws), &nparts, hs);
    if (e != hipSuccess) return set_hip_error(e, "tensor list launch");
    return one ? ZSP_OK : finish(nc, nparts, hs);
}

zsp_status zsp_tensor_list_clip(const zsp_tensor_list* list, const zsp_clip* clip, void* stream) {
    using namespace zsp;
    zsp_status st = check_device(list);
    if (st == ZSP_OK) st = check_clip(clip, "clip");
    if (st != ZSP_OK) return st;
    if (list->overlap) return set_error(ZSP_EINVAL, "tensors to clip overlap");
    TensorsLaunch L;
    L.chunks = list->dev;
    L.nchunk = list->nchunk;
    const hipError_t e = launch_list_clip(L, clip, static_cast<hipStream_t>(stream));
    if (e != hipSuccess) return set_hip_error(e, "tensor list launch");
    return ZSP_OK;
}

void zsp_tensor_list_destroy(zsp_tensor_list* list) {
    if (!list) return;
    if (list->dev) (void)hipFree(list->dev);
    delete list;
}

}  // extern "C"
