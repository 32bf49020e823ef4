// Host side of the layer operators: launches, workspaces, checks of arguments.
#pragma once

#include <algorithm>
#include <initializer_list>
#include <new>
#include <string>

#include <cuda_runtime.h>

#include "ccl_internal.h"

namespace ccl {
namespace tensor {

#define TRY_CUDA(call, what)                                                                                   \
    do {                                                                                                       \
        cudaError_t e_ = (call);                                                                               \
        if (e_ != cudaSuccess)                                                                                 \
            return fail(e_ == cudaErrorMemoryAllocation ? CCL_ERR_OOM : CCL_ERR_CUDA,                          \
                        std::string(what) + ": " + cudaGetErrorString(e_));                                    \
    } while (0)
#define TRY(call)                                 \
    do {                                          \
        ccl_status_t s_ = (call);                 \
        if (s_ != CCL_OK) return s_;              \
    } while (0)

// what the router and the row moves, then the cross entropy, have reported on this device (and take it back)
ccl_status_t take_layer_status();
ccl_status_t take_loss_status();

inline int64_t round_up(int64_t v, int64_t m) { return (v + m - 1) / m * m; }
inline bool aligned16(const void* p) { return ((uintptr_t)p & 15) == 0; }

template <typename Arg>
inline ccl_status_t launch(void (*kernel)(const Arg), dim3 grid, int threads, size_t smem, cudaStream_t stream, const Arg& arg,
                           int cluster = 1)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = (unsigned)cluster;
    at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    TRY_CUDA(cudaLaunchKernelEx(&cfg, kernel, arg), "launch");
    return CCL_OK;
}

// Bump allocation from the caller's workspace (a null base only measures).
struct Arena {
    char* base;
    int64_t used = 0;
    template <typename T>
    T* take(int64_t bytes)
    {
        T* p = base ? reinterpret_cast<T*>(base + used) : nullptr;
        used += round_up(bytes, 256);
        return p;
    }
};

inline bool vectors(const void* p, int64_t ld, int64_t bs) { return aligned16(p) && ld % 8 == 0 && bs % 8 == 0; }

// A stride given as 0 means packed; one below the row's length would make rows overlap.
inline ccl_status_t stride(const char* what, int64_t given, int64_t least, int64_t* out)
{
    if (given != 0 && given < least)
        return fail(CCL_ERR_INVALID_ARG, std::string(what) + " stride " + std::to_string(given) + " below " +
                                             std::to_string(least));
    *out = given ? given : least;
    return CCL_OK;
}

inline ccl_status_t pointer(const char* what, const void* p, bool needed)
{
    if (needed && !p) return fail(CCL_ERR_INVALID_ARG, std::string(what) + " is null");
    if ((uintptr_t)p & 1) return fail(CCL_ERR_INVALID_ARG, std::string(what) + " is not aligned to its elements");
    return CCL_OK;
}

// Whether an output that is asked for starts where one of these does.
inline bool same(const void* out, std::initializer_list<const void*> others)
{
    return out && std::find(others.begin(), others.end(), out) != others.end();
}

template <typename Args>
inline ccl_status_t guarded(ccl_status_t (*fn)(const Args*, char*, int64_t*, cudaStream_t), const Args* a, void* ws,
                            int64_t ws_bytes, void* stream)
{
    int64_t need = 0;
    TRY(fn(a, nullptr, &need, nullptr));
    if (need > 0 && (!ws || ws_bytes < need))
        return fail(CCL_ERR_INVALID_ARG, "workspace of " + std::to_string(need) + " bytes needed, " +
                                             std::to_string(ws ? ws_bytes : 0) + " given");
    if (need > 0 && ((uintptr_t)ws & 255)) return fail(CCL_ERR_INVALID_ARG, "workspace not aligned to 256 bytes");
    return fn(a, (char*)ws, nullptr, (cudaStream_t)stream);
}

template <typename Args>
inline ccl_status_t measured(ccl_status_t (*fn)(const Args*, char*, int64_t*, cudaStream_t), const Args* a, int64_t* out)
{
    if (!out) return fail(CCL_ERR_INVALID_ARG, "null size");
    int64_t need = 0;
    TRY(fn(a, nullptr, &need, nullptr));
    *out = need;
    return CCL_OK;
}

}  // namespace tensor
}  // namespace ccl

// no exception leaves the library
#define C_ENTRY(...)                                                     \
    try {                                                                \
        return (__VA_ARGS__);                                            \
    } catch (const std::bad_alloc&) {                                    \
        return CCL_ERR_OOM;                                              \
    } catch (...) {                                                      \
        return CCL_ERR_INTERNAL;                                         \
    }
