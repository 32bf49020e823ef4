// Element access shared by the router, the row moves and the norm.
#pragma once

#include <cstdint>

#include "../../include/ccl.h"
#include "ccl_tensor.cuh"

namespace ccl {
namespace tensor {

// Element types by their CCL_* code: Bytes per element, elements of 16 bytes,
// conversions from and to 32 bits.
template <int T>
struct Type;
template <>
struct Type<CCL_F32> {
    typedef float Raw;
    static constexpr int kVec = 4;
    static __device__ __forceinline__ float load(const Raw* p) { return *p; }
    static __device__ __forceinline__ void store(Raw* p, float v) { *p = v; }
    static __device__ __forceinline__ void unpack(const uint4& u, float* v)
    {
        v[0] = __uint_as_float(u.x), v[1] = __uint_as_float(u.y), v[2] = __uint_as_float(u.z), v[3] = __uint_as_float(u.w);
    }
    static __device__ __forceinline__ uint4 pack(const float* v)
    {
        return make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
    }
};
template <bool BF>
struct Type16 {
    typedef uint16_t Raw;
    static constexpr int kVec = 8;
    static __device__ __forceinline__ float load(const Raw* p) { return load1(p, BF); }
    static __device__ __forceinline__ void store(Raw* p, float v) { store1(p, v, BF); }
    static __device__ __forceinline__ void unpack(const uint4& u, float* v) { unpack8(u, BF, v); }
    static __device__ __forceinline__ uint4 pack(const float* v)
    {
        return make_uint4(pack2<BF>(v[0], v[1]), pack2<BF>(v[2], v[3]), pack2<BF>(v[4], v[5]), pack2<BF>(v[6], v[7]));
    }
};
template <>
struct Type<CCL_BF16> : Type16<true> {};
template <>
struct Type<CCL_F16> : Type16<false> {};

__device__ __forceinline__ float warp_sum(float v)
{
#pragma unroll
    for (int d = 16; d; d >>= 1) v += __shfl_xor_sync(~0u, v, d);
    return v;
}
__device__ __forceinline__ float warp_max(float v)       // NaN counts for nothing
{
    float r;
    asm("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
    return r;
}

}  // namespace tensor
}  // namespace ccl
