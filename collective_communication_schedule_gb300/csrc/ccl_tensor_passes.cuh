// Elementwise passes beside the tensor products: what all users of the products
// share of the activation's gradient, and copies of matrices that TMA cannot address.
#pragma once

#include <cstdint>

#include "ccl_internal.h"
#include "ccl_tensor.cuh"

namespace ccl {
namespace tensor {

// [0]: a ccl_status_t of a failed launch on this device, 0 if none.  Every translation
// unit has its own; ccl_tensor_status asks all of them.
static __device__ int g_status[4];

// An expert's offsets that decrease or leave the rows are reported, once.
__device__ __forceinline__ void check_offsets(const int32_t* offsets, int e, int rows)
{
    if (offsets[e] < 0 || offsets[e + 1] < offsets[e] || offsets[e + 1] > rows)
        atomicCAS(&g_status[0], 0, (int)CCL_ERR_INVALID_ARG);
}

// Rows of a partial column sum of the activation's gradient (act_grad_kernel).
constexpr int kGradRows = 32;

struct GradPass {
    const uint16_t *dy, *z;
    uint16_t* dz;                  // may be null (sums only)
    float* partial;                // may be null (no bias gradient)
    uint16_t* db;
    const int32_t* offsets;        // null: one expert with all rows
    int64_t ld_dy, ld_z, ld_dz, bs_db;
    int64_t ld_part;
    int32_t rows, n, groups, act, bf, vec;
};

__device__ __forceinline__ int64_t chunk_base(const GradPass& G, int e, int lo) { return lo / kGradRows + e; }

__device__ __forceinline__ void grad_range(const GradPass& G, int e, int& lo, int& len)
{
    lo = 0;
    len = G.rows;
    if (G.offsets) {
        lo = min(max(G.offsets[e], 0), G.rows);
        len = min(max(G.offsets[e + 1], lo), G.rows) - lo;
    }
}

// The sums of bias_grad_kernel in its order beside the products of a pair, 32 columns
// of one expert at a time.
[[maybe_unused]] static __device__ __noinline__ void add_chunks(const GradPass& G, int lane)
{
    const int columns = (G.n + 31) / 32;
    for (int item = blockIdx.x; item < G.groups * columns; item += gridDim.x) {
        const int e = item / columns, c = item % columns * 32 + lane;
        int lo, len;
        grad_range(G, e, lo, len);
        if (c >= G.n) continue;
        const int chunks = (len + kGradRows - 1) / kGradRows;
        const float* p = G.partial + chunk_base(G, e, lo) * G.ld_part + c;
        float s[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        int i = 0;
        for (; i + 8 <= chunks; i += 8)
#pragma unroll
            for (int j = 0; j < 8; ++j) s[j] += p[(i + j) * G.ld_part];
#pragma unroll
        for (int j = 0; j < 7; ++j)
            if (i + j < chunks) s[j] += p[(i + j) * G.ld_part];
#pragma unroll
        for (int j = 1; j < 8; ++j) s[0] += s[j];
        store1(G.db + e * G.bs_db + c, s[0], G.bf);
    }
}

struct PackArgs {
    uint16_t* dst;
    const uint16_t* src;
    int64_t ld_dst, bs_dst, ld_src, bs_src, rows, cols;
};
// Copy a matrix whose base or row stride TMA cannot address (not a multiple
// of 16 bytes) into rows padded to 8 elements, 2 bytes a thread: a weight of 4096 x
// 4095 in 34 us (1.0 TB/s), three times what its product with one row takes.
static __global__ void __launch_bounds__(256) pack_rows_kernel(const PackArgs a)
{
    let_next_in();
    wait_for_previous();
    for (int64_t r = blockIdx.x; r < a.rows; r += gridDim.x) {
        const uint16_t* s = a.src + blockIdx.y * a.bs_src + r * a.ld_src;
        uint16_t* d = a.dst + blockIdx.y * a.bs_dst + r * a.ld_dst;
        for (int64_t i = threadIdx.x; i < a.cols; i += blockDim.x) d[i] = s[i];
    }
}

}  // namespace tensor
}  // namespace ccl
