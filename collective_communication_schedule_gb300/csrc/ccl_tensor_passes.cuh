// Elementwise passes beside the tensor products: the activation's gradient
// with its column sums, and copies of matrices that TMA cannot address.
#pragma once

#include <cstdint>

#include "ccl_internal.h"
#include "ccl_tensor.cuh"

namespace ccl {
namespace tensor {

// [0]: a ccl_status_t of a failed launch on this device, 0 if none
__device__ int g_status[4];

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

// dz = dy * act'(z), and the column sums of dz that make the bias gradient.
// A threadblock takes 256 columns of up to kGradRows rows of one expert
// (dense: one expert with all rows); 32 threads cover the columns, 8 each,
// and 8 groups of threads take 4 rows each, all loads ahead of the
// arithmetic.  Bound by DRAM, 6 bytes an element: 4096 x 4096 with gelu in 20 us
// (5.0 TB/s; 35 us with the loads of two rows at a time).  Rows that 16-byte loads
// cannot address are read 32 neighbouring elements at a time instead.  The
// sums go, in 32 bits and a fixed order, to partial[chunk][column]; an
// expert's chunks are added up in order afterwards.  Chunks of expert e start
// at offsets[e] / kGradRows + e, which leaves every expert room for its rows.
__global__ void __launch_bounds__(256) act_grad_kernel(const GradPass G)
{
    __shared__ float sums[8][256 + 8];
    let_next_in();
    wait_for_previous();
    // the last expert whose first chunk is at or before this one (first chunks strictly increase)
    const int chunk = blockIdx.x;
    int e = 0, lo, len;
    if (G.offsets) {
        int a = 0, b = G.groups - 1;
        while (a < b) {
            const int mid = (a + b + 1) >> 1;
            grad_range(G, mid, lo, len);
            if (chunk_base(G, mid, lo) <= chunk)
                a = mid;
            else
                b = mid - 1;
        }
        e = a;
    }
    grad_range(G, e, lo, len);
    const int64_t first = (chunk - chunk_base(G, e, lo)) * kGradRows;
    if (first < 0 || first >= len) return;
    constexpr int kRows = kGradRows / 8;
    const int nrows = (int)min((int64_t)kGradRows, len - first);
    const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5, col = blockIdx.y * 256;
    const int64_t row0 = lo + first + ty;
    if (G.vec) {
        const int c = col + tx * 8;
        float sum[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        if (c < G.n) {              // n is a multiple of 8
            uint4 y[kRows], z[kRows];
#pragma unroll
            for (int j = 0; j < kRows; ++j)
                if (ty + 8 * j < nrows) {
                    y[j] = *reinterpret_cast<const uint4*>(G.dy + (row0 + 8 * j) * G.ld_dy + c);
                    if (G.act) z[j] = *reinterpret_cast<const uint4*>(G.z + (row0 + 8 * j) * G.ld_z + c);
                }
#pragma unroll
            for (int j = 0; j < kRows; ++j)
                if (ty + 8 * j < nrows) {
                    float v[8];
                    unpack8(y[j], G.bf, v);
                    if (G.act) {
                        float w[8];
                        unpack8(z[j], G.bf, w);
#pragma unroll
                        for (int i = 0; i < 8; ++i) v[i] *= activate_grad(w[i], G.act);
                    }
                    if (G.dz) store8(G.dz + (row0 + 8 * j) * G.ld_dz + c, G.bf, 8, v);
#pragma unroll
                    for (int i = 0; i < 8; ++i) sum[i] += v[i];
                }
        }
        if (G.partial) {
#pragma unroll
            for (int i = 0; i < 8; ++i) sums[ty][tx * 8 + i] = sum[i];
        }
    } else {
#pragma unroll 1
        for (int i = 0; i < 8; ++i) {
            const int c = col + i * 32 + tx;
            float sum = 0.f;
            if (c < G.n) {
                float y[kRows], z[kRows];
#pragma unroll
                for (int j = 0; j < kRows; ++j)
                    if (ty + 8 * j < nrows) {
                        y[j] = load1(G.dy + (row0 + 8 * j) * G.ld_dy + c, G.bf);
                        if (G.act) z[j] = load1(G.z + (row0 + 8 * j) * G.ld_z + c, G.bf);
                    }
#pragma unroll
                for (int j = 0; j < kRows; ++j)
                    if (ty + 8 * j < nrows) {
                        if (G.act) y[j] *= activate_grad(z[j], G.act);
                        if (G.dz) store1(G.dz + (row0 + 8 * j) * G.ld_dz + c, y[j], G.bf);
                        sum += y[j];
                    }
            }
            if (G.partial) sums[ty][i * 32 + tx] = sum;
        }
    }
    if (!G.partial) return;
    __syncthreads();
    const int c = col + threadIdx.x;
    if (c < G.n) {
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) s += sums[i][threadIdx.x];
        G.partial[(int64_t)chunk * G.ld_part + c] = s;
    }
}

// 32 columns per threadblock; 8 groups of threads take an expert's chunks in
// turn, and their sums are added in order.
__global__ void __launch_bounds__(256) bias_grad_kernel(const GradPass G)
{
    __shared__ float sums[8][32];
    let_next_in();
    wait_for_previous();
    const int e = blockIdx.y, tx = threadIdx.x & 31, ty = threadIdx.x >> 5, c = blockIdx.x * 32 + tx;
    int lo, len;
    grad_range(G, e, lo, len);
    // (no product may follow that checks them)
    if (G.offsets && blockIdx.x == 0 && threadIdx.x == 0) check_offsets(G.offsets, e, G.rows);
    const int chunks = (len + kGradRows - 1) / kGradRows;
    float s = 0.f;
    if (c < G.n) {
        const float* p = G.partial + chunk_base(G, e, lo) * G.ld_part + c;
#pragma unroll 4
        for (int i = ty; i < chunks; i += 8) s += p[i * G.ld_part];
    }
    sums[ty][tx] = s;
    __syncthreads();
    if (ty == 0 && c < G.n) {
#pragma unroll
        for (int i = 1; i < 8; ++i) s += sums[i][tx];
        store1(G.db + e * G.bs_db + c, s, G.bf);
    }
}

// The same sums in the same order beside the products of a pair, 32 columns of
// one expert at a time.
__device__ __noinline__ void add_chunks(const GradPass& G, int lane)
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
__global__ void __launch_bounds__(256) pack_rows_kernel(const PackArgs a)
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
