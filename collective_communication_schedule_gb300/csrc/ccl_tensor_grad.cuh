// The activation's gradient with its column sums, for the gradients of linear layers.
#pragma once

#include "ccl_tensor_passes.cuh"

namespace ccl {
namespace tensor {

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

}  // namespace tensor
}  // namespace ccl
