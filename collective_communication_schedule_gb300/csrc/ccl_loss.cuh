// Passes around the products of the cross entropy.
#pragma once

#include "ccl_tensor_passes.cuh"
#include "ccl_tensor_product.cuh"

namespace ccl {
namespace tensor {

struct LossRows {
    const void* target;
    int64_t ignore;
    int64_t rows, vocab;
    int32_t wide;
    // forward: the tiles' parts, the targets' values
    const float2* part;
    const float* picked;
    float *loss, *lse;
    int64_t tiles;
    // backward
    const float *dloss, *dlse, *lse_in;
    float4* coef;
    float* scale;                  // [0]: of the derivatives (a power of two), [1]: its inverse
    int32_t* dirty;                // not 0: a row that counts for nothing holds Inf or NaN
    const uint16_t* x;             // null: nobody asks
    uint16_t* clean;
    int64_t ld_x, ld_clean, k;
    int32_t f16;
};

// A row's target, -1 where it counts for nothing; one that is neither is reported.
__device__ __forceinline__ int64_t target_of(const LossRows& L, int64_t row)
{
    const int64_t t = L.wide ? ((const int64_t*)L.target)[row] : ((const int32_t*)L.target)[row];
    if (t == L.ignore) return -1;
    if (t < 0 || t >= L.vocab) {
        atomicCAS(&g_status[0], 0, (int)CCL_ERR_INVALID_ARG);
        return -1;
    }
    return t;
}

// The parts of a row's tiles put together, in an order that the sizes fix:
// lse = m + log(sum), loss = log(sum) + (m - the target's value), which keeps
// the digits of a small loss.  32 rows a threadblock; 16 groups of threads take
// the tiles in turn.
static __global__ void __launch_bounds__(512) loss_kernel(const LossRows L)
{
    __shared__ float2 parts[16][32];
    let_next_in();
    wait_for_previous();
    const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
    const int64_t row = (int64_t)blockIdx.x * 32 + tx;
    float2 s = make_float2(-INFINITY, 0.f);
    if (row < L.rows) {
        for (int64_t t = ty; t < L.tiles; t += 64) {
            float2 p[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                p[i] = t + i * 16 < L.tiles ? L.part[(t + i * 16) * L.rows + row] : make_float2(-INFINITY, 0.f);
#pragma unroll
            for (int i = 0; i < 4; ++i) s = join(s, p[i]);
        }
    }
    parts[ty][tx] = s;
    __syncthreads();
    if (ty == 0 && row < L.rows) {
#pragma unroll
        for (int i = 1; i < 16; ++i) s = join(s, parts[i][tx]);
        float loss = 0.f, lse = 0.f;
        if (target_of(L, row) >= 0) {
            const float l = logf(s.y);
            loss = l + (s.x - L.picked[row]);
            lse = s.x + l;
        }
        L.loss[row] = loss;
        if (L.lse) L.lse[row] = lse;
    }
}

// Before a backward pass, one threadblock: no row is known to be dirty, and for
// f16 the scale that brings the largest factor of a row to below 2^14 (sums of
// two below 2^15; f16 then holds what is 2^-38 of it to half a unit).
static __global__ void __launch_bounds__(1024) loss_scale_kernel(const LossRows L)
{
    __shared__ float most[32];
    let_next_in();
    wait_for_previous();
    float m = 0.f;
    if (L.f16)
        for (int64_t row = threadIdx.x; row < L.rows; row += 1024) {
            if (target_of(L, row) < 0) continue;
            const float b = L.dloss[row], a = L.dlse ? b + L.dlse[row] : b;
            if (fabsf(a) < INFINITY) m = fmaxf(m, fabsf(a));
            if (fabsf(b) < INFINITY) m = fmaxf(m, fabsf(b));
        }
#pragma unroll
    for (int d = 16; d; d >>= 1) m = fmaxf(m, __shfl_xor_sync(~0u, m, d));
    if ((threadIdx.x & 31) == 0) most[threadIdx.x >> 5] = m;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int i = 1; i < 32; ++i) m = fmaxf(m, most[i]);
        int e = 0;
        if (m > 0.f) frexpf(m, &e);            // m < 2^e
        const int shift = L.f16 && m > 0.f ? max(-100, min(100, 14 - e)) : 0;
        L.scale[0] = ldexpf(1.f, shift);
        L.scale[1] = ldexpf(1.f, -shift);
        *L.dirty = 0;
    }
}

// A row's coefficients for the products' epilogue, a warp a row, and whether a
// row that counts for nothing holds Inf or NaN (0 times which would reach dw).
static __global__ void __launch_bounds__(256) loss_rows_kernel(const LossRows L)
{
    let_next_in();
    wait_for_previous();
    const int lane = threadIdx.x & 31;
    const int64_t row = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
    if (row >= L.rows) return;
    const int64_t t = target_of(L, row);
    const float b = t < 0 ? 0.f : L.dloss[row], a = t >= 0 && L.dlse ? b + L.dlse[row] : b;
    if (lane == 0) {
        const float s = L.scale[0];
        L.coef[row] = make_float4(t < 0 ? 0.f : L.lse_in[row], a * s, b * s,
                                  __int_as_float(t < 0 ? -1 : (int)t));
    }
    if (L.x && a == 0.f && b == 0.f) {
        bool bad = false;
        for (int64_t c = lane; c < L.k; c += 32) {
            const float v = load1(L.x + row * L.ld_x + c, !L.f16);
            bad |= !(fabsf(v) < INFINITY);
        }
        if (bad) *L.dirty = 1;
    }
}

// x without the rows that count for nothing, where one of them is dirty.
static __global__ void __launch_bounds__(256) loss_clean_kernel(const LossRows L)
{
    let_next_in();
    wait_for_previous();
    if (!*L.dirty) return;
    for (int64_t row = blockIdx.x; row < L.rows; row += gridDim.x) {
        const float4 k = L.coef[row];
        const bool dead = k.y == 0.f && k.z == 0.f;
        for (int64_t c = threadIdx.x; c < L.k; c += 256)
            L.clean[row * L.ld_clean + c] = dead ? (uint16_t)0 : L.x[row * L.ld_x + c];
    }
}

}  // namespace tensor
}  // namespace ccl
