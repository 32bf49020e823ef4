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
    float2* block;                 // by 8 rows: the largest factor; not 0 if a row that counts for nothing holds Inf or NaN
    int32_t* dirty;                // not 0 if one of all rows does
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

// A row's parts put together, in an order that the sizes fix:
// lse = m + log(sum), loss = log(sum) + (m - the target's value), which keeps
// the digits of a small loss.  8 rows a threadblock; 32 groups of threads take
// the parts in turn, a warp a row puts the groups' together.
static __global__ void __launch_bounds__(256) loss_kernel(const LossRows L)
{
    __shared__ float2 parts[32][9];
    let_next_in();
    wait_for_previous();
    const int tx = threadIdx.x & 7, ty = threadIdx.x >> 3, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t row = (int64_t)blockIdx.x * 8 + tx, mine = (int64_t)blockIdx.x * 8 + warp;
    const bool live = lane == 0 && mine < L.rows && target_of(L, mine) >= 0;
    const float picked = live ? L.picked[mine] : 0.f;
    float2 s = make_float2(-INFINITY, 0.f);
    if (row < L.rows) {
        for (int64_t t = ty; t < L.tiles; t += 256) {
            float2 p[8];
#pragma unroll
            for (int i = 0; i < 8; ++i)
                p[i] = t + i * 32 < L.tiles ? __ldcg(L.part + (t + i * 32) * L.rows + row) : make_float2(-INFINITY, 0.f);
#pragma unroll
            for (int n = 4; n; n /= 2)
#pragma unroll
                for (int i = 0; i < n; ++i) p[i] = join(p[i], p[i + n]);
            s = join(s, p[0]);
        }
    }
    parts[ty][tx] = s;
    __syncthreads();
    s = parts[lane][warp];
#pragma unroll
    for (int d = 16; d; d /= 2) s = join(s, make_float2(__shfl_xor_sync(~0u, s.x, d), __shfl_xor_sync(~0u, s.y, d)));
    if (lane == 0 && mine < L.rows) {
        const float l = logf(s.y);
        L.loss[mine] = live ? l + (s.x - picked) : 0.f;
        if (L.lse) L.lse[mine] = live ? s.x + l : 0.f;
    }
}

// A row's coefficients for the products' epilogue, a warp a row, whether a row
// that counts for nothing holds Inf or NaN (0 times which would reach dw), and the
// largest factor of 8 rows.  This and the next kernel are launch and latency, about 2 us
// each of a backward pass.
static __global__ void __launch_bounds__(256) loss_rows_kernel(const LossRows L)
{
    __shared__ float2 found[8];
    let_next_in();
    wait_for_previous();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t row = (int64_t)blockIdx.x * 8 + warp;
    float most = 0.f;
    bool bad = false;
    if (row < L.rows) {
        const int64_t t = target_of(L, row);
        const float b = t < 0 ? 0.f : L.dloss[row], a = t >= 0 && L.dlse ? b + L.dlse[row] : b;
        if (lane == 0) L.coef[row] = make_float4(t < 0 ? 0.f : L.lse_in[row], a, b, __int_as_float(t < 0 ? -1 : (int)t));
        if (fabsf(a) < INFINITY) most = fabsf(a);
        if (fabsf(b) < INFINITY) most = fmaxf(most, fabsf(b));
        if (L.x && a == 0.f && b == 0.f) {
            // (x is in rows on 16 bytes here)
            const uint16_t* x = L.x + row * L.ld_x;
#pragma unroll 4
            for (int64_t c = lane * 8; c < L.k; c += 256) {
                float v[8];
                load8(x + c, !L.f16, (int)min((int64_t)8, L.k - c), v);
#pragma unroll
                for (int i = 0; i < 8; ++i) bad |= !(fabsf(v[i]) < INFINITY);
            }
        }
    }
    bad = __any_sync(~0u, bad);
    if (lane == 0) found[warp] = make_float2(most, bad ? 1.f : 0.f);
    __syncthreads();
    if (threadIdx.x == 0) {
        float2 all = found[0];
        for (int i = 1; i < 8; ++i) all.x = fmaxf(all.x, found[i].x), all.y = fmaxf(all.y, found[i].y);
        L.block[blockIdx.x] = all;
    }
}

// What the products are told of all rows: for f16 the scale that brings the
// largest factor to below 2^14 (sums of two below 2^15; f16 then holds what is
// 2^-38 of it to half a unit), and whether x is to be read without the rows that
// count for nothing, which is written here where one of them is dirty.
static __global__ void __launch_bounds__(256) loss_ready_kernel(const LossRows L)
{
    __shared__ float2 found[8];
    let_next_in();
    wait_for_previous();
    float2 all = make_float2(0.f, 0.f);
    const int64_t blocks = (L.rows + 7) / 8;
#pragma unroll 8
    for (int64_t i = threadIdx.x; i < blocks; i += 256) {
        const float2 b = L.block[i];
        all.x = fmaxf(all.x, b.x);
        all.y = fmaxf(all.y, b.y);
    }
#pragma unroll
    for (int d = 16; d; d >>= 1) {
        all.x = fmaxf(all.x, __shfl_xor_sync(~0u, all.x, d));
        all.y = fmaxf(all.y, __shfl_xor_sync(~0u, all.y, d));
    }
    if ((threadIdx.x & 31) == 0) found[threadIdx.x >> 5] = all;
    __syncthreads();
    for (int i = 0; i < 8; ++i) all.x = fmaxf(all.x, found[i].x), all.y = fmaxf(all.y, found[i].y);
    const bool dirty = all.y != 0.f;
    if (blockIdx.x == 0 && threadIdx.x == 0) {
        int e = 0;
        if (all.x > 0.f) frexpf(all.x, &e);    // the largest factor < 2^e
        const int shift = L.f16 && all.x > 0.f ? max(-100, min(100, 14 - e)) : 0;
        L.scale[0] = ldexpf(1.f, shift);
        L.scale[1] = ldexpf(1.f, -shift);
        *L.dirty = dirty;
    }
    if (!dirty) return;
    for (int64_t row = blockIdx.x; row < L.rows; row += gridDim.x) {
        const float4 k = L.coef[row];
        const bool dead = k.y == 0.f && k.z == 0.f;
        for (int64_t c = threadIdx.x; c < L.k; c += 256)
            L.clean[row * L.ld_clean + c] = dead ? (uint16_t)0 : L.x[row * L.ld_x + c];
    }
}

// dx from its parts, which the segments of the vocabulary left, added up in order:
// mostly from L2 (777 x 1032 in 12 parts 3 us).
struct LossSum {
    const float* sum;
    uint16_t* dx;
    int64_t rows, k, ld_sum, bs_sum, ld_dx;
    int32_t parts, bf;
};
static __global__ void __launch_bounds__(256) loss_sum_kernel(const LossSum L)
{
    let_next_in();
    wait_for_previous();
    // (rows of the parts are on 16 bytes and padded)
    const int64_t quads = (L.k + 3) / 4, i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= L.rows * quads) return;
    const int64_t row = i / quads, c = (i - row * quads) * 4;
    const float4* p = reinterpret_cast<const float4*>(L.sum + row * L.ld_sum + c);
    float4 v = __ldcg(p);
#pragma unroll 4
    for (int s = 1; s < L.parts; ++s) {
        const float4 u = __ldcg(p + s * (L.bs_sum / 4));
        v.x += u.x, v.y += u.y, v.z += u.z, v.w += u.w;
    }
    uint16_t* o = L.dx + row * L.ld_dx + c;
    const float f[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int e = 0; e < 4; ++e)
        if (c + e < L.k) store1(o + e, f[e], L.bf);
}

}  // namespace tensor
}  // namespace ccl
