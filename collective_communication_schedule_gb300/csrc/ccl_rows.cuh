// Rows of tokens to the places of their experts and back.
#pragma once

#include "ccl_layer_common.cuh"

namespace ccl {
namespace tensor {

// [0]: a ccl_status_t of a failed launch on this device, [1]: what it was (REPORT_*)
static __device__ int g_layer_status[4];

enum { REPORT_PLACE = 1, REPORT_EXPERT = 2 };

__device__ __forceinline__ void report(int what)
{
    if (atomicCAS(&g_layer_status[0], 0, (int)CCL_ERR_INVALID_ARG) == 0) g_layer_status[1] = what;
}

struct Moves {
    const void *x, *r, *residual;  // rows by token; rows by place; by token
    void* out;
    const int32_t* place;          // rows x k: where a choice's row lies, < 0 for none
    const float* weights;          // rows x k (null: 1)
    float* dweights;
    int64_t rows, count, h;
    int64_t ld_x, ld_r, ld_s, ld_out;
    int32_t k, chunks;             // chunks: pieces of a row
};

// the place of choice j of a row, -1 where there is none
__device__ __forceinline__ int64_t place_of(const Moves& M, int64_t row, int j)
{
    const int p = M.place[row * M.k + j];
    if (p >= M.count) {
        report(REPORT_PLACE);
        return -1;
    }
    return p;
}

// out[place[t, j]] = x[t].  A warp takes a piece of 64 loads of one token, two
// a lane, and writes it k times.  VEC: loads of 16 bytes, else of one element.
template <int T, bool VEC>
__global__ void __launch_bounds__(256) dispatch_kernel(const Moves M)
{
    typedef Type<T> E;
    typedef typename E::Raw Raw;
    constexpr int W = VEC ? E::kVec : 1;
    let_next_in();
    wait_for_previous();
    const int64_t item = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    const int64_t t = item / M.chunks;
    if (t >= M.rows) return;
    const int64_t c = ((item - t * M.chunks) * 64 + lane) * W;
    const Raw* x = (const Raw*)M.x + t * M.ld_x + c;
    uint4 v[2];
    Raw s[2];
#pragma unroll
    for (int i = 0; i < 2; ++i)
        if (c + i * 32 * W < M.h) {
            if (VEC)
                v[i] = *reinterpret_cast<const uint4*>(x + i * 32 * W);
            else
                s[i] = x[i * 32];
        }
    for (int j = 0; j < M.k; ++j) {
        const int64_t p = place_of(M, t, j);
        if (p < 0) continue;
        Raw* o = (Raw*)M.out + p * M.ld_out + c;
#pragma unroll
        for (int i = 0; i < 2; ++i)
            if (c + i * 32 * W < M.h) {
                if (VEC)
                    *reinterpret_cast<uint4*>(o + i * 32 * W) = v[i];
                else
                    o[i * 32] = s[i];
            }
    }
}

// y[t] = sum_j w[t, j] r[place[t, j]] (+ residual[t]), in 32 bits, j ascending.
template <int T, bool VEC>
__global__ void __launch_bounds__(256) combine_kernel(const Moves M)
{
    typedef Type<T> E;
    typedef typename E::Raw Raw;
    constexpr int W = VEC ? E::kVec : 1;
    let_next_in();
    wait_for_previous();
    const int64_t item = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    const int64_t t = item / M.chunks;
    if (t >= M.rows) return;
    const int64_t c = ((item - t * M.chunks) * 32 + lane) * W;
    const bool in = c < M.h;
    float acc[W] = {};
#pragma unroll 4
    for (int j = 0; j < M.k; ++j) {
        const int64_t p = place_of(M, t, j);
        if (p < 0 || !in) continue;
        const float w = M.weights ? M.weights[t * M.k + j] : 1.f;
        const Raw* r = (const Raw*)M.r + p * M.ld_r + c;
        float v[W];
        if (VEC)
            E::unpack(*reinterpret_cast<const uint4*>(r), v);
        else
            v[0] = E::load(r);
#pragma unroll
        for (int i = 0; i < W; ++i) acc[i] = fmaf(w, v[i], acc[i]);
    }
    if (!in) return;
    if (M.residual) {
        const Raw* r = (const Raw*)M.residual + t * M.ld_s + c;
        float v[W];
        if (VEC)
            E::unpack(*reinterpret_cast<const uint4*>(r), v);
        else
            v[0] = E::load(r);
#pragma unroll
        for (int i = 0; i < W; ++i) acc[i] += v[i];
    }
    Raw* o = (Raw*)M.out + t * M.ld_out + c;
    if (VEC)
        *reinterpret_cast<uint4*>(o) = E::pack(acc);
    else
        E::store(o, acc[0]);
}

// dr[place[t, j]] = w[t, j] dy[t],  dweights[t, j] = <dy[t], r[place[t, j]]>.
// A threadblock takes a token, a warp a choice; dy is read once from memory and
// by the other warps from L1.  x: dy, out: dr (either output may be null).
template <int T, bool VEC>
__global__ void __launch_bounds__(256) combine_grad_kernel(const Moves M)
{
    typedef Type<T> E;
    typedef typename E::Raw Raw;
    constexpr int W = VEC ? E::kVec : 1;
    let_next_in();
    wait_for_previous();
    const int lane = threadIdx.x & 31;
    const int64_t t = blockIdx.x;
    const Raw* dy = (const Raw*)M.x + t * M.ld_x;
    for (int j = threadIdx.x >> 5; j < M.k; j += blockDim.x >> 5) {
        const int64_t p = place_of(M, t, j);
        float dot = 0.f;
        if (p >= 0) {
            const float w = M.weights ? M.weights[t * M.k + j] : 1.f;
            const Raw* r = (const Raw*)M.r + p * M.ld_r;
            Raw* o = (Raw*)M.out + p * M.ld_out;
#pragma unroll 4
            for (int64_t c = lane * W; c < M.h; c += 32 * W) {
                float g[W], v[W];
                if (VEC) {
                    E::unpack(*reinterpret_cast<const uint4*>(dy + c), g);
                    if (M.dweights) E::unpack(*reinterpret_cast<const uint4*>(r + c), v);
                } else {
                    g[0] = E::load(dy + c);
                    if (M.dweights) v[0] = E::load(r + c);
                }
                if (M.dweights) {
#pragma unroll
                    for (int i = 0; i < W; ++i) dot = fmaf(g[i], v[i], dot);
                }
                if (M.out) {
#pragma unroll
                    for (int i = 0; i < W; ++i) g[i] *= w;
                    if (VEC)
                        *reinterpret_cast<uint4*>(o + c) = E::pack(g);
                    else
                        E::store(o + c, g[0]);
                }
            }
        }
        if (M.dweights) {
            dot = warp_sum(dot);
            if (lane == 0) M.dweights[t * M.k + j] = dot;
        }
    }
}

}  // namespace tensor
}  // namespace ccl
