// Layer norm over rows, and its gradients.
#pragma once

#include "ccl_layer_common.cuh"

namespace ccl {
namespace tensor {

struct Norm {
    const void *x, *dy, *w, *b;
    void *y, *dx, *dw, *db;
    float *mean, *rstd;            // outputs of the forward pass (may be null), inputs of the backward pass
    float* partial;                // blocks x 2 x n: sums of dw and db
    int64_t rows, n;
    int64_t ld_x, ld_y, ld_dy, ld_dx;
    int32_t blocks;                // of the backward pass
    float eps;
};

// Sum over the TPR threads of a row (all of them get it): a warp, or warps of
// a threadblock through shared memory.  buf: 32 floats a row.
template <int TPR>
__device__ __forceinline__ float row_sum(float v, float* buf, int tid)
{
    v = warp_sum(v);
    if (TPR == 32) return v;
    __syncthreads();
    if ((tid & 31) == 0) buf[tid >> 5] = v;
    __syncthreads();
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < TPR / 32; ++i) s += buf[i];
    return s;
}
template <int TPR>
__device__ __forceinline__ float2 row_sum2(float2 v, float2* buf, int tid)
{
    v.x = warp_sum(v.x);
    v.y = warp_sum(v.y);
    if (TPR == 32) return v;
    __syncthreads();
    if ((tid & 31) == 0) buf[tid >> 5] = v;
    __syncthreads();
    float2 s = make_float2(0.f, 0.f);
#pragma unroll
    for (int i = 0; i < TPR / 32; ++i) s.x += buf[i].x, s.y += buf[i].y;
    return s;
}

// W consecutive elements at p (VEC: 16 bytes), in 32 bits
template <typename E, bool VEC, int W>
__device__ __forceinline__ void read(const typename E::Raw* p, float* v)
{
    if (VEC && W == E::kVec) {
        E::unpack(*reinterpret_cast<const uint4*>(p), v);
    } else if (VEC && W == 8 && E::kVec == 4) {
        E::unpack(*reinterpret_cast<const uint4*>(p), v);
        E::unpack(*reinterpret_cast<const uint4*>(p + 4), v + 4);
    } else {
#pragma unroll
        for (int i = 0; i < W; ++i) v[i] = E::load(p + i);
    }
}
template <typename E, bool VEC, int W>
__device__ __forceinline__ void write(typename E::Raw* p, const float* v)
{
    if (VEC && W == E::kVec) {
        *reinterpret_cast<uint4*>(p) = E::pack(v);
    } else if (VEC && W == 8 && E::kVec == 4) {
        *reinterpret_cast<uint4*>(p) = E::pack(v);
        *reinterpret_cast<uint4*>(p + 4) = E::pack(v + 4);
    } else {
#pragma unroll
        for (int i = 0; i < W; ++i) E::store(p + i, v[i]);
    }
}

// A row in the registers of TPR threads, read once: y = (x - mean) rstd w + b
// with the variance summed over differences from the mean.  V pieces of 16
// bytes a thread (VEC) or of one element.
template <int T, int TW, int TPR, int V, bool VEC>
__global__ void __launch_bounds__(TPR < 128 ? 128 : TPR) norm_kernel_rows(const Norm N)
{
    typedef Type<T> E;
    typedef Type<TW> EW;
    constexpr int W = VEC ? E::kVec : 1;
    constexpr int kRows = TPR < 128 ? 128 / TPR : 1;
    __shared__ float buf[2][32];
    let_next_in();
    wait_for_previous();
    const int tid = threadIdx.x % TPR;
    const int64_t row = (int64_t)blockIdx.x * kRows + threadIdx.x / TPR;
    if (kRows > 1 && row >= N.rows) return;
    const typename E::Raw* x = (const typename E::Raw*)N.x + row * N.ld_x;
    float v[V][W];
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int64_t c = (int64_t)(i * TPR + tid) * W;
        if (c < N.n) {
            read<E, VEC, W>(x + c, v[i]);
        } else {
#pragma unroll
            for (int e = 0; e < W; ++e) v[i][e] = 0.f;
        }
    }
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
        for (int e = 0; e < W; ++e) s += v[i][e];
    const float inv = 1.f / (float)N.n;
    const float mean = row_sum<TPR>(s, buf[0], tid) * inv;
    s = 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i)
        if ((int64_t)(i * TPR + tid) * W < N.n) {
#pragma unroll
            for (int e = 0; e < W; ++e) {
                const float d = v[i][e] - mean;
                s = fmaf(d, d, s);
            }
        }
    const float rstd = 1.f / sqrtf(row_sum<TPR>(s, buf[1], tid) * inv + N.eps);
    if (tid == 0) {
        if (N.mean) N.mean[row] = mean;
        if (N.rstd) N.rstd[row] = rstd;
    }
    typename E::Raw* y = (typename E::Raw*)N.y + row * N.ld_y;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int64_t c = (int64_t)(i * TPR + tid) * W;
        if (c < N.n) {
            float o[W];
#pragma unroll
            for (int e = 0; e < W; ++e) o[e] = (v[i][e] - mean) * rstd;
            if (N.w) {
                float w[W];
                read<EW, VEC, W>((const typename EW::Raw*)N.w + c, w);
#pragma unroll
                for (int e = 0; e < W; ++e) o[e] *= w[e];
            }
            if (N.b) {
                float b[W];
                read<EW, VEC, W>((const typename EW::Raw*)N.b + c, b);
#pragma unroll
                for (int e = 0; e < W; ++e) o[e] += b[e];
            }
            write<E, VEC, W>(y + c, o);
        }
    }
}

// Rows too long for registers: three passes over the row, the second and third from L2.
template <int T, int TW>
__global__ void __launch_bounds__(1024) norm_kernel_long(const Norm N)
{
    typedef Type<T> E;
    typedef Type<TW> EW;
    __shared__ float buf[2][32];
    let_next_in();
    wait_for_previous();
    const int tid = threadIdx.x;
    const int64_t row = blockIdx.x;
    const typename E::Raw* x = (const typename E::Raw*)N.x + row * N.ld_x;
    float s = 0.f;
#pragma unroll 4
    for (int64_t c = tid; c < N.n; c += 1024) s += E::load(x + c);
    const float inv = 1.f / (float)N.n;
    const float mean = row_sum<1024>(s, buf[0], tid) * inv;
    s = 0.f;
#pragma unroll 4
    for (int64_t c = tid; c < N.n; c += 1024) {
        const float d = E::load(x + c) - mean;
        s = fmaf(d, d, s);
    }
    const float rstd = 1.f / sqrtf(row_sum<1024>(s, buf[1], tid) * inv + N.eps);
    if (tid == 0) {
        if (N.mean) N.mean[row] = mean;
        if (N.rstd) N.rstd[row] = rstd;
    }
    typename E::Raw* y = (typename E::Raw*)N.y + row * N.ld_y;
#pragma unroll 4
    for (int64_t c = tid; c < N.n; c += 1024) {
        float o = (E::load(x + c) - mean) * rstd;
        if (N.w) o *= EW::load((const typename EW::Raw*)N.w + c);
        if (N.b) o += EW::load((const typename EW::Raw*)N.b + c);
        E::store(y + c, o);
    }
}

// dx = rstd (g - mean(g) - xh mean(g xh)) with g = dy w, and, over this
// block's rows, the sums of dy xh and dy that make dw and db.  Blocks take rows
// in turn, TPR threads a row; sums stay in registers until the last row.
template <int T, int TW, int TPR, int V, bool VEC>
__global__ void __launch_bounds__(TPR < 256 ? 256 : TPR) norm_grad_kernel_rows(const Norm N)
{
    typedef Type<T> E;
    typedef Type<TW> EW;
    constexpr int W = VEC ? E::kVec : 1;
    constexpr int kThreadsHere = TPR < 256 ? 256 : TPR, kRows = kThreadsHere / TPR;
    __shared__ float2 buf[kRows][32];
    __shared__ float sums[kRows > 1 ? kRows : 1][kRows > 1 ? TPR * W : 1];
    let_next_in();
    wait_for_previous();
    const int tid = threadIdx.x % TPR, slot = threadIdx.x / TPR;
    const float inv = 1.f / (float)N.n;
    float w[V][W], dw[V][W], db[V][W];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int64_t c = (int64_t)(i * TPR + tid) * W;
#pragma unroll
        for (int e = 0; e < W; ++e) w[i][e] = 1.f, dw[i][e] = db[i][e] = 0.f;
        if (N.w && c < N.n) read<EW, VEC, W>((const typename EW::Raw*)N.w + c, w[i]);
    }
    for (int64_t first = (int64_t)blockIdx.x * kRows; first < N.rows; first += (int64_t)gridDim.x * kRows) {
        const int64_t row = first + slot;
        const bool live = row < N.rows;
        float x[V][W], g[V][W];
        float2 s = make_float2(0.f, 0.f);
        const float mean = live ? N.mean[row] : 0.f, rstd = live ? N.rstd[row] : 0.f;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int64_t c = (int64_t)(i * TPR + tid) * W;
            if (live && c < N.n) {
                read<E, VEC, W>((const typename E::Raw*)N.x + row * N.ld_x + c, x[i]);
                read<E, VEC, W>((const typename E::Raw*)N.dy + row * N.ld_dy + c, g[i]);
            } else {
#pragma unroll
                for (int e = 0; e < W; ++e) x[i][e] = mean, g[i][e] = 0.f;
            }
        }
#pragma unroll
        for (int i = 0; i < V; ++i)
#pragma unroll
            for (int e = 0; e < W; ++e) {
                x[i][e] = (x[i][e] - mean) * rstd;
                dw[i][e] = fmaf(g[i][e], x[i][e], dw[i][e]);
                db[i][e] += g[i][e];
                g[i][e] *= w[i][e];
                s.x += g[i][e];
                s.y = fmaf(g[i][e], x[i][e], s.y);
            }
        if (N.dx) {
            s = row_sum2<TPR>(s, buf[slot], tid);
            const float a = s.x * inv, b = s.y * inv;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const int64_t c = (int64_t)(i * TPR + tid) * W;
                if (live && c < N.n) {
                    float o[W];
#pragma unroll
                    for (int e = 0; e < W; ++e) o[e] = rstd * (g[i][e] - a - x[i][e] * b);
                    write<E, VEC, W>((typename E::Raw*)N.dx + row * N.ld_dx + c, o);
                }
            }
        }
    }
    if (!N.partial) return;
    float* out = N.partial + (int64_t)blockIdx.x * 2 * N.n;
#pragma unroll
    for (int which = 0; which < 2; ++which)
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int64_t c = (int64_t)(i * TPR + tid) * W;
            float v[W];
#pragma unroll
            for (int e = 0; e < W; ++e) v[e] = which ? db[i][e] : dw[i][e];
            if (kRows > 1) {
                __syncthreads();
#pragma unroll
                for (int e = 0; e < W; ++e) sums[slot][tid * W + e] = v[e];
                __syncthreads();
#pragma unroll
                for (int e = 0; e < W; ++e) {
                    v[e] = 0.f;
#pragma unroll
                    for (int r = 0; r < kRows; ++r) v[e] += sums[r][tid * W + e];
                }
            }
            if (slot == 0 && c < N.n) {
#pragma unroll
                for (int e = 0; e < W; ++e) out[which * N.n + c + e] = v[e];
            }
        }
}

// Rows too long for registers: dx of a row in two passes ...
template <int T, int TW>
__global__ void __launch_bounds__(1024) norm_grad_kernel_long(const Norm N)
{
    typedef Type<T> E;
    typedef Type<TW> EW;
    __shared__ float2 buf[32];
    let_next_in();
    wait_for_previous();
    const int tid = threadIdx.x;
    const int64_t row = blockIdx.x;
    const typename E::Raw *x = (const typename E::Raw*)N.x + row * N.ld_x, *dy = (const typename E::Raw*)N.dy + row * N.ld_dy;
    const typename EW::Raw* w = (const typename EW::Raw*)N.w;
    const float mean = N.mean[row], rstd = N.rstd[row], inv = 1.f / (float)N.n;
    float2 s = make_float2(0.f, 0.f);
#pragma unroll 4
    for (int64_t c = tid; c < N.n; c += 1024) {
        const float g = E::load(dy + c) * (w ? EW::load(w + c) : 1.f);
        s.x += g;
        s.y = fmaf(g, (E::load(x + c) - mean) * rstd, s.y);
    }
    s = row_sum2<1024>(s, buf, tid);
    const float a = s.x * inv, b = s.y * inv;
    typename E::Raw* dx = (typename E::Raw*)N.dx + row * N.ld_dx;
#pragma unroll 4
    for (int64_t c = tid; c < N.n; c += 1024) {
        const float g = E::load(dy + c) * (w ? EW::load(w + c) : 1.f);
        E::store(dx + c, rstd * (g - a - (E::load(x + c) - mean) * rstd * b));
    }
}
// ... and the sums of dw and db, a column a thread, rows of a block in turn.
template <int T>
__global__ void __launch_bounds__(256) norm_sums_kernel_long(const Norm N)
{
    typedef Type<T> E;
    let_next_in();
    wait_for_previous();
    const int64_t c = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (c >= N.n) return;
    float dw = 0.f, db = 0.f;
#pragma unroll 4
    for (int64_t row = blockIdx.y; row < N.rows; row += gridDim.y) {
        const float g = E::load((const typename E::Raw*)N.dy + row * N.ld_dy + c);
        const float xh = (E::load((const typename E::Raw*)N.x + row * N.ld_x + c) - N.mean[row]) * N.rstd[row];
        dw = fmaf(g, xh, dw);
        db += g;
    }
    float* out = N.partial + (int64_t)blockIdx.y * 2 * N.n;
    out[c] = dw;
    out[N.n + c] = db;
}

// The blocks' sums added up in order: 32 columns a threadblock, 16 groups of
// threads take the blocks in turn.  blockIdx.y: dw, db.
template <int TW>
__global__ void __launch_bounds__(512) norm_sums_kernel(const Norm N)
{
    typedef Type<TW> EW;
    __shared__ float sums[16][32];
    let_next_in();
    wait_for_previous();
    const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
    const int64_t c = (int64_t)blockIdx.x * 32 + tx;
    typename EW::Raw* out = (typename EW::Raw*)(blockIdx.y ? N.db : N.dw);
    if (!out) return;
    float s = 0.f;
    if (c < N.n) {
        const float* p = N.partial + blockIdx.y * N.n + c;
#pragma unroll 8
        for (int i = ty; i < N.blocks; i += 16) s += p[(int64_t)i * 2 * N.n];
    }
    sums[ty][tx] = s;
    __syncthreads();
    if (ty == 0 && c < N.n) {
#pragma unroll
        for (int i = 1; i < 16; ++i) s += sums[i][tx];
        EW::store(out + c, s);
    }
}

}  // namespace tensor
}  // namespace ccl
