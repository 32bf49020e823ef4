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

// A lane's pieces of a row: VEC: one of 16 bytes, else 8 elements 32 apart.
// at: the first one's element, of h.
template <typename E, bool VEC>
struct Part {
    static constexpr int kSize = VEC ? E::kVec : 8;        // elements
    static constexpr int kWarp = 32 * kSize;               // of a warp
    uint4 u;
    typename E::Raw r[VEC ? 1 : 8];

    static __device__ __forceinline__ int first(int lane) { return VEC ? lane * E::kVec : lane; }
    __device__ __forceinline__ void load(const typename E::Raw* p, int64_t at, int64_t h)
    {
        if constexpr (VEC) {
            if (at < h) u = *reinterpret_cast<const uint4*>(p + at);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (at + i * 32 < h) r[i] = p[at + i * 32];
        }
    }
    // copied as it is
    __device__ __forceinline__ void store(typename E::Raw* p, int64_t at, int64_t h) const
    {
        if constexpr (VEC) {
            if (at < h) *reinterpret_cast<uint4*>(p + at) = u;
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (at + i * 32 < h) p[at + i * 32] = r[i];
        }
    }
    // in 32 bits (0 beyond the row)
    __device__ __forceinline__ void get(float (&v)[kSize], int64_t at, int64_t h) const
    {
        if constexpr (VEC) {
            if (at < h) {
                E::unpack(u, v);
            } else {
#pragma unroll
                for (int i = 0; i < kSize; ++i) v[i] = 0.f;
            }
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = at + i * 32 < h ? E::load(r + i) : 0.f;
        }
    }
    static __device__ __forceinline__ void put(typename E::Raw* p, const float (&v)[kSize], int64_t at, int64_t h)
    {
        if constexpr (VEC) {
            if (at < h) *reinterpret_cast<uint4*>(p + at) = E::pack(v);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (at + i * 32 < h) E::store(p + at + i * 32, v[i]);
        }
    }
};

// out[place[t, j]] = x[t].  A warp takes a part of a token (16 bytes a lane) and
// writes it k times; written bytes bound it.  8190 rows of 2048 bf16 to 4 places each:
// 26 us, 6.4 TB/s; 24 rows to 8 places 2.2 us.  Two parts a warp took as long at
// the large size, 14.4 us instead of 12.5 for 4096 rows of 1024 to 8 places and 14.7
// instead of 15.0 for 4097 rows of 1544 to 6.
template <int T, bool VEC>
__global__ void __launch_bounds__(256) dispatch_kernel(const Moves M)
{
    typedef Type<T> E;
    typedef typename E::Raw Raw;
    typedef Part<E, VEC> P;
    let_next_in();
    wait_for_previous();
    const int64_t item = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    const int64_t t = item / M.chunks;
    if (t >= M.rows) return;
    const int64_t c = (item - t * M.chunks) * P::kWarp + P::first(lane);
    P v;
    v.load((const Raw*)M.x + t * M.ld_x, c, M.h);
#pragma unroll 4
    for (int j = 0; j < M.k; ++j) {
        const int64_t p = place_of(M, t, j);
        if (p < 0) continue;
        v.store((Raw*)M.out + p * M.ld_out, c, M.h);
    }
}

// y[t] = sum_j w[t, j] r[place[t, j]] (+ residual[t]), in 32 bits, j ascending.  A
// warp takes a part of a token, its choices one after another (places and weights
// come from L1): the 32 registers of a thread do not hold the loads of four choices,
// and a choice without a place is a branch between two of them.  8190 rows of 2048 bf16
// from 4 places 33 us, 5.1 TB/s, where dispatch writes at 6.4: too few loads on their way.
// Few rows are bound by the chain of place, row and launch: 24 rows from 8 places 3.6 us.
template <int T, bool VEC>
__global__ void __launch_bounds__(256) combine_kernel(const Moves M)
{
    typedef Type<T> E;
    typedef typename E::Raw Raw;
    typedef Part<E, VEC> P;
    let_next_in();
    wait_for_previous();
    const int64_t item = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    const int64_t t = item / M.chunks;
    if (t >= M.rows) return;
    const int64_t c = (item - t * M.chunks) * P::kWarp + P::first(lane);
    float acc[P::kSize] = {};
#pragma unroll 4
    for (int j = 0; j < M.k; ++j) {
        const int64_t p = place_of(M, t, j);
        if (p < 0) continue;
        const float w = M.weights ? M.weights[t * M.k + j] : 1.f;
        P part;
        float v[P::kSize];
        part.load((const Raw*)M.r + p * M.ld_r, c, M.h);
        part.get(v, c, M.h);
#pragma unroll
        for (int i = 0; i < P::kSize; ++i) acc[i] = fmaf(w, v[i], acc[i]);
    }
    if (M.residual) {
        P part;
        float v[P::kSize];
        part.load((const Raw*)M.residual + t * M.ld_s, c, M.h);
        part.get(v, c, M.h);
#pragma unroll
        for (int i = 0; i < P::kSize; ++i) acc[i] += v[i];
    }
    P::put((Raw*)M.out + t * M.ld_out, acc, c, M.h);
}

// dr[place[t, j]] = w[t, j] dy[t],  dweights[t, j] = <dy[t], r[place[t, j]]>, for
// rows of up to 16 bytes a lane.  `across` lanes (a power of two) lie along a row, and
// take four choices with all loads on their way at a time: a warp a choice spends its
// time on the chain of place, row and sum (128000 choices of 128 bf16 15.6 us, 4.4
// TB/s, instead of 36).
template <int T>
__global__ void __launch_bounds__(256) combine_grad_short_kernel(const Moves M)
{
    typedef Type<T> E;
    typedef typename E::Raw Raw;
    constexpr int W = E::kVec, kEach = 4;
    let_next_in();
    wait_for_previous();
    const int across = M.chunks, lane = threadIdx.x & (across - 1), c = lane * W, h = (int)M.h;
    const int64_t all = M.rows * M.k, first = ((int64_t)blockIdx.x * 256 + threadIdx.x) / across * kEach;
    int64_t p[kEach];
    float w[kEach], dot[kEach];
    uint4 g[kEach], r[kEach];
#pragma unroll
    for (int q = 0; q < kEach; ++q) p[q] = first + q < all ? place_of(M, 0, (int)(first + q)) : -1;
#pragma unroll
    for (int q = 0; q < kEach; ++q) {
        dot[q] = 0.f;
        if (p[q] < 0) continue;
        w[q] = M.weights ? M.weights[first + q] : 1.f;
        if (c >= h) continue;
        g[q] = *reinterpret_cast<const uint4*>((const Raw*)M.x + (int)(first + q) / M.k * M.ld_x + c);
        if (M.dweights) r[q] = *reinterpret_cast<const uint4*>((const Raw*)M.r + p[q] * M.ld_r + c);
    }
#pragma unroll
    for (int q = 0; q < kEach; ++q) {
        if (p[q] < 0 || c >= h) continue;
        float a[W], b[W];
        E::unpack(g[q], a);
        if (M.dweights) {
            E::unpack(r[q], b);
#pragma unroll
            for (int i = 0; i < W; ++i) dot[q] = fmaf(a[i], b[i], dot[q]);
        }
        if (M.out) {
#pragma unroll
            for (int i = 0; i < W; ++i) a[i] *= w[q];
            *reinterpret_cast<uint4*>((Raw*)M.out + p[q] * M.ld_out + c) = E::pack(a);
        }
    }
    if (!M.dweights) return;
#pragma unroll
    for (int q = 0; q < kEach; ++q) {
        for (int d = across / 2; d; d /= 2) dot[q] += __shfl_xor_sync(~0u, dot[q], d);
        if (lane == 0 && first + q < all) M.dweights[first + q] = dot[q];
    }
}

// The same for rows of any length.  A warp takes a choice; neighbouring warps take choices of one token, whose dy is
// read once from memory and by the others from L1.  x: dy, out: dr (either output
// may be null).  8190 rows of 2048 bf16 at 4 places 54 us (5.6 TB/s).  dr may lie
// anywhere, so a step's loads wait for the stores of the step before, and with a step
// for less than a warp or choices without a place there is less on its way: f16, 4097
// rows at 6 places, 1536 wide (6 steps) 32.5 us (5.0 TB/s), 1544 (a seventh for one lane)
// 34.6 (4.8), and with a fifth of the places none 28.9 (4.6) and 30.8 (4.4).
template <int T, bool VEC>
__global__ void __launch_bounds__(256) combine_grad_kernel(const Moves M)
{
    typedef Type<T> E;
    typedef typename E::Raw Raw;
    let_next_in();
    wait_for_previous();
    const int lane = threadIdx.x & 31;
    const int64_t item = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
    if (item >= M.rows * M.k) return;
    const int t = (int)item / M.k, h = (int)M.h;           // (fewer than 2^31 choices)
    const int64_t p = place_of(M, 0, (int)item);
    float dot = 0.f;
    if (p >= 0) {
        const Raw* dy = (const Raw*)M.x + t * M.ld_x;
        const float w = M.weights ? M.weights[item] : 1.f;
        const Raw* r = (const Raw*)M.r + p * M.ld_r;
        Raw* o = (Raw*)M.out + p * M.ld_out;
        if constexpr (VEC) {
            constexpr int W = E::kVec;
#pragma unroll 4
            for (int c = lane * W; c < h; c += 32 * W) {
                float g[W], v[W];
                E::unpack(*reinterpret_cast<const uint4*>(dy + c), g);
                if (M.dweights) {
                    E::unpack(*reinterpret_cast<const uint4*>(r + c), v);
#pragma unroll
                    for (int i = 0; i < W; ++i) dot = fmaf(g[i], v[i], dot);
                }
                if (M.out) {
#pragma unroll
                    for (int i = 0; i < W; ++i) g[i] *= w;
                    *reinterpret_cast<uint4*>(o + c) = E::pack(g);
                }
            }
        } else {
            // 8 elements a lane on their way at a time
            for (int c0 = lane; c0 < h; c0 += 8 * 32) {
                Raw v[8], g[8];
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (c0 + i * 32 < h) {
                        if (M.dweights) v[i] = r[c0 + i * 32];
                        g[i] = dy[c0 + i * 32];
                    }
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (c0 + i * 32 < h) {
                        const float a = E::load(g + i);
                        if (M.dweights) dot = fmaf(a, E::load(v + i), dot);
                        if (M.out) E::store(o + c0 + i * 32, a * w);
                    }
            }
        }
    }
    if (M.dweights) {
        dot = warp_sum(dot);
        if (lane == 0) M.dweights[item] = dot;
    }
}

}  // namespace tensor
}  // namespace ccl
