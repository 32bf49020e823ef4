// The orthogonalisation's own kernels: norm and scaling passes, and all of the
// iteration in one launch for matrices with a short side.
#pragma once

#include <cstdint>

#include "ccl_tensor.cuh"
#include "ccl_tensor_passes.cuh"

namespace ccl {
namespace tensor {

// The iteration keeps x, A and B in f16: 11 bits instead of bf16's 8, at the
// same matrix rate, and their range is known (singular values of x stay
// near 1), so fixed powers of two keep the entries clear of both ends.
constexpr float kScaleX = 4096.f, kScaleA = 1024.f;
constexpr int kNormBlocks = 256;

struct NormPass {
    const void* g;
    __half* x;
    float *partial, *kappa, *kappa2;
    int64_t ld_g, bs_g, ld_x, bs_x;
    int64_t run;                   // elements of a run of consecutive ones: a row, or the whole matrix
    int32_t p, q, type, runs, blocks;
    float eps;
};

__device__ __forceinline__ float load_any(const void* p, int64_t i, int type)
{
    if (type == CCL_F32) return ((const float*)p)[i];
    return load1((const uint16_t*)p + i, type == CCL_BF16);
}

// 8 elements from i on, i any index
__device__ __forceinline__ void load_any8(const void* p, int64_t i, int type, float v[8])
{
    if (type == CCL_F32) {
        const float* f = (const float*)p + i;
        if (((uintptr_t)f & 15) == 0) {
            const float4 a = ((const float4*)f)[0], b = ((const float4*)f)[1];
            v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = f[e];
        }
    } else {
        const uint16_t* h = (const uint16_t*)p + i;
        if (((uintptr_t)h & 15) == 0) {
            unpack8(*reinterpret_cast<const uint4*>(h), type == CCL_BF16, v);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = load1(h + e, type == CCL_BF16);
        }
    }
}

__device__ __forceinline__ float block_sum(float v, float* sm)
{
#pragma unroll
    for (int d = 16; d; d >>= 1) v += __shfl_xor_sync(~0u, v, d);
    if ((threadIdx.x & 31) == 0) sm[threadIdx.x >> 5] = v;
    __syncthreads();
    float s = 0.f;
    for (int i = 0; i < (int)blockDim.x / 32; ++i) s += sm[i];
    return s;
}

// Sums of squares (DRAM: 4 x 2048 x 4096 bf16 in 14 us): threadblocks take groups of 8 elements of all runs in
// turn (one run where the matrix is packed), so the order is fixed.
__global__ void __launch_bounds__(256) norm_kernel(const NormPass N)
{
    __shared__ float sm[8];
    let_next_in();
    wait_for_previous();
    const int64_t base = blockIdx.y * N.bs_g, per = (N.run + 7) / 8, all = per * N.runs;
    const int64_t stride = (int64_t)gridDim.x * 256;
    float s = 0.f;
    int64_t i = blockIdx.x * 256 + threadIdx.x;
    if (N.runs == 1 && N.type != CCL_F32 && ((uintptr_t)((const uint16_t*)N.g + base) & 15) == 0) {
        // packed 16-bit matrices on a 16-byte boundary: eight loads in flight
        const uint4* p = (const uint4*)((const uint16_t*)N.g + base);
        for (; i + 7 * stride < N.run / 8; i += 8 * stride) {
            uint4 u[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) u[j] = p[i + j * stride];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                float v[8], t = 0.f;
                unpack8(u[j], N.type == CCL_BF16, v);
#pragma unroll
                for (int e = 0; e < 8; ++e) t = fmaf(v[e], v[e], t);
                s += t;
            }
        }
    }
#pragma unroll 4
    for (; i < all; i += stride) {
        const int64_t r = N.runs == 1 ? 0 : i / per, c = (i - r * per) * 8, at = base + r * N.ld_g + c;
        float v[8];
        if (c + 8 <= N.run) {
            load_any8(N.g, at, N.type, v);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = c + e < N.run ? load_any(N.g, at + e, N.type) : 0.f;
        }
        float t = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) t = fmaf(v[e], v[e], t);
        s += t;
    }
    s = block_sum(s, sm);
    if (threadIdx.x == 0) N.partial[blockIdx.y * kNormBlocks + blockIdx.x] = s;
}

// x0 = g * 2^e in f16 (exact for bf16 gradients) with the power of two that
// brings the norm to kScaleX / 2 .. kScaleX; the remaining factor kappa of
// x0 = kScaleX * g / (norm + eps) is applied in 32 bits by the epilogues of
// the first step.
__device__ __forceinline__ void norm_scale(float sum, float eps, float& kappa, float& f1, float& f2)
{
    const float norm = sqrtf(sum);
    int e = 0;
    if (norm > 0.f && norm <= 3.4e38f) {
        int x;
        frexpf(norm, &x);            // norm in [2^(x-1), 2^x)
        e = 12 - x;                  // kScaleX = 2^12
    }
    kappa = ldexpf(1.f, 12 - e) / (norm + eps);
    f1 = ldexpf(1.f, e / 2);         // 2^e may leave the range of 32 bits: in two factors
    f2 = ldexpf(1.f, e - e / 2);
}

__global__ void __launch_bounds__(256) scale_kernel(const NormPass N)
{
    __shared__ float sm[8];
    let_next_in();
    wait_for_previous();
    float s = (int)threadIdx.x < N.blocks ? N.partial[blockIdx.y * kNormBlocks + threadIdx.x] : 0.f;
    s = block_sum(s, sm);
    float kappa, f1, f2;
    norm_scale(s, N.eps, kappa, f1, f2);
    if (blockIdx.x == 0 && threadIdx.x == 0) {
        N.kappa[blockIdx.y] = kappa;
        N.kappa2[blockIdx.y] = kappa * kappa;
    }
    const int per = (N.q + 7) / 8;
    const int64_t all = (int64_t)per * N.p;
#pragma unroll 2
    for (int64_t i = blockIdx.x * 256 + threadIdx.x; i < all; i += (int64_t)gridDim.x * 256) {
        const int64_t r = i / per, c = (i - r * per) * 8, at = blockIdx.y * N.bs_g + r * N.ld_g + c;
        float v[8];
        if (c + 8 <= N.q) {
            load_any8(N.g, at, N.type, v);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = c + e < N.q ? load_any(N.g, at + e, N.type) : 0.f;
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = v[e] * f1 * f2;
        store8((uint16_t*)N.x + blockIdx.y * N.bs_x + r * N.ld_x + c, false, 8, v);   // rows are padded
    }
}

// All of the iteration for matrices with a side of at most 128, in one launch
// and without leaving the SM: x, A and B live in shared memory in the layout
// the matrix instructions read, accumulators in tensor memory, and a step is
// three products with a threadblock barrier after each.  A long side is cut
// over the threadblocks of a cluster, `width` columns of x each: they add up
// their parts of A = x x^T through distributed shared memory (each reads 128 /
// size rows of all, sums them in rank order, and hands them to all: 128 x 1024
// in 45 us, 53 when the parts were pushed from the accumulators, where a
// store of a warp went to 32 rows), the rest of the step stays within a threadblock.  A tall matrix is transposed as it is loaded
// and stored.  Bound by the latency of 3 x steps products in a row: 128 x 128 in
// 19 us, 2.5 us a step; one launch per product took 87 us.
//
// Rows of 64 elements (128 bytes) in 1024-byte atoms of 8 rows, 16-byte pieces
// exchanged by the row's index: element (i, j) of x is at piece (j / 8 % 8) ^
// (i % 8) of row i of block j / 64.  The same bytes are x with the reduction
// along its columns (x x^T) and along its rows (B x).
constexpr int kSmallSide = 128;
constexpr int kSmallThreads = 512;
constexpr int kSmallCluster = 16;
constexpr int kSmallBlock = kSmallSide * 128;          // bytes of a block of 64 columns
constexpr int kSharePitch = kSmallSide + 4;            // floats; rows 4 banks apart

struct Small {
    const void* g;
    uint16_t* out;
    int64_t ld_g, bs_g, ld_out, bs_out;
    int32_t side, length;          // short and long side
    int32_t tall, type, out_bf, steps;
    int32_t size, width, vec_g, vec_out;
    float a, b, c, eps, scale;
};

__device__ __forceinline__ uint32_t small_at(int i, int j)
{
    return (uint32_t)(j >> 6) * kSmallBlock + i * 128 + (((j >> 3) & 7) ^ (i & 7)) * 16;
}

__device__ __forceinline__ void store_cluster8(uint32_t addr, uint2 v)
{
    asm volatile("st.shared::cluster.v2.b32 [%0], {%1, %2};" ::"r"(addr), "r"(v.x), "r"(v.y) : "memory");
}

__device__ __forceinline__ float4 load_cluster16(uint32_t addr)
{
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(addr)
                 : "memory");
    return v;
}

// use(i, j, v) for the pieces of 8 columns j.. of row i of a threadblock's part
// of g (or of its transpose), zeros outside of it.  Neighbouring threads take
// neighbouring elements in memory.  Four pieces are loaded before the first is
// used: TYPE and the way of loading are settled outside of the loops, or each
// piece would wait for the one before.
template <int TYPE, class Use>
__device__ __forceinline__ void small_pieces(const Small& S, int64_t base, int col0, int cols, Use use)
{
    const int pieces = S.width / 8, items = pieces * kSmallSide;
    auto element = [&](int i, int j) {
        const int64_t at = S.tall ? base + (int64_t)(col0 + j) * S.ld_g + i : base + i * S.ld_g + col0 + j;
        return load_any(S.g, at, TYPE);
    };
    const bool vector = !S.tall && S.vec_g;
    for (int n0 = threadIdx.x; n0 < items; n0 += 4 * kSmallThreads) {
        float v[4][8];
        int row[4], col[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int n = n0 + u * kSmallThreads;
            row[u] = S.tall ? n % kSmallSide : n / pieces;
            col[u] = S.tall ? n / kSmallSide * 8 : n % pieces * 8;
        }
        if (vector) {
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const bool in = row[u] < S.side;
                if (in && col[u] + 8 <= cols) {
                    load_any8(S.g, base + row[u] * S.ld_g + col0 + col[u], TYPE, v[u]);
                } else {
#pragma unroll
                    for (int e = 0; e < 8; ++e) v[u][e] = in && col[u] + e < cols ? element(row[u], col[u] + e) : 0.f;
                }
            }
        } else {
            // the last element stands in for those outside
#pragma unroll
            for (int u = 0; u < 4; ++u)
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    v[u][e] = cols > 0 ? element(min(row[u], S.side - 1), min(col[u] + e, cols - 1)) : 0.f;
#pragma unroll
            for (int u = 0; u < 4; ++u)
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    if (row[u] >= S.side || col[u] + e >= cols) v[u][e] = 0.f;
        }
#pragma unroll
        for (int u = 0; u < 4; ++u)
            if (n0 + u * kSmallThreads < items) use(row[u], col[u], v[u]);
    }
}

template <class Use>
__device__ __forceinline__ void small_pieces_of(const Small& S, int64_t base, int col0, int cols, Use use)
{
    if (S.type == CCL_F32)
        small_pieces<CCL_F32>(S, base, col0, cols, use);
    else if (S.type == CCL_BF16)
        small_pieces<CCL_BF16>(S, base, col0, cols, use);
    else
        small_pieces<CCL_F16>(S, base, col0, cols, use);
}

// MOST: threadblocks of a matrix at most -- 1, 8 (2, 4 or 8 of them) or 16
// (always 16); one kernel for all took 1 us longer for one and 3 us for 16.
template <int MOST>
__global__ void __launch_bounds__(kSmallThreads, 1) small_ortho_kernel(const __grid_constant__ Small S)
{
    __shared__ __align__(8) uint64_t done;
    __shared__ uint32_t tmem_slot;
    __shared__ int failed;
    __shared__ float sm[16], norms[kSmallCluster];
    extern __shared__ unsigned char raw[];
    unsigned char* dyn = raw + ((1024 - (smem_addr(raw) & 1023)) & 1023);
    const int size = MOST == 8 ? S.size : MOST;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, quad = warp & 3, group = warp >> 2;
    const int rank = MOST > 1 ? (int)cluster_rank() : 0, entry = blockIdx.x / size;
    const int width = S.width, col0 = rank * width, cols = max(0, min(width, S.length - col0));
    unsigned char *x = dyn, *A = x + (size_t)width / 64 * kSmallBlock, *B = A + 2 * kSmallBlock;
    float* share = reinterpret_cast<float*>(B + 2 * kSmallBlock);   // size > 1: this threadblock's part of A
    const uint32_t bar = smem_addr(&done);
    if (threadIdx.x == 0) {
        bar_init(bar, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        failed = 0;
    }
    if (warp == 1) {
        tmem_alloc<1>(smem_addr(&tmem_slot), 512);
        let_next_in();              // not before: the next kernel could take the tensor memory and wait for this one
    }
    wait_for_previous();

    const int64_t base = (int64_t)entry * S.bs_g;
    float sum = 0.f;
    small_pieces_of(S, base, col0, cols, [&](int, int, const float v[8]) {
        float t = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) t = fmaf(v[e], v[e], t);
        sum += t;
    });
    sum = block_sum(sum, sm);
    if constexpr (MOST > 1) {
        cluster_sync();            // the others' shared memory is live from here on
        if ((int)threadIdx.x < size) store_cluster(cluster_addr(smem_addr(&norms[rank]), threadIdx.x), sum);
        cluster_sync();
        sum = 0.f;
        for (int i = 0; i < size; ++i) sum += norms[i];
    }
    float kappa, f1, f2;
    norm_scale(sum, S.eps, kappa, f1, f2);
    small_pieces_of(S, base, col0, cols, [&](int i, int j, const float v[8]) {
        uint4 u;
        uint32_t* w = &u.x;
#pragma unroll
        for (int e = 0; e < 4; ++e) w[e] = pack2<false>(v[2 * e] * f1 * f2, v[2 * e + 1] * f1 * f2);
        *reinterpret_cast<uint4*>(x + small_at(i, j)) = u;
    });
    fence_async();
    fence_before();
    __syncthreads();
    fence_after();
    const uint32_t tmem = tmem_slot, lanes = (uint32_t)(quad * 32) << 16;
    const uint32_t x_at = (smem_addr(x) & 0x3ffff) >> 4, a_at = (smem_addr(A) & 0x3ffff) >> 4,
                   b_at = (smem_addr(B) & 0x3ffff) >> 4;
    const uint64_t along = operand_desc(0, 0, 1024), across = operand_desc(0, kSmallBlock, 1024);
    const uint32_t square = mma_desc(false, false, false, kSmallSide, kSmallSide);
    constexpr uint32_t to_x = kSmallSide;       // tensor memory: columns 0.. A or B, 128.. x
    const int row = quad * 32 + lane;
    uint32_t parity = 0;
    // an accumulator's 32 columns from `col` of this thread's row, once all products issued so far are done
    auto finish = [&]() {
        if (!bar_wait(bar, parity, &failed)) failed = 1;
        parity ^= 1;
        fence_after();
    };

    for (int step = 0; step < S.steps; ++step) {
        const bool first = step == 0, last = step + 1 == S.steps;
        // A = x x^T
        if (warp == 0) {
            if (elect_one()) {
                for (int k = 0; k < width / 16; ++k) {
                    const uint32_t at = x_at + ((k >> 2) * kSmallBlock + (k & 3) * 32 >> 4);
                    mma_f16<1>(tmem, along | at, along | at, square, k > 0);
                }
                mma_commit<1>(bar);
            }
            __syncwarp();
        }
        finish();
        const float alpha = kScaleA / (kScaleX * kScaleX) * (first ? kappa * kappa : 1.f);
        {
            uint32_t u[32];
            tmem_load32(tmem + lanes + group * 32, u);
            if constexpr (MOST == 1) {
#pragma unroll
                for (int c = 0; c < 32; c += 8) {
                    uint4 h;
                    uint32_t* w = &h.x;
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        w[e] = pack2<false>(alpha * __uint_as_float(u[c + 2 * e]), alpha * __uint_as_float(u[c + 2 * e + 1]));
                    *reinterpret_cast<uint4*>(A + small_at(row, group * 32 + c)) = h;
                }
            } else {
                float* at = share + row * kSharePitch + group * 32;
#pragma unroll
                for (int c = 0; c < 32; c += 4)
                    *reinterpret_cast<uint4*>(at + c) = make_uint4(u[c], u[c + 1], u[c + 2], u[c + 3]);
            }
        }
        if constexpr (MOST > 1) {
            cluster_sync();
            const int own = kSmallSide / size;
            for (int n = threadIdx.x; n < own * (kSmallSide / 4); n += kSmallThreads) {
                const int r = rank * own + n / (kSmallSide / 4), c = n % (kSmallSide / 4) * 4;
                const uint32_t from = smem_addr(share + r * kSharePitch + c), at = smem_addr(A + small_at(r, c)) + (c & 4) * 2;
                float4 v = {0.f, 0.f, 0.f, 0.f};
                auto gather = [&](int first_rank) {
                    float4 p[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        if (first_rank + i < size) p[i] = load_cluster16(cluster_addr(from, first_rank + i));
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        if (first_rank + i < size) v.x += p[i].x, v.y += p[i].y, v.z += p[i].z, v.w += p[i].w;
                };
                gather(0);
                if constexpr (MOST > 8) gather(8);
                const uint2 h = {pack2<false>(alpha * v.x, alpha * v.y), pack2<false>(alpha * v.z, alpha * v.w)};
                auto hand_out = [&](int first_rank) {
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        if (first_rank + i < size) store_cluster8(cluster_addr(at, first_rank + i), h);
                };
                hand_out(0);
                if constexpr (MOST > 8) hand_out(8);
            }
            asm volatile("fence.proxy.async;" ::: "memory");
            fence_before();
            cluster_sync();
            fence_after();
        } else {
            fence_async();
            fence_before();
            __syncthreads();
            fence_after();
        }
        // B = b A + c A A (A is symmetric)
        if (warp == 0) {
            if (elect_one()) {
                fence_async();
#pragma unroll
                for (int k = 0; k < kSmallSide / 16; ++k) {
                    const uint32_t at = a_at + ((k >> 2) * kSmallBlock + (k & 3) * 32 >> 4);
                    mma_f16<1>(tmem, along | at, along | at, square, k > 0);
                }
                mma_commit<1>(bar);
            }
            __syncwarp();
        }
        finish();
        {
            uint32_t u[32];
            tmem_load32(tmem + lanes + group * 32, u);
            const float beta = S.b, gamma = S.c / kScaleA;
#pragma unroll
            for (int c = 0; c < 32; c += 8) {
                const uint32_t at = small_at(row, group * 32 + c);
                float o[8];
                unpack8(*reinterpret_cast<const uint4*>(A + at), false, o);
                uint4 h;
                uint32_t* w = &h.x;
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    w[e] = pack2<false>(gamma * __uint_as_float(u[c + 2 * e]) + beta * o[2 * e],
                                        gamma * __uint_as_float(u[c + 2 * e + 1]) + beta * o[2 * e + 1]);
                *reinterpret_cast<uint4*>(B + at) = h;
            }
        }
        fence_async();
        fence_before();
        __syncthreads();
        fence_after();
        // x <- a x + B x
        if (warp == 0) {
            if (elect_one()) {
                for (int n = 0; n < width; n += 256) {
                    const uint32_t idesc = mma_desc(false, false, true, kSmallSide, min(256, width - n));
#pragma unroll
                    for (int k = 0; k < kSmallSide / 16; ++k)
                        mma_f16<1>(tmem + to_x + n, along | (b_at + ((k >> 2) * kSmallBlock + (k & 3) * 32 >> 4)),
                                   across | (x_at + (n / 64 * kSmallBlock + k * 2048 >> 4)), idesc, k > 0);
                }
                mma_commit<1>(bar);
            }
            __syncwarp();
        }
        finish();
        const float unscale = (last ? S.scale / kScaleX : 1.f) * (first ? kappa : 1.f);
        const float beta = S.a * unscale, gamma = unscale / kScaleA;
        for (int c0 = group * 32; c0 < width; c0 += 128) {
            uint32_t u[32], w[16];
            tmem_load32(tmem + lanes + to_x + c0, u);
#pragma unroll
            for (int c = 0; c < 32; c += 8) {
                unsigned char* p = x + small_at(row, c0 + c);
                float o[8];
                unpack8(*reinterpret_cast<const uint4*>(p), false, o);
#pragma unroll
                for (int e = 0; e < 8; ++e) o[e] = gamma * __uint_as_float(u[c + e]) + beta * o[e];
                const bool bf = last && S.out_bf;
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    w[c / 2 + e] = bf ? pack2<true>(o[2 * e], o[2 * e + 1]) : pack2<false>(o[2 * e], o[2 * e + 1]);
                if (!last || !S.tall)
                    *reinterpret_cast<uint4*>(p) = make_uint4(w[c / 2], w[c / 2 + 1], w[c / 2 + 2], w[c / 2 + 3]);
            }
            if (last && S.tall && row < S.side) {
                const int n = cols - c0;         // columns of this thread's 32 that exist
                uint16_t* o = S.out + (int64_t)entry * S.bs_out + (int64_t)(col0 + c0) * S.ld_out + row;
#pragma unroll
                for (int e = 0; e < 32; ++e, o += S.ld_out)
                    if (e < n) *o = (uint16_t)(w[e / 2] >> (e & 1) * 16);
            }
        }
        fence_async();
        fence_before();
        __syncthreads();
        fence_after();
    }
    if (!S.tall && cols > 0) {
        // out of shared memory along the rows: from the accumulators, a store of
        // a warp would touch 32 rows (with the batched loads: 128 x 385 in 52 us, 82 before)
        uint16_t* o = S.out + (int64_t)entry * S.bs_out + col0;
        const int whole = S.vec_out ? cols / 8 : 0, rest = cols - whole * 8;
        for (int n = threadIdx.x; n < whole * S.side; n += kSmallThreads) {
            const int i = n / whole, j = n % whole * 8;
            *reinterpret_cast<uint4*>(o + i * S.ld_out + j) = *reinterpret_cast<const uint4*>(x + small_at(i, j));
        }
        for (int n = threadIdx.x; n < rest * S.side; n += kSmallThreads) {
            const int i = n / rest, j = whole * 8 + n % rest;
            o[i * S.ld_out + j] = reinterpret_cast<const uint16_t*>(x + small_at(i, j))[j & 7];
        }
    }
    if (failed && threadIdx.x == 0) atomicCAS(&g_status[0], 0, (int)CCL_ERR_TIMEOUT);
    if constexpr (MOST > 1) cluster_sync();     // nobody leaves while another may still write to it
    if (warp == 1) tmem_free<1>(tmem, 512);
}

}  // namespace tensor
}  // namespace ccl
