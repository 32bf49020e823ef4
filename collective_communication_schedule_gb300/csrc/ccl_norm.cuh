// Layer norm over rows, and its gradients.
#pragma once

#include "ccl_layer_common.cuh"

namespace ccl {
namespace tensor {

// Blocks of a backward pass that keep sums of dw and db: by the sizes alone, so
// that the order of the sums is.
constexpr int kNormBlocks = 152;
// Rows that the backward pass has on their way.  us with 1, 2 and 3: bf16 8192 x 4096
// 57.7, 42.2 and 44.8, 8192 x 8192 126, 81.2 and 81.9, f32 8192 x 4096 110, 71.1 and 70.5.
constexpr int kRowsAhead = 2;

struct Norm {
    const void *x, *dy, *w, *b;
    void *y, *dx, *dw, *db;
    float *mean, *rstd;            // outputs of the forward pass (may be null), inputs of the backward pass
    float* partial;                // blocks x 2 x n: sums of dw and db
    int64_t rows, n;
    int64_t ld_x, ld_y, ld_dy, ld_dx;
    int32_t blocks;                // of the backward pass
    float eps;
    int32_t apart;                 // rows of y lie otherwise to 16 bytes than those of x
};

// Sum over the TPR threads of a row (all of them get it): a warp, or a
// threadblock through shared memory.  buf: 32 words, not read by a slower warp any
// more (calls take turns with two, each behind the other's barrier).
template <int TPR>
__device__ __forceinline__ float row_sum(float v, float* buf, int tid)
{
    v = warp_sum(v);
    if (TPR == 32) return v;
    if ((tid & 31) == 0) buf[tid >> 5] = v;
    __syncthreads();
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < TPR / 32; i += 4) {
        const float4 p = *reinterpret_cast<const float4*>(buf + i);
        s += (p.x + p.y) + (p.z + p.w);
    }
    return s;
}

// W consecutive elements at p, in 32 bits: at a time where they fill 8 or 16 bytes (VEC), else one by one.
template <typename E, bool VEC, int W>
__device__ __forceinline__ void read(const typename E::Raw* p, float* v)
{
    if (VEC && W == 8 && E::kVec == 8) {
        E::unpack(*reinterpret_cast<const uint4*>(p), v);
    } else if (VEC && E::kVec == 4) {
#pragma unroll
        for (int i = 0; i < W; i += 4) E::unpack(*reinterpret_cast<const uint4*>(p + i), v + i);
    } else {
#pragma unroll
        for (int i = 0; i < W; ++i) v[i] = E::load(p + i);
    }
}
template <typename E, bool VEC, int W>
__device__ __forceinline__ void write(typename E::Raw* p, const float* v)
{
    if (VEC && W == 8 && E::kVec == 8) {
        *reinterpret_cast<uint4*>(p) = E::pack(v);
    } else if (VEC && E::kVec == 4) {
#pragma unroll
        for (int i = 0; i < W; i += 4) *reinterpret_cast<uint4*>(p + i) = E::pack(v + i);
    } else {
#pragma unroll
        for (int i = 0; i < W; ++i) E::store(p + i, v[i]);
    }
}

// A row in the registers of TPR threads, read once: y = (x - mean) rstd w + b
// with the variance summed over differences from the mean.  V pieces of 16
// bytes a thread (VEC) or of one element.  DRAM bounds it where rows are on 16
// bytes: 8192 x 4096 bf16 22 us (6.1 TB/s), f32 40.4 us (6.6 TB/s).
template <int T, int TW, int TPR, int V, bool VEC>
__global__ void __launch_bounds__(TPR < 128 ? 128 : TPR) norm_kernel_rows(const Norm N)
{
    typedef Type<T> E;
    typedef Type<TW> EW;
    typedef typename E::Raw Raw;
    constexpr int W = VEC ? E::kVec : 1;
    constexpr int kRows = TPR < 128 ? 128 / TPR : 1;
    __shared__ __align__(16) float buf[2][32];
    let_next_in();
    wait_for_previous();
    const int tid = threadIdx.x % TPR, n = (int)N.n;
    const int64_t row = (int64_t)blockIdx.x * kRows + threadIdx.x / TPR;
    if (kRows > 1 && row >= N.rows) return;
    const Raw* x = (const Raw*)N.x + row * N.ld_x;
    Raw* y = (Raw*)N.y + row * N.ld_y;
    const typename EW::Raw *w = (const typename EW::Raw*)N.w, *b = (const typename EW::Raw*)N.b;
    const float inv = 1.f / (float)n;
    if constexpr (VEC) {
        float v[V][W], t = 0.f;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            if ((i * TPR + tid) * W < n) {
                read<E, VEC, W>(x + (i * TPR + tid) * W, v[i]);
            } else {
#pragma unroll
                for (int e = 0; e < W; ++e) v[i][e] = 0.f;
            }
        }
#pragma unroll
        for (int i = 0; i < V; ++i)
#pragma unroll
            for (int e = 0; e < W; ++e) t += v[i][e];
        const float mean = row_sum<TPR>(t, buf[0], tid) * inv;
        t = 0.f;
#pragma unroll
        for (int i = 0; i < V; ++i)
            if ((i * TPR + tid) * W < n) {
#pragma unroll
                for (int e = 0; e < W; ++e) {
                    v[i][e] -= mean;
                    t = fmaf(v[i][e], v[i][e], t);
                }
            }
        const float rstd = 1.f / sqrtf(row_sum<TPR>(t, buf[1], tid) * inv + N.eps);
        if (tid == 0) {
            if (N.mean) N.mean[row] = mean;
            if (N.rstd) N.rstd[row] = rstd;
        }
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int c = (i * TPR + tid) * W;
            if (c < n) {
                float k[W];
#pragma unroll
                for (int e = 0; e < W; ++e) v[i][e] *= rstd;
                if (w) {
                    read<EW, VEC, W>(w + c, k);
#pragma unroll
                    for (int e = 0; e < W; ++e) v[i][e] *= k[e];
                }
                if (b) {
                    read<EW, VEC, W>(b + c, k);
#pragma unroll
                    for (int e = 0; e < W; ++e) v[i][e] += k[e];
                }
                write<E, VEC, W>(y + c, v[i]);
            }
        }
    } else {
        const int used = (n + TPR - 1) / TPR;              // elements that anybody has
        Raw raw[V];
        float v[V], t = 0.f;
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (i < used && i * TPR + tid < n) raw[i] = x[i * TPR + tid];
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (i < used && i * TPR + tid < n) {
                v[i] = E::load(raw + i);
                t += v[i];
            }
        const float mean = row_sum<TPR>(t, buf[0], tid) * inv;
        t = 0.f;
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (i < used && i * TPR + tid < n) {
                v[i] -= mean;
                t = fmaf(v[i], v[i], t);
            }
        const float rstd = 1.f / sqrtf(row_sum<TPR>(t, buf[1], tid) * inv + N.eps);
        if (tid == 0) {
            if (N.mean) N.mean[row] = mean;
            if (N.rstd) N.rstd[row] = rstd;
        }
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int c = i * TPR + tid;
            if (i >= used || c >= n) continue;
            float o = v[i] * rstd;
            if (w) o *= EW::load(w + c);
            if (b) o += EW::load(b + c);
            E::store(y + c, o);
        }
    }
}

// Rows off 16 bytes: what lies on 16 bytes of each is read and written so, and
// the up to 2 (W - 1) elements before and behind go to a thread each.  A thread's
// elements of w and b then lie anywhere, so the threadblock keeps both as W
// planes in shared memory (element i in plane i mod W), of which neighbouring
// lanes read neighbouring places whatever the row's distance from 16 bytes.  Where
// rows of y have another distance they go through shared memory too, and out by
// elements (bf16 8191 x 2057 24.8 us instead of 19.6, 4096 x 5001 47.3 instead of 24.4).
// The threadblock's groups of TPR threads take rows in turn.
//
// Instructions bound it (1750 a row of 2057, most SM cycles issue one).  Element
// by element, us, and so: bf16 8191 x 2057 26.3 and 19.8 (3.4 TB/s), 4097 x 4097
// 48.5 and 23.4, 1000 x 10007 26.9 and 18.6, f16 20000 x 517 29.5 and 12.8, bf16
// 20000 x 131 10.1 and 9.3, but 8191 x 100 3.6 and 5.2, so up to 128 elements
// stay one by one, and f32, which has half as many elements in the same bytes: 8191
// x 2057 27.3 and 37.5.
constexpr int kShiftedThreads = 256;
// Blocks of an SM that registers allow, by the elements that a thread holds.  Shared
// memory allows one less for 256 threads of 5 pieces (82 KB of w and b) and, with rows
// of y apart, for 256 of 3; the blocks beyond those follow as a second turn.
__host__ __device__ constexpr int shifted_blocks(int each) { return each > 24 ? 3 : 4; }
template <int W, int TPR, int V>
__host__ __device__ constexpr int plane_of() { return V * TPR + 16 / W; }    // pairs (one behind the last; spread over the banks)
template <int T, int TW, int TPR, int V>
__global__ void __launch_bounds__(kShiftedThreads, shifted_blocks(V * Type<T>::kVec)) norm_kernel_shifted(const Norm N)
{
    typedef Type<T> E;
    typedef Type<TW> EW;
    typedef typename E::Raw Raw;
    constexpr int W = E::kVec, P = plane_of<W, TPR, V>(), kRows = kShiftedThreads / TPR;
    __shared__ float buf[2][kShiftedThreads / 32];
    extern __shared__ __align__(16) float2 planes[];       // w and b
    let_next_in();
    wait_for_previous();
    const int tid = threadIdx.x % TPR, group = threadIdx.x / TPR, n = (int)N.n;
    const typename EW::Raw *w = (const typename EW::Raw*)N.w, *b = (const typename EW::Raw*)N.b;
    uint4* stage = reinterpret_cast<uint4*>(planes + W * P) + group * (V * TPR);
    const float inv = 1.f / (float)n;
    auto sync = [&]() {            // the row's threads
        if (TPR == 32)
            __syncwarp();
        else
            named_sync(1 + group, TPR);
    };
    auto sum = [&](float t, float* at) {
        t = warp_sum(t);
        if (TPR == 32) return t;
        if ((threadIdx.x & 31) == 0) at[threadIdx.x >> 5] = t;
        sync();
        t = 0.f;
#pragma unroll
        for (int i = 0; i < TPR / 32; ++i) t += at[group * (TPR / 32) + i];
        return t;
    };
    const int64_t step = (int64_t)gridDim.x * kRows;
    int64_t row = (int64_t)blockIdx.x * kRows + group;
    uint4 raw[V];
    Raw one;
    int head = 0, full = 0, own = n;       // elements before the first 16 bytes, pieces, this thread's element of the rest
    auto fetch = [&]() {
        const Raw* x = (const Raw*)N.x + row * N.ld_x;
        head = min((int)(-(uintptr_t)x & 15) / (int)sizeof(Raw), n);
        full = (n - head) / W;
        own = tid < W ? (tid < head ? tid : n) : tid < 2 * W ? head + full * W + tid - W : n;
        if (own < n) one = x[own];
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (i * TPR + tid < full) raw[i] = *reinterpret_cast<const uint4*>(x + head + (i * TPR + tid) * W);
    };
    if (row < N.rows) fetch();
    for (int i0 = threadIdx.x; i0 < n; i0 += 8 * kShiftedThreads) {
        float kw[8], kb[8];        // all on their way at a time
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int i = min(i0 + j * kShiftedThreads, n - 1);
            kw[j] = w ? EW::load(w + i) : 1.f;
            kb[j] = b ? EW::load(b + i) : 0.f;
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int i = i0 + j * kShiftedThreads;
            if (i < n) planes[i % W * P + i / W] = make_float2(kw[j], kb[j]);
        }
    }
    __syncthreads();
    while (row < N.rows) {
        float v[V][W], z = own < n ? E::load(&one) : 0.f, t = z;
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (i * TPR + tid < full) {
                E::unpack(raw[i], v[i]);
#pragma unroll
                for (int e = 0; e < W; ++e) t += v[i][e];
            }
        const float mean = sum(t, buf[0]) * inv;
        z -= mean;
        t = own < n ? z * z : 0.f;
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (i * TPR + tid < full) {
#pragma unroll
                for (int e = 0; e < W; ++e) {
                    v[i][e] -= mean;
                    t = fmaf(v[i][e], v[i][e], t);
                }
            }
        const float rstd = 1.f / sqrtf(sum(t, buf[1]) * inv + N.eps);
        if (tid == 0) {
            if (N.mean) N.mean[row] = mean;
            if (N.rstd) N.rstd[row] = rstd;
        }
        Raw* y = (Raw*)N.y + row * N.ld_y;
        if (own < n) {
            const float2 k = planes[own % W * P + own / W];
            E::store(y + own, fmaf(z * rstd, k.x, k.y));
        }
        int at[W];                 // its elements of w and b
#pragma unroll
        for (int e = 0; e < W; ++e) at[e] = ((e + head) & (W - 1)) * P + tid + (e + head >= W);
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (i * TPR + tid < full) {
#pragma unroll
                for (int e = 0; e < W; ++e) {
                    const float2 k = planes[at[e] + i * TPR];
                    v[i][e] = fmaf(v[i][e] * rstd, k.x, k.y);
                }
                if (N.apart)
                    stage[i * TPR + tid] = E::pack(v[i]);
                else
                    *reinterpret_cast<uint4*>(y + head + (i * TPR + tid) * W) = E::pack(v[i]);
            }
        if (N.apart) {
            sync();
            const Raw* held = reinterpret_cast<const Raw*>(stage);
            for (int i = tid; i < full * W; i += TPR) y[head + i] = held[i];
            sync();
        }
        row += step;
        if (row < N.rows) fetch();
    }
}

// Rows too long for registers: three passes over the row, the second and third from L2.
template <int T, int TW>
__global__ void __launch_bounds__(1024) norm_kernel_long(const Norm N)
{
    typedef Type<T> E;
    typedef Type<TW> EW;
    __shared__ __align__(16) float buf[2][32];
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

__device__ __forceinline__ void copy16(uint32_t to, const void* from)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
}
__device__ __forceinline__ void copies_end() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int LEFT>
__device__ __forceinline__ void copies_wait()
{
    asm volatile("cp.async.wait_group %0;" ::"n"(LEFT) : "memory");
}

// Sums of two numbers over the ACROSS threads of a group (all of them get
// both).  part: 32 pairs, not read by a slower warp any more.
template <int ACROSS>
__device__ __forceinline__ float2 group_sums(float2 s, float* part, int group, int warp, int lane)
{
    // the halves of a warp take one sum each
    const bool up = lane & 16;
    float v = (up ? s.y : s.x) + __shfl_xor_sync(~0u, up ? s.x : s.y, 16);
#pragma unroll
    for (int d = 8; d; d /= 2) v += __shfl_xor_sync(~0u, v, d);
    if (ACROSS > 32) {
        // sums of x in part[0..31], of y in part[32..63], by warp
        if ((lane & 15) == 0) part[(up ? 32 : 0) + warp] = v;
        named_sync(1 + group, ACROSS);
        constexpr int width = ACROSS / 32;
        const int l = lane & 15;
        const float* p = part + (up ? 32 : 0) + group * width;
        v = p[l & (width - 1)];
        if (width == 32) v += p[l + 16];
#pragma unroll
        for (int d = width < 16 ? width / 2 : 8; d; d /= 2) v += __shfl_xor_sync(~0u, v, d);
    }
    return make_float2(__shfl_sync(~0u, v, 0), __shfl_sync(~0u, v, 16));
}

// dx = rstd (g - mean(g) - xh mean(g xh)) with g = dy w, and, over this
// block's rows, the sums of dy xh and dy that make dw and db.  ACROSS threads (a
// warp, or a power of two from 128 up) lie across a row and own its columns, V
// pieces each, whose sums they keep in registers; the block's groups of them take
// rows in turn.  VEC: pieces of 16 bytes, which every thread copies for itself into
// its own places in shared memory some rows before it needs them; else of
// one element, read a row ahead.
//
// Instructions bound it, about 300 of a warp a row for 8 elements a lane (the
// schedulers issue in 7 cycles of 10): 8192 x 4096 bf16 42 us with dw and db
// (4.8 TB/s), f32 with half as many elements in the same bytes 71 us (5.7 TB/s).
// Elements are unpacked twice instead of kept: 1024 threads have 64 registers each, of
// which w, dw and db take 24.  Few rows: 85 x 15656 14 us, of which the sums and their
// way through memory take two thirds (dx alone 4.8).  Rows off 16 bytes: 8191 x 2057 bf16 34 us; columns belong
// to threads, so rows cannot be taken by the pieces of 16 bytes that they touch.
template <int T, int TW, int THREADS, int ACROSS, int V, bool VEC>
__global__ void __launch_bounds__(THREADS) norm_grad_kernel_rows(const Norm N)
{
    typedef Type<T> E;
    typedef Type<TW> EW;
    typedef typename E::Raw Raw;
    constexpr int W = VEC ? E::kVec : 1, kAhead = kRowsAhead;
    __shared__ float part[2][64];
    extern __shared__ __align__(16) unsigned char dyn[];
    let_next_in();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, n = (int)N.n;
    constexpr int across = ACROSS, groups = THREADS / ACROSS;
    const int group = threadIdx.x / across, tid = threadIdx.x & (across - 1);
    const float inv = 1.f / (float)n;
    const int step = gridDim.x * groups, row = blockIdx.x * groups + group;
    int left = row < (int)N.rows ? ((int)N.rows - row - 1) / step + 1 : 0;       // rows of this group
    // places of this thread: [row ahead][x, dy][piece], 16 bytes each, neighbours for neighbouring threads
    unsigned char* place = dyn + threadIdx.x * 16;
    const uint32_t place0 = smem_addr(place);
    constexpr int kPlace = THREADS * 16;
    bool mine[V];
#pragma unroll
    for (int i = 0; i < V; ++i) mine[i] = (i * across + tid) * W < n;
    const Raw *px = (const Raw*)N.x + row * N.ld_x + tid * W, *pd = (const Raw*)N.dy + row * N.ld_dy + tid * W;
    const int64_t next_x = step * N.ld_x, next_d = step * N.ld_dy;
    wait_for_previous();
    auto fetch = [&](int slot, bool any) {
        if (any) {
#pragma unroll
            for (int i = 0; i < V; ++i)
                if (mine[i]) {
                    copy16(place0 + ((slot * 2 + 0) * V + i) * kPlace, px + i * across * W);
                    copy16(place0 + ((slot * 2 + 1) * V + i) * kPlace, pd + i * across * W);
                }
        }
        copies_end();
        px += next_x;
        pd += next_d;
    };
    Raw nx[VEC ? 1 : V], nd[VEC ? 1 : V];
    auto fetch1 = [&](bool any) {
        if (any) {
#pragma unroll
            for (int i = 0; i < V; ++i)
                if (mine[i]) {
                    nx[VEC ? 0 : i] = px[i * across];
                    nd[VEC ? 0 : i] = pd[i * across];
                }
        }
        px += next_x;
        pd += next_d;
    };
    if constexpr (VEC) {
#pragma unroll
        for (int i = 0; i < kAhead; ++i) fetch(i, i < left);
    } else {
        fetch1(left > 0);
    }
    constexpr bool kHeld = !VEC || V * W <= 16;            // w in registers; else read for every row (from L1)
    float held[kHeld ? V : 1][W], dw[V][W], db[V][W];
    auto weights = [&](int i, float (&w)[W]) {
#pragma unroll
        for (int e = 0; e < W; ++e) w[e] = 1.f;
        if (N.w && mine[i]) read<EW, VEC, W>((const typename EW::Raw*)N.w + (i * across + tid) * W, w);
    };
#pragma unroll
    for (int i = 0; i < V; ++i) {
#pragma unroll
        for (int e = 0; e < W; ++e) dw[i][e] = db[i][e] = 0.f;
        if (kHeld) weights(i, held[kHeld ? i : 0]);
    }
    const float *pm = N.mean + row, *pr = N.rstd + row;
    float next_mean = left > 0 ? *pm : 0.f, next_rstd = left > 0 ? *pr : 0.f;
    Raw* dx = N.dx ? (Raw*)N.dx + row * N.ld_dx + tid * W : nullptr;
    const int64_t next_o = step * N.ld_dx;
    int slot = 0, turn = 0;
    for (; left > 0; --left, turn ^= 1) {
        const float mean = next_mean, rstd = next_rstd;
        if (left > 1) next_mean = *(pm += step), next_rstd = *(pr += step);
        // (16-byte pieces are read again from shared memory for dx, single elements kept)
        float xh[V][W], g[V][W];
        const unsigned char* at = place + slot * 2 * V * kPlace;
        if constexpr (VEC) {
            copies_wait<kAhead - 1>();
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i)
                if (mine[i]) xh[i][0] = E::load(nx + i), g[i][0] = E::load(nd + i);
            fetch1(left > 1);
        }
        float2 s = make_float2(0.f, 0.f);
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (mine[i]) {
                if constexpr (VEC) {
                    read<E, VEC, W>((const Raw*)(at + i * kPlace), xh[i]);
                    read<E, VEC, W>((const Raw*)(at + (V + i) * kPlace), g[i]);
                }
                float own[W];
                if (!kHeld) weights(i, own);
                const float (&w)[W] = kHeld ? held[kHeld ? i : 0] : own;
#pragma unroll
                for (int e = 0; e < W; ++e) {
                    xh[i][e] = (xh[i][e] - mean) * rstd;
                    dw[i][e] = fmaf(g[i][e], xh[i][e], dw[i][e]);
                    db[i][e] += g[i][e];
                    g[i][e] *= w[e];
                    s.x += g[i][e];
                    s.y = fmaf(g[i][e], xh[i][e], s.y);
                }
            }
        if (dx) {
            s = group_sums<ACROSS>(s, part[turn], group, warp, lane);
            // rstd (g - a - xh b) = g rstd - a rstd - xh (b rstd)
            const float ka = -s.x * inv * rstd, kb = -s.y * inv * rstd;
#pragma unroll
            for (int i = 0; i < V; ++i)
                if (mine[i]) {
                    if constexpr (VEC) {
                        asm volatile("" ::: "memory");
                        read<E, VEC, W>((const Raw*)(at + i * kPlace), xh[i]);
                        read<E, VEC, W>((const Raw*)(at + (V + i) * kPlace), g[i]);
                        float own[W];
                        if (!kHeld) weights(i, own);
                        const float (&w)[W] = kHeld ? held[kHeld ? i : 0] : own;
#pragma unroll
                        for (int e = 0; e < W; ++e) xh[i][e] = (xh[i][e] - mean) * rstd, g[i][e] *= w[e];
                    }
#pragma unroll
                    for (int e = 0; e < W; ++e) g[i][e] = fmaf(xh[i][e], kb, fmaf(g[i][e], rstd, ka));
                    write<E, VEC, W>(dx + i * across * W, g[i]);
                }
            dx += next_o;
        }
        if constexpr (VEC) {
            fetch(slot, left > kAhead);
            slot = slot + 1 == kAhead ? 0 : slot + 1;
        }
    }
    if (!N.partial) return;
    if (VEC) copies_wait<0>();
    // the groups' sums, in turn through the places' memory
    float* sums = reinterpret_cast<float*>(dyn);
    float* out = N.partial + (int64_t)blockIdx.x * 2 * n;
#pragma unroll
    for (int which = 0; which < 2; ++which)
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int c = (i * across + tid) * W;
            float v[W];
#pragma unroll
            for (int e = 0; e < W; ++e) v[e] = which ? db[i][e] : dw[i][e];
            if (groups > 1) {
                __syncthreads();
#pragma unroll
                for (int e = 0; e < W; ++e) sums[(group * W + e) * across + tid] = v[e];
                __syncthreads();
                if (group > 0) continue;
#pragma unroll
                for (int e = 0; e < W; ++e) {
                    v[e] = 0.f;
#pragma unroll 4
                    for (int r = 0; r < groups; ++r) v[e] += sums[(r * W + e) * across + tid];
                }
            }
            if (c < n) {
                if constexpr (VEC) {       // (n is a multiple of W)
#pragma unroll
                    for (int e = 0; e < W; e += 4)
                        *reinterpret_cast<float4*>(out + which * n + c + e) = make_float4(v[e], v[e + 1], v[e + 2], v[e + 3]);
                } else {
                    out[which * n + c] = v[0];
                }
            }
        }
}

// Rows too long for registers: dx of a row in two passes ...
template <int T, int TW>
__global__ void __launch_bounds__(1024) norm_grad_kernel_long(const Norm N)
{
    typedef Type<T> E;
    typedef Type<TW> EW;
    __shared__ __align__(16) float buf[2][32];
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
    s.x = row_sum<1024>(s.x, buf[0], tid);
    s.y = row_sum<1024>(s.y, buf[1], tid);
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

// The blocks' sums added up in order: 32 columns a threadblock, 32 groups of
// threads take the blocks in turn.  blockIdx.y: dw, db.
template <int TW>
__global__ void __launch_bounds__(1024) norm_sums_kernel(const Norm N)
{
    typedef Type<TW> EW;
    __shared__ float sums[32][32];
    let_next_in();
    wait_for_previous();
    const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
    const int64_t c = (int64_t)blockIdx.x * 32 + tx;
    typename EW::Raw* out = (typename EW::Raw*)(blockIdx.y ? N.db : N.dw);
    if (!out) return;
    float s = 0.f;
    if (c < N.n) {
        const float* p = N.partial + blockIdx.y * N.n + c;
        // (at most kNormBlocks / 32 loads a thread, all on their way at a time)
        float v[(kNormBlocks + 31) / 32];
#pragma unroll
        for (int i = 0; i < (kNormBlocks + 31) / 32; ++i) v[i] = i * 32 + ty < N.blocks ? __ldcg(p + (int64_t)(i * 32 + ty) * 2 * N.n) : 0.f;
#pragma unroll
        for (int i = 0; i < (kNormBlocks + 31) / 32; ++i) s += v[i];
    }
    sums[ty][tx] = s;
    __syncthreads();
    if (ty == 0 && c < N.n) {
#pragma unroll
        for (int i = 1; i < 32; ++i) s += sums[i][tx];
        EW::store(out + c, s);
    }
}

}  // namespace tensor
}  // namespace ccl
