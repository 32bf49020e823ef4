// The matrix-product kernel of the dense and expert products, their gradients
// and the orthogonalisation.
#pragma once

#include <cstdint>

#include "ccl_tensor.cuh"
#include "ccl_tensor_passes.cuh"

namespace ccl {
namespace tensor {

// ======================================================================
// The product kernel
//
//   out[n, m] = act(alpha * sum_k A[m, k] B[n, k] + bias[m]) + beta * C[n, m]
//
// m runs along the contiguous axis of the output (features), n along its
// rows (tokens), so a thread that owns accumulator lane m writes neighbours
// of its warp's other lanes.  A and B are 16-bit matrices in either storage
// order; a leading index g selects the matrix of a batch or an expert.
// Ragged forms: RAGGED_ROWS (rows n of all experts in one matrix, offsets
// give every expert's range) and RAGGED_REDUCE (the reduction runs over an
// expert's rows).
//
// A threadblock owns 128 features x bn rows of the output at a time.  Warp 0
// streams 128-wide slices of the reduction axis into a ring of shared-memory
// stages with TMA, warp 1 issues tcgen05 matrix instructions into one of two
// accumulators in tensor memory, warps 4..19 drain the other one through the
// epilogue, so that an epilogue costs nothing as long as it is shorter than
// the next tile's products.  Warp 3 clears what a ragged reduction must not
// see.  Two ways to use a cluster:
//   CG = 2: a pair of threadblocks on neighbouring SMs works on 256 features
//     x bn rows with one matrix instruction stream (cta_group::2); each
//     loads its 128 features and half of the rows, so an operand byte taken
//     from L2 feeds twice the products.  For large outputs.
//   split > 1 (CG = 1): the reduction of one tile is cut over the cluster's
//     threadblocks; each then sums its share of the tile's rows, sent by the
//     others through distributed shared memory, in rank order.  For outputs
//     with fewer tiles than SMs.
//
// What bounds it and what it measured (bf16, GB300, GPU time in a graph):
//   many rows: the matrix instructions, at 256 x 256 tiles 620 clocks per 64
//     reduction elements where the instructions alone take 512; 8192 x 8192 x
//     4096 with gelu and both outputs 301 us, 1830 TFLOP/s.  Slices of 128
//     instead of 64 halved the cost of handing slices over (338 -> 304 us),
//     whole warps in the issuing loops keep addresses in uniform registers.
//   few rows: DRAM and the start of a launch; 1 x 4096 x 4096 (33.6 MB) 12 us,
//     37 x 8192 x 2048 11 us, 24 rows over 64 experts of 2048 x 1024 (74 MB for the
//     18 experts that have rows) 19 us.
//   short reductions: the epilogue, about 5000 clocks for 256 x 256 outputs
//     that are only rounded (4096 x 4096 outputs of 64 products each: 15 us),
//     twice that with an activation or a residual (22 and 24 us); sixteen warps,
//     since eight took 1.3 times as long.
//   between: whole waves of tiles (4096 x 4096 x 4096: 78 us, 1750 TFLOP/s),
//     rows that start off a cache line (a 128-byte row of a tile then costs
//     two: 1001 x 5003 takes 30 us at k = 2056, 24 at 2048).
// ======================================================================
constexpr int kTileM = 128;
constexpr int kSliceK = 128;      // reduction elements per stage: two swizzled rows of 64, or 128 rows
constexpr int kMaxStages = 6;
constexpr int kMaxGroups = 1024;
constexpr int kEpilogueWarps = 16;
constexpr int kThreads = 128 + 32 * kEpilogueWarps;
constexpr int kBlockRows = 16;                  // an epilogue warp's block: 16 rows x 32 features
constexpr int kStagingBytes = kEpilogueWarps * kBlockRows * 64;
constexpr int kSmemBudget = 227 * 1024 - 5 * 1024;   // dynamic part; the rest is static

enum { DENSE = 0, RAGGED_ROWS = 1, RAGGED_REDUCE = 2 };

// What a product is, but for its maps: loops keep a copy in registers, since
// a parameter read again after every barrier costs more than it.
struct Scalars {
    int32_t m, n, k, groups;
    int32_t bn, stages, split, tiles_m, tiles_n;
    int32_t per, total;            // tiles of a batch entry, of all (RAGGED_ROWS: counted on the device)
    int32_t ragged, symmetric, act;
    int32_t in_bf, out_bf;
    int32_t a_mn, b_mn;            // stored with consecutive rows (features, or rows of the output) instead of
                                   // consecutive reduction elements
    int32_t tma_out, tma_pre;
    int32_t vec;                   // rows of out, pre, c and bias allow 16-byte accesses
    int32_t pad_c;                 // rows of c are padded to multiples of 8 elements
    int32_t fast;                  // fast_blocks() can take whole tiles
    float alpha, beta;
    const int32_t* offsets;
    uint16_t *out, *pre;           // pre: the sum before the activation (may be null)
    const uint16_t *c, *bias;
    const float *alpha_of, *beta_of;   // device factors per batch entry (may be null)
    int64_t ld_out, bs_out, ld_pre, ld_c, bs_c, bs_bias;
};

struct Product : Scalars {
    CUtensorMap ma, mb, mo, mp;    // operands; out and pre where TMA can store them
};

// The two products of a backward pass in one launch: they read the same dz and
// do not depend on each other, so the second one's tiles fill the places that
// the first one's last wave leaves, and warp 2 of every threadblock, idle
// otherwise, adds up the bias gradient.
struct Pair {
    int32_t width, stages;         // the wider tile's rows; stages of that width
    GradPass sums;                 // sums.db: null if there is no bias gradient
    Product p[2];
};

struct TileAt {
    int g, za, zb;          // group, and its index in the operand maps
    int m0, n0;             // first feature, first row within the group
    int live;               // rows of this tile
    int row0;               // row of the group's first row in the matrices
    int k0, klen;           // reduction range
};

struct Shared {
    uint64_t full[kMaxStages], empty[kMaxStages], acc_full[2], acc_empty[2];
    uint64_t land[kMaxStages], fixed[kMaxStages];   // a ragged reduction's last slice: loaded, cleared
    uint64_t got, taken;           // split: every share has arrived here, every share sent has been read
    uint32_t tmem;
    int failed;
    int total;                     // RAGGED_ROWS: tiles of all experts
    int second;                    // pair: this cluster's first tile of the second product
    int seg_end[kMaxGroups];       // RAGGED_ROWS: tiles of the experts up to each one
};

__device__ __forceinline__ void group_range(const Scalars& P, int g, int limit, int& lo, int& len)
{
    lo = min(max(P.offsets[g], 0), limit);
    len = min(max(P.offsets[g + 1], lo), limit) - lo;
}

// Before the products of a launch with offsets: a check of the offsets, and for
// RAGGED_ROWS the tiles of the experts up to each one.
__device__ __forceinline__ void prepare_tiles(const Scalars& P, Shared* sh)
{
    if (!P.offsets) return;
    const int lane = threadIdx.x & 31;
    if (blockIdx.x == 0) {
        const int limit = P.ragged == RAGGED_ROWS ? P.n : P.k;
        for (int s = threadIdx.x; s < P.groups; s += kThreads) check_offsets(P.offsets, s, limit);
    }
    if (P.ragged == RAGGED_ROWS && threadIdx.x < 32) {
        long long base = 0;
        for (int s = 0; s < P.groups; s += 32) {
            long long v = 0;
            if (s + lane < P.groups) {
                int lo, len;
                group_range(P, s + lane, P.n, lo, len);
                v = P.tiles_m * ((len + P.bn - 1) / P.bn);
            }
#pragma unroll
            for (int d = 1; d < 32; d *= 2) {
                const long long u = __shfl_up_sync(~0u, v, d);
                if (lane >= d) v += u;
            }
            if (s + lane < P.groups) sh->seg_end[s + lane] = (int)(base + v);
            base += __shfl_sync(~0u, v, 31);
        }
        // (only overlapping ranges, reported above, can come to more tiles than there are indexes: none is run)
        if (lane == 0) sh->total = base > INT32_MAX ? 0 : (int)base;
    }
}

__device__ __forceinline__ int find_segment(const Shared* sh, int n, int t)
{
    int lo = 0, hi = n - 1;
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (t < sh->seg_end[mid])
            hi = mid;
        else
            lo = mid + 1;
    }
    return lo;
}

// Position of tile t; tiles are CG * 128 features x bn rows.
template <int CG>
__device__ __forceinline__ TileAt tile_at(const Scalars& P, const Shared* sh, int t)
{
    TileAt q;
    int rows = P.n;
    q.row0 = 0;
    q.k0 = 0;
    q.klen = P.k;
    if (P.ragged == RAGGED_ROWS) {
        q.g = find_segment(sh, P.groups, t);
        const int l = t - (q.g ? sh->seg_end[q.g - 1] : 0);
        group_range(P, q.g, P.n, q.row0, rows);
        // an expert's row tiles of one feature tile are neighbours: they share its weights
        const int tn = (rows + P.bn - 1) / P.bn;
        q.m0 = l / tn * (CG * kTileM);
        q.n0 = l % tn * P.bn;
        q.za = q.g;
        q.zb = 0;
    } else {
        q.g = P.groups == 1 ? 0 : t / P.per;
        int l = t - q.g * P.per;
        if (P.symmetric) {
            // columns of tiles, each from the diagonal on
            int s = 0, first = 0;
            while (l >= P.tiles_n - first) {
                l -= P.tiles_n - first;
                ++s;
                first = s * (CG * kTileM) / P.bn;
            }
            q.m0 = s * (CG * kTileM);
            q.n0 = (first + l) * P.bn;
        } else {
            // bands of feature tiles (2048 features), row tiles inside: the
            // tiles in flight at one time form a compact block of the output
            const int band_w = 16 / CG, area = band_w * P.tiles_n;
            const int band = P.tiles_m <= band_w ? 0 : l / area, r = l - band * area;
            const int width = min(band_w, P.tiles_m - band * band_w), x = r / width;
            q.m0 = (band * band_w + r - x * width) * (CG * kTileM);
            q.n0 = x * P.bn;
        }
        q.za = q.zb = q.g;
        if (P.ragged == RAGGED_REDUCE) {
            group_range(P, q.g, P.k, q.k0, q.klen);
            q.za = q.zb = 0;
        }
    }
    q.live = min(P.bn, rows - q.n0);
    return q;
}

// A threadblock's slices of a tile's reduction: [first, last) of all of them.
__device__ __forceinline__ void slices(const TileAt& q, int parts, int rank, int& first, int& last)
{
    const int ns = (q.klen + kSliceK - 1) / kSliceK;
    first = parts == 1 ? 0 : (int)((int64_t)ns * rank / parts);
    last = parts == 1 ? ns : (int)((int64_t)ns * (rank + 1) / parts);
}
// a slice that runs into the next expert's rows has to be cleared there
__device__ __forceinline__ bool partial(const TileAt& q, int s) { return q.klen - s * kSliceK < kSliceK; }
// rows of a tile that are worth multiplying: a multiple of what one instruction takes
template <int CG>
__device__ __forceinline__ int used_rows(const Scalars& P, const TileAt& q)
{
    return P.ragged == RAGGED_ROWS ? min(P.bn, (q.live + 16 * CG - 1) / (16 * CG) * (16 * CG)) : P.bn;
}

// The part of the epilogue after alpha, for the first `hi` of 8 consecutive
// features f.. of row n, where 16-byte accesses are possible.
__device__ __forceinline__ void finish8(const Scalars& P, float v[8], int g, int64_t n, int f, int hi, float beta)
{
    float w[8];
    if (P.bias) {
        load8(P.bias + g * P.bs_bias + f, P.in_bf, hi, w);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] += w[i];
    }
    if (P.pre) store8(P.pre + n * P.ld_pre + f, P.in_bf, hi, v);
    if (P.act) {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = activate(v[i], P.act);
    }
    if (P.c) {
        load8(P.c + g * P.bs_c + n * P.ld_c + f, P.in_bf, hi, w);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] += beta * w[i];
    }
    store8(P.out + g * P.bs_out + n * P.ld_out + f, P.out_bf, hi, v);
}

__device__ __forceinline__ void finish1(const Scalars& P, float v, int g, int64_t n, int f, float beta, float bias,
                                        float c)
{
    v += bias;
    if (P.pre) store1(P.pre + n * P.ld_pre + f, v, P.in_bf);
    if (P.act) v = activate(v, P.act);
    store1(P.out + g * P.bs_out + n * P.ld_out + f, v + beta * c, P.out_bf);
}

// A block's rows of C at one feature per lane: 64 neighbouring bytes a row and
// warp, whatever the alignment.
__device__ __forceinline__ void fetch_c(const Scalars& P, uint16_t c[kBlockRows], int g, int64_t row, int nrows, int f)
{
    const uint16_t* p = P.c + g * P.bs_c + row * P.ld_c + f;
#pragma unroll
    for (int i = 0; i < kBlockRows; ++i, p += P.ld_c) c[i] = f < P.m && i < nrows ? __ldcg(p) : (uint16_t)0;
}

// A block of 16 rows x 32 features (one feature per lane, two rows per word)
// to global memory: through shared memory and a TMA store where the whole
// block may be written (the parts of it outside the matrix are cut off by
// TMA), else 64 neighbouring bytes of a row at a time.  buf: this warp's 1 KB
// of shared memory.
__device__ __forceinline__ void store_block(const CUtensorMap* map, uint16_t* p, int64_t ld, const uint32_t w[kBlockRows / 2],
                                            unsigned char* buf, bool tma, int lane, int x, int y, int z, int nrows,
                                            int nfeat)
{
    if (tma && nfeat > 0) {
        if (lane == 0) tma_stores_read<0>();
        __syncwarp();
        uint16_t* b = reinterpret_cast<uint16_t*>(buf) + lane;
#pragma unroll
        for (int i = 0; i < kBlockRows / 2; ++i) {
            b[i * 64] = (uint16_t)w[i];
            b[i * 64 + 32] = (uint16_t)(w[i] >> 16);
        }
        fence_async();
        __syncwarp();
        if (lane == 0) tma_store(map, smem_addr(buf), x, y, z);
    } else if (lane < nfeat) {
#pragma unroll
        for (int i = 0; i < kBlockRows; ++i, p += ld)
            if (i < nrows) *p = (uint16_t)(w[i / 2] >> (i & 1) * 16);
    }
}

__device__ __forceinline__ void pack_block(const float v[kBlockRows], uint32_t w[kBlockRows / 2], bool bf)
{
    if (bf) {
#pragma unroll
        for (int i = 0; i < kBlockRows / 2; ++i) w[i] = pack2<true>(v[2 * i], v[2 * i + 1]);
    } else {
#pragma unroll
        for (int i = 0; i < kBlockRows / 2; ++i) w[i] = pack2<false>(v[2 * i], v[2 * i + 1]);
    }
}

// A warp's whole blocks of a tile whose outputs TMA can store (and whose C, if
// any, can be read in pieces of 16 bytes), with what varies between products
// decided beforehand: half the instructions of the general way.  C is read a
// block ahead, two pieces of 8 features a lane, and turned through the block's
// shared memory to a feature a lane.  SYM: a symmetric output, of which blocks
// above the diagonal are left out, blocks that touch it are written as they are
// (together they hold both sides of it: tiles start at multiples of 32), and
// blocks below it are written with their mirror images.
template <int ACT, bool ADD, bool SYM = false>
__device__ __forceinline__ void fast_blocks(const Scalars& P, const CUtensorMap* map, uint32_t from, int first, int live,
                                            int stride, float alpha, float bias, float beta, unsigned char* buf, int lane,
                                            int x, int nfeat, int64_t row, int g, int z)
{
    const uint32_t at = smem_addr(buf) + lane * 2, piece = smem_addr(buf) + lane * 16;
    const bool out_bf = P.out_bf, in_bf = P.in_bf;
    const uint16_t* pc = nullptr;
    int64_t ld = 0;
    uint4 c0, c1;
    const int cr = lane >> 2, ck = (lane & 3) * 8;
    auto fetch = [&](int c) {
        c0 = c1 = make_uint4(0, 0, 0, 0);
        if (ck < nfeat) {               // a piece that the matrix cuts short lies in its row's padding
            const uint16_t* p = pc + c * ld;
            if (c + cr < live) c0 = __ldcg(reinterpret_cast<const uint4*>(p));
            if (c + cr + 8 < live) c1 = __ldcg(reinterpret_cast<const uint4*>(p + 8 * ld));
        }
    };
    if (ADD) {
        ld = P.ld_c;
        pc = P.c + g * P.bs_c + (row + cr) * ld + x + ck;
        fetch(first);
    }
#pragma unroll 1
    for (int c = first; c < live; c += stride) {
        const int over = x + 31 - ((int)row + c);        // > 0 where the block reaches above the diagonal
        if (SYM && over >= 31 + kBlockRows) {
            if (ADD && c + stride < live) fetch(c + stride);
            continue;
        }
        float v[kBlockRows];
        {
            uint32_t u[kBlockRows];
            tmem_load16(from + c, u);
#pragma unroll
            for (int i = 0; i < kBlockRows; ++i) v[i] = fmaf(alpha, __uint_as_float(u[i]), bias);
        }
        if (ACT) {
#pragma unroll
            for (int i = 0; i < kBlockRows; ++i) v[i] = activate(v[i], ACT);
        }
        if (lane == 0) tma_stores_read<0>();
        __syncwarp();
        if (ADD) {
            asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};\n\tst.shared.v4.b32 [%0 + 512], {%5, %6, %7, %8};" ::"r"(piece),
                         "r"(c0.x), "r"(c0.y), "r"(c0.z), "r"(c0.w), "r"(c1.x), "r"(c1.y), "r"(c1.z), "r"(c1.w)
                         : "memory");
            __syncwarp();
            if (c + stride < live) fetch(c + stride);
#pragma unroll
            for (int i = 0; i < kBlockRows; ++i) {
                uint16_t h;
                asm volatile("ld.shared.b16 %0, [%1];" : "=h"(h) : "r"(at + i * 64));
                v[i] += beta * (in_bf ? __uint_as_float((uint32_t)h << 16) : __half2float(__ushort_as_half(h)));
            }
            __syncwarp();
        }
        uint32_t w[kBlockRows / 2];
        pack_block(v, w, out_bf);
#pragma unroll
        for (int i = 0; i < kBlockRows; i += 2)
            asm volatile("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\t"
                         "st.shared.b16 [%0], l;\n\tst.shared.b16 [%0 + 64], h;\n\t}" ::"r"(at + i * 64), "r"(w[i / 2])
                         : "memory");
        fence_async();
        __syncwarp();
        if (lane == 0) tma_store(map, smem_addr(buf), x, (int)row + c, z);
        if (SYM && over <= 0 && lane < nfeat) {
            // a lane's 16 values are neighbours in the row of its feature; rows are padded to multiples of 8 (with zeros)
            uint4* m = reinterpret_cast<uint4*>(P.out + g * P.bs_out + (int64_t)(x + lane) * P.ld_out + row + c);
            m[0] = make_uint4(w[0], w[1], w[2], w[3]);
            if (c + 8 < live) m[1] = make_uint4(w[4], w[5], w[6], w[7]);
        }
    }
}

// FORM: storage of the operands (a pair: A_MN, then BOTH_MN)
enum { BOTH_K = 0, A_MN = 1, BOTH_MN = 2 };

// MODE: one product, or the two of a Pair
enum { SINGLE = 0, PAIR = 1 };

template <int MODE>
struct Sequence {
    const Product* list;
    __device__ int width() const { return list->bn; }
    __device__ int stages() const { return list->stages; }
    __device__ int split() const { return list->split; }
    __device__ int phases() const { return 1; }
    __device__ const Product& at(int) const { return *list; }
};
template <>
struct Sequence<PAIR> {
    const Pair* pair;
    __device__ int width() const { return pair->width; }
    __device__ int stages() const { return pair->stages; }
    __device__ int split() const { return 1; }
    __device__ int phases() const { return 2; }
    __device__ const Product& at(int ph) const { return pair->p[ph]; }
};

// A threadblock's share of the tiles of a sequence of products.
template <int CG, int FORM, int MODE>
__device__ __forceinline__ void products(const Sequence<MODE> seq)
{
    __shared__ __align__(8) Shared sh;
    extern __shared__ unsigned char raw[];
    unsigned char* dyn = raw + ((1024 - (smem_addr(raw) & 1023)) & 1023);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int size = CG == 2 ? 2 : seq.split();             // threadblocks of the cluster
    const int rank = size > 1 ? (int)cluster_rank() : 0;
    const int cluster = blockIdx.x / size, clusters = gridDim.x / size;
    const int width = seq.width(), stages = seq.stages(), phases = seq.phases();
    const uint32_t bytes_a = kTileM * kSliceK * 2;
    const uint32_t step = bytes_a + width / CG * kSliceK * 2;          // from one stage to the next
    unsigned char* staging = dyn + (size_t)stages * step;
    float* shares = reinterpret_cast<float*>(staging + kStagingBytes);   // split: [source][row][feature], own rows
    uint32_t tcols = 64;
    while (tcols < 2u * width) tcols *= 2;

    if (threadIdx.x < kMaxStages) {
        const int i = threadIdx.x;
        bar_init(smem_addr(&sh.full[i]), 1);
        bar_init(smem_addr(&sh.empty[i]), 1);
        bar_init(smem_addr(&sh.land[i]), 1);
        bar_init(smem_addr(&sh.fixed[i]), CG);
        if (i < 2) {
            bar_init(smem_addr(&sh.acc_full[i]), 1);
            bar_init(smem_addr(&sh.acc_empty[i]), CG * kEpilogueWarps);
        }
        if (i == 2) bar_init(smem_addr(&sh.got), size * kEpilogueWarps);
        if (i == 3) bar_init(smem_addr(&sh.taken), size * kEpilogueWarps);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (threadIdx.x == 32) {
        sh.failed = 0;
        tma_prefetch(&seq.at(0).ma);
        tma_prefetch(&seq.at(0).mb);
    }
    if (seq.at(0).offsets) wait_for_previous();
    prepare_tiles(seq.at(0), &sh);
    if (MODE == PAIR && threadIdx.x == 0) {
        const int total = seq.at(0).ragged == RAGGED_ROWS ? sh.total : seq.at(0).total;
        sh.second = (cluster + clusters - total % clusters) % clusters;
    }
    if (size > 1)
        cluster_sync();
    else
        __syncthreads();
    volatile int* failed = &sh.failed;
    // Loads start while tensor memory is being allocated; everything up to
    // here overlaps the end of the kernel before this one, on SMs that it has
    // left (two of these kernels need more registers than an SM has).  The next
    // kernel is let in only when this one holds its tensor memory: on a shared
    // SM it could otherwise take it first and wait for this one to end.
    uint32_t tmem = 0;
    if (warp == 2) {
        tmem_alloc<CG>(smem_addr(&sh.tmem), tcols);
        let_next_in();
    }
    if (warp != 0 && warp != 3) {
        fence_before();
        named_sync(1, 64 + 32 * kEpilogueWarps);
        fence_after();
        tmem = sh.tmem;
    }

    // This threadblock's (cluster's) tiles of the next product: every
    // `clusters`-th one, so that tiles in flight at a time share operands
    // (ranges of consecutive tiles, balanced by their cost, took 168 us
    // instead of 117 for 8190 rows over 32 experts of 4096 x 2048; row tiles of
    // equal length changed nothing there: the weights' 440 MB bound it).  In a pair
    // the second product's go on where the first one's stopped.
    struct Run {
        int begin, end;
    };
    auto next_run = [&](const Scalars& P, int ph) {
        return Run{MODE == PAIR && ph ? sh.second : cluster, P.ragged == RAGGED_ROWS ? sh.total : P.total};
    };

    const uint32_t ring = smem_addr(dyn), full0 = smem_addr(sh.full), empty0 = smem_addr(sh.empty);

    // A wait that fails does not change the way through these loops: it only
    // keeps them from issuing anything more, and later waits return at once.
    if (warp == 0) {
        int s = 0, loaded = 0;
        uint32_t phase = 0;                // of the current stage
        uint32_t flips = 0, used = 0;      // per stage: parity of its uses for cleared slices, whether any
        bool good = true;
        for (int ph = 0; ph < phases; ++ph) {
            const Product& maps = seq.at(ph);
            const Scalars P = maps;
            if (MODE != SINGLE && ph + 1 < phases && lane == 0) {
                tma_prefetch(&seq.at(ph + 1).ma);
                tma_prefetch(&seq.at(ph + 1).mb);
            }
            const bool a_mn = MODE == PAIR || FORM != BOTH_K;
            const bool b_mn = MODE == PAIR ? ph == 1 : FORM == BOTH_MN;
            const uint32_t bytes_b = P.bn / CG * kSliceK * 2;
            const uint32_t part_b = bytes_b / 2;      // one of a slice's two halves of B (reduction 0..63, 64..127)
            const uint32_t bytes = bytes_a + bytes_b;
            const bool reduce_rows = b_mn && P.ragged == RAGGED_REDUCE;
            const int bn = P.bn;
            // the first tile is found before the wait for what it reads
            TileAt q;
            const Run run = next_run(P, ph);
            if (run.begin < run.end) q = tile_at<CG>(P, &sh, run.begin);
            if (ph == 0) wait_for_previous();
            for (int t = run.begin; t < run.end; t += clusters) {
                if (t != run.begin) q = tile_at<CG>(P, &sh, t);
                const int m0 = q.m0 + (CG == 2 ? rank * kTileM : 0);
                const int n0 = q.n0 + (CG == 2 ? rank * (used_rows<CG>(P, q) / 2) : 0);
                int first, last;
                slices(q, CG == 2 ? 1 : size, rank, first, last);
                for (int j = first; j < last; ++j) {
                    const int k = j * kSliceK;
                    if (good) good = bar_wait(empty0 + s * 8, phase ^ 1, failed);
                    const uint32_t a = ring + s * step, b = a + bytes_a;
                    uint32_t bar = full0 + s * 8;
                    const bool clear = reduce_rows && partial(q, j);
                    if (elect_one() && good) {
                        if (clear) {
                            // lands on a barrier of this threadblock, for warp 3
                            if (rank == 0 || CG == 1) bar_arrive(bar);
                            bar = smem_addr(&sh.land[s]);
                            bar_expect(bar, bytes);
                        } else if (CG == 1) {
                            bar_expect(bar, bytes);
                        } else {
                            if (rank == 0) bar_expect(bar, 2 * bytes);
                            bar = cluster_addr(bar, 0);
                        }
                        auto load = [&](uint32_t dst, const CUtensorMap* map, int x, int y, int z) {
                            if (CG == 1)
                                tma_load(dst, map, bar, x, y, z);
                            else
                                tma_load_pair(dst, map, bar, x, y, z);
                        };
                        if (a_mn) {
                            load(a, &maps.ma, m0, q.k0 + k, q.za);
                            load(a + kSliceK * 128, &maps.ma, m0 + 64, q.k0 + k, q.za);
                        } else {
                            load(a, &maps.ma, k, m0, q.za);
                            load(a + kTileM * 128, &maps.ma, k + 64, m0, q.za);
                        }
                        if (b_mn) {
                            for (int i = 0; i < bn / CG; i += 64)
                                load(b + i * (kSliceK * 2), &maps.mb, n0 + i, q.k0 + k, q.zb);
                        } else {
                            load(b, &maps.mb, k, q.row0 + n0, q.zb);
                            load(b + part_b, &maps.mb, k + 64, q.row0 + n0, q.zb);
                        }
                    }
                    if (clear && good) flips ^= 1u << s, used |= 1u << s;
                    if (good) ++loaded;
                    if (++s == stages) s = 0, phase ^= 1;
                }
            }
        }
        // copies in flight write this threadblock's shared memory: see the
        // last one of every stage land before leaving
        int none = 0;
        if (CG == 1 || rank == 0)
            for (int i = max(0, loaded - stages); i < loaded; ++i)
                bar_wait(full0 + i % stages * 8, i / stages & 1, &none);
        for (int i = 0; i < stages; ++i)
            if (used >> i & 1) bar_wait(smem_addr(&sh.land[i]), (flips >> i & 1) ^ 1, &none);
        __syncwarp();
    } else if (warp == 1) {
        if (CG == 1 || rank == 0) {
            const uint32_t lead = kSliceK * 128;
            const uint64_t base = operand_desc(0, lead, 1024);
            // (in a cluster the upper bits of a shared-memory address tell the threadblock)
            const uint32_t ring_at = (ring & 0x3ffff) >> 4;
            const uint32_t acc_full0 = smem_addr(sh.acc_full), acc_empty0 = smem_addr(sh.acc_empty);
            int s = 0, issued = 0, done = 0;
            uint32_t phase = 0, flips = 0;
            bool good = true;
            for (int ph = 0; ph < phases; ++ph) {
                const Scalars P = seq.at(ph);
                const bool a_mn = MODE == PAIR || FORM != BOTH_K;
                const bool b_mn = MODE == PAIR ? ph == 1 : FORM == BOTH_MN;
                const uint32_t bytes_b = P.bn / CG * kSliceK * 2;
                const uint32_t part_b = bytes_b / 2;      // one of a slice's two halves of B (reduction 0..63, 64..127)
                const bool reduce_rows = b_mn && P.ragged == RAGGED_REDUCE;
                const Run run = next_run(P, ph);
                for (int t = run.begin; t < run.end; t += clusters) {
                    const TileAt q = tile_at<CG>(P, &sh, t);
                    int first, last;
                    slices(q, CG == 2 ? 1 : size, rank, first, last);
                    if (first >= last) continue;
                    const uint32_t idesc = mma_desc(P.in_bf, a_mn, b_mn, CG * kTileM, used_rows<CG>(P, q));
                    const int acc = done & 1;
                    const uint32_t d = tmem + acc * width;
                    if (good) good = bar_wait(acc_empty0 + acc * 8, ((done >> 1) & 1) ^ 1, failed);
                    fence_after();
                    for (int j = first; j < last; ++j) {
                        if (good) good = bar_wait(full0 + s * 8, phase, failed);
                        if (reduce_rows && partial(q, j)) {
                            if (good) good = bar_wait<CG == 2>(smem_addr(&sh.fixed[s]), flips >> s & 1, failed);
                            flips ^= 1u << s;
                        }
                        const uint32_t a = ring_at + s * (step >> 4), b = a + (bytes_a >> 4);
                        const int steps = min(kSliceK / 16, (q.klen - j * kSliceK + 15) / 16);   // of 16 reduction elements
                        if (elect_one() && good) {
#pragma unroll
                            for (int i = 0; i < kSliceK / 16; ++i) {
                                // 16 reduction elements: 16 rows of 128 bytes, or 32 bytes along a row of 64
                                const uint32_t at_a = a + ((a_mn ? i * 2048 : i / 4 * (kTileM * 128) + i % 4 * 32) >> 4);
                                const uint32_t at_b = b + (b_mn ? i * 2048 >> 4 : (i / 4) * (part_b >> 4) + (i % 4 * 32 >> 4));
                                if (i < steps) mma_f16<CG>(d, base | at_a, base | at_b, idesc, j > first || i > 0);
                            }
                            mma_commit<CG>(empty0 + s * 8);
                            if (j + 1 == last) mma_commit<CG>(acc_full0 + acc * 8);
                        }
                        if (good) ++issued;
                        if (++s == stages) s = 0, phase ^= 1;
                    }
                    ++done;
                }
            }
            if (!good && issued) {
                // matrix instructions still in flight read shared memory and
                // write tensor memory: wait (bounded) until all have finished
                int none = 0;
                bar_wait(empty0 + (issued - 1) % stages * 8, (issued - 1) / stages & 1, &none);
            }
        }
        __syncwarp();
    } else if (warp == 2 && MODE == PAIR) {
        if constexpr (MODE == PAIR) {
            if (seq.pair->sums.db) {
                wait_for_previous();
                add_chunks(seq.pair->sums, lane);
            }
        }
        __syncwarp();
    } else if (warp == 3 && (MODE == PAIR || FORM == BOTH_MN) && seq.at(phases - 1).ragged == RAGGED_REDUCE) {
        // 0 x Inf or NaN would not be 0: both operands are cleared
        int it = 0;
        uint32_t flips = 0;
        bool good = true;
        for (int ph = 0; ph < phases; ++ph) {
            const Scalars P = seq.at(ph);
            const Run run = next_run(P, ph);
            for (int t = run.begin; good && t < run.end; t += clusters) {
                const TileAt q = tile_at<CG>(P, &sh, t);
                int first, last;
                slices(q, CG == 2 ? 1 : size, rank, first, last);
                if (first >= last) continue;
                it += last - first;
                if (P.ragged != RAGGED_REDUCE || !partial(q, last - 1)) continue;
                const int s = (it - 1) % stages;
                good = __all_sync(~0u, bar_wait(smem_addr(&sh.land[s]), flips >> s & 1, failed));
                if (!good) break;
                flips ^= 1u << s;
                unsigned char* at = dyn + (size_t)s * step;
                // only as far as the matrix instructions reach: 16 rows at a time
                const int left = q.klen - (last - 1) * kSliceK, dead = -left & 15;
                for (int i = lane; i < (P.bn / CG + kTileM) / 64 * dead * 8; i += 32) {
                    const int blk = i / (dead * 8), o = i % (dead * 8);
                    *reinterpret_cast<uint4*>(at + blk * (kSliceK * 128) + left * 128 + o * 16) = make_uint4(0, 0, 0, 0);
                }
                fence_async();
                __syncwarp();
                if (lane == 0) {
                    if (CG == 2)
                        bar_arrive_cluster(cluster_addr(smem_addr(&sh.fixed[s]), 0));
                    else
                        bar_arrive(smem_addr(&sh.fixed[s]));
                }
            }
        }
        __syncwarp();
    } else if (warp >= 4) {
        const int quad = warp & 3, slot = (warp - 4) >> 2;
        constexpr int kStride = kEpilogueWarps / 4 * kBlockRows;     // rows that the warps of a quadrant take at once
        // the products of a pair are only rounded: no bias, activation, C, split or mirror image
        constexpr bool kAll = MODE == SINGLE;
        unsigned char* st = staging + (warp - 4) * (kBlockRows * 64);
        uint32_t release[2];
        for (int i = 0; i < 2; ++i)
            release[i] = CG == 2 ? cluster_addr(smem_addr(&sh.acc_empty[i]), 0) : smem_addr(&sh.acc_empty[i]);
        int done = 0, round = 0;
        for (int ph = 0; ph < phases; ++ph) {
            const Product& maps = seq.at(ph);
            const Scalars P = maps;
            const int side = kAll && P.symmetric ? 1 : 0;
            TileAt q;
            const Run run = next_run(P, ph);
            if (run.begin < run.end) q = tile_at<CG>(P, &sh, run.begin);
            if (ph == 0) wait_for_previous();
            for (int t = run.begin; t < run.end; t += clusters) {
                if (t != run.begin) q = tile_at<CG>(P, &sh, t);
                int first, last;
                slices(q, CG == 2 ? 1 : size, rank, first, last);
                const bool some = first < last;
                const int acc = done & 1;
                const int feat = q.m0 + (CG == 2 ? rank * kTileM : 0) + quad * 32, nfeat = P.m - feat, f = feat + lane;
                const int64_t row = (int64_t)q.row0 + q.n0;
                const float alpha = P.alpha * (kAll && P.alpha_of ? P.alpha_of[q.g] : 1.f);
                const float beta = P.beta * (P.beta_of ? P.beta_of[q.g] : 1.f);
                const float bias = kAll && P.bias && f < P.m ? load1(P.bias + q.g * P.bs_bias + f, P.in_bf) : 0.f;
                const bool whole = P.ragged != RAGGED_ROWS;
                const int zo = P.ragged == RAGGED_ROWS ? 0 : q.g;
                // rows that the short way takes: an expert's last rows may end inside a block, and TMA cuts rows off at
                // the end of the matrix only
                const int short_to = !(some && P.fast && nfeat > 0) ? 0 : whole ? q.live : q.live & -kBlockRows;
                int c = slot * kBlockRows;          // this warp's next block
                uint16_t cv[kBlockRows];
                // the general way reads C a block ahead of its use, the short way reads it by itself
                if (kAll && P.c && size == CG && !short_to) fetch_c(P, cv, q.g, row + c, q.live - c, f);
                if (some) {
                    if (!__all_sync(~0u, bar_wait(smem_addr(&sh.acc_full[acc]), (done >> 1) & 1, failed))) break;
                    fence_after();
                }
                if (kAll && size > CG) {
                    // shares of the last tile have been read by their owners
                    if (!__all_sync(~0u, bar_wait<true>(smem_addr(&sh.taken), (round & 1) ^ 1, failed))) break;
                }
                const uint32_t from = tmem + ((uint32_t)(quad * 32) << 16) + acc * width;
                if (short_to) {
#define FAST(...)                                                                                                       \
    fast_blocks<__VA_ARGS__>(P, &maps.mo, from, c, short_to, kStride, alpha, bias, beta, st, lane, feat, nfeat, row, q.g, zo)
                    if (kAll && side) {
                        if (P.c && c < short_to) FAST(ACT_NONE, true, true);
                        if (!P.c) FAST(ACT_NONE, false, true);
                    } else if (!kAll) {
                        FAST(ACT_NONE, false);
                    } else if (P.c) {
                        if (c < short_to) FAST(ACT_NONE, true);
                    } else if (P.act == ACT_NONE) {
                        FAST(ACT_NONE, false);
                    } else if (P.act == ACT_RELU) {
                        FAST(ACT_RELU, false);
                    } else if (P.act == ACT_GELU) {
                        FAST(ACT_GELU, false);
                    } else {
                        FAST(ACT_SILU, false);
                    }
#undef FAST
                    while (c < short_to) c += kStride;
                    if (kAll && P.c && c < q.live) fetch_c(P, cv, q.g, row + c, q.live - c, f);
                }
                for (; c < q.live; c += kStride) {
                    uint32_t u[kBlockRows];
                    if (some) {
                        tmem_load16(from + c, u);
                    } else {
#pragma unroll
                        for (int i = 0; i < kBlockRows; ++i) u[i] = 0;
                    }
                    const int nrows = q.live - c;
                    if (kAll && size > CG) {
                        const int own = P.bn / size;
                        const uint32_t at = smem_addr(shares + (size_t)rank * own * kTileM + quad * 32 + lane);
                        // own is a power of two from 4 up: 4 rows at a time go to one owner
#pragma unroll
                        for (int i = 0; i < kBlockRows; i += 4) {
                            const int r = c + i;
                            const uint32_t to = cluster_addr(at + r % own * (kTileM * 4), r / own);
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                if (i + e < nrows) store_cluster(to + e * (kTileM * 4), __uint_as_float(u[i + e]));
                        }
                        continue;
                    }
                    float v[kBlockRows];
                    uint32_t w[kBlockRows / 2];
#pragma unroll
                    for (int i = 0; i < kBlockRows; ++i) v[i] = fmaf(alpha, __uint_as_float(u[i]), bias);
                    if (kAll && P.pre) {
                        pack_block(v, w, P.in_bf);
                        store_block(&maps.mp, P.pre + (row + c) * P.ld_pre + f, P.ld_pre, w, st,
                                    P.tma_pre && (whole || nrows >= kBlockRows), lane, feat, (int)row + c, 0, nrows, nfeat);
                    }
                    if (kAll && P.act == ACT_RELU) {
#pragma unroll
                        for (int i = 0; i < kBlockRows; ++i) v[i] = activate(v[i], ACT_RELU);
                    } else if (kAll && P.act == ACT_GELU) {
#pragma unroll
                        for (int i = 0; i < kBlockRows; ++i) v[i] = activate(v[i], ACT_GELU);
                    } else if (kAll && P.act == ACT_SILU) {
#pragma unroll
                        for (int i = 0; i < kBlockRows; ++i) v[i] = activate(v[i], ACT_SILU);
                    }
                    if (kAll && P.c) {
                        if (P.in_bf) {
#pragma unroll
                            for (int i = 0; i < kBlockRows; ++i) v[i] += beta * __uint_as_float((uint32_t)cv[i] << 16);
                        } else {
#pragma unroll
                            for (int i = 0; i < kBlockRows; ++i) v[i] += beta * __half2float(__ushort_as_half(cv[i]));
                        }
                        if (c + kStride < q.live) fetch_c(P, cv, q.g, row + c + kStride, nrows - kStride, f);
                    }
                    pack_block(v, w, P.out_bf);
                    store_block(&maps.mo, P.out + q.g * P.bs_out + (row + c) * P.ld_out + f, P.ld_out, w, st,
                                P.tma_out && (whole || nrows >= kBlockRows), lane, feat, (int)row + c, zo, nrows, nfeat);
                }
                if (some) {
                    fence_before();
                    if (lane == 0) {
                        if (CG == 2)
                            bar_arrive_cluster(release[acc]);
                        else
                            bar_arrive(release[acc]);
                    }
                    ++done;
                }
                if (kAll && size > CG) {
                    __syncwarp();
                    if (lane < size) bar_arrive_cluster(cluster_addr(smem_addr(&sh.got), lane));
                    if (!__all_sync(~0u, bar_wait<true>(smem_addr(&sh.got), round & 1, failed))) break;
                    // sum the shares of this threadblock's rows in rank order
                    const int own = P.bn / size, base = rank * own, mine = min(own, q.live - base);
                    const int id = (warp - 4) * 32 + lane;
                    if (P.vec) {
                        for (int i = id; i < mine * (kTileM / 8); i += 32 * kEpilogueWarps) {
                            const int r = i / (kTileM / 8), f = i % (kTileM / 8) * 8, hi = min(8, P.m - q.m0 - f);
                            if (hi <= 0) continue;
                            float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
                            for (int s = 0; s < size; ++s) {
                                const float4* p =
                                    reinterpret_cast<const float4*>(shares + ((size_t)s * own + r) * kTileM + f);
                                const float4 a = p[0], b = p[1];
                                v[0] += a.x, v[1] += a.y, v[2] += a.z, v[3] += a.w;
                                v[4] += b.x, v[5] += b.y, v[6] += b.z, v[7] += b.w;
                            }
#pragma unroll
                            for (int e = 0; e < 8; ++e) v[e] *= alpha;
                            finish8(P, v, q.g, row + base + r, q.m0 + f, hi, beta);
                        }
                    } else {
                        for (int i = id; i < mine * kTileM; i += 32 * kEpilogueWarps) {
                            const int r = i / kTileM, f = q.m0 + i % kTileM;
                            const int64_t n = row + base + r;
                            if (f >= P.m) continue;
                            float v = 0.f;
                            for (int s = 0; s < size; ++s) v += shares[((size_t)s * own + r) * kTileM + i % kTileM];
                            finish1(P, alpha * v, q.g, n, f, beta,
                                    P.bias ? load1(P.bias + q.g * P.bs_bias + f, P.in_bf) : 0.f,
                                    P.c ? load1(P.c + q.g * P.bs_c + n * P.ld_c + f, P.in_bf) : 0.f);
                        }
                    }
                    __syncwarp();
                    if (lane < size) bar_arrive_cluster(cluster_addr(smem_addr(&sh.taken), lane));
                    ++round;
                }
            }
        }
        fence_before();
        if (CG == 1) named_arrive(2, 32 + 32 * kEpilogueWarps);
        if (lane == 0) tma_stores_read<0>();
    }
    if (CG == 1 && warp == 2) {
        // tensor memory is free as soon as the last accumulator has been read
        named_sync(2, 32 + 32 * kEpilogueWarps);
        fence_after();
        tmem_free<1>(tmem, tcols);
    }
    if (sh.failed && lane == 0) atomicCAS(&g_status[0], 0, (int)CCL_ERR_TIMEOUT);
    __syncwarp();
    // no threadblock leaves while another one of its cluster may still reach
    // its memory or its barriers
    if (size > 1)
        cluster_sync();
    else
        __syncthreads();
    if (CG == 2 && warp == 2) {
        fence_after();
        tmem_free<2>(tmem, tcols);
    }
}

template <int CG, int FORM>
__global__ void __launch_bounds__(kThreads, 1) product_kernel(const __grid_constant__ Product P)
{
    products<CG, FORM, SINGLE>({&P});
}
template <int CG>
__global__ void __launch_bounds__(kThreads, 1) pair_kernel(const __grid_constant__ Pair P)
{
    products<CG, A_MN, PAIR>({&P});
}

}  // namespace tensor
}  // namespace ccl
