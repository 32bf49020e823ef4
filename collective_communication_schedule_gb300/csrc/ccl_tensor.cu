// Tensor products of language-model layers: dense products with a fused
// epilogue, products grouped by expert over ragged rows, and the
// Newton-Schulz orthogonalisation of gradient matrices.  C ABI in
// include/ccl.h; PTX building blocks in ccl_tensor.cuh.
#include <algorithm>
#include <cmath>
#include <cstring>
#include <mutex>
#include <string>

#include <cuda_runtime.h>

#include "ccl_internal.h"
#include "ccl_tensor.cuh"

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

// The two products of a backward pass in one launch: they read the same dz and
// do not depend on each other, so the second one's tiles fill the places that
// the first one's last wave leaves, and warp 2 of every threadblock, idle
// otherwise, adds up the bias gradient.
struct Pair {
    int32_t width, stages;         // the wider tile's rows; stages of that width
    GradPass sums;                 // sums.db: null if there is no bias gradient
    Product p[2];
};

// [0]: a ccl_status_t of a failed launch on this device, 0 if none
__device__ int g_status[4];

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
        for (int s = threadIdx.x; s < P.groups; s += kThreads)
            if (P.offsets[s] < 0 || P.offsets[s + 1] < P.offsets[s] || P.offsets[s + 1] > limit)
                atomicCAS(&g_status[0], 0, (int)CCL_ERR_INVALID_ARG);
    }
    if (P.ragged == RAGGED_ROWS && threadIdx.x < 32) {
        int base = 0;
        for (int s = 0; s < P.groups; s += 32) {
            int v = 0;
            if (s + lane < P.groups) {
                int lo, len;
                group_range(P, s + lane, P.n, lo, len);
                v = P.tiles_m * ((len + P.bn - 1) / P.bn);
            }
#pragma unroll
            for (int d = 1; d < 32; d *= 2) {
                const int u = __shfl_up_sync(~0u, v, d);
                if (lane >= d) v += u;
            }
            if (s + lane < P.groups) sh->seg_end[s + lane] = base + v;
            base += __shfl_sync(~0u, v, 31);
        }
        if (lane == 0) sh->total = base;
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

// FORM: storage of the operands (a pair: A_MN, then BOTH_MN)
enum { BOTH_K = 0, A_MN = 1, BOTH_MN = 2 };

// Sum a bias gradient's chunks, 32 columns of one expert at a time.
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
        float s = 0.f;
#pragma unroll 8
        for (int i = 0; i < chunks; ++i) s += p[i * G.ld_part];
        store1(G.db + e * G.bs_db + c, s, G.bf);
    }
}

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
    let_next_in();
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
    // loads start while tensor memory is being allocated; everything up to
    // here overlaps the end of the kernel before this one
    uint32_t tmem = 0;
    if (warp == 2) tmem_alloc<CG>(smem_addr(&sh.tmem), tcols);
    if (warp != 0 && warp != 3) {
        fence_before();
        named_sync(1, 64 + 32 * kEpilogueWarps);
        fence_after();
        tmem = sh.tmem;
    }

    // This threadblock's (cluster's) tiles of the next product: every
    // `clusters`-th one, so that tiles in flight at a time share operands
    // (ranges of consecutive tiles, balanced by their cost, took 168 us
    // instead of 117 for 8190 rows over 32 experts of 4096 x 2048).  In a pair
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
            __syncwarp();
        }
    } else if (warp == 3 && (MODE == PAIR || FORM == BOTH_MN) &&
               seq.at(phases - 1).ragged == RAGGED_REDUCE) {
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
        // what the products of a mode can have
        constexpr bool kLayer = MODE == SINGLE, kAdds = MODE != PAIR;
        unsigned char* st = staging + (warp - 4) * (kBlockRows * 64);
        uint32_t release[2];
        for (int i = 0; i < 2; ++i)
            release[i] = CG == 2 ? cluster_addr(smem_addr(&sh.acc_empty[i]), 0) : smem_addr(&sh.acc_empty[i]);
        int done = 0, round = 0;
        for (int ph = 0; ph < phases; ++ph) {
            const Product& maps = seq.at(ph);
            const Scalars P = maps;
            const int side = kAdds && P.symmetric ? 1 : 0;
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
                const float alpha = P.alpha * (kAdds && P.alpha_of ? P.alpha_of[q.g] : 1.f);
                const float beta = P.beta * (P.beta_of ? P.beta_of[q.g] : 1.f);
                const float bias = kLayer && P.bias && f < P.m ? load1(P.bias + q.g * P.bs_bias + f, P.in_bf) : 0.f;
                const bool whole = P.ragged != RAGGED_ROWS;    // TMA may cut rows off at the end of the matrix only
                const int zo = P.ragged == RAGGED_ROWS ? 0 : q.g;
                uint16_t cv[kBlockRows];
                // C is read a block ahead of its use
                if (kAdds && P.c && size == CG) fetch_c(P, cv, q.g, row + slot * kBlockRows, q.live - slot * kBlockRows, f);
                if (some) {
                    if (!__all_sync(~0u, bar_wait(smem_addr(&sh.acc_full[acc]), (done >> 1) & 1, failed))) break;
                    fence_after();
                }
                if (kLayer && size > CG) {
                    // shares of the last tile have been read by their owners
                    if (!__all_sync(~0u, bar_wait<true>(smem_addr(&sh.taken), (round & 1) ^ 1, failed))) break;
                }
                const uint32_t from = tmem + ((uint32_t)(quad * 32) << 16) + acc * width;
                for (int c = slot * kBlockRows; c < q.live; c += kStride) {
                    uint32_t u[kBlockRows];
                    if (some) {
                        tmem_load16(from + c, u);
                    } else {
#pragma unroll
                        for (int i = 0; i < kBlockRows; ++i) u[i] = 0;
                    }
                    const int nrows = q.live - c;
                    if (kLayer && size > CG) {
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
                    if (kLayer && P.pre) {
                        pack_block(v, w, P.in_bf);
                        store_block(&maps.mp, P.pre + (row + c) * P.ld_pre + f, P.ld_pre, w, st,
                                    P.tma_pre && (whole || nrows >= kBlockRows), lane, feat, (int)row + c, 0, nrows, nfeat);
                    }
                    if (!kLayer) {
                    } else if (P.act == ACT_RELU) {
#pragma unroll
                        for (int i = 0; i < kBlockRows; ++i) v[i] = activate(v[i], ACT_RELU);
                    } else if (P.act == ACT_GELU) {
#pragma unroll
                        for (int i = 0; i < kBlockRows; ++i) v[i] = activate(v[i], ACT_GELU);
                    } else if (P.act == ACT_SILU) {
#pragma unroll
                        for (int i = 0; i < kBlockRows; ++i) v[i] = activate(v[i], ACT_SILU);
                    }
                    if (kAdds && P.c) {
                        if (P.in_bf) {
#pragma unroll
                            for (int i = 0; i < kBlockRows; ++i) v[i] += beta * __uint_as_float((uint32_t)cv[i] << 16);
                        } else {
#pragma unroll
                            for (int i = 0; i < kBlockRows; ++i) v[i] += beta * __half2float(__ushort_as_half(cv[i]));
                        }
                        if (c + kStride < q.live) fetch_c(P, cv, q.g, row + c + kStride, nrows - kStride, f);
                    }
                    // Symmetric outputs: blocks above the diagonal are left out, blocks that touch it are written as
                    // they are (together they hold both sides of it: tiles start at multiples of 32), blocks below
                    // it are written with their mirror images.
                    const int over = feat + 31 - (q.n0 + c);      // > 0 where the block reaches above the diagonal
                    if (side && over >= 31 + kBlockRows) continue;
                    pack_block(v, w, P.out_bf);
                    store_block(&maps.mo, P.out + q.g * P.bs_out + (row + c) * P.ld_out + f, P.ld_out, w, st,
                                P.tma_out && (whole || nrows >= kBlockRows), lane, feat, (int)row + c, zo, nrows, nfeat);
                    if (side && over <= 0 && lane < nfeat) {
                        // a lane's 16 values are neighbours in row f; rows are padded to multiples of 8 (with zeros)
                        uint4* m = reinterpret_cast<uint4*>(P.out + q.g * P.bs_out + (int64_t)f * P.ld_out + q.n0 + c);
                        m[0] = make_uint4(w[0], w[1], w[2], w[3]);
                        if (nrows > 8) m[1] = make_uint4(w[4], w[5], w[6], w[7]);
                    }
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
                if (kLayer && size > CG) {
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

// ======================================================================
// Elementwise passes
// ======================================================================

// dz = dy * act'(z), and the column sums of dz that make the bias gradient.
// A threadblock takes 256 columns of up to kGradRows rows of one expert
// (dense: one expert with all rows); 32 threads cover the columns, 8 each,
// and 8 groups of threads take 4 rows each, all loads ahead of the
// arithmetic (bound by DRAM: 6 bytes an element).  Rows that 16-byte loads
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

// ---------------------------------------------- orthogonalisation passes
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

// Sums of squares: threadblocks take groups of 8 elements of all runs in
// turn (one run where the matrix is packed), so the order is fixed.
__global__ void __launch_bounds__(256) norm_kernel(const NormPass N)
{
    __shared__ float sm[8];
    let_next_in();
    wait_for_previous();
    const int64_t base = blockIdx.y * N.bs_g, per = (N.run + 7) / 8, all = per * N.runs;
    float s = 0.f;
#pragma unroll 4
    for (int64_t i = blockIdx.x * 256 + threadIdx.x; i < all; i += (int64_t)gridDim.x * 256) {
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
// their parts of A = x x^T through distributed shared memory (each sums 128 /
// size rows, in rank order, and hands them to all), the rest of the step
// stays within a threadblock.  A tall matrix is transposed as it is loaded
// and stored.  Bound by the latency of 3 x steps products in a row.
//
// Rows of 64 elements (128 bytes) in 1024-byte atoms of 8 rows, 16-byte pieces
// exchanged by the row's index: element (i, j) of x is at piece (j / 8 % 8) ^
// (i % 8) of row i of block j / 64.  The same bytes are x with the reduction
// along its columns (x x^T) and along its rows (B x).
constexpr int kSmallSide = 128;
constexpr int kSmallThreads = 512;
constexpr int kSmallBlock = kSmallSide * 128;          // bytes of a block of 64 columns
constexpr int kSharePitch = kSmallSide + 4;            // floats; rows 4 banks apart

struct Small {
    const void* g;
    uint16_t* out;
    int64_t ld_g, bs_g, ld_out, bs_out;
    int32_t side, length;          // short and long side
    int32_t tall, type, out_bf, steps;
    int32_t size, width, vec_out;
    float a, b, c, eps, scale;
};

__device__ __forceinline__ uint32_t small_at(int i, int j)
{
    return (uint32_t)(j >> 6) * kSmallBlock + i * 128 + (((j >> 3) & 7) ^ (i & 7)) * 16;
}

__device__ __forceinline__ void store_cluster16(uint32_t addr, uint4 v)
{
    asm volatile("st.shared::cluster.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w)
                 : "memory");
}

__global__ void __launch_bounds__(kSmallThreads, 1) small_ortho_kernel(const __grid_constant__ Small S)
{
    __shared__ __align__(8) uint64_t done;
    __shared__ uint32_t tmem_slot;
    __shared__ int failed;
    __shared__ float sm[16], norms[8];
    extern __shared__ unsigned char raw[];
    unsigned char* dyn = raw + ((1024 - (smem_addr(raw) & 1023)) & 1023);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, quad = warp & 3, group = warp >> 2;
    const int rank = S.size > 1 ? (int)cluster_rank() : 0, entry = blockIdx.x / S.size;
    const int width = S.width, col0 = rank * width, cols = max(0, min(width, S.length - col0));
    unsigned char *x = dyn, *A = x + (size_t)width / 64 * kSmallBlock, *B = A + 2 * kSmallBlock;
    float* shares = reinterpret_cast<float*>(B + 2 * kSmallBlock);   // size > 1: [source][own row][column of A]
    const uint32_t bar = smem_addr(&done);
    if (threadIdx.x == 0) {
        bar_init(bar, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        failed = 0;
    }
    if (warp == 1) tmem_alloc<1>(smem_addr(&tmem_slot), 512);
    let_next_in();
    wait_for_previous();

    // 8 columns j.. of row i of g (or of its transpose)
    const int64_t base = (int64_t)entry * S.bs_g;
    auto fetch = [&](int i, int j, float v[8]) {
        if (i >= S.side || j >= cols) {
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = 0.f;
        } else if (S.tall) {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                v[e] = j + e < cols ? load_any(S.g, base + (int64_t)(col0 + j + e) * S.ld_g + i, S.type) : 0.f;
        } else if (j + 8 <= cols) {
            load_any8(S.g, base + i * S.ld_g + col0 + j, S.type, v);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                v[e] = j + e < cols ? load_any(S.g, base + i * S.ld_g + col0 + j + e, S.type) : 0.f;
        }
    };
    // neighbouring threads take neighbouring elements in memory
    const int pieces = width / 8, items = pieces * kSmallSide;
    auto place = [&](int n, int& i, int& j) {
        if (S.tall) {
            i = n % kSmallSide;
            j = n / kSmallSide * 8;
        } else {
            i = n / pieces;
            j = n % pieces * 8;
        }
    };
    float sum = 0.f;
#pragma unroll 2
    for (int n = threadIdx.x; n < items; n += kSmallThreads) {
        int i, j;
        place(n, i, j);
        float v[8], t = 0.f;
        fetch(i, j, v);
#pragma unroll
        for (int e = 0; e < 8; ++e) t = fmaf(v[e], v[e], t);
        sum += t;
    }
    sum = block_sum(sum, sm);
    if (S.size > 1) {
        cluster_sync();            // the others' shared memory is live from here on
        if ((int)threadIdx.x < S.size) store_cluster(cluster_addr(smem_addr(&norms[rank]), threadIdx.x), sum);
        cluster_sync();
        sum = 0.f;
        for (int i = 0; i < S.size; ++i) sum += norms[i];
    }
    float kappa, f1, f2;
    norm_scale(sum, S.eps, kappa, f1, f2);
#pragma unroll 2
    for (int n = threadIdx.x; n < items; n += kSmallThreads) {
        int i, j;
        place(n, i, j);
        float v[8];
        fetch(i, j, v);
        uint4 u;
        uint32_t* w = &u.x;
#pragma unroll
        for (int e = 0; e < 4; ++e) w[e] = pack2<false>(v[2 * e] * f1 * f2, v[2 * e + 1] * f1 * f2);
        *reinterpret_cast<uint4*>(x + small_at(i, j)) = u;
    }
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
            if (S.size == 1) {
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
                const int own = kSmallSide / S.size, to = row / own;
                const uint32_t at = cluster_addr(
                    smem_addr(shares + ((size_t)rank * own + row % own) * kSharePitch + group * 32), to);
#pragma unroll
                for (int c = 0; c < 32; c += 4) store_cluster16(at + c * 4, make_uint4(u[c], u[c + 1], u[c + 2], u[c + 3]));
            }
        }
        if (S.size > 1) {
            cluster_sync();
            const int own = kSmallSide / S.size;
            for (int n = threadIdx.x; n < own * (kSmallSide / 8); n += kSmallThreads) {
                const int r = n / (kSmallSide / 8), c = n % (kSmallSide / 8) * 8;
                float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
                for (int s = 0; s < S.size; ++s) {
                    const float4* p = reinterpret_cast<const float4*>(shares + ((size_t)s * own + r) * kSharePitch + c);
                    const float4 l = p[0], h = p[1];
                    v[0] += l.x, v[1] += l.y, v[2] += l.z, v[3] += l.w;
                    v[4] += h.x, v[5] += h.y, v[6] += h.z, v[7] += h.w;
                }
                uint4 h;
                uint32_t* w = &h.x;
#pragma unroll
                for (int e = 0; e < 4; ++e) w[e] = pack2<false>(alpha * v[2 * e], alpha * v[2 * e + 1]);
                const uint32_t at = smem_addr(A + small_at(rank * own + r, c));
                for (int s = 0; s < S.size; ++s) store_cluster16(cluster_addr(at, s), h);
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
                if (!last)
                    *reinterpret_cast<uint4*>(p) = make_uint4(w[c / 2], w[c / 2 + 1], w[c / 2 + 2], w[c / 2 + 3]);
            }
            if (last && row < S.side) {
                const int n = cols - c0;         // columns of this thread's 32 that exist
                uint16_t* o = S.out + (int64_t)entry * S.bs_out;
                if (S.tall) {
                    o += (int64_t)(col0 + c0) * S.ld_out + row;
#pragma unroll
                    for (int e = 0; e < 32; ++e, o += S.ld_out)
                        if (e < n) *o = (uint16_t)(w[e / 2] >> (e & 1) * 16);
                } else {
                    o += row * S.ld_out + col0 + c0;
                    if (S.vec_out && n >= 32) {
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            reinterpret_cast<uint4*>(o)[e] = make_uint4(w[4 * e], w[4 * e + 1], w[4 * e + 2], w[4 * e + 3]);
                    } else {
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            if (e < n) o[e] = (uint16_t)(w[e / 2] >> (e & 1) * 16);
                    }
                }
            }
        }
        fence_async();
        fence_before();
        __syncthreads();
        fence_after();
    }
    if (failed && threadIdx.x == 0) atomicCAS(&g_status[0], 0, (int)CCL_ERR_TIMEOUT);
    if (S.size > 1) cluster_sync();     // nobody leaves while another may still write to it
    if (warp == 1) tmem_free<1>(tmem, 512);
}

// ======================================================================
// Host side
// ======================================================================
#define TRY_CUDA(call, what)                                                                                   \
    do {                                                                                                       \
        cudaError_t e_ = (call);                                                                               \
        if (e_ != cudaSuccess)                                                                                 \
            return fail(e_ == cudaErrorMemoryAllocation ? CCL_ERR_OOM : CCL_ERR_CUDA,                          \
                        std::string(what) + ": " + cudaGetErrorString(e_));                                    \
    } while (0)
#define TRY(call)                                 \
    do {                                          \
        ccl_status_t s_ = (call);                 \
        if (s_ != CCL_OK) return s_;              \
    } while (0)

static int64_t round_up(int64_t v, int64_t m) { return (v + m - 1) / m * m; }
static bool aligned16(const void* p) { return ((uintptr_t)p & 15) == 0; }

typedef CUresult (*EncodeFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                             const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                             CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

static void (*const kKernels[2][3])(Product) = {
    {product_kernel<1, BOTH_K>, product_kernel<1, A_MN>, product_kernel<1, BOTH_MN>},
    {product_kernel<2, BOTH_K>, product_kernel<2, A_MN>, product_kernel<2, BOTH_MN>}};

// What the launches need to know of a device, looked up once per device.
struct Device {
    bool ready = false;
    int sms = 0;
    EncodeFn encode = nullptr;
};

static ccl_status_t device(const Device** out)
{
    static std::mutex mu;
    static Device all[64];
    int d = 0;
    TRY_CUDA(cudaGetDevice(&d), "cudaGetDevice");
    if (d < 0 || d >= 64) return fail(CCL_ERR_UNSUPPORTED, "device index above 63");
    std::lock_guard<std::mutex> lock(mu);
    if (!all[d].ready) {
        TRY_CUDA(cudaDeviceGetAttribute(&all[d].sms, cudaDevAttrMultiProcessorCount, d), "SM count");
        void* fn = nullptr;
        cudaDriverEntryPointQueryResult q;
        TRY_CUDA(cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &q),
                 "cuTensorMapEncodeTiled");
        if (q != cudaDriverEntryPointSuccess || !fn) return fail(CCL_ERR_CUDA, "the driver has no tensor maps");
        all[d].encode = (EncodeFn)fn;
        for (auto& forms : kKernels)
            for (auto kernel : forms)
                TRY_CUDA(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBudget),
                         "shared memory of the product kernel");
        for (auto kernel : {pair_kernel<1>, pair_kernel<2>})
            TRY_CUDA(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBudget),
                     "shared memory of the pair kernel");
        TRY_CUDA(cudaFuncSetAttribute(small_ortho_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBudget),
                 "shared memory of the small orthogonalisation kernel");
        all[d].ready = true;
    }
    *out = &all[d];
    return CCL_OK;
}

template <typename Arg>
static ccl_status_t launch(void (*kernel)(const Arg), dim3 grid, int threads, size_t smem, cudaStream_t stream, const Arg& arg,
                           int cluster = 1)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = (unsigned)cluster;
    at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    TRY_CUDA(cudaLaunchKernelEx(&cfg, kernel, arg), "launch");
    return CCL_OK;
}

// A 16-bit matrix (or a stack of them): rows of `cols` consecutive elements.
struct Matrix {
    const void* p = nullptr;
    int64_t rows = 0, cols = 0, ld = 0, count = 1, stride = 0;
    bool loadable() const
    {
        return aligned16(p) && ld % 8 == 0 && (count <= 1 || stride % 8 == 0);
    }
    int64_t packed_ld() const { return round_up(cols, 8); }
    int64_t packed_bytes() const { return loadable() ? 0 : round_up(count * rows * packed_ld() * 2, 256); }
};

// Bump allocation from the caller's workspace (a null base only measures).
struct Arena {
    char* base;
    int64_t used = 0;
    template <typename T>
    T* take(int64_t bytes)
    {
        T* p = base ? reinterpret_cast<T*>(base + used) : nullptr;
        used += round_up(bytes, 256);
        return p;
    }
};

struct PackArgs {
    uint16_t* dst;
    const uint16_t* src;
    int64_t ld_dst, bs_dst, ld_src, bs_src, rows, cols;
};
// Copy a matrix whose base or row stride TMA cannot address (not a multiple
// of 16 bytes) into rows padded to 8 elements.
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

// The matrix itself, or a copy in the workspace that TMA can address.
static ccl_status_t loadable(Matrix* m, Arena* ws, cudaStream_t stream)
{
    if (m->loadable()) return CCL_OK;
    uint16_t* d = ws->take<uint16_t>(m->packed_bytes());
    PackArgs a = {d, (const uint16_t*)m->p, m->packed_ld(), m->rows * m->packed_ld(), m->ld, m->stride, m->rows, m->cols};
    m->p = d;
    m->ld = a.ld_dst;
    m->stride = a.bs_dst;
    if (!ws->base) return CCL_OK;
    return launch(pack_rows_kernel, dim3((unsigned)std::min<int64_t>(a.rows, 4096), (unsigned)m->count), 256, 0, stream, a);
}

static ccl_status_t encode(const Device* dev, CUtensorMap* map, const Matrix& m, int box_cols, int box_rows,
                           CUtensorMapSwizzle swizzle = CU_TENSOR_MAP_SWIZZLE_128B)
{
    const cuuint64_t dims[3] = {(cuuint64_t)m.cols, (cuuint64_t)m.rows, (cuuint64_t)m.count};
    const cuuint64_t strides[2] = {(cuuint64_t)m.ld * 2, (cuuint64_t)(m.count > 1 ? m.stride : m.ld * m.rows) * 2};
    const cuuint32_t box[3] = {(cuuint32_t)box_cols, (cuuint32_t)box_rows, 1};
    const cuuint32_t unit[3] = {1, 1, 1};
    const CUresult r = dev->encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT16, 3, const_cast<void*>(m.p), dims, strides, box,
                                   unit, CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle,
                                   CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) return fail(CCL_ERR_INVALID_ARG, "a matrix cannot be described to TMA (size or stride)");
    return CCL_OK;
}

static bool vectors(const void* p, int64_t ld, int64_t bs) { return aligned16(p) && ld % 8 == 0 && bs % 8 == 0; }

static void set_out(Product* P, void* out, int64_t ld, int64_t bs, bool bf)
{
    P->out = (uint16_t*)out;
    P->ld_out = ld;
    P->bs_out = bs;
    P->out_bf = bf;
}
static void set_c(Product* P, const void* c, int64_t ld, int64_t bs, float beta)
{
    P->c = (const uint16_t*)c;
    P->ld_c = ld;
    P->bs_c = bs;
    P->beta = beta;
}
// how the epilogue may access its matrices (once all of them are set)
static void set_vec(Product* P)
{
    P->vec = vectors(P->out, P->ld_out, P->bs_out) && (!P->pre || vectors(P->pre, P->ld_pre, 0)) &&
             (!P->c || vectors(P->c, P->ld_c, P->bs_c)) && (!P->bias || vectors(P->bias, 0, P->bs_bias));
}

// How a product is cut up.
struct Shape {
    int cg, bn, split;
    double cost;
};

// The cheapest way by an estimate in clocks: waves of tiles over the SMs (or
// pairs, or clusters), each tile the longer of its products with their loads
// and of its epilogue, and never less than DRAM takes for the operands.  The
// constants are fits to measured times (bf16, 1.9 GHz, 4096 x 4096 x 4096
// unless noted).  Per 64 reduction elements: pairs 620, 540, 378 and 278
// clocks for 256, 192, 128 and 64 rows; single threadblocks 864, 476 and 300
// for 256, 128 and 64; no SM gets more than about 68 bytes a clock from L2,
// all together 8000.  An exchange of shares costs about 5000 clocks and 60 per
// row (1 x 4096 x 4096: 15.1, 12.9, 11.7 and 19 us cut in 1, 2, 4 and 8; x x^T
// of 1024 x 4096: 40 us more when cut in 4), and clusters of 4 and 8 leave SMs
// unused.
struct Choices {
    Shape best, single, pairs;     // of all; of single threadblocks without a split; of pairs
};

static Choices choose(const Product& P, int sms)
{
    const bool ragged_rows = P.ragged == RAGGED_ROWS, ragged_reduce = P.ragged == RAGGED_REDUCE;
    const int64_t rows = ragged_rows ? std::max(1, P.n / P.groups) : P.n;
    const int64_t groups = ragged_rows ? std::min(P.n, P.groups) : P.groups;
    const int64_t reduce = ragged_reduce ? std::max(1, P.k / P.groups) : P.k;
    const int64_t slices = (reduce + kSliceK - 1) / kSliceK;
    const double least = 2.0 * P.k * ((double)P.m * (ragged_reduce ? 1 : groups) + P.n) / 3400;
    Choices c = {};
    for (int cg = 1; cg <= 2; ++cg) {
        const int64_t tiles_m = (P.m + (int64_t)cg * kTileM - 1) / (cg * kTileM);
        for (int bn : {256, 192, 128, 64, 32}) {
            const int unit = P.b_mn ? 64 * cg : 32;       // rows are loaded 64 at a time where they are consecutive
            if (bn % unit || (bn > unit && bn / 2 >= rows)) continue;
            const int64_t tiles_n = (rows + bn - 1) / bn;
            const int64_t tiles = P.symmetric ? groups * (tiles_m * tiles_n + std::max(tiles_m, tiles_n)) / 2
                                              : groups * tiles_m * tiles_n;
            const double bytes = (kTileM + bn / cg) * 128.0;
            const double busy = (double)std::min<int64_t>(tiles * cg, sms);
            const double block = 400 + 16.0 * std::min<int64_t>(bn, rows);
            for (int split = 1; split <= (cg == 2 || bn > 128 || P.symmetric ? 1 : 8); split *= 2) {
                if (split > 1 && (split * 2 > slices || tiles * split > 2 * sms)) break;
                const double slice = std::max({cg == 2 ? 150 + 1.85 * bn : 130 + 2.8 * bn, bytes / 68,
                                               bytes * std::min<double>(sms, busy * split) / 8000});
                const double main = (double)((slices + split - 1) / split) * 2 * slice;
                const double epilogue = split == 1 ? block : 400 + (block - 400) / split + 5000 + 60.0 * std::min<int64_t>(bn, rows);
                const int places = cg == 2 ? sms / 2 : split == 4 ? sms / 4 - 2 : split == 8 ? sms / 8 - 3 : sms / split;
                const double cost = (double)((tiles + places - 1) / places) * std::max(main, epilogue) +
                                    std::min(main, epilogue);
                const Shape s = {cg, bn, split, std::max(cost, least) + 0.1 * cost};
                if (c.best.cg == 0 || s.cost < c.best.cost) c.best = s;
                Shape& own = cg == 1 ? c.single : c.pairs;
                if (split == 1 && (own.cg == 0 || s.cost < own.cost)) own = s;
            }
        }
    }
    return c;
}

// Complete a product for a shape: tiles and maps.
static ccl_status_t complete(const Device* dev, Product* P, const Shape& sh, const Matrix& a, const Matrix& b)
{
    set_vec(P);
    P->bn = sh.bn;
    P->split = sh.split;
    const int64_t tiles_m = (P->m + (int64_t)sh.cg * kTileM - 1) / (sh.cg * kTileM);
    const int64_t tiles_n = (P->n + (int64_t)P->bn - 1) / P->bn;
    int64_t per = tiles_m * tiles_n;
    if (P->symmetric) {
        per = 0;
        for (int64_t s = 0; s < tiles_m; ++s) per += tiles_n - s * sh.cg * kTileM / P->bn;
    }
    // ragged rows: at most one more row tile per expert than full tiles
    const int64_t most = P->ragged == RAGGED_ROWS ? tiles_m * (tiles_n + P->groups) : per * P->groups;
    if (most > INT32_MAX) return fail(CCL_ERR_UNSUPPORTED, "too many tiles");
    P->tiles_m = (int32_t)tiles_m;
    P->tiles_n = (int32_t)tiles_n;
    P->per = (int32_t)per;
    P->total = (int32_t)most;
    TRY(encode(dev, &P->ma, a, 64, P->a_mn ? kSliceK : kTileM));
    TRY(encode(dev, &P->mb, b, 64, P->b_mn ? kSliceK : P->bn / sh.cg));
    if (sh.split == 1) {
        const int64_t count = P->ragged == RAGGED_ROWS ? 1 : P->groups;
        P->tma_out = vectors(P->out, P->ld_out, P->bs_out);
        if (P->tma_out)
            TRY(encode(dev, &P->mo, Matrix{P->out, P->n, P->m, P->ld_out, count, P->bs_out}, 32, kBlockRows,
                       CU_TENSOR_MAP_SWIZZLE_NONE));
        P->tma_pre = P->pre && vectors(P->pre, P->ld_pre, 0);
        if (P->tma_pre)
            TRY(encode(dev, &P->mp, Matrix{P->pre, P->n, P->m, P->ld_pre}, 32, kBlockRows, CU_TENSOR_MAP_SWIZZLE_NONE));
    }
    return CCL_OK;
}

// Complete a product and launch it.
static ccl_status_t run(const Device* dev, Product P, const Shape& sh, const Matrix& a, const Matrix& b, cudaStream_t stream)
{
    TRY(complete(dev, &P, sh, a, b));
    const int size = sh.cg == 2 ? 2 : sh.split;
    const int bytes = (kTileM + P.bn / sh.cg) * kSliceK * 2;
    const int fixed = 1024 + kStagingBytes + (sh.split > 1 ? P.bn * kTileM * 4 : 0);
    P.stages = std::min(kMaxStages, (kSmemBudget - fixed) / bytes);
    // one tile each: no more stages than it has slices, so that the next
    // kernel's threadblocks find room beside this one's
    if (P.total <= dev->sms / size)
        P.stages = (int)std::min<int64_t>(P.stages, ((P.k + kSliceK - 1) / kSliceK + P.split - 1) / P.split);
    const size_t smem = fixed + (size_t)P.stages * bytes;
    const int clusters = std::min(P.total, dev->sms / size);
    return launch(kKernels[sh.cg - 1][P.b_mn ? BOTH_MN : P.a_mn ? A_MN : BOTH_K], dim3((unsigned)(clusters * size)),
                  kThreads, smem, stream, P, size);
}

// Launch a pair of products that do not depend on each other.
static ccl_status_t run_pair(const Device* dev, Pair* R, const Shape sh[2], const Matrix a[2], const Matrix b[2],
                             cudaStream_t stream)
{
    const int cg = sh[0].cg;
    int64_t most = 0;
    for (int i = 0; i < 2; ++i) {
        TRY(complete(dev, &R->p[i], sh[i], a[i], b[i]));
        R->width = std::max(R->width, sh[i].bn);
        most += R->p[i].total;
    }
    if (most > INT32_MAX) return fail(CCL_ERR_UNSUPPORTED, "too many tiles");
    const int bytes = (kTileM + R->width / cg) * kSliceK * 2, fixed = 1024 + kStagingBytes;
    R->stages = std::min(kMaxStages, (kSmemBudget - fixed) / bytes);
    const int clusters = (int)std::min<int64_t>(most, dev->sms / cg);
    return launch(cg == 2 ? pair_kernel<2> : pair_kernel<1>, dim3((unsigned)(clusters * cg)), kThreads,
                  fixed + (size_t)R->stages * bytes, stream, *R, cg);
}

// --------------------------------------------------------- linear layers
static std::string dims(int64_t rows, int64_t n, int64_t k)
{
    return "rows " + std::to_string(rows) + ", n " + std::to_string(n) + ", k " + std::to_string(k);
}

static ccl_status_t check_shape(const char* who, int64_t rows, int64_t n, int64_t k, int32_t dtype, int32_t act,
                                int32_t experts, const void* offsets)
{
    auto refuse = [&](ccl_status_t st, const std::string& why) { return fail(st, std::string(who) + ": " + why); };
    if (dtype != CCL_BF16 && dtype != CCL_F16)
        return refuse(CCL_ERR_UNSUPPORTED, "products take bf16 and f16 (dtype " + std::to_string(dtype) + ")");
    const int64_t top = (int64_t)1 << 30;
    if (rows < 0 || n < 1 || k < 1 || rows > top || n > top || k > top)
        return refuse(CCL_ERR_INVALID_ARG, "sizes out of range (" + dims(rows, n, k) + ")");
    if (act < CCL_ACT_NONE || act > CCL_ACT_SILU)
        return refuse(CCL_ERR_INVALID_ARG, "unknown activation " + std::to_string(act));
    if (experts < 0 || experts > kMaxGroups)
        return refuse(CCL_ERR_INVALID_ARG, "experts outside 0.." + std::to_string(kMaxGroups));
    if (experts > 0 && !offsets) return refuse(CCL_ERR_INVALID_ARG, "experts without offsets");
    return CCL_OK;
}

// A stride given as 0 means packed; one below the row's length would make rows overlap.
static ccl_status_t stride(const char* what, int64_t given, int64_t least, int64_t* out)
{
    if (given != 0 && given < least)
        return fail(CCL_ERR_INVALID_ARG, std::string(what) + " stride " + std::to_string(given) + " below " +
                                             std::to_string(least));
    *out = given ? given : least;
    return CCL_OK;
}

static ccl_status_t pointer(const char* what, const void* p, bool needed)
{
    if (needed && !p) return fail(CCL_ERR_INVALID_ARG, std::string(what) + " is null");
    if ((uintptr_t)p & 1) return fail(CCL_ERR_INVALID_ARG, std::string(what) + " is not aligned to its elements");
    return CCL_OK;
}

static ccl_status_t linear(const ccl_linear_t* a, char* base, int64_t* need, cudaStream_t stream)
{
    if (!a) return fail(CCL_ERR_INVALID_ARG, "ccl_linear: null arguments");
    TRY(check_shape("ccl_linear", a->rows, a->n, a->k, a->dtype, a->act, a->experts, a->offsets));
    int64_t ldx, ldw, ldr, ldy, ldz, sw, sb;
    TRY(stride("x", a->ldx, a->k, &ldx));
    TRY(stride("w", a->ldw, a->k, &ldw));
    TRY(stride("residual", a->ldr, a->n, &ldr));
    TRY(stride("y", a->ldy, a->n, &ldy));
    TRY(stride("z", a->ldz, a->n, &ldz));
    TRY(stride("w expert", a->w_stride, (a->n - 1) * ldw + a->k, &sw));
    if (!a->w_stride) sw = a->n * ldw;
    TRY(stride("bias expert", a->bias_stride, a->n, &sb));
    Arena ws = {base};
    const int64_t count = a->experts > 0 ? a->experts : 1;
    Matrix w = {a->w, a->n, a->k, ldw, count, sw}, x = {a->x, a->rows, a->k, ldx};
    if (!need) {
        const bool some = a->rows > 0;
        TRY(pointer("x", a->x, some));
        TRY(pointer("w", a->w, some));
        TRY(pointer("y", a->y, some));
        TRY(pointer("z", a->z, false));
        TRY(pointer("bias", a->bias, false));
        TRY(pointer("residual", a->residual, false));
        if (some && (a->y == a->x || a->y == a->w || (a->z && a->z == a->y)))
            return fail(CCL_ERR_INVALID_ARG, "ccl_linear: an output is also an operand");
        if (!some) return CCL_OK;
    }
    if (need) {
        *need = w.packed_bytes() + x.packed_bytes();
        return CCL_OK;
    }
    TRY(loadable(&w, &ws, stream));
    TRY(loadable(&x, &ws, stream));
    Product P = {};
    P.m = (int32_t)a->n;
    P.n = (int32_t)a->rows;
    P.k = (int32_t)a->k;
    P.groups = (int32_t)count;
    P.ragged = a->experts > 0 ? RAGGED_ROWS : DENSE;
    P.offsets = a->experts > 0 ? a->offsets : nullptr;
    P.alpha = 1.f;
    P.act = a->act;
    P.in_bf = a->dtype == CCL_BF16;
    set_out(&P, a->y, ldy, 0, P.in_bf);
    if (a->residual) set_c(&P, a->residual, ldr, 0, 1.f);
    if (a->z) {
        P.pre = (uint16_t*)a->z;
        P.ld_pre = ldz;
    }
    if (a->bias) {
        P.bias = (const uint16_t*)a->bias;
        P.bs_bias = count > 1 ? sb : 0;
    }
    const Device* dev = nullptr;
    TRY(device(&dev));
    return run(dev, P, choose(P, dev->sms).best, w, x, stream);
}

static ccl_status_t linear_grad(const ccl_linear_grad_t* a, char* base, int64_t* need, cudaStream_t stream)
{
    if (!a) return fail(CCL_ERR_INVALID_ARG, "ccl_linear_grad: null arguments");
    TRY(check_shape("ccl_linear_grad", a->rows, a->n, a->k, a->dtype, a->act, a->experts, a->offsets));
    int64_t lddy, ldx, ldw, ldz, lddx, lddw, sw, sdw, sdb;
    TRY(stride("dy", a->lddy, a->n, &lddy));
    TRY(stride("x", a->ldx, a->k, &ldx));
    TRY(stride("w", a->ldw, a->k, &ldw));
    TRY(stride("z", a->ldz, a->n, &ldz));
    TRY(stride("dx", a->lddx, a->k, &lddx));
    TRY(stride("dw", a->lddw, a->k, &lddw));
    TRY(stride("w expert", a->w_stride, (a->n - 1) * ldw + a->k, &sw));
    if (!a->w_stride) sw = a->n * ldw;
    TRY(stride("dw expert", a->dw_stride, (a->n - 1) * lddw + a->k, &sdw));
    if (!a->dw_stride) sdw = a->n * lddw;
    TRY(stride("db expert", a->db_stride, a->n, &sdb));
    const int64_t count = a->experts > 0 ? a->experts : 1;
    if (!need) {
        const bool some = a->rows > 0;
        TRY(pointer("dy", a->dy, some));
        TRY(pointer("x", a->x, some && a->dw));
        TRY(pointer("w", a->w, some && a->dx));
        TRY(pointer("z", a->z, some && a->act != CCL_ACT_NONE));
        TRY(pointer("dx", a->dx, false));
        TRY(pointer("dw", a->dw, false));
        TRY(pointer("db", a->db, false));
        if ((a->dx && (a->dx == a->dy || a->dx == a->w)) || (a->dw && (a->dw == a->dy || a->dw == a->x)))
            return fail(CCL_ERR_INVALID_ARG, "ccl_linear_grad: an output is also an operand");
        if (!some) {
            if (a->dw)
                for (int64_t e = 0; e < count; ++e)
                    TRY_CUDA(cudaMemset2DAsync((uint16_t*)a->dw + e * sdw, lddw * 2, 0, a->k * 2, a->n, stream), "dw");
            if (a->db)
                TRY_CUDA(cudaMemset2DAsync(a->db, sdb * 2, 0, a->n * 2, count, stream), "db");
            return CCL_OK;
        }
    }
    // dz: dy itself where there is no activation and TMA can read it
    const bool own_dz = a->act != CCL_ACT_NONE || !aligned16(a->dy) || lddy % 8 != 0;
    Arena ws = {base};
    Matrix dz = {a->dy, a->rows, a->n, lddy}, x = {a->x, a->rows, a->k, ldx}, w = {a->w, a->n, a->k, ldw, count, sw};
    if (!a->dx) w.p = nullptr, w.ld = 8;
    if (!a->dw) x.p = nullptr, x.ld = 8;
    GradPass G = {};
    const int64_t chunks = a->rows / kGradRows + count;
    G.ld_part = round_up(a->n, 64);
    G.ld_dz = round_up(a->n, 8);
    if (own_dz) {
        G.dz = ws.take<uint16_t>(a->rows * G.ld_dz * 2);
        dz.p = G.dz;
        dz.ld = G.ld_dz;
    }
    if (a->db) G.partial = ws.take<float>(chunks * G.ld_part * 4);
    if (need) {
        *need = ws.used + w.packed_bytes() + x.packed_bytes();
        return CCL_OK;
    }
    const bool bf = a->dtype == CCL_BF16;
    if (own_dz || a->db) {
        G.dy = (const uint16_t*)a->dy;
        G.z = (const uint16_t*)a->z;
        G.db = (uint16_t*)a->db;
        G.offsets = a->experts > 0 ? a->offsets : nullptr;
        G.ld_dy = lddy;
        G.ld_z = ldz;
        G.bs_db = sdb;
        G.rows = (int32_t)a->rows;
        G.n = (int32_t)a->n;
        G.groups = (int32_t)count;
        G.act = a->act;
        G.bf = bf;
        G.vec = a->n % 8 == 0 && vectors(a->dy, lddy, 0) && (a->act == CCL_ACT_NONE || vectors(a->z, ldz, 0));
        TRY(launch(act_grad_kernel, dim3((unsigned)chunks, (unsigned)((a->n + 255) / 256)), 256, 0, stream, G));
    }
    Product P = {};
    P.groups = (int32_t)count;
    P.offsets = a->experts > 0 ? a->offsets : nullptr;
    P.alpha = 1.f;
    P.in_bf = bf;
    Product px = P, pw = P;
    if (a->dx) {   // dx[t, k] = sum_n w[n, k] dz[t, n]
        TRY(loadable(&w, &ws, stream));
        px.m = (int32_t)a->k;
        px.n = (int32_t)a->rows;
        px.k = (int32_t)a->n;
        px.ragged = a->experts > 0 ? RAGGED_ROWS : DENSE;
        px.a_mn = 1;
        set_out(&px, a->dx, lddx, 0, bf);
    }
    if (a->dw) {   // dw[n, k] = sum_t x[t, k] dz[t, n]
        TRY(loadable(&x, &ws, stream));
        pw.m = (int32_t)a->k;
        pw.n = (int32_t)a->n;
        pw.k = (int32_t)a->rows;
        pw.ragged = a->experts > 0 ? RAGGED_REDUCE : DENSE;
        pw.a_mn = pw.b_mn = 1;
        set_out(&pw, a->dw, lddw, sdw, bf);
    }
    const Device* dev = nullptr;
    TRY(device(&dev));
    const Choices cx = a->dx ? choose(px, dev->sms) : Choices(), cw = a->dw ? choose(pw, dev->sms) : Choices();
    if (a->dx && a->dw) {
        // one launch for both unless splitting or shapes of their own are worth more than the launch (9500 clocks)
        const double one = cx.single.cost + cw.single.cost, two = cx.pairs.cost + cw.pairs.cost;
        if (std::min(one, two) < cx.best.cost + cw.best.cost + 9500) {
            Pair R = {};
            R.p[0] = px;
            R.p[1] = pw;
            if (a->db) R.sums = G;
            const Shape sh[2] = {two <= one ? cx.pairs : cx.single, two <= one ? cw.pairs : cw.single};
            const Matrix left[2] = {w, x}, right[2] = {dz, dz};
            return run_pair(dev, &R, sh, left, right, stream);
        }
    }
    if (a->db) TRY(launch(bias_grad_kernel, dim3((unsigned)((a->n + 31) / 32), (unsigned)count), 256, 0, stream, G));
    if (a->dx) TRY(run(dev, px, cx.best, w, dz, stream));
    if (a->dw) TRY(run(dev, pw, cw.best, x, dz, stream));
    return CCL_OK;
}

// ------------------------------------------------------ orthogonalisation
static ccl_status_t orthogonalize(const ccl_ortho_t* a, char* base, int64_t* need, cudaStream_t stream)
{
    const std::string who = "ccl_orthogonalize: ";
    if (!a) return fail(CCL_ERR_INVALID_ARG, who + "null arguments");
    if (a->dtype != CCL_F32 && a->dtype != CCL_BF16 && a->dtype != CCL_F16)
        return fail(CCL_ERR_UNSUPPORTED, who + "gradients are f32, bf16 or f16");
    if (a->out_dtype != CCL_BF16 && a->out_dtype != CCL_F16)
        return fail(CCL_ERR_UNSUPPORTED, who + "the update is bf16 or f16");
    if (a->batch < 0 || a->batch > 65535 || a->p < 1 || a->q < 1 || a->p > (1 << 30) || a->q > (1 << 30) ||
        std::min(a->p, a->q) > kMaxGroups * kTileM)
        return fail(CCL_ERR_INVALID_ARG, who + "sizes out of range (batch " + std::to_string(a->batch) + ", " +
                                             std::to_string(a->p) + " x " + std::to_string(a->q) + ")");
    if (a->steps < 1 || a->steps > 64) return fail(CCL_ERR_INVALID_ARG, who + "steps outside 1..64");
    if (!(a->eps >= 0.f)) return fail(CCL_ERR_INVALID_ARG, who + "eps is negative");
    int64_t ldg, ldo, sg, so;
    TRY(stride("g", a->ldg, a->q, &ldg));
    TRY(stride("out", a->ldo, a->q, &ldo));
    TRY(stride("g matrix", a->g_stride, (a->p - 1) * ldg + a->q, &sg));
    if (!a->g_stride) sg = a->p * ldg;
    TRY(stride("out matrix", a->out_stride, (a->p - 1) * ldo + a->q, &so));
    if (!a->out_stride) so = a->p * ldo;
    const int64_t r = std::min(a->p, a->q);
    const bool tall = a->p > a->q;
    // threadblocks that a matrix with a short side of up to 128 takes: each
    // holds up to 384 columns, or 256 beside the others' shares of A
    const int64_t longer = std::max(a->p, a->q);
    int size = 1;
    while (size < 8 && longer > (size == 1 ? 384 : 256 * size)) size *= 2;
    const bool small = r <= kSmallSide && longer <= (size == 1 ? 384 : 256 * size);
    Arena ws = {base};
    Matrix x[2], A, B;
    // rows start on cache lines: a 128-byte row of a tile would touch two of them otherwise
    const int64_t ldx = round_up(a->q, 64), lda = round_up(r, 64);
    for (int i = 0; i < 2; ++i) {
        x[i] = {nullptr, a->p, a->q, ldx, a->batch, a->p * ldx};
        x[i].p = ws.take<void>(a->batch * a->p * ldx * 2);
    }
    A = B = {nullptr, r, r, lda, a->batch, r * lda};
    A.p = ws.take<void>(a->batch * r * lda * 2);
    B.p = ws.take<void>(a->batch * r * lda * 2);
    NormPass N = {};
    N.partial = ws.take<float>(a->batch * kNormBlocks * 4);
    N.kappa = ws.take<float>(a->batch * 4);
    N.kappa2 = ws.take<float>(a->batch * 4);
    if (need) {
        *need = small ? 0 : ws.used;
        return CCL_OK;
    }
    if (a->batch == 0) return CCL_OK;
    if (!a->g || !a->out) return fail(CCL_ERR_INVALID_ARG, who + "null matrix");
    if ((uintptr_t)a->g % (a->dtype == CCL_F32 ? 4 : 2) || (uintptr_t)a->out % 2)
        return fail(CCL_ERR_INVALID_ARG, who + "a matrix is not aligned to its elements");
    if (small) {
        Small S = {};
        S.g = a->g;
        S.out = (uint16_t*)a->out;
        S.ld_g = ldg;
        S.bs_g = sg;
        S.ld_out = ldo;
        S.bs_out = so;
        S.side = (int32_t)r;
        S.length = (int32_t)longer;
        S.tall = tall;
        S.type = a->dtype;
        S.out_bf = a->out_dtype == CCL_BF16;
        S.steps = a->steps;
        S.size = size;
        S.width = (int32_t)round_up((longer + size - 1) / size, 64);
        S.vec_out = vectors(a->out, ldo, so);
        S.a = a->a;
        S.b = a->b;
        S.c = a->c;
        S.eps = a->eps;
        S.scale = a->scale;
        const Device* dev = nullptr;
        TRY(device(&dev));
        const size_t smem = 1024 + (size_t)S.width / 64 * kSmallBlock + 4 * kSmallBlock +
                            (size > 1 ? (size_t)kSmallSide * kSharePitch * 4 : 0);
        return launch(small_ortho_kernel, dim3((unsigned)(a->batch * size)), kSmallThreads, smem, stream, S, size);
    }
    N.g = a->g;
    N.x = (__half*)x[0].p;
    N.ld_g = ldg;
    N.bs_g = sg;
    N.ld_x = ldx;
    N.bs_x = a->p * ldx;
    N.p = (int32_t)a->p;
    N.q = (int32_t)a->q;
    N.type = a->dtype;
    N.eps = a->eps;
    N.runs = ldg == a->q ? 1 : (int32_t)a->p;
    N.run = N.runs == 1 ? a->p * a->q : a->q;
    const int64_t groups = a->p * ((a->q + 7) / 8);   // of 8 elements
    N.blocks = (int32_t)std::min<int64_t>(kNormBlocks, (groups + 1023) / 1024);
    TRY(launch(norm_kernel, dim3(N.blocks, (unsigned)a->batch), 256, 0, stream, N));
    TRY(launch(scale_kernel, dim3((unsigned)std::min<int64_t>(1216, (groups + 511) / 512), (unsigned)a->batch), 256, 0,
               stream, N));
    // The products of a step, by the place their operands are in: kind 0 is
    // A = x x^T (or x^T x of a tall x), kind 1 is B = b A + c A A, kind 2 is
    // x <- a x + B x (or a x + x B).
    struct Step {
        Product p;
        const Matrix *a, *b;
    };
    auto product = [&](int kind, int from, bool first, bool last) {
        Step s = {};
        Product& P = s.p;
        P.groups = (int32_t)a->batch;
        P.m = P.n = (int32_t)r;
        if (kind == 0) {
            P.k = (int32_t)(tall ? a->p : a->q);
            P.a_mn = P.b_mn = tall;
            P.symmetric = 1;
            P.alpha = kScaleA / (kScaleX * kScaleX);
            P.alpha_of = first ? N.kappa2 : nullptr;
            set_out(&P, const_cast<void*>(A.p), lda, r * lda, false);
            s.a = s.b = &x[from];
        } else if (kind == 1) {
            P.k = (int32_t)r;
            P.symmetric = 1;
            P.alpha = a->c / kScaleA;
            set_c(&P, A.p, lda, r * lda, a->b);
            set_out(&P, const_cast<void*>(B.p), lda, r * lda, false);
            s.a = s.b = &A;
        } else {
            P.m = (int32_t)a->q;
            P.n = (int32_t)a->p;
            P.k = (int32_t)r;
            const float unscale = last ? a->scale / kScaleX : 1.f;
            P.alpha = unscale / kScaleA;
            P.alpha_of = P.beta_of = first ? N.kappa : nullptr;
            set_c(&P, x[from].p, ldx, a->p * ldx, a->a * unscale);
            if (last)
                set_out(&P, a->out, ldo, so, a->out_dtype == CCL_BF16);
            else
                set_out(&P, const_cast<void*>(x[from ^ 1].p), ldx, a->p * ldx, false);
            P.a_mn = !tall;            // wide: out[p, q] = sum_r x[r, q] B[p, r]
            s.a = tall ? &B : &x[from];   // tall: out[p, q] = sum_r B[q, r] x[p, r], B symmetric
            s.b = tall ? &x[from] : &B;
        }
        return s;
    };
    const Device* dev = nullptr;
    TRY(device(&dev));
    Shape shapes[3];
    for (int kind = 0; kind < 3; ++kind) shapes[kind] = choose(product(kind, 0, false, false).p, dev->sms).best;
    for (int i = 0; i < 3 * a->steps; ++i) {
        const Step s = product(i % 3, i / 3 & 1, i < 3, i / 3 + 1 == a->steps);
        TRY(run(dev, s.p, shapes[i % 3], *s.a, *s.b, stream));
    }
    return CCL_OK;
}

template <typename Args>
static ccl_status_t guarded(ccl_status_t (*fn)(const Args*, char*, int64_t*, cudaStream_t), const Args* a, void* ws,
                            int64_t ws_bytes, void* stream)
{
    int64_t need = 0;
    TRY(fn(a, nullptr, &need, nullptr));
    if (need > 0 && (!ws || ws_bytes < need))
        return fail(CCL_ERR_INVALID_ARG, "workspace of " + std::to_string(need) + " bytes needed, " +
                                             std::to_string(ws ? ws_bytes : 0) + " given");
    if (need > 0 && ((uintptr_t)ws & 255)) return fail(CCL_ERR_INVALID_ARG, "workspace not aligned to 256 bytes");
    return fn(a, (char*)ws, nullptr, (cudaStream_t)stream);
}

template <typename Args>
static ccl_status_t measured(ccl_status_t (*fn)(const Args*, char*, int64_t*, cudaStream_t), const Args* a, int64_t* out)
{
    if (!out) return fail(CCL_ERR_INVALID_ARG, "null size");
    int64_t need = 0;
    TRY(fn(a, nullptr, &need, nullptr));
    *out = need;
    return CCL_OK;
}

}  // namespace tensor
}  // namespace ccl

using namespace ccl;

// no exception leaves the library
#define C_ENTRY(...)                                                     \
    try {                                                                \
        return (__VA_ARGS__);                                            \
    } catch (const std::bad_alloc&) {                                    \
        return CCL_ERR_OOM;                                              \
    } catch (...) {                                                      \
        return CCL_ERR_INTERNAL;                                         \
    }

extern "C" {

ccl_status_t ccl_linear_workspace(const ccl_linear_t* a, int64_t* bytes)
{
    C_ENTRY(tensor::measured(tensor::linear, a, bytes));
}
ccl_status_t ccl_linear(const ccl_linear_t* a, void* ws, int64_t ws_bytes, void* stream)
{
    C_ENTRY(tensor::guarded(tensor::linear, a, ws, ws_bytes, stream));
}
ccl_status_t ccl_linear_grad_workspace(const ccl_linear_grad_t* a, int64_t* bytes)
{
    C_ENTRY(tensor::measured(tensor::linear_grad, a, bytes));
}
ccl_status_t ccl_linear_grad(const ccl_linear_grad_t* a, void* ws, int64_t ws_bytes, void* stream)
{
    C_ENTRY(tensor::guarded(tensor::linear_grad, a, ws, ws_bytes, stream));
}
ccl_status_t ccl_orthogonalize_workspace(const ccl_ortho_t* a, int64_t* bytes)
{
    C_ENTRY(tensor::measured(tensor::orthogonalize, a, bytes));
}
ccl_status_t ccl_orthogonalize(const ccl_ortho_t* a, void* ws, int64_t ws_bytes, void* stream)
{
    C_ENTRY(tensor::guarded(tensor::orthogonalize, a, ws, ws_bytes, stream));
}

ccl_status_t ccl_tensor_status(void)
{
    C_ENTRY([]() -> ccl_status_t {
        int st[4] = {0, 0, 0, 0};
        TRY_CUDA(cudaDeviceSynchronize(), "cudaDeviceSynchronize");
        TRY_CUDA(cudaMemcpyFromSymbol(st, tensor::g_status, sizeof(st)), "status word");
        if (st[0] == 0) return CCL_OK;
        const int zero[4] = {0, 0, 0, 0};
        TRY_CUDA(cudaMemcpyToSymbol(tensor::g_status, zero, sizeof(zero)), "status word");
        return fail((ccl_status_t)st[0], st[0] == CCL_ERR_TIMEOUT ? "a wait inside a tensor product ran out of time"
                                                                  : "expert offsets decrease or leave the rows");
    }());
}

}  // extern "C"
