// Host side of the product kernels: matrices, tensor maps, the choice of tiles.
#pragma once

#include <algorithm>
#include <string>

#include "ccl_tensor_host.h"
#include "ccl_tensor_passes.cuh"
#include "ccl_tensor_product.cuh"

namespace ccl {
namespace tensor {

typedef CUresult (*EncodeFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                             const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                             CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// What the launches need to know of a device, looked up once per device.
struct Device {
    bool ready = false;
    int sms = 0;
    int small_clusters[5] = {};    // of 2^i threadblocks of the small orthogonalisation kernel that run at once
    EncodeFn encode = nullptr;
};

// What every user of the product kernels needs of the current device.
inline ccl_status_t look_up(Device* dev, int d)
{
    TRY_CUDA(cudaDeviceGetAttribute(&dev->sms, cudaDevAttrMultiProcessorCount, d), "SM count");
    void* fn = nullptr;
    cudaDriverEntryPointQueryResult q;
    TRY_CUDA(cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &q),
             "cuTensorMapEncodeTiled");
    if (q != cudaDriverEntryPointSuccess || !fn) return fail(CCL_ERR_CUDA, "the driver has no tensor maps");
    dev->encode = (EncodeFn)fn;
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

// The matrix itself, or a copy in the workspace that TMA can address.
[[maybe_unused]] static ccl_status_t loadable(Matrix* m, Arena* ws, cudaStream_t stream)
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

[[maybe_unused]] static ccl_status_t encode(const Device* dev, CUtensorMap* map, const Matrix& m, int box_cols, int box_rows,
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

inline void set_out(Product* P, void* out, int64_t ld, int64_t bs, bool bf)
{
    P->out = (uint16_t*)out;
    P->ld_out = ld;
    P->bs_out = bs;
    P->out_bf = bf;
}
inline void set_c(Product* P, const void* c, int64_t ld, int64_t bs, float beta)
{
    P->c = (const uint16_t*)c;
    P->ld_c = ld;
    P->bs_c = bs;
    P->beta = beta;
}
// how the epilogue may access its matrices (once all of them are set)
inline void set_vec(Product* P)
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
// clocks for 256, 192, 128 and 64 rows; single threadblocks 476 and 300 for
// 128 and 64; no SM gets more than about 68 bytes a clock from L2, all
// together 8000.  Widths between the powers of two fit the waves: 4096 x 4096
// x 4096 takes 78 us in tiles of 224 rows (four whole waves), 81 of 256, 88 of
// 192.  An exchange of shares costs about 5000 clocks and 60 per row (1 x 4096
// x 4096: 15.1, 12.9, 11.7 and 19 us cut in 1, 2, 4 and 8; x x^T of 1024 x
// 4096: 40 us more when cut in 4), and clusters of 4 and 8 leave SMs unused.
struct Choices {
    Shape best;                    // of all
    Shape single, pairs;           // beside another product in one launch: of single threadblocks, of pairs
};

inline Choices choose_anew(const Product& P, int sms, int max_split)
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
        // single threadblocks lose to pairs on wide tiles: only what few rows want
        for (int bn = cg == 2 ? 256 : 128; bn >= 32; bn = cg == 2 ? bn - 32 : bn / 2) {
            const int unit = P.b_mn ? 64 * cg : 32;       // rows are loaded 64 at a time where they are consecutive
            if (bn % unit || (bn > unit && bn - unit >= rows)) continue;
            const int64_t tiles_n = (rows + bn - 1) / bn;
            const int64_t tiles = P.symmetric ? groups * (tiles_m * tiles_n + std::max(tiles_m, tiles_n)) / 2
                                              : groups * tiles_m * tiles_n;
            const double bytes = (kTileM + bn / cg) * 128.0;
            const double busy = (double)std::min<int64_t>(tiles * cg, sms);
            const double block = 400 + 16.0 * std::min<int64_t>(bn, rows);
            for (int split = 1; split <= (cg == 2 || P.symmetric ? 1 : max_split); split *= 2) {
                if (split > 1 && (split * 2 > slices || tiles * split > 2 * sms)) break;
                const double slice = std::max(std::max(cg == 2 ? 150 + 1.85 * bn : 130 + 2.8 * bn, bytes / 68),
                                              bytes * std::min<double>(sms, busy * split) / 8000);
                const double main = (double)((slices + split - 1) / split) * 2 * slice;
                const double epilogue = split == 1 ? block : 400 + (block - 400) / split + 5000 + 60.0 * std::min<int64_t>(bn, rows);
                const int places = cg == 2 ? sms / 2 : split == 4 ? sms / 4 - 2 : split == 8 ? sms / 8 - 3 : sms / split;
                const double cost = (double)((tiles + places - 1) / places) * std::max(main, epilogue) +
                                    std::min(main, epilogue);
                const Shape s = {cg, bn, split, std::max(cost, least) + 0.1 * cost};
                if (c.best.cg == 0 || s.cost < c.best.cost) c.best = s;
                if (split > 1) continue;
                // beside another product whole waves do not matter
                const double beside = std::max(1.0, (double)tiles / places) * std::max(main, epilogue);
                Shape& own = cg == 1 ? c.single : c.pairs;
                if (own.cg == 0 || beside < own.cost) own = {cg, bn, 1, beside};
            }
        }
    }
    return c;
}

// The same, remembered by the sizes that it depends on: an estimate takes about a
// microsecond, a gradient asks for ten, and calls come again with the same sizes.
inline Choices choose(const Product& P, int sms, int max_split = 8)
{
    struct Entry {
        int32_t key[10];
        Choices choices;
    };
    static thread_local Entry known[64];
    const int32_t key[10] = {P.m, P.n, P.k, P.groups, P.ragged, P.symmetric, P.b_mn, sms, max_split, 1};
    uint32_t h = 0;
    for (int32_t v : key) h = (h ^ (uint32_t)v) * 0x9e3779b1u, h ^= h >> 15;
    Entry& e = known[h % 64];
    if (!std::equal(key, key + 10, e.key)) {
        e.choices = choose_anew(P, sms, max_split);
        std::copy(key, key + 10, e.key);
    }
    return e.choices;
}

// Complete a product for a shape: tiles and maps.  alt: A as P->alt's flag has it read.
[[maybe_unused]] static ccl_status_t complete(const Device* dev, Product* P, const Shape& sh, const Matrix& a, const Matrix& b,
                                              const Matrix* alt = nullptr)
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
    if (alt) TRY(encode(dev, &P->mp, *alt, 64, P->a_mn ? kSliceK : kTileM));
    if (sh.split == 1) {
        const int64_t count = P->ragged == RAGGED_ROWS ? 1 : P->groups;
        P->tma_out = P->out && !P->sum && vectors(P->out, P->ld_out, P->bs_out);
        if (P->tma_out)
            TRY(encode(dev, &P->mo, Matrix{P->out, P->n, P->m, P->ld_out, count, P->bs_out}, 32, kBlockRows,
                       CU_TENSOR_MAP_SWIZZLE_NONE));
        P->tma_pre = P->pre && vectors(P->pre, P->ld_pre, 0);
        if (P->tma_pre)
            TRY(encode(dev, &P->mp, Matrix{P->pre, P->n, P->m, P->ld_pre}, 32, kBlockRows, CU_TENSOR_MAP_SWIZZLE_NONE));
        const bool pieces = P->c && vectors(P->c, P->ld_c, P->bs_c) && (P->m % 8 == 0 || P->pad_c);
        P->fast = P->tma_out && !P->pre && !P->sum && (!P->c || (pieces && P->act == CCL_ACT_NONE));
    }
    if (P->symmetric && !P->fast) return fail(CCL_ERR_INTERNAL, "a symmetric product whose rows TMA cannot store");
    return CCL_OK;
}

// A single product on the current device (ccl_tensor.cu).
ccl_status_t run_product(const Product& P, const Shape& sh, const Matrix& a, const Matrix& b, const Matrix* alt,
                         cudaStream_t stream);

}  // namespace tensor
}  // namespace ccl
