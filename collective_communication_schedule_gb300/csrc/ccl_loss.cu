// Softmax cross entropy of x w^T against target classes without its values in
// memory, and its gradients.  C ABI in include/ccl.h.
#include <algorithm>
#include <mutex>
#include <string>

#include <cuda_runtime.h>

#include "ccl_loss.cuh"
#include "ccl_tensor_launch.cuh"

namespace ccl {
namespace tensor {

static ccl_status_t loss_device(const Device** out)
{
    static std::mutex mu;
    static Device all[64];
    int d = 0;
    TRY_CUDA(cudaGetDevice(&d), "cudaGetDevice");
    if (d < 0 || d >= 64) return fail(CCL_ERR_UNSUPPORTED, "device index above 63");
    std::lock_guard<std::mutex> lock(mu);
    if (!all[d].ready) {
        TRY(look_up(&all[d], d));
        for (auto kernel : {rowwise_kernel<1, STATS>, rowwise_kernel<2, STATS>, rowwise_kernel<1, SLOPE>, rowwise_kernel<2, SLOPE>,
                            rowwise_kernel<1, STATS_TURNED>, rowwise_kernel<1, SLOPE_TURNED>})
            TRY_CUDA(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBudget),
                     "shared memory of the rowwise kernel");
        TRY_CUDA(cudaFuncSetAttribute(sum_pairs<2>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBudget),
                 "shared memory of the pair kernel");
        all[d].ready = true;
    }
    *out = &all[d];
    return CCL_OK;
}

// Shapes are chosen for the SMs of a GB300, so that workspaces and the order of
// sums depend on the sizes alone.
constexpr int kShapeSms = 152;

// Up to this many rows, rows of w lie along the lanes.  Forward, 32003 x 2048
// weights, us turned and not: 1 row 25.3 and 41.5 (all tiles read the one row of x),
// 8 rows 25.6 and 39.9, 32 rows 27.2 and 28.0, 64 rows 31.0 and 28.1.  The whole
// backward pass: 1 row 101 and 116, 64 rows 101 and 104, 128 rows 107 and 108.
static bool turns(int mode, int64_t rows) { return rows <= (mode == STATS ? 32 : 128); }

// The product x w^T, in either orientation, and its shape.
static Product values_of(int mode, int64_t rows, int64_t vocab, int64_t k, bool bf, Shape* sh)
{
    Product P = {};
    const bool turned = turns(mode, rows);
    P.m = (int32_t)(turned ? vocab : rows);
    P.n = (int32_t)(turned ? rows : vocab);
    P.k = (int32_t)k;
    P.groups = 1;
    P.alpha = 1.f;
    P.in_bf = P.out_bf = bf;
    if (turned) {                  // all rows of x in one tile
        *sh = {1, 32, 1, 0.};
        while (sh->bn < rows) sh->bn *= 2;
    } else if (rows <= kTileM) {
        // one tile of rows: single threadblocks, all SMs busy (128 x 32003 x 2048 28.3 us, 30.6 in pairs)
        *sh = {1, 128, 1, 0.};
        while (sh->bn > 32 && (vocab + sh->bn - 1) / sh->bn < kShapeSms) sh->bn /= 2;
    } else {
        *sh = choose(P, kShapeSms, 1).best;
    }
    return P;
}
// Parts of a row's statistics: by tile, or by cluster where one tile holds all rows.
static int64_t parts_of(const Product& P, const Shape& sh, bool turned, int sms, bool* whole)
{
    const int64_t across = (P.m + sh.cg * kTileM - 1) / (sh.cg * kTileM), along = (P.n + sh.bn - 1) / sh.bn;
    *whole = turned || across == 1;
    if (!*whole) return along;
    return std::min<int64_t>(across * along, sms / sh.cg);
}

// mode: STATS or SLOPE
static ccl_status_t run_rowwise(const Device* dev, int mode, Rowwise* R, const Shape& sh, const Matrix& x, const Matrix& w,
                                uint16_t* out, int64_t ld_out, cudaStream_t stream)
{
    const bool turned = turns(mode, x.rows);
    if (turned) set_out(&R->p, out, ld_out, 0, R->p.out_bf);
    TRY(complete(dev, &R->p, sh, turned ? w : x, turned ? x : w));
    R->p.out = out;
    R->p.ld_out = ld_out;
    const int bytes = (kTileM + sh.bn / sh.cg) * kSliceK * 2, fixed = 1024 + kStagingBytes;
    R->p.stages = std::min(kMaxStages, (kSmemBudget - fixed) / bytes);
    const int clusters = std::min(R->p.total, std::min(dev->sms, kShapeSms) / sh.cg);
    // lanes along x: single threadblocks or pairs; turned: single ones
    void (*const kernels[2][3])(Rowwise) = {{rowwise_kernel<1, STATS>, rowwise_kernel<2, STATS>, rowwise_kernel<1, STATS_TURNED>},
                                            {rowwise_kernel<1, SLOPE>, rowwise_kernel<2, SLOPE>, rowwise_kernel<1, SLOPE_TURNED>}};
    return launch(kernels[mode == SLOPE][turned ? 2 : sh.cg - 1], dim3((unsigned)(clusters * sh.cg)), kThreads,
                  fixed + (size_t)R->p.stages * bytes, stream, *R, sh.cg);
}

static ccl_status_t check_loss(const std::string& who, int64_t rows, int64_t vocab, int64_t k, int dtype, int target_bits)
{
    if (dtype != CCL_BF16 && dtype != CCL_F16)
        return fail(CCL_ERR_UNSUPPORTED, who + "products take bf16 and f16 (dtype " + std::to_string(dtype) + ")");
    const int64_t top = (int64_t)1 << 30;
    if (rows < 0 || vocab < 1 || k < 1 || rows > top || vocab > top || k > top)
        return fail(CCL_ERR_INVALID_ARG, who + "sizes out of range (rows " + std::to_string(rows) + ", vocab " +
                                             std::to_string(vocab) + ", k " + std::to_string(k) + ")");
    if (target_bits != 32 && target_bits != 64) return fail(CCL_ERR_INVALID_ARG, who + "targets of neither 32 nor 64 bits");
    return CCL_OK;
}

static ccl_status_t words(const std::string& who, const char* what, const void* p, bool needed, int bytes = 4)
{
    if (needed && !p) return fail(CCL_ERR_INVALID_ARG, who + what + " is null");
    if ((uintptr_t)p % bytes) return fail(CCL_ERR_INVALID_ARG, who + what + " is not aligned to its elements");
    return CCL_OK;
}

static ccl_status_t cross_entropy(const ccl_cross_entropy_t* a, char* base, int64_t* need, cudaStream_t stream)
{
    const std::string who = "ccl_cross_entropy: ";
    if (!a) return fail(CCL_ERR_INVALID_ARG, who + "null arguments");
    TRY(check_loss(who, a->rows, a->vocab, a->k, a->dtype, a->target_bits));
    int64_t ldx, ldw;
    TRY(stride("x", a->ldx, a->k, &ldx));
    TRY(stride("w", a->ldw, a->k, &ldw));
    Arena ws = {base};
    Matrix x = {a->x, a->rows, a->k, ldx}, w = {a->w, a->vocab, a->k, ldw};
    Rowwise R = {};
    LossRows L = {};
    Shape sh = {};
    bool whole = false;
    if (a->rows > 0) {
        R.p = values_of(STATS, a->rows, a->vocab, a->k, a->dtype == CCL_BF16, &sh);
        L.tiles = parts_of(R.p, sh, turns(STATS, a->rows), kShapeSms, &whole);
        R.part = ws.take<float2>(L.tiles * a->rows * sizeof(float2));
        R.picked = ws.take<float>(a->rows * 4);
    }
    if (need) {
        *need = a->rows > 0 ? ws.used + w.packed_bytes() + x.packed_bytes() : 0;
        return CCL_OK;
    }
    if (a->rows == 0) return CCL_OK;
    TRY(pointer("x", a->x, true));
    TRY(pointer("w", a->w, true));
    TRY(words(who, "target", a->target, true, a->target_bits / 8));
    TRY(words(who, "loss", a->loss, true));
    TRY(words(who, "lse", a->lse, false));
    if (same(a->loss, {a->x, a->w, a->target, a->lse}) || same(a->lse, {a->x, a->w, a->target}))
        return fail(CCL_ERR_INVALID_ARG, who + "an output is also an operand or another output");
    const Device* dev = nullptr;
    TRY(loss_device(&dev));
    TRY(loadable(&w, &ws, stream));
    TRY(loadable(&x, &ws, stream));
    R.whole = whole;
    L.tiles = parts_of(R.p, sh, turns(STATS, a->rows), std::min(dev->sms, kShapeSms), &whole);
    R.target = L.target = a->target;
    R.wide = L.wide = a->target_bits == 64;
    TRY(run_rowwise(dev, STATS, &R, sh, x, w, nullptr, 0, stream));
    L.ignore = a->ignore_index;
    L.rows = a->rows;
    L.vocab = a->vocab;
    L.part = R.part;
    L.picked = R.picked;
    L.loss = a->loss;
    L.lse = a->lse;
    return launch(loss_kernel, dim3((unsigned)((a->rows + 7) / 8)), 256, 0, stream, L);
}

// Rows of w whose derivatives are held at a time: what keeps them within 256 MB
// (but at least 1024).  us with 64, 256 and 1024 MB: 4096 x 65536 x 4096 3758, 3438 and
// 3396, 2048 x 128000 x 1024 1230, 970 and 958: more memory gains 1 %.
constexpr int64_t kPieceBytes = 256ll << 20;
static int64_t piece_of(int64_t rows, int64_t vocab)
{
    const int64_t most = std::max<int64_t>(1024, kPieceBytes / 2 / std::max<int64_t>(1, rows) / 256 * 256);
    const int64_t pieces = (vocab + most - 1) / most;
    return pieces == 1 ? vocab : round_up((vocab + pieces - 1) / pieces, 256);
}

// dx of a piece: the product's shape, and the segments of the piece's classes
// that are reduced side by side where its tiles alone would leave SMs idle: 777 x
// 32003 x 1032, whose dx is 25 tiles, 176 us instead of 251; 4096 x 65536 x 4096 takes
// one segment.
struct DxShape {
    Shape shape;
    int32_t segment, parts;
};
static DxShape dx_shape(int64_t rows, int64_t k, int64_t width)
{
    Product P = {};
    P.m = (int32_t)k;
    P.n = (int32_t)rows;
    P.a_mn = 1;
    DxShape best = {};
    double least = 0;
    for (int parts : {1, 2, 3, 4, 6, 8, 12, 16}) {
        const int64_t segment = round_up((width + parts - 1) / parts, kSliceK);
        if (parts > 1 && (segment < 8 * kSliceK || (parts - 1) * segment >= width)) break;
        P.groups = parts;
        P.k = (int32_t)std::min(segment, width);
        const Choices c = choose(P, kShapeSms, 1);
        const Shape& sh = c.pairs;
        // whole waves of tiles, and the parts' way through memory and back at 3400 bytes a clock
        const int64_t tiles = (k + 2 * kTileM - 1) / (2 * kTileM) * ((rows + sh.bn - 1) / sh.bn) * parts;
        const double one = sh.cost / std::max(1.0, (double)tiles / (kShapeSms / 2));
        const double cost = (double)((tiles + kShapeSms / 2 - 1) / (kShapeSms / 2)) * one + (parts > 1 ? 8.0 * parts * rows * k / 3400 + 4000 : 0);
        if (best.parts == 0 || cost < least) best = {sh, parts > 1 ? (int32_t)segment : 0, parts}, least = cost;
    }
    return best;
}

static ccl_status_t cross_entropy_grad(const ccl_cross_entropy_grad_t* a, char* base, int64_t* need, cudaStream_t stream)
{
    const std::string who = "ccl_cross_entropy_grad: ";
    if (!a) return fail(CCL_ERR_INVALID_ARG, who + "null arguments");
    TRY(check_loss(who, a->rows, a->vocab, a->k, a->dtype, a->target_bits));
    int64_t ldx, ldw, lddx, lddw;
    TRY(stride("x", a->ldx, a->k, &ldx));
    TRY(stride("w", a->ldw, a->k, &ldw));
    TRY(stride("dx", a->lddx, a->k, &lddx));
    TRY(stride("dw", a->lddw, a->k, &lddw));
    Arena ws = {base};
    Matrix x = {a->x, a->rows, a->k, ldx}, w = {a->w, a->vocab, a->k, ldw};
    const int64_t piece = piece_of(a->rows, a->vocab), ld_dl = round_up(piece, 64), ld_sum = round_up(a->k, 32);
    const bool several = piece < a->vocab, bf = a->dtype == CCL_BF16, some = a->rows > 0 && (a->dx || a->dw);
    LossRows L = {};
    DxShape dxs = {};
    uint16_t* dl = nullptr;
    float* sum = nullptr;
    Matrix clean = {nullptr, a->rows, a->k, round_up(a->k, 8)};
    if (some) {
        L.coef = ws.take<float4>(a->rows * sizeof(float4));
        L.scale = ws.take<float>(16);
        L.block = ws.take<float2>((a->rows + 7) / 8 * sizeof(float2));
        dl = ws.take<uint16_t>(a->rows * ld_dl * 2);
        if (a->dx) {
            dxs = dx_shape(a->rows, a->k, piece);
            if (several || dxs.parts > 1) sum = ws.take<float>(dxs.parts * a->rows * ld_sum * 4);
        }
        if (a->dw) clean.p = ws.take<uint16_t>(a->rows * clean.ld * 2);
    }
    if (need) {
        *need = some ? ws.used + w.packed_bytes() + x.packed_bytes() : 0;
        return CCL_OK;
    }
    TRY(pointer("dx", a->dx, false));
    TRY(pointer("dw", a->dw, false));
    if (a->rows == 0) {
        if (a->dw) TRY_CUDA(cudaMemset2DAsync(a->dw, lddw * 2, 0, a->k * 2, a->vocab, stream), "dw");
        return CCL_OK;
    }
    if (!some) return CCL_OK;
    TRY(pointer("x", a->x, true));
    TRY(pointer("w", a->w, true));
    TRY(words(who, "target", a->target, true, a->target_bits / 8));
    TRY(words(who, "dloss", a->dloss, true));
    TRY(words(who, "dlse", a->dlse, false));
    TRY(words(who, "lse", a->lse, true));
    // pieces are written while x and w are still read
    for (const void* out : {(const void*)a->dx, (const void*)a->dw})
        if (same(out, {a->x, a->w, a->target, a->dloss, a->dlse, a->lse}))
            return fail(CCL_ERR_INVALID_ARG, who + "an output is also an operand");
    if (same(a->dx, {a->dw})) return fail(CCL_ERR_INVALID_ARG, who + "an output is also another output");
    const Device* dev = nullptr;
    TRY(loss_device(&dev));
    TRY(loadable(&w, &ws, stream));
    TRY(loadable(&x, &ws, stream));
    L.target = a->target;
    L.ignore = a->ignore_index;
    L.rows = a->rows;
    L.vocab = a->vocab;
    L.wide = a->target_bits == 64;
    L.dloss = a->dloss;
    L.dlse = a->dlse;
    L.lse_in = a->lse;
    L.dirty = (int32_t*)(L.scale + 2);
    L.k = a->k;
    L.f16 = !bf;
    if (a->dw) {
        L.x = (const uint16_t*)x.p;
        L.ld_x = x.ld;
        L.clean = (uint16_t*)clean.p;
        L.ld_clean = clean.ld;
    }
    TRY(launch(loss_rows_kernel, dim3((unsigned)((a->rows + 7) / 8)), 256, 0, stream, L));
    TRY(launch(loss_ready_kernel, dim3((unsigned)(a->dw ? std::min<int64_t>(a->rows, 152) : 1)), 256, 0, stream, L));
    for (int64_t first = 0; first < a->vocab; first += piece) {
        const int64_t width = std::min(piece, a->vocab - first);
        Matrix wp = w, dlp = {dl, a->rows, width, ld_dl};
        wp.p = (const uint16_t*)w.p + first * w.ld;
        wp.rows = width;
        Rowwise R = {};
        Shape shape;
        R.p = values_of(SLOPE, a->rows, width, a->k, bf, &shape);
        R.coef = L.coef;
        R.scale = L.scale;
        R.first = (int32_t)first;
        TRY(run_rowwise(dev, SLOPE, &R, shape, x, wp, dl, ld_dl, stream));
        Product P = {};
        P.groups = 1;
        P.alpha = 1.f;
        P.alpha_of = L.scale + 1;
        P.in_bf = bf;
        Product px = P, pw = P;
        if (a->dx) {   // dx[t, k] = sum_v w[v, k] dl[t, v]
            px.m = (int32_t)a->k;
            px.n = (int32_t)a->rows;
            px.k = (int32_t)width;
            px.a_mn = 1;
            set_out(&px, a->dx, lddx, 0, bf);
            px.sum = sum;
            px.ld_sum = ld_sum;
            px.bs_sum = a->rows * ld_sum;
            px.sum_first = first == 0;
            if (dxs.parts > 1) {
                px.groups = dxs.parts;
                px.segment = dxs.segment;
            }
        }
        if (a->dw) {   // dw[v, k] = sum_t x[t, k] dl[t, v]
            pw.m = (int32_t)a->k;
            pw.n = (int32_t)width;
            pw.k = (int32_t)a->rows;
            pw.a_mn = pw.b_mn = 1;
            pw.alt = L.dirty;
            set_out(&pw, (uint16_t*)a->dw + first * lddw, lddw, 0, bf);
        }
        if (!a->dx) {
            TRY(run_product(pw, choose(pw, kShapeSms).best, x, dlp, &clean, stream));
            continue;
        }
        // both in one launch: the tiles of dw fill the places that those of dx leave
        Pair S = {};
        S.p[0] = px;
        TRY(complete(dev, &S.p[0], dxs.shape, wp, dlp));
        int64_t most = S.p[0].total;
        S.width = dxs.shape.bn;
        if (a->dw) {
            const Shape sw = choose(pw, kShapeSms).pairs;
            S.p[1] = pw;
            TRY(complete(dev, &S.p[1], sw, x, dlp, &clean));
            S.width = std::max(S.width, sw.bn);
            most += S.p[1].total;
        } else {
            S.p[1] = S.p[0];
            S.p[1].total = 0;
        }
        if (most > INT32_MAX) return fail(CCL_ERR_UNSUPPORTED, who + "too many tiles");
        const int bytes = (kTileM + S.width / 2) * kSliceK * 2, fixed = 1024 + kStagingBytes;
        S.stages = std::min(kMaxStages, (kSmemBudget - fixed) / bytes);
        const int clusters = (int)std::min<int64_t>(most, dev->sms / 2);
        TRY(launch(sum_pairs<2>, dim3((unsigned)(clusters * 2)), kThreads, fixed + (size_t)S.stages * bytes, stream, S, 2));
    }
    if (sum) {
        LossSum Q = {sum, (uint16_t*)a->dx, a->rows, a->k, ld_sum, a->rows * ld_sum, lddx, dxs.parts, bf};
        const int64_t blocks = (a->rows * ((a->k + 3) / 4) + 255) / 256;
        if (blocks > INT32_MAX) return fail(CCL_ERR_UNSUPPORTED, who + "dx is too large");
        TRY(launch(loss_sum_kernel, dim3((unsigned)blocks), 256, 0, stream, Q));
    }
    return CCL_OK;
}

ccl_status_t take_loss_status()
{
    int st[4] = {0, 0, 0, 0};
    TRY_CUDA(cudaMemcpyFromSymbol(st, g_status, sizeof(st)), "status word");
    if (st[0] == 0) return CCL_OK;
    const int zero[4] = {0, 0, 0, 0};
    TRY_CUDA(cudaMemcpyToSymbol(g_status, zero, sizeof(zero)), "status word");
    return fail((ccl_status_t)st[0], st[0] == CCL_ERR_TIMEOUT ? "a wait inside a product of the cross entropy ran out of time"
                                                              : "a target outside the vocabulary");
}

}  // namespace tensor
}  // namespace ccl

using namespace ccl;

extern "C" {

ccl_status_t ccl_cross_entropy_workspace(const ccl_cross_entropy_t* a, int64_t* bytes)
{
    C_ENTRY(tensor::measured(tensor::cross_entropy, a, bytes));
}
ccl_status_t ccl_cross_entropy(const ccl_cross_entropy_t* a, void* ws, int64_t ws_bytes, void* stream)
{
    C_ENTRY(tensor::guarded(tensor::cross_entropy, a, ws, ws_bytes, stream));
}
ccl_status_t ccl_cross_entropy_grad_workspace(const ccl_cross_entropy_grad_t* a, int64_t* bytes)
{
    C_ENTRY(tensor::measured(tensor::cross_entropy_grad, a, bytes));
}
ccl_status_t ccl_cross_entropy_grad(const ccl_cross_entropy_grad_t* a, void* ws, int64_t ws_bytes, void* stream)
{
    C_ENTRY(tensor::guarded(tensor::cross_entropy_grad, a, ws, ws_bytes, stream));
}

}  // extern "C"
