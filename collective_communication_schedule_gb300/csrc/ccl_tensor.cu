// Tensor products of language-model layers: dense products with a fused
// epilogue, products grouped by expert over ragged rows, and the
// Newton-Schulz orthogonalisation of gradient matrices.  C ABI in
// include/ccl.h; PTX building blocks in ccl_tensor.cuh.
#include <algorithm>
#include <mutex>
#include <string>

#include <cuda_runtime.h>

#include "ccl_tensor_grad.cuh"
#include "ccl_tensor_launch.cuh"
#include "ccl_tensor_ortho.cuh"

namespace ccl {
namespace tensor {

// ======================================================================
// Host side
// ======================================================================
static void (*const kKernels[2][3])(Product) = {
    {product_kernel<1, BOTH_K>, product_kernel<1, A_MN>, product_kernel<1, BOTH_MN>},
    {product_kernel<2, BOTH_K>, product_kernel<2, A_MN>, product_kernel<2, BOTH_MN>}};

// the small orthogonalisation kernel for `size` threadblocks a matrix, and its shared memory
static void (*small_kernel(int size))(Small)
{
    return size == 1 ? small_ortho_kernel<1> : size <= 8 ? small_ortho_kernel<8> : small_ortho_kernel<16>;
}
static size_t small_smem(int size, int width)
{
    return 1024 + (size_t)width / 64 * kSmallBlock + 4 * kSmallBlock + (size > 1 ? (size_t)kSmallSide * kSharePitch * 4 : 0);
}

static ccl_status_t device(const Device** out)
{
    static std::mutex mu;
    static Device all[64];
    int d = 0;
    TRY_CUDA(cudaGetDevice(&d), "cudaGetDevice");
    if (d < 0 || d >= 64) return fail(CCL_ERR_UNSUPPORTED, "device index above 63");
    std::lock_guard<std::mutex> lock(mu);
    if (!all[d].ready) {
        TRY(look_up(&all[d], d));
        for (auto& forms : kKernels)
            for (auto kernel : forms)
                TRY_CUDA(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBudget),
                         "shared memory of the product kernel");
        for (auto kernel : {pair_kernel<1>, pair_kernel<2>})
            TRY_CUDA(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBudget),
                     "shared memory of the pair kernel");
        for (auto kernel : {small_ortho_kernel<1>, small_ortho_kernel<8>, small_ortho_kernel<16>})
            TRY_CUDA(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBudget),
                     "shared memory of the small orthogonalisation kernel");
        TRY_CUDA(cudaFuncSetAttribute(small_ortho_kernel<16>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1),
                 "clusters of 16 of the small orthogonalisation kernel");
        all[d].small_clusters[0] = all[d].sms;
        for (int i = 1; 1 << i <= kSmallCluster; ++i) {
            cudaLaunchConfig_t cfg = {};
            cudaLaunchAttribute at;
            at.id = cudaLaunchAttributeClusterDimension;
            at.val.clusterDim.x = 1u << i;
            at.val.clusterDim.y = at.val.clusterDim.z = 1;
            cfg.gridDim = dim3(1u << i);
            cfg.blockDim = dim3(kSmallThreads);
            cfg.dynamicSmemBytes = small_smem(1 << i, 256);
            cfg.attrs = &at;
            cfg.numAttrs = 1;
            TRY_CUDA(cudaOccupancyMaxActiveClusters(&all[d].small_clusters[i], small_kernel(1 << i), &cfg),
                     "clusters of the small orthogonalisation kernel");
        }
        all[d].ready = true;
    }
    *out = &all[d];
    return CCL_OK;
}

// Complete a product and launch it.
static ccl_status_t run(const Device* dev, Product P, const Shape& sh, const Matrix& a, const Matrix& b, cudaStream_t stream,
                        const Matrix* alt = nullptr)
{
    TRY(complete(dev, &P, sh, a, b, alt));
    const int size = sh.cg == 2 ? 2 : sh.split;
    const int bytes = (kTileM + P.bn / sh.cg) * kSliceK * 2;
    const int fixed = 1024 + kStagingBytes + (sh.split > 1 ? P.bn * kTileM * 4 : 0);
    P.stages = std::min(kMaxStages, (kSmemBudget - fixed) / bytes);
    const size_t smem = fixed + (size_t)P.stages * bytes;
    const int clusters = std::min(P.total, dev->sms / size);
    return launch(kKernels[sh.cg - 1][P.b_mn ? BOTH_MN : P.a_mn ? A_MN : BOTH_K], dim3((unsigned)(clusters * size)),
                  kThreads, smem, stream, P, size);
}

ccl_status_t run_product(const Product& P, const Shape& sh, const Matrix& a, const Matrix& b, const Matrix* alt,
                         cudaStream_t stream)
{
    const Device* dev = nullptr;
    TRY(device(&dev));
    return run(dev, P, sh, a, b, stream, alt);
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
        if (some && (same(a->y, {a->x, a->w, a->bias, a->z}) || same(a->z, {a->x, a->w, a->bias, a->residual})))
            return fail(CCL_ERR_INVALID_ARG, "ccl_linear: an output is also an operand or another output");
        // in place, a row of y may be written while the rows after it are read
        if (a->rows > 1 && same(a->y, {a->residual}) && ldr != ldy)
            return fail(CCL_ERR_INVALID_ARG, "ccl_linear: y over a residual of another row stride");
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
    if (a->n > 256 * 65535) return fail(CCL_ERR_UNSUPPORTED, "ccl_linear_grad: n above " + std::to_string(256 * 65535));
    if (!need) {
        const bool some = a->rows > 0;
        TRY(pointer("dy", a->dy, some));
        TRY(pointer("x", a->x, some && a->dw));
        TRY(pointer("w", a->w, some && a->dx));
        TRY(pointer("z", a->z, some && a->act != CCL_ACT_NONE));
        TRY(pointer("dx", a->dx, false));
        TRY(pointer("dw", a->dw, false));
        TRY(pointer("db", a->db, false));
        // the two products and the bias gradient run at one time: none may write what another one reads
        const void *x_read = a->dw ? a->x : nullptr, *w_read = a->dx ? a->w : nullptr;
        if (same(a->dx, {a->dy, a->w, x_read}) || same(a->dw, {a->dy, a->x, w_read}) || same(a->db, {a->dy, x_read, w_read}))
            return fail(CCL_ERR_INVALID_ARG, "ccl_linear_grad: an output is also an operand");
        if (same(a->dx, {a->dw, a->db}) || same(a->dw, {a->db}))
            return fail(CCL_ERR_INVALID_ARG, "ccl_linear_grad: an output is also another output");
        if (!some) {
            if (a->dw)
                for (int64_t e = 0; e < count; ++e)
                    TRY_CUDA(cudaMemset2DAsync((uint16_t*)a->dw + e * sdw, lddw * 2, 0, a->k * 2, a->n, stream), "dw");
            if (a->db)
                TRY_CUDA(cudaMemset2DAsync(a->db, sdb * 2, 0, a->n * 2, count, stream), "db");
            return CCL_OK;
        }
    }
    if (!a->dx && !a->dw && !a->db) {
        if (need) *need = 0;
        return CCL_OK;
    }
    // dz, for the products: dy itself where there is no activation and TMA can read it
    const bool own_dz = (a->dx || a->dw) && (a->act != CCL_ACT_NONE || !aligned16(a->dy) || lddy % 8 != 0);
    Arena ws = {base};
    Matrix dz = {a->dy, a->rows, a->n, lddy}, x = {a->x, a->rows, a->k, ldx}, w = {a->w, a->n, a->k, ldw, count, sw};
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
        *need = ws.used + (a->dx ? w.packed_bytes() : 0) + (a->dw ? x.packed_bytes() : 0);
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
        // by the sizes alone: the small kernel leaves it unused, but which
        // kernel runs is no part of what a caller has to know
        *need = ws.used;
        return CCL_OK;
    }
    if (a->batch == 0) return CCL_OK;
    if (!a->g || !a->out) return fail(CCL_ERR_INVALID_ARG, who + "null matrix");
    if ((uintptr_t)a->g % (a->dtype == CCL_F32 ? 4 : 2) || (uintptr_t)a->out % 2)
        return fail(CCL_ERR_INVALID_ARG, who + "a matrix is not aligned to its elements");
    // a matrix of a batch is written while others may not have been read: in
    // place each must stay within its own bytes
    if (a->out == a->g && a->batch > 1 && (a->dtype == CCL_F32 || sg != so))
        return fail(CCL_ERR_INVALID_ARG, who + "in place with another element size or matrix stride");
    const Device* dev = nullptr;
    TRY(device(&dev));
    // Threadblocks that a matrix with a short side of up to 128 takes: each
    // holds up to 384 columns, or 256 beside its part of A.
    const int64_t longer = std::max(a->p, a->q);
    int log = 0;
    while (1 << log < kSmallCluster && longer > (log == 0 ? 384 : 256 << log)) ++log;
    const int size = 1 << log, at_once = dev->small_clusters[log];
    bool small = r <= kSmallSide && longer <= (log == 0 ? 384 : 256 << log) && at_once > 0;
    if (small && size > 1) {
        // A matrix holds `size` SMs for all of its steps, so a large batch goes
        // around several times, while one launch per product fills the machine.
        // Fits in us to five steps, small against general: 128 x 4096 56 and 120,
        // batch 64 576 and 441; 24 x 4096 batch 16 157 and 155, batch 64 519 and
        // 284; 32 x 700 batch 64 99 and 115, batch 128 193 and 152; 128 x 2048
        // batch 32 155 and 176, batch 128 496 and 429; 128 x 1024 batch 256 387
        // and 452.  Single threadblocks always win (128 x 384 batch 512: 151, 438).
        const float kilo = longer / 1024.f, rounds = (float)((a->batch + at_once - 1) / at_once);
        small = rounds * (46.f + 4.f * kilo) < 75.f + 12.f * kilo + a->batch * kilo * (0.56f + 0.0067f * r);
    }
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
        const int64_t each = a->dtype == CCL_F32 ? 4 : 8;      // elements of 16 bytes
        S.vec_g = aligned16(a->g) && ldg % each == 0 && sg % each == 0;
        S.a = a->a;
        S.b = a->b;
        S.c = a->c;
        S.eps = a->eps;
        S.scale = a->scale;
        return launch(small_kernel(size), dim3((unsigned)(a->batch * size)), kSmallThreads, small_smem(size, S.width), stream,
                      S, size);
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
            P.pad_c = 1;
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
            P.pad_c = 1;
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
    Shape shapes[3];
    for (int kind = 0; kind < 3; ++kind) shapes[kind] = choose(product(kind, 0, false, false).p, dev->sms).best;
    for (int i = 0; i < 3 * a->steps; ++i) {
        const Step s = product(i % 3, i / 3 & 1, i < 3, i / 3 + 1 == a->steps);
        TRY(run(dev, s.p, shapes[i % 3], *s.a, *s.b, stream));
    }
    return CCL_OK;
}

}  // namespace tensor
}  // namespace ccl

using namespace ccl;

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
        if (st[0] == 0) return tensor::take_layer_status();
        const int zero[4] = {0, 0, 0, 0};
        TRY_CUDA(cudaMemcpyToSymbol(tensor::g_status, zero, sizeof(zero)), "status word");
        return fail((ccl_status_t)st[0], st[0] == CCL_ERR_TIMEOUT ? "a wait inside a tensor product ran out of time"
                                                                  : "expert offsets decrease or leave the rows");
    }());
}

}  // extern "C"
