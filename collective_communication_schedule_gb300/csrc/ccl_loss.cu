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
        for (auto kernel : {rowwise_kernel<1, STATS>, rowwise_kernel<2, STATS>, rowwise_kernel<1, SLOPE>, rowwise_kernel<2, SLOPE>})
            TRY_CUDA(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBudget),
                     "shared memory of the rowwise kernel");
        for (auto kernel : {sum_pair_kernel<1>, sum_pair_kernel<2>})
            TRY_CUDA(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBudget),
                     "shared memory of the pair kernel");
        all[d].ready = true;
    }
    *out = &all[d];
    return CCL_OK;
}

// Shapes are chosen for the SMs of a GB300, so that workspaces and the order of
// sums depend on the sizes alone.
constexpr int kShapeSms = 152;

static Product values_of(int64_t rows, int64_t vocab, int64_t k, bool bf)
{
    Product P = {};
    P.m = (int32_t)rows;
    P.n = (int32_t)vocab;
    P.k = (int32_t)k;
    P.groups = 1;
    P.alpha = 1.f;
    P.in_bf = P.out_bf = bf;
    return P;
}

static ccl_status_t run_rowwise(const Device* dev, int mode, Rowwise* R, const Shape& sh, const Matrix& x, const Matrix& w,
                                uint16_t* out, int64_t ld_out, cudaStream_t stream)
{
    TRY(complete(dev, &R->p, sh, x, w));
    R->p.out = out;
    R->p.ld_out = ld_out;
    const int bytes = (kTileM + sh.bn / sh.cg) * kSliceK * 2, fixed = 1024 + kStagingBytes;
    R->p.stages = std::min(kMaxStages, (kSmemBudget - fixed) / bytes);
    const int clusters = std::min(R->p.total, dev->sms / sh.cg);
    void (*const kernels[2][2])(Rowwise) = {{rowwise_kernel<1, STATS>, rowwise_kernel<2, STATS>},
                                            {rowwise_kernel<1, SLOPE>, rowwise_kernel<2, SLOPE>}};
    return launch(kernels[mode == SLOPE][sh.cg - 1], dim3((unsigned)(clusters * sh.cg)), kThreads,
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
    R.p = values_of(a->rows, a->vocab, a->k, a->dtype == CCL_BF16);
    LossRows L = {};
    Shape sh = {};
    if (a->rows > 0) {
        sh = choose(R.p, kShapeSms, 1).best;
        L.tiles = (a->vocab + sh.bn - 1) / sh.bn;
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
    return launch(loss_kernel, dim3((unsigned)((a->rows + 31) / 32)), 512, 0, stream, L);
}

// Rows of w whose derivatives are held at a time: what keeps them within 256 MB.
constexpr int64_t kPieceBytes = 256ll << 20;
static int64_t piece_of(int64_t rows, int64_t vocab)
{
    const int64_t most = std::max<int64_t>(1024, kPieceBytes / 2 / std::max<int64_t>(1, rows) / 256 * 256);
    const int64_t pieces = (vocab + most - 1) / most;
    return pieces == 1 ? vocab : round_up((vocab + pieces - 1) / pieces, 256);
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
    uint16_t* dl = nullptr;
    float* sum = nullptr;
    Matrix clean = {nullptr, a->rows, a->k, round_up(a->k, 8)};
    if (some) {
        L.coef = ws.take<float4>(a->rows * sizeof(float4));
        L.scale = ws.take<float>(16);
        dl = ws.take<uint16_t>(a->rows * ld_dl * 2);
        if (several && a->dx) sum = ws.take<float>(a->rows * ld_sum * 4);
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
    TRY(launch(loss_scale_kernel, dim3(1), 1024, 0, stream, L));
    TRY(launch(loss_rows_kernel, dim3((unsigned)((a->rows + 7) / 8)), 256, 0, stream, L));
    if (a->dw) TRY(launch(loss_clean_kernel, dim3((unsigned)std::min<int64_t>(a->rows, 608)), 256, 0, stream, L));
    for (int64_t first = 0; first < a->vocab; first += piece) {
        const int64_t width = std::min(piece, a->vocab - first);
        Matrix wp = w, dlp = {dl, a->rows, width, ld_dl};
        wp.p = (const uint16_t*)w.p + first * w.ld;
        wp.rows = width;
        Rowwise R = {};
        R.p = values_of(a->rows, width, a->k, bf);
        R.coef = L.coef;
        R.first = (int32_t)first;
        TRY(run_rowwise(dev, SLOPE, &R, choose(R.p, kShapeSms, 1).best, x, wp, dl, ld_dl, stream));
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
            px.sum_first = first == 0;
            px.sum_last = first + piece >= a->vocab;
        }
        if (a->dw) {   // dw[v, k] = sum_t x[t, k] dl[t, v]
            pw.m = (int32_t)a->k;
            pw.n = (int32_t)width;
            pw.k = (int32_t)a->rows;
            pw.a_mn = pw.b_mn = 1;
            pw.alt = L.dirty;
            set_out(&pw, (uint16_t*)a->dw + first * lddw, lddw, 0, bf);
        }
        const Choices cx = a->dx ? choose(px, kShapeSms) : Choices(), cw = a->dw ? choose(pw, kShapeSms) : Choices();
        // one launch for both unless splitting or shapes of their own are worth more than the launch (9500 clocks)
        const double one = cx.single.cost + cw.single.cost, two = cx.pairs.cost + cw.pairs.cost;
        if (sum || (a->dx && a->dw && std::min(one, two) < cx.best.cost + cw.best.cost + 9500)) {
            Pair S = {};
            const Shape sx = two <= one ? cx.pairs : cx.single, sw = two <= one ? cw.pairs : cw.single;
            S.p[0] = px;
            TRY(complete(dev, &S.p[0], sx, wp, dlp));
            int64_t most = S.p[0].total;
            S.width = sx.bn;
            if (a->dw) {
                S.p[1] = pw;
                TRY(complete(dev, &S.p[1], sw, x, dlp, &clean));
                S.width = std::max(S.width, sw.bn);
                most += S.p[1].total;
            } else {
                S.p[1] = S.p[0];
                S.p[1].total = 0;
            }
            if (most > INT32_MAX) return fail(CCL_ERR_UNSUPPORTED, who + "too many tiles");
            const int cg = sx.cg, bytes = (kTileM + S.width / cg) * kSliceK * 2, fixed = 1024 + kStagingBytes;
            S.stages = std::min(kMaxStages, (kSmemBudget - fixed) / bytes);
            const int clusters = (int)std::min<int64_t>(most, dev->sms / cg);
            TRY(launch(cg == 2 ? sum_pair_kernel<2> : sum_pair_kernel<1>, dim3((unsigned)(clusters * cg)), kThreads,
                       fixed + (size_t)S.stages * bytes, stream, S, cg));
            continue;
        }
        if (a->dx) TRY(run_product(px, cx.best, wp, dlp, nullptr, stream));
        if (a->dw) TRY(run_product(pw, cw.best, x, dlp, &clean, stream));
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
