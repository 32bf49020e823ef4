// Layer norm and its gradients.  C ABI in include/ccl.h.
#include <algorithm>
#include <mutex>
#include <string>
#include <vector>

#include <cuda_runtime.h>

#include "ccl_norm_kernels.cuh"
#include "ccl_tensor_host.h"

namespace ccl {
namespace tensor {

#define NORM_KERNELS(t, tw) const NormKernels& norm_kernels_##t##_##tw()
NORM_KERNELS(f32, f32);
NORM_KERNELS(bf16, bf16);
NORM_KERNELS(bf16, f32);
NORM_KERNELS(f16, f16);
NORM_KERNELS(f16, f32);
#undef NORM_KERNELS

static const NormKernels& norm_kernels(int t, int tw)
{
    if (t == CCL_F32) return norm_kernels_f32_f32();
    if (t == CCL_BF16) return tw == CCL_F32 ? norm_kernels_bf16_f32() : norm_kernels_bf16_bf16();
    return tw == CCL_F32 ? norm_kernels_f16_f32() : norm_kernels_f16_f16();
}

// Shared memory of a backward pass: what its threads have on their way, or what
// the sums of its groups go through.
static size_t grad_smem(const NormKernels::Backward& r)
{
    return std::max<size_t>(r.each > 1 ? (size_t)kRowsAhead * 2 * r.pieces * r.threads * 16 : 0, (size_t)r.threads * r.each * 4);
}

// Once per device: the kernels of a pair of types may use that much.
static ccl_status_t norm_device(const NormKernels& k)
{
    static std::mutex mu;
    static std::vector<const NormKernels*> known[64];
    int d = 0;
    TRY_CUDA(cudaGetDevice(&d), "cudaGetDevice");
    if (d < 0 || d >= 64) return fail(CCL_ERR_UNSUPPORTED, "device index above 63");
    std::lock_guard<std::mutex> lock(mu);
    if (std::find(known[d].begin(), known[d].end(), &k) != known[d].end()) return CCL_OK;
    for (const auto& form : k.backward)
        for (const auto& r : form)
            TRY_CUDA(cudaFuncSetAttribute(r.kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)grad_smem(r)),
                     "shared memory of a norm's gradient");
    for (const auto& r : k.forward[1])
        if (r.blocks)
            TRY_CUDA(cudaFuncSetAttribute(r.kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, r.smem + r.stage), "shared memory of a norm");
    known[d].push_back(&k);
    return CCL_OK;
}

static ccl_status_t check_norm(const std::string& who, int64_t rows, int64_t n, int dtype, int wdtype)
{
    if (dtype != CCL_F32 && dtype != CCL_BF16 && dtype != CCL_F16)
        return fail(CCL_ERR_UNSUPPORTED, who + "takes f32, bf16 and f16 (dtype " + std::to_string(dtype) + ")");
    if (wdtype != dtype && wdtype != CCL_F32)
        return fail(CCL_ERR_UNSUPPORTED, who + "weight and bias have the type of x or are f32");
    if (rows < 0 || rows > INT32_MAX || n < 1 || n > (int64_t)1 << 24)
        return fail(CCL_ERR_INVALID_ARG, who + "sizes out of range (rows " + std::to_string(rows) + ", n " + std::to_string(n) + ")");
    return CCL_OK;
}

static ccl_status_t norm_array(const std::string& who, const char* what, const void* p, bool needed, int dtype)
{
    if (needed && !p) return fail(CCL_ERR_INVALID_ARG, who + what + " is null");
    if ((uintptr_t)p % (dtype == CCL_F32 ? 4 : 2)) return fail(CCL_ERR_INVALID_ARG, who + what + " is not aligned to its elements");
    return CCL_OK;
}

static ccl_status_t layer_norm(const ccl_layer_norm_t* a, cudaStream_t stream)
{
    const std::string who = "ccl_layer_norm: ";
    if (!a) return fail(CCL_ERR_INVALID_ARG, who + "null arguments");
    TRY(check_norm(who, a->rows, a->n, a->dtype, a->wdtype));
    if (!(a->eps >= 0.f)) return fail(CCL_ERR_INVALID_ARG, who + "eps is negative");
    Norm N = {};
    TRY(stride("x", a->ldx, a->n, &N.ld_x));
    TRY(stride("y", a->ldy, a->n, &N.ld_y));
    if (a->rows == 0) return CCL_OK;
    TRY(norm_array(who, "x", a->x, true, a->dtype));
    TRY(norm_array(who, "y", a->y, true, a->dtype));
    TRY(norm_array(who, "w", a->w, false, a->wdtype));
    TRY(norm_array(who, "b", a->b, false, a->wdtype));
    TRY(norm_array(who, "mean", a->mean, false, CCL_F32));
    TRY(norm_array(who, "rstd", a->rstd, false, CCL_F32));
    if (same(a->y, {a->w, a->b, a->mean, a->rstd}) || same(a->mean, {a->x, a->w, a->b, a->rstd}) || same(a->rstd, {a->x, a->w, a->b}))
        return fail(CCL_ERR_INVALID_ARG, who + "an output is also an operand or another output");
    if (a->rows > 1 && same(a->y, {a->x}) && N.ld_x != N.ld_y)
        return fail(CCL_ERR_INVALID_ARG, who + "y over an x of another row stride");
    N.x = a->x;
    N.y = a->y;
    N.w = a->w;
    N.b = a->b;
    N.mean = a->mean;
    N.rstd = a->rstd;
    N.rows = a->rows;
    N.n = a->n;
    N.eps = a->eps;
    const NormKernels& k = norm_kernels(a->dtype, a->wdtype);
    const int64_t each = a->dtype == CCL_F32 ? 4 : 8;
    const bool vec = a->n % each == 0 && aligned16(a->x) && aligned16(a->y) && aligned16(a->w) && aligned16(a->b) &&
                     N.ld_x % each == 0 && N.ld_y % each == 0;
    const int64_t es = a->dtype == CCL_F32 ? 4 : 2;
    N.apart = ((uintptr_t)a->x - (uintptr_t)a->y) % 16 != 0 || (a->rows > 1 && (N.ld_x - N.ld_y) * es % 16 != 0);
    for (const auto& r : k.forward[!vec]) {
        if (a->n > r.width) continue;
        int64_t blocks = (a->rows + r.rows - 1) / r.rows;
        if (r.blocks) {
            TRY(norm_device(k));
            blocks = std::min<int64_t>(blocks, (int64_t)kNormBlocks * r.blocks);
        }
        return launch(r.kernel, dim3((unsigned)blocks), r.threads, r.smem + (N.apart ? r.stage : 0), stream, N);
    }
    return launch(k.forward_long, dim3((unsigned)a->rows), 1024, 0, stream, N);
}

static int norm_blocks(int64_t rows, int64_t at_once)
{
    return (int)std::min<int64_t>(kNormBlocks, std::max<int64_t>(1, (rows + at_once - 1) / at_once));
}

static ccl_status_t layer_norm_grad(const ccl_layer_norm_grad_t* a, char* base, int64_t* need, cudaStream_t stream)
{
    const std::string who = "ccl_layer_norm_grad: ";
    if (!a) return fail(CCL_ERR_INVALID_ARG, who + "null arguments");
    TRY(check_norm(who, a->rows, a->n, a->dtype, a->wdtype));
    Norm N = {};
    TRY(stride("dy", a->lddy, a->n, &N.ld_dy));
    TRY(stride("x", a->ldx, a->n, &N.ld_x));
    TRY(stride("dx", a->lddx, a->n, &N.ld_dx));
    const bool sums = a->dw || a->db;
    Arena ws = {base};
    const int most = norm_blocks(a->rows, 1);
    if (sums && a->rows > 0) N.partial = ws.take<float>((int64_t)most * 2 * a->n * 4);
    if (need) {
        *need = ws.used;
        return CCL_OK;
    }
    const int wt = a->wdtype;
    TRY(norm_array(who, "dw", a->dw, false, wt));
    TRY(norm_array(who, "db", a->db, false, wt));
    if (same(a->dw, {a->db})) return fail(CCL_ERR_INVALID_ARG, who + "an output is also another output");
    if (a->rows == 0) {
        const size_t bytes = a->n * (wt == CCL_F32 ? 4 : 2);
        if (a->dw) TRY_CUDA(cudaMemsetAsync(a->dw, 0, bytes, stream), "dw");
        if (a->db) TRY_CUDA(cudaMemsetAsync(a->db, 0, bytes, stream), "db");
        return CCL_OK;
    }
    if (!a->dx && !sums) return CCL_OK;
    TRY(norm_array(who, "dy", a->dy, true, a->dtype));
    TRY(norm_array(who, "x", a->x, true, a->dtype));
    TRY(norm_array(who, "w", a->w, false, wt));
    TRY(norm_array(who, "mean", a->mean, true, CCL_F32));
    TRY(norm_array(who, "rstd", a->rstd, true, CCL_F32));
    TRY(norm_array(who, "dx", a->dx, false, a->dtype));
    for (const void* out : {(const void*)a->dx, (const void*)a->dw, (const void*)a->db})
        if (same(out, {a->dy, a->x, a->w, a->mean, a->rstd}))
            return fail(CCL_ERR_INVALID_ARG, who + "an output is also an operand");
    if (same(a->dx, {a->dw, a->db})) return fail(CCL_ERR_INVALID_ARG, who + "an output is also another output");
    N.dy = a->dy;
    N.x = a->x;
    N.w = a->w;
    N.mean = const_cast<float*>(a->mean);
    N.rstd = const_cast<float*>(a->rstd);
    N.dx = a->dx;
    N.dw = a->dw;
    N.db = a->db;
    N.rows = a->rows;
    N.n = a->n;
    const NormKernels& k = norm_kernels(a->dtype, wt);
    const int64_t each = a->dtype == CCL_F32 ? 4 : 8;
    const bool vec = a->n % each == 0 && aligned16(a->x) && aligned16(a->dy) && aligned16(a->dx) && aligned16(a->w) &&
                     N.ld_x % each == 0 && N.ld_dy % each == 0 && N.ld_dx % each == 0;
    TRY(norm_device(k));
    const NormKernels::Backward* fit = nullptr;
    for (const auto& r : k.backward[!vec])
        if (!fit && a->n <= r.width) fit = &r;
    if (fit) {
        N.blocks = norm_blocks(a->rows, fit->threads / fit->across);
        TRY(launch(fit->kernel, dim3(N.blocks), fit->threads, grad_smem(*fit), stream, N));
    } else {
        if (a->dx) TRY(launch(k.backward_long, dim3((unsigned)a->rows), 1024, 0, stream, N));
        N.blocks = norm_blocks(a->rows, 32);
        if (sums) TRY(launch(k.sums_long, dim3((unsigned)((a->n + 255) / 256), N.blocks), 256, 0, stream, N));
    }
    if (sums) TRY(launch(k.sums, dim3((unsigned)((a->n + 31) / 32), 2), 1024, 0, stream, N));
    return CCL_OK;
}

}  // namespace tensor
}  // namespace ccl

using namespace ccl;

extern "C" {

ccl_status_t ccl_layer_norm(const ccl_layer_norm_t* a, void* stream)
{
    C_ENTRY(tensor::layer_norm(a, (cudaStream_t)stream));
}
ccl_status_t ccl_layer_norm_grad_workspace(const ccl_layer_norm_grad_t* a, int64_t* bytes)
{
    C_ENTRY(tensor::measured(tensor::layer_norm_grad, a, bytes));
}
ccl_status_t ccl_layer_norm_grad(const ccl_layer_norm_grad_t* a, void* ws, int64_t ws_bytes, void* stream)
{
    C_ENTRY(tensor::guarded(tensor::layer_norm_grad, a, ws, ws_bytes, stream));
}

}  // extern "C"
