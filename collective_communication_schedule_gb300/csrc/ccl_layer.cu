// The router, the order of rows by expert, and the rows' way to their experts
// and back.  C ABI in include/ccl.h.
#include <algorithm>
#include <mutex>
#include <string>

#include <cuda_runtime.h>

#include "ccl_route.cuh"
#include "ccl_rows.cuh"
#include "ccl_tensor_host.h"

namespace ccl {
namespace tensor {

static int element_bytes(int dtype) { return dtype == CCL_F32 ? 4 : 2; }

static ccl_status_t check_type(const std::string& who, int dtype)
{
    if (dtype != CCL_F32 && dtype != CCL_BF16 && dtype != CCL_F16)
        return fail(CCL_ERR_UNSUPPORTED, who + "takes f32, bf16 and f16 (dtype " + std::to_string(dtype) + ")");
    return CCL_OK;
}

// an array of 32-bit words, or of elements of another size
static ccl_status_t array(const std::string& who, const char* what, const void* p, bool needed, int bytes = 4)
{
    if (needed && !p) return fail(CCL_ERR_INVALID_ARG, who + what + " is null");
    if ((uintptr_t)p % bytes) return fail(CCL_ERR_INVALID_ARG, who + what + " is not aligned to its elements");
    return CCL_OK;
}

// ---------------------------------------------------------------- router
constexpr int kOrderThreads = 1024;
constexpr int kRouteSmem = 34 * kMostRouted * 4;       // counts of 32 warps and two of the block (more than 16 warps' values)

// The kernels for every number of experts a lane, from the smallest up: widths
// that usual numbers of experts fill, so that groups of them are whole lanes.
struct RouteKernel {
    int vpl;
    void (*route)(const Route);
    void (*grad)(const Route);
};
#define ROUTE(vpl) {vpl, route_kernel<vpl>, route_grad_kernel<vpl>}
static const RouteKernel kRoute[] = {ROUTE(1), ROUTE(2), ROUTE(3), ROUTE(4),  ROUTE(5),
                                     ROUTE(6), ROUTE(8), ROUTE(12), ROUTE(16), ROUTE(32)};
#undef ROUTE
static const RouteKernel& route_kernel_for(int64_t experts)
{
    const RouteKernel* k = kRoute;
    while (32 * k->vpl < experts) ++k;
    return *k;
}

// once per device: kernels that take more than 48 KB of shared memory are told so
static ccl_status_t layer_device()
{
    static std::mutex mu;
    static bool known[64];
    int d = 0;
    TRY_CUDA(cudaGetDevice(&d), "cudaGetDevice");
    if (d < 0 || d >= 64) return fail(CCL_ERR_UNSUPPORTED, "device index above 63");
    std::lock_guard<std::mutex> lock(mu);
    if (known[d]) return CCL_OK;
    for (const RouteKernel& k : kRoute)
        TRY_CUDA(cudaFuncSetAttribute(k.route, cudaFuncAttributeMaxDynamicSharedMemorySize, kRouteSmem),
                 "shared memory of the router");
    for (auto kernel : {place_kernel<true>, place_kernel<false>})
        TRY_CUDA(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kRouteSmem),
                 "shared memory of the row order");
    known[d] = true;
    return CCL_OK;
}

// Blocks of a router call whose rows are ordered too, and of an order alone, at
// least `least` rows or slots each: by the sizes, so that the workspace does not
// depend on the device.  A block's place in the order costs the same whatever it
// holds, so small calls take few.
constexpr int kOrderBlocks = 152;
static int order_blocks(int64_t items, int least)
{
    return (int)std::min<int64_t>(kOrderBlocks, (items + least - 1) / least);
}
static size_t order_smem(int experts, int threads) { return (size_t)(threads / 32 + 2) * experts * 4; }
static int64_t hist_bytes(int blocks, int64_t experts) { return blocks * round_up(experts, 4) * 4; }

static ccl_status_t check_router(const std::string& who, int64_t rows, int64_t experts, int k, int dtype, int score)
{
    TRY(check_type(who, dtype));
    if (experts < 1 || experts > kMostRouted)
        return fail(CCL_ERR_INVALID_ARG, who + "experts outside 1.." + std::to_string(kMostRouted));
    if (k < 1 || k > kMostChoices || k > experts)
        return fail(CCL_ERR_INVALID_ARG, who + "choices outside 1.." + std::to_string(std::min<int64_t>(kMostChoices, experts)));
    if (rows < 0 || rows > INT32_MAX / k) return fail(CCL_ERR_INVALID_ARG, who + "rows out of range");
    if (score != CCL_SCORE_SOFTMAX && score != CCL_SCORE_SIGMOID)
        return fail(CCL_ERR_INVALID_ARG, who + "unknown score " + std::to_string(score));
    return CCL_OK;
}

// As many rows go to one threadblock, which orders them as well: us in one launch
// and in two, 64 experts, choose 6: 1 row 4.6 and 7.0, 24 rows 6.3 and 7.3, 32 rows 7.1
// and 7.4; 256 experts, choose 8: 6.8 and 8.6, 8.6 and 9.3, 10.2 and 9.6.
constexpr int kRowsOfOne = 24;

static ccl_status_t route(const ccl_route_t* a, char* base, int64_t* need, cudaStream_t stream)
{
    const std::string who = "ccl_route: ";
    if (!a) return fail(CCL_ERR_INVALID_ARG, who + "null arguments");
    TRY(check_router(who, a->rows, a->experts, a->k, a->dtype, a->score));
    if (a->groups < 0 || a->groups > kMostExpertGroups || (a->groups > 1 && a->experts % a->groups))
        return fail(CCL_ERR_INVALID_ARG, who + "groups outside 1.." + std::to_string(kMostExpertGroups) + " or no divisor of the experts");
    const int groups = a->groups > 1 ? a->groups : 1;
    if (groups > 1) {
        if (a->top_groups < 1 || a->top_groups > groups) return fail(CCL_ERR_INVALID_ARG, who + "top_groups outside 1..groups");
        if (a->group_best < 1 || a->group_best > 2) return fail(CCL_ERR_INVALID_ARG, who + "group_best is neither 1 nor 2");
        if (a->experts / groups * a->top_groups < a->k)
            return fail(CCL_ERR_INVALID_ARG, who + "more choices than experts in the best groups");
    }
    int64_t ld;
    TRY(stride("logits", a->ld, a->experts, &ld));
    const bool order = a->offsets || a->place;
    if (order && !(a->offsets && (a->place || a->rows == 0))) return fail(CCL_ERR_INVALID_ARG, who + "offsets and place go together");
    Arena ws = {base};
    Route R = {};
    const bool one = a->rows <= kRowsOfOne;
    R.blocks = one ? 1 : order_blocks(a->rows, 16);
    if (order && !one) R.hist = ws.take<int32_t>(hist_bytes(R.blocks, a->experts));
    if (need) {
        *need = ws.used;
        return CCL_OK;
    }
    const bool some = a->rows > 0;
    TRY(array(who, "logits", a->logits, some, element_bytes(a->dtype)));
    TRY(array(who, "bias", a->bias, false));
    TRY(array(who, "weights", a->weights, some));
    TRY(array(who, "chosen", a->chosen, some));
    TRY(array(who, "offsets", a->offsets, false));
    TRY(array(who, "place", a->place, false));
    if (!some) {
        if (order) TRY_CUDA(cudaMemsetAsync(a->offsets, 0, (a->experts + 1) * 4, stream), "offsets");
        return CCL_OK;
    }
    if (same(a->weights, {a->logits, a->bias, a->chosen, a->place, a->offsets}) || same(a->chosen, {a->logits, a->bias, a->place, a->offsets}) ||
        same(a->place, {a->logits, a->bias, a->offsets}) || same(a->offsets, {a->logits, a->bias}))
        return fail(CCL_ERR_INVALID_ARG, who + "an output is also an operand or another output");
    R.logits = a->logits;
    R.bias = a->bias;
    R.weights = a->weights;
    R.chosen = a->chosen;
    R.offsets = a->offsets;
    R.place = a->place;
    R.rows = a->rows;
    R.ld = ld;
    R.slots = a->rows * a->k;
    R.experts = (int32_t)a->experts;
    R.k = a->k;
    R.type = a->dtype;
    R.score = a->score;
    R.groups = groups;
    R.top_groups = a->top_groups;
    R.group_best = groups > 1 ? a->group_best : 1;
    R.renormalize = a->renormalize != 0;
    R.scored = a->bias || R.group_best == 2;
    R.scale = a->scale;
    TRY(layer_device());
    const int64_t each = 16 / element_bytes(a->dtype);
    R.vec = aligned16(a->logits) && ld % each == 0 && a->experts % each == 0;
    const RouteKernel& k = route_kernel_for(a->experts);
    R.vec_b = aligned16(a->bias) && a->experts % 4 == 0;
    if (groups > 1) {
        R.group_size = R.experts / groups;
        R.group_lanes = R.group_size % k.vpl ? 0 : R.group_size / k.vpl;
    }
    const int most = route_threads(k.vpl);
    // values in 64 bits (and groups that are not whole lanes) need shared memory: for a warp each
    const bool held = a->bias || groups > 1;
    auto values = [&](int threads) { return held ? (size_t)threads / 32 * a->experts * 8 : 0; };
    if (!order) {
        const int threads = 256;
        const int64_t blocks = (a->rows + 7) / 8;
        R.per_block = 8;
        return launch(k.route, dim3((unsigned)blocks), threads, values(threads), stream, R);
    }
    if (one) {
        const int threads = (int)std::min<int64_t>(most, round_up(std::max<int64_t>(a->rows, 4), 4) * 32);
        R.order = 1;
        R.per_block = a->rows;
        return launch(k.route, dim3(1), threads, std::max(values(threads), order_smem(R.experts, threads)), stream, R);
    }
    R.order = 2;
    R.per_block = (a->rows + R.blocks - 1) / R.blocks;
    R.blocks = (int32_t)((a->rows + R.per_block - 1) / R.per_block);
    const int threads = (int)std::min<int64_t>(most, round_up(R.per_block, 4) * 32);
    TRY(launch(k.route, dim3(R.blocks), threads, round_up(a->experts * 4, 8) + values(threads), stream, R));
    R.per_block *= a->k;
    return launch(place_kernel<false>, dim3(R.blocks), kOrderThreads, order_smem(R.experts, kOrderThreads), stream, R);
}

static ccl_status_t expert_order(const ccl_expert_order_t* a, char* base, int64_t* need, cudaStream_t stream)
{
    const std::string who = "ccl_expert_order: ";
    if (!a) return fail(CCL_ERR_INVALID_ARG, who + "null arguments");
    if (a->experts < 1 || a->experts > kMostRouted)
        return fail(CCL_ERR_INVALID_ARG, who + "experts outside 1.." + std::to_string(kMostRouted));
    if (a->slots < 0 || a->slots > INT32_MAX) return fail(CCL_ERR_INVALID_ARG, who + "slots out of range");
    Arena ws = {base};
    Route R = {};
    // one threadblock for what takes it no longer than a second launch (256 experts, us in one and
    // several: 1024 slots 5.0 and 5.4, 2048 slots 7.2 and 5.5, 8192 slots 19.1 and 5.7)
    R.blocks = a->slots <= kOrderThreads ? 1 : order_blocks(a->slots, 512);
    if (R.blocks > 1) R.hist = ws.take<int32_t>(hist_bytes(R.blocks, a->experts));
    if (need) {
        *need = ws.used;
        return CCL_OK;
    }
    const bool some = a->slots > 0;
    TRY(array(who, "chosen", a->chosen, some));
    TRY(array(who, "place", a->place, some));
    TRY(array(who, "offsets", a->offsets, true));
    if (same(a->place, {a->chosen, a->offsets}) || same(a->offsets, {a->chosen}))
        return fail(CCL_ERR_INVALID_ARG, who + "an output is also an operand or another output");
    if (!some) {
        TRY_CUDA(cudaMemsetAsync(a->offsets, 0, (a->experts + 1) * 4, stream), "offsets");
        return CCL_OK;
    }
    R.chosen = const_cast<int32_t*>(a->chosen);
    R.offsets = a->offsets;
    R.place = a->place;
    R.slots = a->slots;
    R.experts = a->experts;
    TRY(layer_device());
    R.per_block = (a->slots + R.blocks - 1) / R.blocks;
    if (R.blocks == 1) return launch(place_kernel<true>, dim3(1), kOrderThreads, order_smem(R.experts, kOrderThreads), stream, R);
    R.blocks = (int32_t)((a->slots + R.per_block - 1) / R.per_block);
    TRY(launch(count_kernel, dim3(R.blocks), 512, a->experts * 4, stream, R));
    return launch(place_kernel<false>, dim3(R.blocks), kOrderThreads, order_smem(R.experts, kOrderThreads), stream, R);
}

static ccl_status_t route_grad(const ccl_route_grad_t* a, cudaStream_t stream)
{
    const std::string who = "ccl_route_grad: ";
    if (!a) return fail(CCL_ERR_INVALID_ARG, who + "null arguments");
    TRY(check_router(who, a->rows, a->experts, a->k, a->dtype, a->score));
    int64_t ld, ldd;
    TRY(stride("logits", a->ld, a->experts, &ld));
    TRY(stride("dlogits", a->ldd, a->experts, &ldd));
    if (a->rows == 0) return CCL_OK;
    const int es = element_bytes(a->dtype);
    TRY(array(who, "logits", a->logits, true, es));
    TRY(array(who, "chosen", a->chosen, true));
    TRY(array(who, "dweights", a->dweights, true));
    TRY(array(who, "dlogits", a->dlogits, true, es));
    if (same(a->dlogits, {a->logits, a->chosen, a->dweights}))
        return fail(CCL_ERR_INVALID_ARG, who + "the output is also an operand");
    Route R = {};
    R.logits = a->logits;
    R.chosen = const_cast<int32_t*>(a->chosen);
    R.dweights = a->dweights;
    R.dlogits = a->dlogits;
    R.rows = a->rows;
    R.ld = ld;
    R.ld_d = ldd;
    R.experts = (int32_t)a->experts;
    R.k = a->k;
    R.type = a->dtype;
    R.score = a->score;
    R.renormalize = a->renormalize != 0;
    R.scale = a->scale;
    const int64_t each = 16 / es;
    R.vec = aligned16(a->logits) && ld % each == 0 && a->experts % each == 0;
    R.vec_d = aligned16(a->dlogits) && ldd % each == 0 && a->experts % each == 0;
    return launch(route_kernel_for(a->experts).grad, dim3((unsigned)((a->rows + 7) / 8)), 256, 0, stream, R);
}

// ------------------------------------------------------------- row moves
#define BY_TYPE(kernel, dtype, vec)                                                                     \
    ((dtype) == CCL_F32 ? ((vec) ? kernel<CCL_F32, true> : kernel<CCL_F32, false>)                      \
     : (dtype) == CCL_BF16 ? ((vec) ? kernel<CCL_BF16, true> : kernel<CCL_BF16, false>)                 \
                           : ((vec) ? kernel<CCL_F16, true> : kernel<CCL_F16, false>))

static ccl_status_t check_moves(const std::string& who, int64_t rows, int64_t count, int64_t h, int k, int dtype)
{
    TRY(check_type(who, dtype));
    if (k < 1 || k > kMostChoices) return fail(CCL_ERR_INVALID_ARG, who + "choices outside 1.." + std::to_string(kMostChoices));
    if (rows < 0 || rows > INT32_MAX / k || count < 0 || count > INT32_MAX || h < 1 || h > 1 << 24)
        return fail(CCL_ERR_INVALID_ARG, who + "sizes out of range (rows " + std::to_string(rows) + ", places " +
                                             std::to_string(count) + ", width " + std::to_string(h) + ")");
    return CCL_OK;
}

// whether rows can be read 16 bytes at a time
static bool by_vectors(int64_t h, int dtype, std::initializer_list<std::pair<const void*, int64_t>> rows)
{
    const int64_t each = 16 / element_bytes(dtype);
    bool ok = h % each == 0;
    for (auto& m : rows) ok = ok && (!m.first || (aligned16(m.first) && m.second % each == 0));
    return ok;
}

// A warp's pieces of all rows; the grid is one-dimensional.
static ccl_status_t pieces(const std::string& who, Moves* M, int width, dim3* grid)
{
    M->chunks = (int32_t)((M->h + width - 1) / width);
    const int64_t blocks = (M->rows * M->chunks + 7) / 8;
    if (blocks > INT32_MAX) return fail(CCL_ERR_UNSUPPORTED, who + "too many pieces of rows");
    *grid = dim3((unsigned)blocks);
    return CCL_OK;
}

static ccl_status_t dispatch(const ccl_dispatch_t* a, cudaStream_t stream)
{
    const std::string who = "ccl_dispatch: ";
    if (!a) return fail(CCL_ERR_INVALID_ARG, who + "null arguments");
    TRY(check_moves(who, a->rows, a->count, a->h, a->k, a->dtype));
    Moves M = {};
    TRY(stride("x", a->ldx, a->h, &M.ld_x));
    TRY(stride("out", a->ldo, a->h, &M.ld_out));
    if (a->rows == 0) return CCL_OK;
    const int es = element_bytes(a->dtype);
    TRY(array(who, "x", a->x, true, es));
    TRY(array(who, "out", a->out, a->count > 0, es));
    TRY(array(who, "place", a->place, true));
    if (same(a->out, {a->x, a->place})) return fail(CCL_ERR_INVALID_ARG, who + "the output is also an operand");
    M.x = a->x;
    M.out = a->out;
    M.place = a->place;
    M.rows = a->rows;
    M.count = a->count;
    M.h = a->h;
    M.k = a->k;
    const bool vec = by_vectors(a->h, a->dtype, {{a->x, M.ld_x}, {a->out, M.ld_out}});
    dim3 grid;
    TRY(pieces(who, &M, 32 * (vec ? 16 / es : 8), &grid));
    return launch(BY_TYPE(dispatch_kernel, a->dtype, vec), grid, 256, 0, stream, M);
}

static ccl_status_t combine(const ccl_combine_t* a, cudaStream_t stream)
{
    const std::string who = "ccl_combine: ";
    if (!a) return fail(CCL_ERR_INVALID_ARG, who + "null arguments");
    TRY(check_moves(who, a->rows, a->count, a->h, a->k, a->dtype));
    Moves M = {};
    TRY(stride("r", a->ldr, a->h, &M.ld_r));
    TRY(stride("residual", a->lds, a->h, &M.ld_s));
    TRY(stride("y", a->ldy, a->h, &M.ld_out));
    if (a->rows == 0) return CCL_OK;
    const int es = element_bytes(a->dtype);
    TRY(array(who, "r", a->r, a->count > 0, es));
    TRY(array(who, "y", a->y, true, es));
    TRY(array(who, "residual", a->residual, false, es));
    TRY(array(who, "place", a->place, true));
    TRY(array(who, "weights", a->weights, false));
    if (same(a->y, {a->r, a->place, a->weights})) return fail(CCL_ERR_INVALID_ARG, who + "the output is also an operand");
    if (a->rows > 1 && same(a->y, {a->residual}) && M.ld_s != M.ld_out)
        return fail(CCL_ERR_INVALID_ARG, who + "y over a residual of another row stride");
    M.r = a->r;
    M.residual = a->residual;
    M.out = a->y;
    M.place = a->place;
    M.weights = a->weights;
    M.rows = a->rows;
    M.count = a->count;
    M.h = a->h;
    M.k = a->k;
    const bool vec = by_vectors(a->h, a->dtype, {{a->r, M.ld_r}, {a->y, M.ld_out}, {a->residual, M.ld_s}});
    dim3 grid;
    TRY(pieces(who, &M, 32 * (vec ? 16 / es : 8), &grid));
    return launch(BY_TYPE(combine_kernel, a->dtype, vec), grid, 256, 0, stream, M);
}

static ccl_status_t combine_grad(const ccl_combine_grad_t* a, cudaStream_t stream)
{
    const std::string who = "ccl_combine_grad: ";
    if (!a) return fail(CCL_ERR_INVALID_ARG, who + "null arguments");
    TRY(check_moves(who, a->rows, a->count, a->h, a->k, a->dtype));
    Moves M = {};
    TRY(stride("dy", a->lddy, a->h, &M.ld_x));
    TRY(stride("r", a->ldr, a->h, &M.ld_r));
    TRY(stride("dr", a->lddr, a->h, &M.ld_out));
    if (a->rows == 0 || (!a->dr && !a->dweights)) return CCL_OK;
    const int es = element_bytes(a->dtype);
    TRY(array(who, "dy", a->dy, true, es));
    TRY(array(who, "r", a->r, a->dweights && a->count > 0, es));
    TRY(array(who, "dr", a->dr, false, es));
    TRY(array(who, "place", a->place, true));
    TRY(array(who, "weights", a->weights, false));
    TRY(array(who, "dweights", a->dweights, false));
    if (same(a->dr, {a->dy, a->dweights ? a->r : nullptr, a->place, a->weights, a->dweights}) ||
        same(a->dweights, {a->dy, a->r, a->place, a->weights}))
        return fail(CCL_ERR_INVALID_ARG, who + "an output is also an operand or another output");
    M.x = a->dy;
    M.r = a->r;
    M.out = a->dr;
    M.place = a->place;
    M.weights = a->weights;
    M.dweights = a->dweights;
    M.rows = a->rows;
    M.count = a->count;
    M.h = a->h;
    M.k = a->k;
    const bool vec = by_vectors(a->h, a->dtype, {{a->dy, M.ld_x}, {a->dweights ? a->r : nullptr, M.ld_r}, {a->dr, M.ld_out}});
    const int64_t all = a->rows * a->k;
    // four short rows at a time from 16384 choices on, us so and a warp a choice: h = 128 bf16, 8192 choices
    // 4.2 and 3.0, 16384 4.7 and 4.7, 32768 4.9 and 8.3, 128000 15.6 and 36.3
    if (vec && a->h * es <= 32 * 16 && all > 16384) {
        M.chunks = 1;
        while (M.chunks * 16 < a->h * es) M.chunks *= 2;
        const int64_t each = 256 / M.chunks * 4;
        auto kernel = a->dtype == CCL_F32 ? combine_grad_short_kernel<CCL_F32>
                      : a->dtype == CCL_BF16 ? combine_grad_short_kernel<CCL_BF16> : combine_grad_short_kernel<CCL_F16>;
        return launch(kernel, dim3((unsigned)((all + each - 1) / each)), 256, 0, stream, M);
    }
    return launch(BY_TYPE(combine_grad_kernel, a->dtype, vec), dim3((unsigned)((all + 7) / 8)), 256, 0, stream, M);
}

ccl_status_t take_layer_status()
{
    int st[4] = {0, 0, 0, 0};
    TRY_CUDA(cudaMemcpyFromSymbol(st, g_layer_status, sizeof(st)), "status word");
    if (st[0] == 0) return take_loss_status();
    const int zero[4] = {0, 0, 0, 0};
    TRY_CUDA(cudaMemcpyToSymbol(g_layer_status, zero, sizeof(zero)), "status word");
    return fail((ccl_status_t)st[0], st[1] == REPORT_PLACE ? "a place beyond the rows" : "a chosen expert beyond the experts");
}

}  // namespace tensor
}  // namespace ccl

using namespace ccl;

extern "C" {

ccl_status_t ccl_route_workspace(const ccl_route_t* a, int64_t* bytes) { C_ENTRY(tensor::measured(tensor::route, a, bytes)); }
ccl_status_t ccl_route(const ccl_route_t* a, void* ws, int64_t ws_bytes, void* stream)
{
    C_ENTRY(tensor::guarded(tensor::route, a, ws, ws_bytes, stream));
}
ccl_status_t ccl_route_grad(const ccl_route_grad_t* a, void* stream)
{
    C_ENTRY(tensor::route_grad(a, (cudaStream_t)stream));
}
ccl_status_t ccl_expert_order_workspace(const ccl_expert_order_t* a, int64_t* bytes)
{
    C_ENTRY(tensor::measured(tensor::expert_order, a, bytes));
}
ccl_status_t ccl_expert_order(const ccl_expert_order_t* a, void* ws, int64_t ws_bytes, void* stream)
{
    C_ENTRY(tensor::guarded(tensor::expert_order, a, ws, ws_bytes, stream));
}
ccl_status_t ccl_dispatch(const ccl_dispatch_t* a, void* stream) { C_ENTRY(tensor::dispatch(a, (cudaStream_t)stream)); }
ccl_status_t ccl_combine(const ccl_combine_t* a, void* stream) { C_ENTRY(tensor::combine(a, (cudaStream_t)stream)); }
ccl_status_t ccl_combine_grad(const ccl_combine_grad_t* a, void* stream)
{
    C_ENTRY(tensor::combine_grad(a, (cudaStream_t)stream));
}

}  // extern "C"
