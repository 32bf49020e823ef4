// The router: scores, groups, the best experts of every row, their weights,
// the order of the rows by expert, and the weights' gradient.
#pragma once

#include "ccl_layer_common.cuh"
#include "ccl_rows.cuh"

namespace ccl {
namespace tensor {

constexpr int kMostChoices = 32;       // a lane each
constexpr int kMostRouted = 1024;      // experts: 32 a lane
constexpr int kMostExpertGroups = 32;  // a lane each

struct Route {
    const void* logits;
    const float* bias;
    float* weights;
    int32_t *chosen, *offsets, *place;
    int32_t* hist;                 // blocks x experts: choices of a block's rows by expert (several blocks)
    const float* dweights;         // gradient
    void* dlogits;
    int64_t rows, ld, ld_d;
    int64_t slots, per_block;      // rows x k; rows of a block (route), slots of a block (order)
    int32_t experts, k, type, score, groups, top_groups, group_best, renormalize, blocks;
    float scale;
};

__device__ __forceinline__ float load_as(const void* p, int64_t i, int type)
{
    return type == CCL_F32 ? ((const float*)p)[i] : load1((const uint16_t*)p + i, type == CCL_BF16);
}
__device__ __forceinline__ void store_as(void* p, int64_t i, int type, float v)
{
    if (type == CCL_F32)
        ((float*)p)[i] = v;
    else
        store1((uint16_t*)p + i, v, type == CCL_BF16);
}

__device__ __forceinline__ float sigmoid32(float l) { return 1.f / (1.f + expf(-l)); }

// Keys: unsigned numbers in the order of the values.  0 is a closed expert
// (logit or bias -inf), which nothing but another closed one ties with; NaN comes
// behind every number.
__device__ __forceinline__ uint32_t key_of(float v)
{
    const uint32_t b = __float_as_uint(v != v ? -3.402823466e38f : v == 0.f ? 0.f : v);
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ unsigned long long key_of(double v)
{
    const unsigned long long b = (unsigned long long)__double_as_longlong(v != v ? -1.7976931348623157e308 : v == 0. ? 0. : v);
    return b >> 63 ? ~b : b | 1ull << 63;
}
__device__ __forceinline__ uint32_t warp_most(uint32_t v) { return __reduce_max_sync(~0u, v); }
__device__ __forceinline__ unsigned long long warp_most(unsigned long long v)
{
    const uint32_t hi = __reduce_max_sync(~0u, (uint32_t)(v >> 32));
    const uint32_t lo = __reduce_max_sync(~0u, (uint32_t)(v >> 32) == hi ? (uint32_t)v : 0u);
    return (unsigned long long)hi << 32 | lo;
}

// Close the experts of all but the best groups.  val: the row's values in
// shared memory.  Returns whether the border between the groups is nearer
// than `near` (never without scores: values are exact then).
template <int VPL, typename F, typename K>
__device__ __forceinline__ bool keep_groups(const Route& R, const F (&v)[VPL], K (&key)[VPL], F* val, int lane, F near)
{
    const int size = R.experts / R.groups;
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
        const int e = i * 32 + lane;
        if (e < R.experts) val[e] = key[i] ? v[i] : (F)-INFINITY;
    }
    __syncwarp();
    // a lane a group: its largest value, or the sum of the two largest
    F a = (F)-INFINITY, b = (F)-INFINITY;
    if (lane < R.groups) {
        for (int i = 0; i < size; ++i) {
            F u = val[lane * size + i];
            if (u != u) u = (F)-3.402823466e38f;
            if (u > a)
                b = a, a = u;
            else if (u > b)
                b = u;
        }
    }
    __syncwarp();
    const bool open = a != (F)-INFINITY;
    if (R.group_best == 2 && b != (F)-INFINITY) a += b;
    int rank = 0;
    for (int g = 0; g < R.groups; ++g) {
        const F u = __shfl_sync(~0u, a, g);
        rank += u > a || (u == a && g < lane);
    }
    const bool kept = lane < R.groups && rank < R.top_groups;
    const uint32_t mask = __ballot_sync(~0u, kept);
    // the worst kept and the best dropped group, where both are open
    const uint32_t worst = __ballot_sync(~0u, lane < R.groups && rank == R.top_groups - 1);
    const uint32_t next = __ballot_sync(~0u, lane < R.groups && rank == R.top_groups);
    bool close = false;
    if (next) {
        const F u = __shfl_sync(~0u, a, __ffs(worst) - 1), w = __shfl_sync(~0u, a, __ffs(next) - 1);
        const bool both = __shfl_sync(~0u, (int)open, __ffs(next) - 1);
        close = both && !(u - w >= near);
    }
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
        const int e = i * 32 + lane;
        if (e < R.experts && !(mask >> e / size & 1)) key[i] = 0;
    }
    return close;
}

// The `count` largest keys of a row, ties to the lower expert; lane j gets the
// j-th one's expert (-1: none left) and key.
template <int VPL, typename K>
__device__ __forceinline__ void pick(K (&key)[VPL], int count, int lane, int& expert, K& found)
{
    expert = -1;
    found = 0;
    K best = 0;
    int at = 0;
#pragma unroll
    for (int i = 0; i < VPL; ++i)
        if (key[i] > best) best = key[i], at = i;
    for (int j = 0; j < count; ++j) {
        const K most = warp_most(best);
        if (most == 0) break;
        const uint32_t e = __reduce_min_sync(~0u, best == most ? (uint32_t)(at * 32 + lane) : ~0u);
        if (lane == j) expert = (int)e, found = most;
        if ((e & 31) == lane) {
            best = 0;
#pragma unroll
            for (int i = 0; i < VPL; ++i) {
                if (i == (int)(e >> 5)) key[i] = 0;
                if (key[i] > best) best = key[i], at = i;
            }
        }
    }
}

// A row's choices in 64 bits, for rows whose values lie too near to each other.
template <int VPL>
__device__ __noinline__ int choose64(const Route& R, int64_t row, double* val, int lane)
{
    double v[VPL];
    unsigned long long key[VPL];
    double most = -INFINITY;
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
        const int e = i * 32 + lane;
        v[i] = e < R.experts ? (double)load_as(R.logits, row * R.ld + e, R.type) : -INFINITY;
        key[i] = v[i] == -INFINITY ? 0 : 1;
        most = fmax(most, v[i]);
    }
#pragma unroll
    for (int d = 16; d; d >>= 1) most = fmax(most, __shfl_xor_sync(~0u, most, d));
    double sum = 0;
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
        v[i] = R.score == CCL_SCORE_SIGMOID ? 1 / (1 + exp(-v[i])) : exp(v[i] - most);
        sum += key[i] ? v[i] : 0;
    }
#pragma unroll
    for (int d = 16; d; d >>= 1) sum += __shfl_xor_sync(~0u, sum, d);
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
        if (!key[i]) continue;
        if (R.score != CCL_SCORE_SIGMOID) v[i] /= sum;
        if (R.bias) v[i] += (double)R.bias[i * 32 + lane];
        key[i] = v[i] == -INFINITY ? 0 : key_of(v[i]);
    }
    if (R.groups > 1) keep_groups<VPL>(R, v, key, val, lane, 0.);
    int expert;
    unsigned long long found;
    pick<VPL>(key, R.k, lane, expert, found);
    return expert;
}

// The choices of a row (lane j: the j-th) and their weights.
//
// Which experts come first is decided as in 64 bits.  Without a bias and sums
// of two, scores order the experts as the logits do, and the logits are
// compared.  Else values are computed in 32 bits with an error bound `near`; a
// row with two neighbours in the order (or two groups at the border) nearer
// than that is done again in 64 bits, about one in a thousand.
//   sigmoid: exp within 2 units, a sum, a division: 2^-21.4 of a score; two of
//     them, 2^-20 with the rounding of the comparison;
//   softmax: the sum is off by up to 37 roundings and scales all scores alike,
//     exp within 2 units, and l - max rounds to 2^-24 |l - max| of a score, at
//     most 2^-24 / e: 2^-18 of the largest score;
//   adding the bias rounds to 2^-24 of the value, twice.
template <int VPL>
__device__ __forceinline__ void route_row(const Route& R, int64_t row, double* val, int lane, int& expert, float& weight)
{
    float l[VPL], v[VPL];
    uint32_t key[VPL];
    bool poison = false;
    float most = -INFINITY;
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
        const int e = i * 32 + lane;
        l[i] = e < R.experts ? load_as(R.logits, row * R.ld + e, R.type) : -INFINITY;
    }
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
        most = fmaxf(most, l[i]);
        poison |= l[i] != l[i];
        v[i] = l[i];
    }
    most = warp_max(most);
    const bool softmax = R.score != CCL_SCORE_SIGMOID;
    const bool scored = R.bias || (R.groups > 1 && R.group_best == 2);
    poison = __any_sync(~0u, poison);
    float sum = 1.f, near = 0.f;
    if (softmax && (scored || !R.renormalize)) {
        sum = 0.f;
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
            const float p = l[i] == -INFINITY ? 0.f : expf(l[i] - most);
            if (scored) v[i] = p;
            sum += p;
        }
        sum = warp_sum(sum);
    }
    if (scored) {
        float top = 0.f, far = 0.f;
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
            const int e = i * 32 + lane;
            v[i] = softmax ? v[i] / sum : sigmoid32(l[i]);
            if (l[i] != -INFINITY) top = fmaxf(top, v[i]);
            if (R.bias && e < R.experts) v[i] += R.bias[e];
            if (l[i] != -INFINITY && fabsf(v[i]) < INFINITY) far = fmaxf(far, fabsf(v[i]));
        }
        near = warp_max(top) * (softmax ? 0x1p-18f : 0x1p-20f) + warp_max(far) * 0x1p-22f;
    }
#pragma unroll
    for (int i = 0; i < VPL; ++i) key[i] = l[i] == -INFINITY || v[i] == -INFINITY ? 0u : key_of(v[i]);
    bool again = false;
    if (R.groups > 1) again = keep_groups<VPL>(R, v, key, (float*)val, lane, scored ? 2.f * near : 0.f) && scored;
    uint32_t found;
    pick<VPL>(key, min(R.k + (scored ? 1 : 0), 32), lane, expert, found);
    float own = expert < 0 ? 0.f : load_as(R.logits, row * R.ld + expert, R.type);
    if (scored) {
        // neighbours in the order: near, and not for the same logit and bias
        const uint32_t below = __shfl_down_sync(~0u, found, 1);
        const float b = expert < 0 || !R.bias ? 0.f : R.bias[expert];
        const float own_below = __shfl_down_sync(~0u, own, 1), b_below = __shfl_down_sync(~0u, b, 1);
        const float value = __uint_as_float(found >> 31 ? found ^ 0x80000000u : ~found);
        const float next = __uint_as_float(below >> 31 ? below ^ 0x80000000u : ~below);
        again |= lane < R.k && lane < 31 && found && below && !(value - next >= near) && (own != own_below || b != b_below);
        // (with 32 choices the one behind the last is not looked at above)
        again |= R.k == 32 && R.experts > 32;
        if (__any_sync(~0u, again)) {
            __syncwarp();
            expert = choose64<VPL>(R, row, val, lane);
            own = expert < 0 ? 0.f : load_as(R.logits, row * R.ld + expert, R.type);
        }
    }
    if (lane >= R.k) expert = -1;
    // weights of the choices
    const bool on = expert >= 0;
    float w;
    if (!R.renormalize) {
        w = !softmax ? sigmoid32(own) : expf(own - most) / sum;
    } else if (softmax) {
        const float top = warp_max(on ? own : -INFINITY);
        w = on ? expf(own - top) : 0.f;
        w /= warp_sum(w);
    } else {
        // sigmoids over their sum, scaled by the largest exp(min(l, 0)): no sum that underflows
        const float a = fminf(own, 0.f), top = warp_max(on ? a : -INFINITY);
        w = on ? expf(a - top) / (1.f + expf(-fabsf(own))) : 0.f;
        w /= warp_sum(w);
    }
    if (softmax && poison) w = NAN;
    weight = on ? w * R.scale : 0.f;
}

// Slots in the order of their experts: place[s] is the slot's position when all
// slots are sorted by expert, slots of one expert in order; -1 where a slot has
// none.  A threadblock takes `per_block` consecutive slots; the slots of the
// blocks before it come from their counts in hist.  at: warps x experts words
// of shared memory, then experts.
__device__ __forceinline__ int expert_at(const Route& R, int64_t s)
{
    const int e = R.chosen[s];
    if (e >= R.experts) {
        report(REPORT_EXPERT);
        return -1;
    }
    return e;
}
// warps' counts of the experts of their slots
__device__ __forceinline__ void count_slots(const Route& R, int64_t from, int64_t to, int32_t* mine, int lane)
{
    for (int64_t s = from + lane; s - lane < to; s += 32) {
        const int e = s < to ? expert_at(R, s) : -1;
        const uint32_t peers = __match_any_sync(~0u, e);
        if (e >= 0 && lane == __ffs(peers) - 1) mine[e] += __popc(peers);
        __syncwarp();
    }
}

template <bool SINGLE>
__device__ __forceinline__ void place_slots(const Route& R, int block, int32_t* at)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5, E = R.experts;
    int32_t *total = at + warps * E, *before = total + E;
    const int64_t first = block * R.per_block, last = min(first + R.per_block, R.slots);
    const int64_t each = ((last - first + warps - 1) / warps + 31) / 32 * 32;
    const int64_t from = min(first + warp * each, last), to = min(from + each, last);
    for (int i = threadIdx.x; i < warps * E; i += blockDim.x) at[i] = 0;
    __syncthreads();
    count_slots(R, from, to, at + warp * E, lane);
    __syncthreads();
    // of every expert: slots of all blocks, of the blocks before this one
    if (SINGLE) {
        for (int e = threadIdx.x; e < E; e += blockDim.x) {
            int all = 0;
            for (int w = 0; w < warps; ++w) all += at[w * E + e];
            total[e] = all;
            before[e] = 0;
        }
    } else {
        // several threads an expert, each some of the blocks
        int width = 32;
        while (width < E && width < (int)blockDim.x) width *= 2;
        const int part = threadIdx.x / width, parts = blockDim.x / width;
        for (int e = threadIdx.x; e < E; e += blockDim.x) total[e] = before[e] = 0;
        __syncthreads();
        for (int e = threadIdx.x % width; e < E; e += width) {
            int all = 0, less = 0;
#pragma unroll 8
            for (int b = part; b < R.blocks; b += parts) {
                const int n = R.hist[(int64_t)b * E + e];
                all += n;
                less += b < block ? n : 0;
            }
            atomicAdd(&total[e], all);         // (whole numbers: any order gives the same sum)
            atomicAdd(&before[e], less);
        }
    }
    __syncthreads();
    if (warp == 0) {
        int base = 0;
        for (int e0 = 0; e0 < E; e0 += 32) {
            const int e = e0 + lane, n = e < E ? total[e] : 0;
            int v = n;
#pragma unroll
            for (int d = 1; d < 32; d *= 2) {
                const int u = __shfl_up_sync(~0u, v, d);
                if (lane >= d) v += u;
            }
            if (e < E) {
                before[e] += base + v - n;
                if (block == 0) R.offsets[e] = base + v - n;
            }
            base += __shfl_sync(~0u, v, 31);
        }
        if (block == 0 && lane == 0) R.offsets[E] = base;
    }
    __syncthreads();
    for (int e = threadIdx.x; e < E; e += blockDim.x) {
        int p = before[e];
        for (int w = 0; w < warps; ++w) {
            const int n = at[w * E + e];
            at[w * E + e] = p;
            p += n;
        }
    }
    __syncthreads();
    int32_t* next = at + warp * E;
    for (int64_t s = from + lane; s - lane < to; s += 32) {
        const int e = s < to ? expert_at(R, s) : -1;
        const uint32_t peers = __match_any_sync(~0u, e);
        const int p = e >= 0 ? next[e] + __popc(peers & ((1u << lane) - 1)) : -1;
        __syncwarp();
        if (e >= 0 && lane == __ffs(peers) - 1) next[e] += __popc(peers);
        __syncwarp();
        if (s < to) R.place[s] = p;
    }
}

// A warp a row, a threadblock `per_block` consecutive rows.  ORDER: 0 choices
// and weights only; 1 one threadblock, which orders the rows as well; 2 every
// threadblock leaves its counts for place_kernel.
template <int VPL, int ORDER>
__global__ void __launch_bounds__(512) route_kernel(const Route R)
{
    extern __shared__ __align__(16) unsigned char smem[];
    let_next_in();
    wait_for_previous();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    int32_t* hist = reinterpret_cast<int32_t*>(smem);
    double* val = reinterpret_cast<double*>(smem + (ORDER == 2 ? (R.experts * 4 + 7) & ~7 : 0)) +
                  (R.groups > 1 ? warp * R.experts : 0);
    if (ORDER == 2) {
        for (int e = threadIdx.x; e < R.experts; e += blockDim.x) hist[e] = 0;
        __syncthreads();
    }
    const int64_t first = blockIdx.x * R.per_block, last = min(first + R.per_block, R.rows);
    for (int64_t row = first + warp; row < last; row += warps) {
        int expert;
        float weight;
        route_row<VPL>(R, row, val, lane, expert, weight);
        if (lane < R.k) {
            R.chosen[row * R.k + lane] = expert;
            R.weights[row * R.k + lane] = weight;
        }
        if (ORDER == 2 && expert >= 0) atomicAdd(&hist[expert], 1);
    }
    if (ORDER == 0) return;
    __syncthreads();
    if (ORDER == 1) {
        Route S = R;
        S.per_block = R.slots;
        place_slots<true>(S, 0, hist);
    } else {
        for (int e = threadIdx.x; e < R.experts; e += blockDim.x) R.hist[(int64_t)blockIdx.x * R.experts + e] = hist[e];
    }
}

__global__ void __launch_bounds__(512) count_kernel(const Route R)
{
    extern __shared__ __align__(16) unsigned char smem[];
    int32_t* hist = reinterpret_cast<int32_t*>(smem);
    let_next_in();
    wait_for_previous();
    for (int e = threadIdx.x; e < R.experts; e += blockDim.x) hist[e] = 0;
    __syncthreads();
    const int64_t first = blockIdx.x * R.per_block, last = min(first + R.per_block, R.slots);
    for (int64_t s = first + threadIdx.x; s < last; s += blockDim.x) {
        const int e = expert_at(R, s);
        if (e >= 0) atomicAdd(&hist[e], 1);
    }
    __syncthreads();
    for (int e = threadIdx.x; e < R.experts; e += blockDim.x) R.hist[(int64_t)blockIdx.x * R.experts + e] = hist[e];
}

template <bool SINGLE>
__global__ void __launch_bounds__(512) place_kernel(const Route R)
{
    extern __shared__ __align__(16) unsigned char smem[];
    let_next_in();
    wait_for_previous();
    place_slots<SINGLE>(R, blockIdx.x, reinterpret_cast<int32_t*>(smem));
}

// The gradient of a row's logits from those of its weights, for the choices as they are:
//   softmax                 dl = p (g - sum g p)        (all experts)
//   softmax, renormalised   dl = w (g - sum g w)        (the chosen, w their weights)
//   sigmoid                 dl = g s (1 - s)            (the chosen)
//   sigmoid, renormalised   dl = w (1 - s)(g - sum g w) (the chosen)
// A warp a row.  An expert chosen twice gets the sum of both.
template <int VPL>
__global__ void __launch_bounds__(256) route_grad_kernel(const Route R)
{
    let_next_in();
    wait_for_previous();
    const int lane = threadIdx.x & 31;
    const int64_t row = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
    if (row >= R.rows) return;
    const bool softmax = R.score != CCL_SCORE_SIGMOID, dense = softmax && !R.renormalize;
    int expert = -1;
    float g = 0.f, own = 0.f;
    if (lane < R.k) {
        expert = expert_at(R, row * R.k + lane);
        if (expert >= 0) {
            g = R.dweights[row * R.k + lane] * R.scale;
            own = load_as(R.logits, row * R.ld + expert, R.type);
        }
    }
    const bool on = expert >= 0;
    float l[VPL], most = 0.f, sum = 1.f;
    if (dense) {
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
            const int e = i * 32 + lane;
            l[i] = e < R.experts ? load_as(R.logits, row * R.ld + e, R.type) : -INFINITY;
        }
        most = l[0];
#pragma unroll
        for (int i = 1; i < VPL; ++i) most = fmaxf(most, l[i]);
        most = warp_max(most);
        sum = 0.f;
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
            l[i] = l[i] == -INFINITY ? 0.f : expf(l[i] - most);
            sum += l[i];
        }
        sum = warp_sum(sum);
#pragma unroll
        for (int i = 0; i < VPL; ++i) l[i] = sum == 0.f ? 0.f : l[i] / sum;
    }
    float part = 0.f;              // of a choice: its own term of the gradient
    float all = 0.f;
    if (dense) {
        all = warp_sum(on ? g * (own == -INFINITY ? 0.f : expf(own - most) / sum) : 0.f);
        part = g;
    } else if (!R.renormalize) {
        part = on ? g * sigmoid32(own) * sigmoid32(-own) : 0.f;
    } else {
        const float a = softmax ? own : fminf(own, 0.f), top = warp_max(on ? a : -INFINITY);
        float w = on ? expf(a - top) / (softmax ? 1.f : 1.f + expf(-fabsf(own))) : 0.f;
        w /= warp_sum(w);
        const float mean = warp_sum(on ? g * w : 0.f);
        part = on ? w * (g - mean) * (softmax ? 1.f : sigmoid32(-own)) : 0.f;
    }
    float d[VPL];
#pragma unroll
    for (int i = 0; i < VPL; ++i) d[i] = 0.f;
    for (int j = 0; j < R.k; ++j) {
        const int e = __shfl_sync(~0u, expert, j);
        const float v = __shfl_sync(~0u, part, j);
#pragma unroll
        for (int i = 0; i < VPL; ++i)
            if (e == i * 32 + lane) d[i] += v;
    }
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
        const int e = i * 32 + lane;
        if (e < R.experts) store_as(R.dlogits, row * R.ld_d + e, R.type, dense ? l[i] * (d[i] - all) : d[i]);
    }
}

}  // namespace tensor
}  // namespace ccl
