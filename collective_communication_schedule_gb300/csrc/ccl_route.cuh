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
    int32_t scored;                // values other than the logits decide something
    int32_t group_size, group_lanes;   // experts of a group; lanes of one where they are whole lanes, else 0
    int32_t vec_b;                 // bias can be read 16 bytes at a time
    int32_t order;                 // 0: choices and weights only, 1: one threadblock, which orders the rows as well, 2: counts for
                                   // place_kernel are left in hist
    int32_t vec, vec_d;            // rows of logits can be read, of dlogits written 16 bytes at a time
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
__device__ __forceinline__ float exp2_near(float x)      // within 2^-22
{
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// Keys: unsigned numbers in the order of the values.  0 is a closed expert
// (logit or bias -inf), which nothing but another closed one ties with; NaN comes
// behind every number.
__device__ __forceinline__ uint32_t key_of(float v)
{
    const uint32_t b = __float_as_uint(fmaxf(v, -3.402823466e38f) + 0.f);     // (+ 0: one zero)
    return v == -INFINITY ? 0u : b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}
__device__ __forceinline__ float value_of(uint32_t key)
{
    return __uint_as_float(key >> 31 ? key ^ 0x80000000u : ~key);
}

// From the groups' values, lane g's group g (a: -inf if all of it is closed),
// which are kept, as a mask; sets `close` where an open group lies nearer behind the
// border than `near` and 2^-21 of what the two were added up from (size).
template <typename F>
__device__ __forceinline__ uint32_t best_groups(const Route& R, F a, F size, int lane, F near, bool& close)
{
    int rank = 0;
#pragma unroll 8
    for (int g = 0; g < R.groups; ++g) {
        const F u = __shfl_sync(~0u, a, g);
        rank += u > a || (u == a && g < lane);
    }
    const bool mine = lane < R.groups;
    const uint32_t worst = __ballot_sync(~0u, mine && rank == R.top_groups - 1);
    const uint32_t next = __ballot_sync(~0u, mine && rank == R.top_groups);
    if (next) {
        const int p = __ffs(worst) - 1, q = __ffs(next) - 1;
        const F u = __shfl_sync(~0u, a, p), w = __shfl_sync(~0u, a, q);
        const F most = max(__shfl_sync(~0u, size, p), __shfl_sync(~0u, size, q));
        close = w != (F)-INFINITY && !(u - w >= near + (F)0x1p-21 * most);
    }
    return __ballot_sync(~0u, mine && rank < R.top_groups);
}

// Close the experts of all but the best groups: their values (-inf: closed)
// become -inf.  A lane holds VPL neighbours; where groups are whole lanes, their
// two largest values are found in registers first, else by a lane a group in
// shared memory (val).
template <int VPL>
__device__ __forceinline__ uint32_t keep_groups(const Route& R, const float (&v)[VPL], float* val, int lane, float near,
                                                bool& close)
{
    const int size = R.group_size, lanes = R.group_lanes;
    float a = -INFINITY, b = -INFINITY;
    if (lanes) {
        float x = -INFINITY, y = -INFINITY;
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
            y = fmaxf(y, fminf(x, v[i]));
            x = fmaxf(x, v[i]);
        }
#pragma unroll 4
        for (int i = 0; i < lanes; ++i) {
            const float u = __shfl_sync(~0u, x, lane * lanes + i), w = __shfl_sync(~0u, y, lane * lanes + i);
            b = fmaxf(fmaxf(b, w), fminf(a, u));
            a = fmaxf(a, u);
        }
    } else {
#pragma unroll
        for (int i = 0; i < VPL; ++i)
            if (lane * VPL + i < R.experts) val[lane * VPL + i] = v[i];
        __syncwarp();
        if (lane < R.groups)
            for (int i = 0; i < size; ++i) {
                const float u = val[lane * size + i];
                b = fmaxf(b, fminf(a, u));
                a = fmaxf(a, u);
            }
        __syncwarp();
    }
    // (a sum of open values stays above -inf, which marks a closed group: NaN stands as the lowest finite number)
    float from = fabsf(a);
    if (R.group_best == 2 && b != -INFINITY) from += fabsf(b), a = fmaxf(a + b, -3.402823466e38f);
    if (lane >= R.groups) a = -INFINITY;
    return best_groups(R, a, R.scored ? from : 0.f, lane, near, close);
}

// The largest keys of a row one after another, ties to the lower expert.  A
// lane knows its two largest and looks for another one only when it has to give
// a third, which happens about once a row.
template <int VPL>
struct Picker {
    uint32_t best = 0, second = 0;
    int at = 0, at2 = 0;
    bool two = true;               // second is the one behind best
    __device__ __forceinline__ explicit Picker(const uint32_t (&key)[VPL])
    {
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
            const bool first = key[i] > best, next = key[i] > second;
            at2 = first ? at : next ? i : at2;
            second = first ? best : next ? key[i] : second;
            at = first ? i : at;
            best = first ? key[i] : best;
        }
    }
    // the largest key that is left (0: none)
    __device__ __forceinline__ uint32_t most() const { return __reduce_max_sync(~0u, best); }
    // takes it away, and says whose it is
    __device__ __forceinline__ int take(const uint32_t (&key)[VPL], uint32_t largest, int lane)
    {
        const int owner = __ffs(__ballot_sync(~0u, best == largest)) - 1;
        const int expert = owner * VPL + __shfl_sync(~0u, at, owner);
        if (lane == owner) {
            if (two) {
                best = second, at = at2, two = false;
            } else {
                uint32_t b = 0;
                int a = 0;
#pragma unroll
                for (int i = 0; i < VPL; ++i)
                    if ((key[i] < best || (key[i] == best && i > at)) && key[i] > b) b = key[i], a = i;
                best = b, at = a;
            }
        }
        return expert;
    }
};

// An expert's score in 64 bits, sum and most being the softmax's.
__device__ __forceinline__ double score64(const Route& R, double l, double most, double sum)
{
    return R.score == CCL_SCORE_SIGMOID ? 1 / (1 + exp(-l)) : exp(l - most) / sum;
}
__device__ __noinline__ double2 softmax64(const Route& R, int64_t row, int lane)
{
    double most = -INFINITY, sum = 0;
    if (R.score != CCL_SCORE_SIGMOID) {
        for (int e = lane; e < R.experts; e += 32) most = fmax(most, (double)load_as(R.logits, row * R.ld + e, R.type));
#pragma unroll
        for (int d = 16; d; d >>= 1) most = fmax(most, __shfl_xor_sync(~0u, most, d));
#pragma unroll 2
        for (int e = lane; e < R.experts; e += 32) {
            const double l = load_as(R.logits, row * R.ld + e, R.type);
            sum += l == -INFINITY ? 0 : exp(l - most);
        }
#pragma unroll
        for (int d = 16; d; d >>= 1) sum += __shfl_xor_sync(~0u, sum, d);
    }
    return make_double2(most, sum);
}

// The order of `n` candidates, lane j's the j-th, decided in 64 bits: lane j
// gets the j-th of that order.
__device__ __noinline__ int order64(const Route& R, int64_t row, int expert, int n, int lane)
{
    const double2 s = softmax64(R, row, lane);
    double c = -INFINITY;
    if (lane < n) {
        c = score64(R, load_as(R.logits, row * R.ld + expert, R.type), s.x, s.y) + (double)R.bias[expert];
        if (c != c) c = -1.7976931348623157e308;
    }
    int rank = 0;
    for (int i = 0; i < n; ++i) {
        const double u = __shfl_sync(~0u, c, i);
        const int e = __shfl_sync(~0u, expert, i);
        rank += u > c || (u == c && e < expert);
    }
    int mine = -1;
    for (int i = 0; i < n; ++i) {
        const int r = __shfl_sync(~0u, rank, i), e = __shfl_sync(~0u, expert, i);
        if (r == lane) mine = e;
    }
    return mine;
}

// Which groups are kept, decided in 64 bits: lane g takes the largest values of
// group g and computes them again.  Says whether it could: not where the third
// value of a group may in truth be among those that the group's value is made of:
// its two largest, or the larger of them.
__device__ __noinline__ bool groups64(const Route& R, int64_t row, int lane, float most, float inv, float near, uint32_t& kept)
{
    const int size = R.group_size;
    const bool softmax = R.score != CCL_SCORE_SIGMOID;
    float a = -INFINITY, b = -INFINITY, third = -INFINITY;
    int at_a = -1, at_b = -1;
    auto near_value = [&](int e, float l) {        // (without a bias the logits are in the scores' order)
        float c = l;
        if (R.bias && l != -INFINITY) c = (softmax ? exp2_near((l - most) * 1.4426950408889634f) * inv : sigmoid(l)) + __ldg(R.bias + e);
        return c != c ? -3.402823466e38f : c;
    };
    if (lane < R.groups) {
#pragma unroll 4
        for (int i = 0; i < size; ++i) {
            const int e = lane * size + i;
            const float c = near_value(e, load_as(R.logits, row * R.ld + e, R.type));
            third = fmaxf(third, fminf(b, c));
            if (c > a)
                b = a, at_b = at_a, a = c, at_a = e;
            else if (c > b)
                b = c, at_b = e;
        }
    }
    const float last = R.group_best == 2 ? b : a, bound = fmaf(fmaxf(fabsf(last), fabsf(third)), 0x1p-22f, near);
    bool unsure = R.bias && third != -INFINITY && !(last - third >= bound);
    if (__any_sync(~0u, unsure)) {
        // one with the last one's logit and bias has its value, whichever of them is taken
        if (unsure) {
            const int of = R.group_best == 2 ? at_b : at_a;
            const float l = load_as(R.logits, row * R.ld + of, R.type), b_of = R.bias[of];
            third = -INFINITY;
            for (int e = lane * size; e < (lane + 1) * size; ++e) {
                const float u = load_as(R.logits, row * R.ld + e, R.type);
                if (e != at_a && e != at_b && !(u == l && R.bias[e] == b_of)) third = fmaxf(third, near_value(e, u));
            }
            unsure = third != -INFINITY && !(last - third >= bound);
        }
        if (__any_sync(~0u, unsure)) return false;
    }
    const double2 s = softmax64(R, row, lane);
    double v = -INFINITY;
    auto value = [&](int e) {
        const double c = score64(R, load_as(R.logits, row * R.ld + e, R.type), s.x, s.y) + (R.bias ? (double)R.bias[e] : 0.);
        return c != c ? -1.7976931348623157e308 : c;
    };
    if (at_a >= 0) {
        v = value(at_a);
        if (at_b >= 0) v = R.group_best == 2 ? fmax(v + value(at_b), -1.7976931348623157e308) : fmax(v, value(at_b));
    }
    bool close = false;
    kept = best_groups(R, v, 0., lane, 0., close);
    return true;
}

// A row's choices all in 64 bits, for values of a group or more candidates than
// lanes too near to each other (rare: a call, with the row's values in shared
// memory).
__device__ __noinline__ int choose64(const Route& R, int64_t row, double* val, int lane)
{
    const int E = R.experts;
    const double2 s = softmax64(R, row, lane);
    __syncwarp();
    for (int e = lane; e < E; e += 32) {
        const double l = load_as(R.logits, row * R.ld + e, R.type);
        double c = -INFINITY;
        if (l != -INFINITY) {
            c = score64(R, l, s.x, s.y) + (R.bias ? (double)R.bias[e] : 0.);
            if (c != c) c = -1.7976931348623157e308;
        }
        val[e] = c;
    }
    __syncwarp();
    if (R.groups > 1) {
        const int size = R.group_size;
        double a = -INFINITY, b = -INFINITY;
        if (lane < R.groups)
            for (int i = 0; i < size; ++i) {
                const double u = val[lane * size + i];
                b = fmax(b, fmin(a, u));
                a = fmax(a, u);
            }
        if (R.group_best == 2 && b != -INFINITY) a = fmax(a + b, -1.7976931348623157e308);
        bool close = false;
        const uint32_t kept = best_groups(R, a, 0., lane, 0., close);
        __syncwarp();
        for (int e = lane; e < E; e += 32) {
            if (!(kept >> e / size & 1)) {
                val[e] = -INFINITY;
            } else if (!R.bias) {          // scores order the experts as the logits do
                const double l = load_as(R.logits, row * R.ld + e, R.type);
                val[e] = l != l ? -1.7976931348623157e308 : l;
            }
        }
        __syncwarp();
    }
    int expert = -1;
    for (int j = 0; j < R.k; ++j) {
        double c = -INFINITY;
        int at = INT32_MAX;
        for (int e = lane; e < E; e += 32)
            if (val[e] > c) c = val[e], at = e;
#pragma unroll
        for (int d = 16; d; d >>= 1) {
            const double u = __shfl_xor_sync(~0u, c, d);
            const int e = __shfl_xor_sync(~0u, at, d);
            if (u > c || (u == c && e < at)) c = u, at = e;
        }
        if (c == -INFINITY) break;
        if (lane == j) expert = at;
        if (lane == (at & 31)) val[at] = -INFINITY;
        __syncwarp();
    }
    __syncwarp();
    return expert;
}

// A lane's VPL neighbours of a row of n; -inf beyond it.
template <int VPL, typename E>
__device__ __forceinline__ void load_row(const typename E::Raw* p, int at, int n, bool vec, float (&l)[VPL])
{
    constexpr int W = E::kVec;
    if (VPL % W == 0 && vec) {         // (rows on 16 bytes, n a multiple of a vector)
#pragma unroll
        for (int i = 0; i < VPL; i += W) {
            if (at + i < n) {
                E::unpack(*reinterpret_cast<const uint4*>(p + at + i), l + i);
            } else {
#pragma unroll
                for (int q = 0; q < (W < VPL ? W : VPL); ++q) l[i + q] = -INFINITY;
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < VPL; ++i) l[i] = at + i < n ? E::load(p + at + i) : -INFINITY;
    }
}
template <int VPL>
__device__ __forceinline__ void load_row(const Route& R, int64_t row, int lane, float (&l)[VPL])
{
    const int at = lane * VPL;
    const int64_t o = row * R.ld;
    if (R.type == CCL_F32)
        load_row<VPL, Type<CCL_F32>>((const float*)R.logits + o, at, R.experts, R.vec, l);
    else if (R.type == CCL_BF16)
        load_row<VPL, Type<CCL_BF16>>((const uint16_t*)R.logits + o, at, R.experts, R.vec, l);
    else
        load_row<VPL, Type<CCL_F16>>((const uint16_t*)R.logits + o, at, R.experts, R.vec, l);
}

template <int VPL, typename E>
__device__ __forceinline__ void store_row(typename E::Raw* p, int at, int n, bool vec, const float (&v)[VPL])
{
    constexpr int W = E::kVec;
    if (VPL % W == 0 && vec) {
#pragma unroll
        for (int i = 0; i < VPL; i += W)
            if (at + i < n) *reinterpret_cast<uint4*>(p + at + i) = E::pack(v + i);
    } else {
#pragma unroll
        for (int i = 0; i < VPL; ++i)
            if (at + i < n) E::store(p + at + i, v[i]);
    }
}

// The choices of a row (lane j: the j-th) and their weights.  A lane holds VPL
// neighbouring experts.
//
// Which experts come first is decided as in 64 bits.  Without a bias, scores
// order the experts as the logits do, and the logits are compared.  Else (and
// for groups by the sum of two) values are computed in 32 bits with an error
// bound: two values nearer than `near` may be in the wrong order.  Where that is so
// for neighbours in the order, all that lie within `near` of the k-th are ordered
// again in 64 bits, about one row in a thousand (6 to 9 of 8190 rows of 256 experts
// with a bias); where it is so for the groups at the border, their values are, and
// where that cannot decide, or for more than 32 candidates, the whole row.
//   sigmoid, in units of 2^-22: 2^(-l log2 e) within 1 of itself, of which
//     s (1 - s) <= 1/4 reaches s; its argument within 1/4 of itself, of which
//     |l| s (1 - s) < 0.23 does; the sum 1/4 and the reciprocal 1/2 of s: less than
//     1.07 in all, twice that for two of them, so 1.125 x 2^-21;
//   softmax: the sum is off by up to 37 roundings and scales all scores alike,
//     the exponential is within 2^-22, and l - max and its product with log2 e
//     round to 2^-24 |l - max| of a score, at most 2^-24: 2^-18 of the largest
//     score, which is 1 / sum;
//   adding the bias, or two values, rounds to 2^-24 of the larger, twice.
template <int VPL>
__device__ __forceinline__ void route_row(const Route& R, int64_t row, double* val, int lane, int group, int& expert,
                                          float& weight)
{
    float l[VPL];
    load_row<VPL>(R, row, lane, l);
    const bool softmax = R.score != CCL_SCORE_SIGMOID;
    bool poison = false;
    float most = 0.f, sum = 1.f;
    if (softmax) {
        most = l[0];
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
            most = fmaxf(most, l[i]);
            poison |= l[i] != l[i];
        }
        most = warp_max(most);
        poison = __any_sync(~0u, poison);
        if (R.scored || !R.renormalize) {
            sum = 0.f;
#pragma unroll
            for (int i = 0; i < VPL; ++i) sum += l[i] == -INFINITY ? 0.f : exp2_near((l[i] - most) * 1.4426950408889634f);
            sum = warp_sum(sum);
        }
    }
    uint32_t key[VPL];
    float near = 0.f;
    bool again = false;
    {
        float v[VPL];
        if (R.scored) {
            const float inv = 1.f / sum;
            near = softmax ? inv * 0x1p-18f : 0x1.2p-21f;
            float bias[VPL];
            if (R.bias)
                load_row<VPL, Type<CCL_F32>>(R.bias, lane * VPL, R.experts, R.vec_b, bias);
#pragma unroll
            for (int i = 0; i < VPL; ++i) {
                float c = softmax ? exp2_near((l[i] - most) * 1.4426950408889634f) * inv : sigmoid(l[i]);
                if (R.bias) c += bias[i];
                v[i] = l[i] == -INFINITY || c == -INFINITY ? -INFINITY : fmaxf(c, -3.402823466e38f);
            }
        } else {
#pragma unroll
            for (int i = 0; i < VPL; ++i) v[i] = l[i] == -INFINITY ? -INFINITY : fmaxf(l[i], -3.402823466e38f);
        }
        uint32_t kept = ~0u;
        if (R.groups > 1) {
            kept = keep_groups<VPL>(R, v, (float*)val, lane, R.scored ? 2.f * near : 0.f, again);
            if (again) again = !groups64(R, row, lane, most, 1.f / sum, near, kept);
        }
#pragma unroll
        for (int i = 0; i < VPL; ++i) key[i] = v[i] == -INFINITY ? 0u : key_of(R.bias ? v[i] : l[i]);
        if (R.group_lanes) {
            if (!(kept >> group & 1)) {
#pragma unroll
                for (int i = 0; i < VPL; ++i) key[i] = 0;
            }
        } else if (R.groups > 1) {
#pragma unroll
            for (int i = 0; i < VPL; ++i)
                if (!(kept >> min((lane * VPL + i) / R.group_size, 31) & 1)) key[i] = 0;
        }
    }
    expert = -1;
    uint32_t found = 0;
    if (!again) {
        Picker<VPL> left(key);
        for (int j = 0; j < R.k; ++j) {
            const uint32_t largest = left.most();
            if (largest == 0) break;
            const int e = left.take(key, largest, lane);
            if (lane == j) expert = e, found = largest;
        }
        if (R.bias) {
            // neighbours in the order that are nearer than the bound, and not for the same logit and bias
            int n = __popc(__ballot_sync(~0u, found != 0));
            uint32_t next = left.most();
            auto unsure = [&](bool same) {
                uint32_t below = __shfl_down_sync(~0u, found, 1);
                if (lane == n - 1) below = next;
                const float own = expert < 0 ? 0.f : load_as(R.logits, row * R.ld + expert, R.type);
                const float b = expert < 0 ? 0.f : __ldg(R.bias + expert);
                const float own_below = __shfl_down_sync(~0u, own, 1), b_below = __shfl_down_sync(~0u, b, 1);
                const float x = value_of(found), y = value_of(below);
                const bool close = lane < (same ? n - 1 : n) && lane < 31 && below &&
                                   !(x - y >= fmaf(fmaxf(fabsf(x), fabsf(y)), 0x1p-22f, near));
                return __any_sync(~0u, close && (lane == n - 1 || own != own_below || b != b_below));
            };
            if (n > 0 && (unsure(false) || n == 32)) {
                // candidates: all down to the k-th value less the bound
                const float kth = value_of(__shfl_sync(~0u, found, n - 1)), to = kth - fmaf(fabsf(kth), 0x1p-22f, near);
                while (n >= R.k && next != 0 && !(value_of(next) < to)) {
                    if (n == 32) {
                        again = true;
                        break;
                    }
                    const int e = left.take(key, next, lane);
                    if (lane == n) expert = e, found = next;
                    ++n;
                    next = left.most();
                }
                if (!again && unsure(true)) expert = order64(R, row, expert, n, lane);
            }
        }
    }
    if (again) expert = choose64(R, row, val, lane);
    float own = value_of(found);       // of a number's key, without a bias, the logit itself
    if (R.bias || again || !(own > -3.402823466e38f)) own = expert < 0 ? 0.f : load_as(R.logits, row * R.ld + expert, R.type);
    if (lane >= R.k) expert = -1;
    // weights of the choices
    const bool on = expert >= 0;
    float w;
    if (!R.renormalize) {
        w = !softmax ? sigmoid32(own) : expf(own - most) / sum;       // (the sum, of exponentials within 2^-22, is within 2^-18)
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
// of shared memory, then experts.  The chain of its steps bounds it, not what it
// moves: 1024 slots of 256 experts 5.0 us, 65536 in two launches 7.4.
__device__ __forceinline__ int expert_at(const Route& R, int64_t s)
{
    const int e = R.chosen[s];
    if (e >= R.experts) {
        report(REPORT_EXPERT);
        return -1;
    }
    return e;
}
// A warp's count of the experts of 32 slots (a lane each, -1: none)
__device__ __forceinline__ void count_32(int e, int32_t* mine, int lane)
{
    const uint32_t peers = __match_any_sync(~0u, e);
    if (e >= 0 && lane == __ffs(peers) - 1) mine[e] += __popc(peers);
    __syncwarp();
}

template <bool SINGLE>
__device__ __forceinline__ void place_slots(const Route& R, int block, int64_t per_block, int32_t* at)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5, E = R.experts;
    int32_t *total = at + warps * E, *before = total + E;
    const int64_t first = block * per_block, last = min(first + per_block, R.slots);
    const int64_t each = ((last - first + warps - 1) / warps + 31) / 32 * 32;
    const int64_t from = min(first + warp * each, last), to = min(from + each, last);
    // (the first 32 slots of a warp, mostly all of them, are read once and early)
    const int own = from + lane < to ? expert_at(R, from + lane) : -1;
    for (int i = threadIdx.x; i < (warps + 2) * E; i += blockDim.x) at[i] = 0;
    __syncthreads();
    count_32(own, at + warp * E, lane);
    for (int64_t s = from + 32 + lane; s - lane < to; s += 32) count_32(s < to ? expert_at(R, s) : -1, at + warp * E, lane);
    // of every expert: slots of all blocks, of the blocks before this one
    if (SINGLE) {
        __syncthreads();
        for (int e = threadIdx.x; e < E; e += blockDim.x) {
            int all = 0;
#pragma unroll 8
            for (int w = 0; w < warps; ++w) all += at[w * E + e];
            total[e] = all;
        }
    } else {
        // four experts a thread (hist has rows of a multiple of four), several threads for them, each some of the blocks
        const int quads = (E + 3) / 4, parts = max(1, (int)blockDim.x / quads);
        for (int i = threadIdx.x; i < quads * parts; i += blockDim.x) {
            const int q = i % quads;
            int4 all = make_int4(0, 0, 0, 0), less = all;
#pragma unroll 8
            for (int b = i / quads; b < R.blocks; b += parts) {
                const int4 n = __ldcg(reinterpret_cast<const int4*>(R.hist + ((int64_t)b * quads + q) * 4));
                all.x += n.x, all.y += n.y, all.z += n.z, all.w += n.w;
                if (b < block) less.x += n.x, less.y += n.y, less.z += n.z, less.w += n.w;
            }
            const int a[4] = {all.x, all.y, all.z, all.w}, l[4] = {less.x, less.y, less.z, less.w};
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (q * 4 + j < E) {
                    atomicAdd(&total[q * 4 + j], a[j]);         // (whole numbers: any order gives the same sum)
                    atomicAdd(&before[q * 4 + j], l[j]);
                }
        }
    }
    __syncthreads();
    // a warp 32 experts: slots of the experts before them, then of each before it
    __shared__ int32_t sums[kMostRouted / 32];
    for (int e0 = warp * 32; e0 < E; e0 += warps * 32) {
        const int n = e0 + lane < E ? total[e0 + lane] : 0, all = __reduce_add_sync(~0u, n);
        if (lane == 0) sums[e0 / 32] = all;
    }
    __syncthreads();
    for (int e0 = warp * 32; e0 < E; e0 += warps * 32) {
        const int base = __reduce_add_sync(~0u, lane < e0 / 32 ? sums[lane] : 0), e = e0 + lane, n = e < E ? total[e] : 0;
        int v = n;
#pragma unroll
        for (int d = 1; d < 32; d *= 2) {
            const int u = __shfl_up_sync(~0u, v, d);
            if (lane >= d) v += u;
        }
        if (e < E) {
            int p = base + v - n;
            if (block == 0) R.offsets[e] = p;
            if (block == 0 && e == E - 1) R.offsets[E] = p + n;
            // where the slots of each of this block's warps begin
            p += before[e];
            for (int w0 = 0; w0 < warps; w0 += 8) {
                int m[8];
#pragma unroll
                for (int w = 0; w < 8; ++w) m[w] = w0 + w < warps ? at[(w0 + w) * E + e] : 0;
#pragma unroll
                for (int w = 0; w < 8; ++w) {
                    if (w0 + w < warps) at[(w0 + w) * E + e] = p;
                    p += m[w];
                }
            }
        }
    }
    __syncthreads();
    int32_t* next = at + warp * E;
    for (int64_t s = from + lane; s - lane < to; s += 32) {
        const int e = s - lane == from ? own : s < to ? expert_at(R, s) : -1;
        const uint32_t peers = __match_any_sync(~0u, e);
        const int p = e >= 0 ? next[e] + __popc(peers & ((1u << lane) - 1)) : -1;
        __syncwarp();
        if (e >= 0 && lane == __ffs(peers) - 1) next[e] += __popc(peers);
        __syncwarp();
        if (s < to) R.place[s] = p;
    }
}

// A block's counts go to its row of hist, padded with zeros to a multiple of four.
__device__ __forceinline__ void leave_counts(const Route& R, const int32_t* counts)
{
    const int width = (R.experts + 3) / 4 * 4;
    for (int e = threadIdx.x; e < width; e += blockDim.x)
        R.hist[(int64_t)blockIdx.x * width + e] = e < R.experts ? counts[e] : 0;
}

// Threads that a block of the router may have.  With 1024 of them, 64 registers
// each, the kernels spill from 3 experts a lane on: 4 to 36 bytes a thread up to 6, 88
// for 8 and 196 for 12; with 512, 148 for 32.
constexpr int route_threads(int vpl) { return vpl < 16 ? 1024 : 512; }

// A warp a row, a threadblock `per_block` consecutive rows.
//
// Instructions bound it, about 1290 a row of 256 experts with bias and groups, some
// of them spills and next to none of them rows in 64 bits, and the schedulers issue in
// 6 cycles of 10.  8190 rows choose 8 of 256 f32: by logits
// alone 9.7 us, in groups 11.7, by sigmoids with a bias 12.5, both 16, and with the
// order of the rows 22; the bytes alone would take 1.4.  A warp a row keeps scores in
// registers, so that a choice is one maximum over the warp; for one row (64
// experts, choose 6, ordered in the same launch: 4.6 us) the chain of these is all
// there is.  Where many values of a row are equal, as bf16 logits without a
// bias are, more rows are decided again in 64 bits: 23 us instead of 16 before the order.
template <int VPL>
__global__ void __launch_bounds__(route_threads(VPL)) route_kernel(const Route R)
{
    extern __shared__ __align__(16) unsigned char smem[];
    let_next_in();
    wait_for_previous();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    int32_t* hist = reinterpret_cast<int32_t*>(smem);
    double* val = reinterpret_cast<double*>(smem + (R.order == 2 ? (R.experts * 4 + 7) & ~7 : 0)) + warp * R.experts;
    if (R.order == 2) {
        for (int e = threadIdx.x; e < R.experts; e += blockDim.x) hist[e] = 0;
        __syncthreads();
    }
    const int group = R.group_lanes ? min(lane / R.group_lanes, 31) : 0;       // of this lane's experts
    const int64_t first = blockIdx.x * R.per_block, last = min(first + R.per_block, R.rows);
    for (int64_t row = first + warp; row < last; row += warps) {
        int expert;
        float weight;
        route_row<VPL>(R, row, val, lane, group, expert, weight);
        if (lane < R.k) {
            R.chosen[row * R.k + lane] = expert;
            R.weights[row * R.k + lane] = weight;
        }
        if (R.order == 2 && expert >= 0) atomicAdd(&hist[expert], 1);
    }
    if (R.order == 0) return;
    __syncthreads();
    if (R.order == 1)
        place_slots<true>(R, 0, R.slots, hist);
    else
        leave_counts(R, hist);
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
    leave_counts(R, hist);
}

template <bool SINGLE>
__global__ void __launch_bounds__(1024) place_kernel(const Route R)
{
    extern __shared__ __align__(16) unsigned char smem[];
    let_next_in();
    wait_for_previous();
    place_slots<SINGLE>(R, blockIdx.x, R.per_block, reinterpret_cast<int32_t*>(smem));
}

// The gradient of a row's logits from those of its weights, for the choices as they are:
//   softmax                 dl = p (g - sum g p)        (all experts)
//   softmax, renormalised   dl = w (g - sum g w)        (the chosen, w their weights)
//   sigmoid                 dl = g s (1 - s)            (the chosen)
//   sigmoid, renormalised   dl = w (1 - s)(g - sum g w) (the chosen)
// A warp a row.  An expert chosen twice gets the sum of both.  8191 rows of 128 bf16,
// choose 4: 5.6 us (bytes 0.7), a single wave of warps whose loads follow one another.
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
        load_row<VPL>(R, row, lane, l);
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
        const float inv = sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll
        for (int i = 0; i < VPL; ++i) l[i] *= inv;
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
        const int e = __shfl_sync(~0u, expert, j) - lane * VPL;
        const float v = __shfl_sync(~0u, part, j);
#pragma unroll
        for (int i = 0; i < VPL; ++i)
            if (e == i) d[i] += v;
    }
    if (dense) {
#pragma unroll
        for (int i = 0; i < VPL; ++i) d[i] = l[i] * (d[i] - all);
    }
    if (R.type == CCL_F32)
        store_row<VPL, Type<CCL_F32>>((float*)R.dlogits + row * R.ld_d, lane * VPL, R.experts, R.vec_d, d);
    else if (R.type == CCL_BF16)
        store_row<VPL, Type<CCL_BF16>>((uint16_t*)R.dlogits + row * R.ld_d, lane * VPL, R.experts, R.vec_d, d);
    else
        store_row<VPL, Type<CCL_F16>>((uint16_t*)R.dlogits + row * R.ld_d, lane * VPL, R.experts, R.vec_d, d);
}

}  // namespace tensor
}  // namespace ccl
