// Routing of given logits to experts, and its gradient.
//
// "moe communication costs", Router design: the k largest scores select the
// experts and are the mixture coefficients; here the score is a softmax over
// the N logits or the logistic function of each logit, a balancing bias may
// take part in the choice (not in the weights), and the choice may be limited
// to a few nodes ("MoE: what it costs to train and serve", Limit how many
// machines a token touches).
//
//   s = softmax(l) or 1 / (1 + e^-l);  v = s + b, or l itself without a bias
//   e_1 .. e_k = the k largest v (of the chosen nodes), ties to the lower index
//   w_j = scale * s_{e_j} (/ sum_j s_{e_j});   p_e = mean_t s_e / sum_e s_e
//
#include <cfloat>
#include <cmath>

#include "common.cuh"
#include "kernels.h"
#include "moe.h"

namespace moe {

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr unsigned kAll = 0xffffffffu;
// Below this logit the logistic function is e^l to the last bit in 32 bits and
// its value may underflow: ratios are formed from e^{l - max} there.
constexpr float kTinyScore = -60.0f;

struct RouteParams {
    const void *logits;
    const float *bias;
    int64_t T, ld;
    int32_t N, k, softmax, renorm, n_groups, topk_groups, group_top;
    int32_t vec;             // rows start on a lane's vector boundary
    int32_t node_lanes;      // lanes that hold a node's values
    int32_t node_direct;     // 1: in the order they are loaded in (else regathered)
    int32_t per_node;
    int32_t want_p;
    float scale;
    int32_t *topk_idx;
    float *topk_w;
    double *p_part;   // [gridDim.x, N] or null
    float *p_mean;    // written by a launch of one block, or null
    uint32_t *status;
};

template <typename T>
__device__ __forceinline__ T warp_sum(T v)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        v += __shfl_xor_sync(kAll, v, o);
    return v;
}

// Over lanes 0-7 (the slots); the other lanes get sums of their own.
__device__ __forceinline__ float slot_sum(float v)
{
#pragma unroll
    for (int o = 4; o > 0; o >>= 1)
        v += __shfl_xor_sync(kAll, v, o);
    return v;
}

__device__ __forceinline__ float slot_max(float v)
{
#pragma unroll
    for (int o = 4; o > 0; o >>= 1)
        v = fmaxf(v, __shfl_xor_sync(kAll, v, o));
    return v;
}

// Bits that order as the values do (no NaN; -0 as +0), all above 0: key 0
// marks what cannot be chosen; an expert that is switched off counts -inf.
__device__ __forceinline__ uint64_t order_key(double v)
{
    const int64_t b = __double_as_longlong(v + 0.0);
    return static_cast<uint64_t>(b ^ ((b >> 63) | static_cast<int64_t>(0x8000000000000000ull)));
}

__device__ __forceinline__ uint32_t order_key(float v)
{
    const int32_t b = __float_as_int(v + 0.0f);
    return static_cast<uint32_t>(b ^ ((b >> 31) | static_cast<int32_t>(0x80000000u)));
}

constexpr uint32_t kOffKey = 0x007FFFFFu;     // of -inf

__device__ __forceinline__ float key_value(uint32_t k)
{
    return __uint_as_float((k >> 31) ? (k & 0x7FFFFFFFu) : ~k);
}

__device__ __forceinline__ uint64_t warp_key_max(uint64_t v)
{
    const uint32_t hi = __reduce_max_sync(kAll, static_cast<uint32_t>(v >> 32));
    const uint32_t lo =
        __reduce_max_sync(kAll, static_cast<uint32_t>(v >> 32) == hi ? static_cast<uint32_t>(v) : 0u);
    return (static_cast<uint64_t>(hi) << 32) | lo;
}

__device__ __forceinline__ float warp_max(float v)
{
    return key_value(__reduce_max_sync(kAll, order_key(v)));
}

// The logit as it counts: NaN as -inf (reported), +inf as the largest finite.
__device__ __forceinline__ float clean_logit(float l, bool &nan)
{
    nan |= l != l;
    return fminf(fmaxf(l, -INFINITY), FLT_MAX);      // the maximum with a NaN is the other operand
}

template <bool BF16>
__device__ __forceinline__ float load_logit(const void *row, int e)
{
    if (BF16)
        return __bfloat162float(static_cast<const __nv_bfloat16 *>(row)[e]);
    return static_cast<const float *>(row)[e];
}

// A lane's VPL logits from e0 on, -inf behind the last expert.  vec: the row's
// first element lies on a boundary of VPL elements (at most 16 bytes).
template <int VPL, bool BF16>
__device__ __forceinline__ void load_logits(const void *row, int e0, int N, bool vec,
                                            float (&l)[VPL])
{
    constexpr int bytes = VPL * (BF16 ? 2 : 4);
    const uint8_t *at = static_cast<const uint8_t *>(row) + static_cast<int64_t>(e0) * (BF16 ? 2 : 4);
    if (VPL >= 4 && vec && e0 + VPL <= N) {
        uint32_t w[bytes >= 8 ? bytes / 4 : 2];
        if (bytes >= 16) {
#pragma unroll
            for (int i = 0; i < bytes / 16; ++i) {
                const uint4 v = reinterpret_cast<const uint4 *>(at)[i];
                w[4 * i] = v.x;
                w[4 * i + 1] = v.y;
                w[4 * i + 2] = v.z;
                w[4 * i + 3] = v.w;
            }
        } else {
            const uint2 v = *reinterpret_cast<const uint2 *>(at);
            w[0] = v.x;
            w[1] = v.y;
        }
#pragma unroll
        for (int i = 0; i < VPL; ++i)
            l[i] = BF16 ? __uint_as_float((i & 1) ? (w[i / 2] & 0xFFFF0000u) : (w[i / 2] << 16))
                        : __uint_as_float(w[BF16 ? 0 : i]);
    } else {
#pragma unroll
        for (int i = 0; i < VPL; ++i)
            l[i] = e0 + i < N ? load_logit<BF16>(row, e0 + i) : -INFINITY;
    }
}

// e^x in 64 bits within 2 ulp, for x <= 0: x = n ln 2 + r with |r| <= ln 2 / 2,
// the Taylor series of e^r to r^13 / 13! (the next term is below 2^-57), scaled
// by 2^n.  Inlined, so a lane's series run side by side; below -708: 0.
__device__ __forceinline__ double exp_64(double x)
{
    const double n = rint(x * 1.4426950408889634);
    double r = fma(n, -0.69314718055994529, x);
    r = fma(n, -2.3190468138462996e-17, r);
    double e = 1.0 / 6227020800.0;
    constexpr double f[13] = {1.0 / 479001600.0, 1.0 / 39916800.0, 1.0 / 3628800.0, 1.0 / 362880.0,
                              1.0 / 40320.0, 1.0 / 5040.0, 1.0 / 720.0, 1.0 / 120.0, 1.0 / 24.0,
                              1.0 / 6.0, 0.5, 1.0, 1.0};
#pragma unroll
    for (int i = 0; i < 13; ++i)
        e = fma(e, r, f[i]);
    const double p = __hiloint2double((static_cast<int>(fmax(n, -1022.0)) + 1023) << 20, 0);
    return x < -708.0 ? 0.0 : e * p;
}

// 1 / x in 64 bits within 2 ulp, for 1 <= x <= 2: Newton's iteration from the
// 32-bit reciprocal (each doubles the right bits).
__device__ __forceinline__ double recip_64(double x)
{
    double y = static_cast<double>(__frcp_rn(static_cast<float>(x)));
    y = fma(y, fma(-x, y, 1.0), y);
    return fma(y, fma(-x, y, 1.0), y);
}

__device__ __forceinline__ uint32_t key_max(uint32_t v) { return __reduce_max_sync(kAll, v); }
__device__ __forceinline__ uint64_t key_max(uint64_t v) { return warp_key_max(v); }

__device__ __forceinline__ float larger(float a, float b) { return fmaxf(a, b); }
__device__ __forceinline__ float smaller(float a, float b) { return fminf(a, b); }
__device__ __forceinline__ double larger(double a, double b) { return a > b ? a : b; }
__device__ __forceinline__ double smaller(double a, double b) { return a > b ? b : a; }

// Inserts v into a list of the M largest values, largest first.
template <int M, typename F>
__device__ __forceinline__ void list_insert(F (&a)[M], F v)
{
#pragma unroll
    for (int i = 0; i < M; ++i) {
        const F hi = larger(v, a[i]);
        v = smaller(v, a[i]);
        a[i] = hi;
    }
}

// Sum of the `m` (at most M) largest of the values of this lane's node, on
// every lane of the node, largest first, and the sum of their absolute values;
// -inf counts as nothing.  The lists of two halves of a node merge entry by
// entry.
template <int M, int VPL, typename F>
__device__ __forceinline__ F node_sum(const F (&v)[VPL], const F *s_node, int count, int lanes,
                                      int m, float &size)
{
    F a[M];
#pragma unroll
    for (int i = 0; i < M; ++i)
        a[i] = -INFINITY;
    if (s_node) {
        for (int i = 0; i < count; ++i)
            list_insert<M, F>(a, s_node[i * lanes]);
    } else {
#pragma unroll
        for (int i = 0; i < VPL; ++i)
            list_insert<M, F>(a, v[i]);
    }
    for (int o = 1; o < lanes; o <<= 1) {
        F b[M];
#pragma unroll
        for (int i = 0; i < M; ++i)
            b[i] = __shfl_xor_sync(kAll, a[i], o);
#pragma unroll
        for (int i = 0; i < M; ++i)
            list_insert<M, F>(a, b[i]);
    }
    F sum = 0;
    size = 0.0f;
#pragma unroll
    for (int i = 0; i < M; ++i)
        if (i < m && a[i] != -INFINITY) {
            sum += a[i];
            size += fabsf(static_cast<float>(a[i]));
        }
    return sum;
}

// Sum of the `m` largest of `per` values in shared memory, for any m: each
// pass finds the largest one below the last taken (or one more equal to it).
template <typename F>
__device__ __forceinline__ F node_sum_any(const F *v, int per, int m, float &size)
{
    size = 0.0f;
    F sum = 0, last = INFINITY;
    int taken = 0;              // of the values equal to `last`
    for (int r = 0; r < m; ++r) {
        F best = -INFINITY;
        int equal = 0;
        for (int i = 0; i < per; ++i) {
            if (v[i] == last)
                ++equal;
            else if (v[i] < last && v[i] > best)
                best = v[i];
        }
        if (equal > taken) {
            best = last;
            ++taken;
        } else {
            last = best;
            taken = 1;
        }
        if (best == -INFINITY)
            break;
        sum += best;
        size += fabsf(static_cast<float>(best));
    }
    return sum;
}

__device__ __forceinline__ float key_value_of(uint32_t k) { return key_value(k); }
__device__ __forceinline__ double key_value_of(uint64_t k)
{
    return __longlong_as_double(static_cast<long long>((k >> 63) ? (k & 0x7FFFFFFFFFFFFFFFull) : ~k));
}

// Whether a >= b are far enough apart to be ordered right.  An expert's value is
// off by at most margin / 2 times 1 + |v|; an infinity is exact, and apart from
// every other value (the bound is kept finite), but not from its like.
template <typename F>
__device__ __forceinline__ bool apart(F a, F b, F margin)
{
    const F size = smaller(larger(a < 0 ? -a : a, b < 0 ? -b : b), F(FLT_MAX));
    return a - b > margin * (F(1) + size);
}

// A key below which every value is apart from `a` (twice the bound covers a
// lower value of larger size).  Experts that are switched off lie below it,
// whatever a is: they come in the order of their indices, which needs no bound.
__device__ __forceinline__ uint32_t not_apart_key(float a, float margin)
{
    const uint32_t k = order_key(a < INFINITY ? a - 2.0f * margin * (1.0f + fabsf(a)) : a);
    return k > kOffKey ? k : kOffKey + 1;
}
__device__ __forceinline__ uint64_t not_apart_key(double, double) { return 0; }   // margin < 0

// The choice: v = s + b of this lane's experts (-inf: switched off), K the key
// type of F.  Lane j gets the j-th best expert in `mine` and its key in
// `my_key`, for the `found` best: p.k of them, or with `margin` >= 0 one more,
// and all (up to 32) that may not be apart() from the k-th.  Returns whether a
// chosen node's score is too near the first one left out, with sums off by
// node_margin times their size.
template <typename F, typename K, int VPL>
__device__ __forceinline__ bool choose(const RouteParams &p, const F (&v)[VPL],
                                       const float (&l)[VPL], F *scratch, F node_margin, F margin,
                                       int &found, int &mine, K &my_key)
{
    const int lane = threadIdx.x & 31;
    const int e0 = lane * VPL;
    const int N = p.N;
    bool near = false;
    K key[VPL];
#pragma unroll
    for (int i = 0; i < VPL; ++i)
        key[i] = e0 + i >= N ? K(0) : order_key(p.bias ? v[i] : static_cast<F>(l[i]));
    if (p.n_groups > 1) {
        const int nl = p.node_lanes, per = p.per_node;
        const bool direct = p.node_direct;
        const int g = lane / nl;
        const F *s_node = nullptr;
        int count = 0;
        if (!direct) {
#pragma unroll
            for (int i = 0; i < VPL; ++i)
                scratch[e0 + i] = v[i];
            __syncwarp();
            const int at = lane - g * nl;
            s_node = scratch + (g < p.n_groups ? g * per + at : 0);
            count = g < p.n_groups ? (per - at + nl - 1) / nl : 0;
        }
        F sum;
        float size;
        if (p.group_top > 4)
            sum = node_sum_any<F>(scratch + (g < p.n_groups ? g * per : 0),
                                  g < p.n_groups ? per : 0, p.group_top, size);
        else if (p.group_top <= 2)
            sum = node_sum<2, VPL, F>(v, s_node, count, nl, p.group_top, size);
        else
            sum = node_sum<4, VPL, F>(v, s_node, count, nl, p.group_top, size);
        K gkey = g < p.n_groups && lane == g * nl ? order_key(sum) : K(0);
        uint32_t chosen = 0;
        K m = 0;
        for (int r = 0; r < p.topk_groups; ++r) {
            m = key_max(gkey);
            const int src = __ffs(__ballot_sync(kAll, gkey == m)) - 1;
            chosen |= 1u << (src / nl);
            if (lane == src)
                gkey = 0;
        }
        if (sizeof(F) == 4) {
            size = warp_max(g < p.n_groups ? size : 0.0f);
            near = !(key_value_of(m) - key_value_of(key_max(gkey)) >
                     node_margin * (static_cast<float>(p.group_top) + 2.0f * size));
        }
        if (direct) {
            if (!((chosen >> g) & 1u)) {
#pragma unroll
                for (int i = 0; i < VPL; ++i)
                    key[i] = 0;
            }
        } else {
#pragma unroll
            for (int i = 0; i < VPL; ++i)
                if (e0 + i < N && !((chosen >> ((e0 + i) / per)) & 1u))
                    key[i] = 0;
            __syncwarp();
        }
    }
    // the best two of each lane; a lane that won twice looks again
    K best = 0, second = 0;
    int bi = 0, si = 0;
    if (p.k > 1) {
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
            const bool first = key[i] > best, other = key[i] > second;
            second = first ? best : (other ? key[i] : second);
            si = first ? bi : (other ? i : si);
            best = first ? key[i] : best;
            bi = first ? i : bi;
        }
    } else {
#pragma unroll
        for (int i = 0; i < VPL; ++i)
            if (key[i] > best) {
                best = key[i];
                bi = i;
            }
    }
    my_key = 0;
    mine = 0;
    K stop = 0;
    uint32_t gone = 0;
    for (found = 0; found < 32;) {
        const K m = key_max(best);
        if (m == 0)
            break;                   // no expert left (p.k of them there always are)
        const int src = __ffs(__ballot_sync(kAll, best == m)) - 1;
        const int e = __shfl_sync(kAll, e0 + bi, src);
        if (lane == found) {
            mine = e;
            my_key = m;
        }
        ++found;
        if (found == p.k) {
            if (margin < 0)
                break;
            stop = not_apart_key(key_value_of(m), margin);
        }
        if (m < stop)
            break;
        const bool won = lane == src;
        gone |= won ? 1u << bi : 0u;
        best = won ? second : best;
        bi = won ? si : bi;
        second = won ? K(0) : second;
        if (won && best == 0 && VPL > 1) {
#pragma unroll
            for (int i = 0; i < VPL; ++i)
                if (!((gone >> i) & 1u) && key[i] > best) {
                    best = key[i];
                    bi = i;
                }
        }
    }
    return near;
}

// Whether all experts that are not switched off have one logit and one bias, so
// that their order is that of their indices in every precision.
template <int VPL, bool BF16>
__device__ __forceinline__ bool row_tied(const RouteParams &p, const void *row)
{
    const int e0 = (threadIdx.x & 31) * VPL;
    bool ignore = false;
    float l[VPL], hi = -INFINITY, low = -INFINITY, b_hi = -INFINITY, b_low = -INFINITY;
    load_logits<VPL, BF16>(row, e0, p.N, p.vec, l);
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
        const float li = clean_logit(l[i], ignore);
        const float b = e0 + i < p.N ? fmaxf(p.bias[e0 + i], -INFINITY) : -INFINITY;
        if (li != -INFINITY && b != -INFINITY) {
            hi = fmaxf(hi, li);
            low = fmaxf(low, -li);
            b_hi = fmaxf(b_hi, b);
            b_low = fmaxf(b_low, -b);
        }
    }
    return warp_max(hi) == -warp_max(low) && warp_max(b_hi) == -warp_max(b_low);
}

// The choice in 64 bits, from the logits: the index of lane j's slot (lanes
// below k).  Taken for tokens whose 32-bit values are too near one another.
// s_val: doubles of this warp.  A token whose experts are all equal keeps its slots
// in `tied` (if not negative).
template <int VPL, bool BF16, bool SOFTMAX>
__device__ __noinline__ int choose_exact(const RouteParams &p, const void *row, double *s_val,
                                         int tied)
{
    if (__any_sync(kAll, tied >= 0) && row_tied<VPL, BF16>(p, row))
        return tied;
    const int lane = threadIdx.x & 31;
    const int e0 = lane * VPL;
    bool ignore = false;
    float l[VPL], mx = -INFINITY;
    load_logits<VPL, BF16>(row, e0, p.N, p.vec, l);
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
        l[i] = clean_logit(l[i], ignore);
        mx = fmaxf(mx, l[i]);
    }
    mx = warp_max(mx);
    // through s_val, a few experts at a time: this runs for a token in hundreds or
    // thousands, whose warp waits for its instructions as much as for its sums
    double z = 0.0;
#pragma unroll
    for (int i = 0; i < VPL; ++i)
        s_val[e0 + i] = l[i];
#pragma unroll 4
    for (int i = 0; i < VPL; ++i) {
        const double li = s_val[e0 + i];
        double si;
        if (SOFTMAX) {
            si = exp_64(li - static_cast<double>(mx));
            si = li == -INFINITY ? 0.0 : si;
            z += si;
        } else {
            const double t = exp_64(-fabs(li));
            const double r = recip_64(1.0 + t);
            si = li > 0.0 ? r : t * r;
        }
        s_val[e0 + i] = si;
    }
    if (SOFTMAX) {
        z = warp_sum(z);
        z = z > 0.0 ? 1.0 / z : 0.0;
    }
    double s[VPL];
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
        float b = (p.bias && e0 + i < p.N) ? p.bias[e0 + i] : 0.0f;
        b = fmaxf(b, -INFINITY);
        s[i] = SOFTMAX ? s_val[e0 + i] * z : s_val[e0 + i];
        s[i] = l[i] == -INFINITY || b == -INFINITY ? -INFINITY : s[i] + static_cast<double>(b);
    }
    int mine, found;
    uint64_t won;
    choose<double, uint64_t, VPL>(p, s, l, s_val, 0.0, -1.0, found, mine, won);
    return mine;
}

// The `n` experts of lanes 0 .. n - 1 in the order of their 64-bit values,
// logistic scores with a bias.
template <bool BF16>
__device__ __noinline__ int order_exact(const RouteParams &p, const void *row, int mine, int n)
{
    const int lane = threadIdx.x & 31;
    bool ignore = false;
    double v = -INFINITY;
    if (lane < n) {
        const float l = clean_logit(load_logit<BF16>(row, mine), ignore);
        const float b = fmaxf(p.bias[mine], -INFINITY);
        const double t = exp_64(-fabs(static_cast<double>(l)));
        const double r = recip_64(1.0 + t);
        if (l != -INFINITY && b != -INFINITY)
            v = (l > 0.0f ? r : t * r) + static_cast<double>(b);
    }
    int rank = 0;
    for (int j = 0; j < n; ++j) {
        const double vj = __shfl_sync(kAll, v, j);
        const int ej = __shfl_sync(kAll, mine, j);
        rank += vj > v || (vj == v && ej < mine) ? 1 : 0;
    }
    int sorted = mine;
    for (int j = 0; j < n; ++j) {
        const int rj = __shfl_sync(kAll, rank, j);
        const int ej = __shfl_sync(kAll, mine, j);
        sorted = rj == lane ? ej : sorted;
    }
    return sorted;
}

// One warp per token, VPL consecutive experts per lane.  What bounds it is not
// the bytes (4 to 7 % of the copy rate).  A prompt's batch is bound by latency:
// a token is one long chain (k rounds of a warp maximum, the exponentials, the
// sums), and 4096 tokens of 256 experts on 444 blocks of 8 warps are two for 544
// of the warps while the others wait (1500 instructions per token, issued at
// 0.47 to 0.48 per cycle, a third of the warps active).  Larger and smaller-gated batches
// come nearer to the issue rate (32771 x 128 top-1: 290 instructions, 0.66 per
// cycle).  So values are formed and compared in 32 bits, and a token whose
// decisions hang on differences near the 32-bit error is decided again in 64 (all
// in 64 bits: 44 us at 4096 x 256 with nodes and a bias, now 16, and 3 for the
// second launch that adds up p; 65536 tokens 111 and 118 us).  Without a bias and nodes the 32-bit keys are
// the logits themselves and decide exactly (32771 x 128 bf16, top-1: 15 us).
template <int VPL, bool BF16, bool SOFTMAX>
__global__ void __launch_bounds__(kThreads, VPL == 8 ? 3 : 4)
    route_kernel(const __grid_constant__ RouteParams p)
{
    grid_dep_wait();
    grid_dep_launch();
    __shared__ double s_val[kWarps][32 * VPL];   // scratch of a token's choice
    __shared__ double s_acc[kWarps][32 * VPL];   // sums of s / sum s, a lane's 32 apart
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int N = p.N, k = p.k;
    const int e0 = lane * VPL;
    const bool values = p.bias != nullptr || p.n_groups > 1;   // the choice needs s + b

    bool bad = false;
    float b[VPL];
    float part[VPL];
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
        b[i] = (p.bias && e0 + i < N) ? p.bias[e0 + i] : 0.0f;
        bad |= b[i] != b[i];
        b[i] = fmaxf(b[i], -INFINITY);
        s_acc[warp][i * 32 + lane] = 0.0;
        part[i] = 0.0f;
    }
    // Half steps of 32 bits (2^-24) that a value v = s + b may be off: a logistic
    // score s (6 (1 - s) + 3) <= 3.4 (6 of the exponential, 3 of sum and
    // reciprocal), a softmax's share 22 (its exponential, a sum of up to 256
    // terms, reciprocal and product), the addition |v|.  Two values are apart if
    // they differ by 8 (64) half steps times 1 + |v|: more than both may be off.
    // A sum of n such values is off by n times as much, and by half a step of
    // each of its partial sums: n / 2 times its size at most.
    constexpr float margin = SOFTMAX ? 0x1p-18f : 0x1p-21f;
    const float node_margin = margin * (1.0f + 0.125f * static_cast<float>(p.group_top));
    const int64_t step = static_cast<int64_t>(gridDim.x) * kWarps;
    const int64_t row_bytes = p.ld * (BF16 ? 2 : 4);
    const int64_t row_step = step * row_bytes;
    int64_t t = static_cast<int64_t>(blockIdx.x) * kWarps + warp;
    const uint8_t *row = static_cast<const uint8_t *>(p.logits) + t * row_bytes;
    int64_t slot = t * k + lane;
    int held = 0;
    float nxt[VPL];
    if (t < p.T)
        load_logits<VPL, BF16>(row, e0, N, p.vec, nxt);
    for (; t < p.T; t += step, row += row_step, slot += step * k) {
        float l[VPL];
        float mx = -INFINITY, all = 0.0f;
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
            l[i] = nxt[i];
            all += l[i];
        }
        if (__any_sync(kAll, !(all < INFINITY))) {      // a NaN or +inf among them
#pragma unroll
            for (int i = 0; i < VPL; ++i)
                l[i] = clean_logit(l[i], bad);
        }
#pragma unroll
        for (int i = 0; i < VPL; ++i)
            mx = fmaxf(mx, l[i]);
        if (t + step < p.T)
            load_logits<VPL, BF16>(row + row_step, e0, N, p.vec, nxt);
        const bool scores = SOFTMAX || p.want_p || values;
        if (scores || p.renorm)
            mx = warp_max(mx);
        const float shift = mx == -INFINITY ? 0.0f : mx;
        const bool tiny = !SOFTMAX && mx < kTinyScore;
        // s, or up to a factor: e^{l - max} for a softmax and below kTinyScore
        float s[VPL], z = 0.0f;
        float rz = 0.0f;
        if (scores) {
            if (SOFTMAX || tiny) {
#pragma unroll
                for (int i = 0; i < VPL; ++i) {
                    s[i] = exp_32(l[i] - shift);
                    z += s[i];
                }
            } else {
#pragma unroll
                for (int i = 0; i < VPL; ++i) {
                    // below -88, -inf too, the reciprocal comes out 0
                    s[i] = recip_32(1.0f + exp_32(fminf(-l[i], 88.0f)));
                    z += s[i];
                }
            }
        }
        if (SOFTMAX || p.want_p) {
            z = warp_sum(z);
            rz = z > 0.0f ? recip_32(z) : 0.0f;
#pragma unroll
            for (int i = 0; i < VPL; ++i) {
                const float q = s[i] * rz;
                part[i] += q;
                if (SOFTMAX)
                    s[i] = q;
            }
        }
        if (++held == 32) {          // 32-bit sums of 32 tokens, then 64
            held = 0;
#pragma unroll
            for (int i = 0; i < VPL; ++i) {
                s_acc[warp][i * 32 + lane] += part[i];
                part[i] = 0.0f;
            }
        }
        int mine, found;
        uint32_t won;
        float le = -INFINITY;
        if (!values) {
            // the keys are the logits: exact, and the slot's logit is its key
#pragma unroll
            for (int i = 0; i < VPL; ++i)
                s[i] = l[i];
            choose<float, uint32_t, VPL>(p, s, l, nullptr, 0.0f, -1.0f, found, mine, won);
            if (lane < k)
                le = key_value(won);
        } else {
            bool exact = tiny;
            int tied = -1;
            if (!exact) {
#pragma unroll
                for (int i = 0; i < VPL; ++i)
                    s[i] = l[i] == -INFINITY ? -INFINITY : s[i] + b[i];
                exact = choose<float, uint32_t, VPL>(p, s, l, reinterpret_cast<float *>(s_val[warp]),
                                                     node_margin, p.bias && k < N ? margin : -1.0f,
                                                     found, mine, won);
                if (p.bias && !exact) {
                    // each of the found experts against the next one
                    const uint32_t nk = __shfl_down_sync(kAll, won, 1);
                    const int ne = __shfl_down_sync(kAll, mine, 1);
                    bool close = lane + 1 < found && nk > kOffKey &&
                                 !apart(key_value(won), key_value(nk), margin);
                    if (close)
                        // equal logits with equal biases are equal in every precision
                        close = won != nk || load_logit<BF16>(row, mine) != load_logit<BF16>(row, ne) ||
                                p.bias[mine] != p.bias[ne];
                    if (__any_sync(kAll, close)) {
                        // the k best are among the found ones, unless those are 32 or
                        // the shares' sum is not known well enough
                        if (!SOFTMAX && found < 32)
                            mine = order_exact<BF16>(p, row, mine, found);
                        else
                            exact = true;
                    } else if (found == 32) {
                        // equal ones as far as was looked: what lies behind may differ
                        exact = true;
                        tied = mine;
                    }
                }
            }
            if (exact)
                mine = choose_exact<VPL, BF16, SOFTMAX>(p, row, s_val[warp], tied);
            bool ignore = false;
            if (lane < k)
                le = clean_logit(load_logit<BF16>(row, mine), ignore);
        }
        // weights: lane j has expert e_j; renormalised ones up to a common factor
        const float mc = p.renorm ? slot_max(le) : shift;
        float w;
        if (SOFTMAX || (p.renorm && mc < kTinyScore))
            w = expf(le - (mc == -INFINITY ? 0.0f : mc)) * (p.renorm ? 1.0f : rz);
        else
            w = __fdividef(1.0f, 1.0f + expf(-le));
        if (p.renorm) {
            const float d = slot_sum(w);
            w = d > 0.0f ? __fdividef(w, d) : 0.0f;
        }
        if (lane < k) {
            p.topk_idx[slot] = mine;
            p.topk_w[slot] = w * p.scale;
        }
    }
    if (bad)
        set_status(p.status, DEV_NAN_LOGIT);
    if (p.want_p) {
        // the block's sums, warp by warp in order
#pragma unroll
        for (int i = 0; i < VPL; ++i)
            s_acc[warp][i * 32 + lane] += part[i];
        __syncthreads();
        for (int e = threadIdx.x; e < N; e += kThreads) {
            double sum = 0.0;
            for (int w = 0; w < kWarps; ++w)
                sum += s_acc[w][e % VPL * 32 + e / VPL];
            if (p.p_mean)
                p.p_mean[e] = static_cast<float>(sum / static_cast<double>(p.T));
            else
                p.p_part[static_cast<int64_t>(blockIdx.x) * N + e] = sum;
        }
    }
}

// p_mean from the blocks' sums (at most kRouteMaxBlocks rows): 8 experts per
// block, every 64th row per thread with all its loads in flight, added in order;
// then the 64 threads of an expert by a warp.
constexpr int kMeanThreads = 512;
__global__ void __launch_bounds__(kMeanThreads)
    route_mean_kernel(const double *__restrict__ p_part, int rows, int N, double inv_t,
                      float *__restrict__ p_mean)
{
    grid_dep_wait();
    __shared__ double s_sum[8][65];
    constexpr int kLoads = (kRouteMaxBlocks + 63) / 64;
    const int x = threadIdx.x & 7, y = threadIdx.x >> 3;
    const int e = blockIdx.x * 8 + x;
    double v[kLoads], sum = 0.0;
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
        const int r = y + 64 * i;
        v[i] = e < N && r < rows ? p_part[static_cast<int64_t>(r) * N + e] : 0.0;
    }
#pragma unroll
    for (int i = 0; i < kLoads; ++i)
        sum += v[i];
    s_sum[x][y] = sum;
    __syncthreads();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (warp < 8) {
        sum = warp_sum(s_sum[warp][lane] + s_sum[warp][lane + 32]);
        if (lane == 0 && blockIdx.x * 8 + warp < N)
            p_mean[blockIdx.x * 8 + warp] = static_cast<float>(sum * inv_t);
    }
}

struct RouteGradParams {
    const void *logits;
    const int32_t *topk_idx;
    const float *dtopk_w;    // or null
    const float *dp_mean;    // or null
    void *dlogits;
    int64_t T, ld;
    int32_t N, k, softmax, renorm;
    int32_t vec;             // both matrices' rows start on a lane's vector boundary
    float scale;
    uint32_t *status;
};

template <bool BF16>
__device__ __forceinline__ void store_logit(void *row, int e, float v)
{
    if (BF16)
        static_cast<__nv_bfloat16 *>(row)[e] = __float2bfloat16_rn(v);
    else
        static_cast<float *>(row)[e] = v;
}

template <int VPL, bool BF16>
__device__ __forceinline__ void store_logits(void *row, int e0, int N, bool vec,
                                             const float (&d)[VPL])
{
    constexpr int bytes = VPL * (BF16 ? 2 : 4);
    uint8_t *at = static_cast<uint8_t *>(row) + static_cast<int64_t>(e0) * (BF16 ? 2 : 4);
    if (VPL >= 4 && vec && e0 + VPL <= N) {
        uint32_t w[bytes >= 8 ? bytes / 4 : 2];
#pragma unroll
        for (int i = 0; i < bytes / 4; ++i)
            w[i] = BF16 ? pack_bf16x2(d[(2 * i) % VPL], d[(2 * i + 1) % VPL]) : __float_as_uint(d[i % VPL]);
        if (bytes >= 16) {
#pragma unroll
            for (int i = 0; i < bytes / 16; ++i)
                reinterpret_cast<uint4 *>(at)[i] =
                    make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
        } else {
            *reinterpret_cast<uint2 *>(at) = make_uint2(w[0], w[1]);
        }
    } else {
#pragma unroll
        for (int i = 0; i < VPL; ++i)
            if (e0 + i < N)
                store_logit<BF16>(row, e0 + i, d[i]);
    }
}

// s and 1 - s of the logistic function, both without cancellation.
__device__ __forceinline__ void logistic(float l, float &s, float &om)
{
    const float t = exp_32(-fabsf(l));
    const float r = recip_32(1.0f + t);
    const float tr = t * r;
    s = l > 0.0f ? r : tr;
    om = l > 0.0f ? tr : r;
}

// The same for every expert of a row: below -88 both come out 0, as does what
// they are multiplied into.
__device__ __forceinline__ void logistic_pair(float l, float &s, float &om)
{
    const float t = exp_32(fminf(-l, 88.0f));
    s = recip_32(1.0f + t);
    om = t * s;
}

// With c = dp_mean / T, q = s / sum s, g = scale * dtopk_w, and over the
// chosen slots r = s / sum s (renormalised):
//   sigmoid: dl_e = (1 - s_e) * (q_e (c_e - sum c q) + [e chosen] u_e),
//            u = r (g - sum g r) renormalised, else s g
//   softmax: dl_e = p_e (c_e - sum c p) + [e chosen] u_e (- p_e sum g p),
//            u = r (g - sum g r) renormalised, else p g (and the last term)
// Ratios of scores below kTinyScore are formed from e^{l - max}, so they do
// not underflow.  One warp per token: the logits are read once and the
// gradient is written once (2 T N values, the bound by bytes), the k chosen
// experts' gradients a second time by the lanes that hold the slots.  65536 x
// 256 fp32 in 36 us, 60 % of a plain copy's rate; bound by issue (0.71 per cycle,
// some 400 instructions per token).
template <int VPL, bool BF16, bool SOFTMAX>
__global__ void __launch_bounds__(kThreads, 4)
    route_grad_kernel(const __grid_constant__ RouteGradParams p)
{
    grid_dep_wait();
    grid_dep_launch();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int N = p.N, k = p.k;
    const int e0 = lane * VPL;
    const float inv_t = 1.0f / static_cast<float>(p.T);
    float c[VPL];
#pragma unroll
    for (int i = 0; i < VPL; ++i)
        c[i] = (p.dp_mean && e0 + i < N) ? p.dp_mean[e0 + i] * inv_t : 0.0f;
    bool bad = false, nan = false;
    const int64_t step = static_cast<int64_t>(gridDim.x) * kWarps;
    const int64_t row_bytes = p.ld * (BF16 ? 2 : 4);
    const int64_t row_step = step * row_bytes;
    int64_t t = static_cast<int64_t>(blockIdx.x) * kWarps + warp;
    const uint8_t *row = static_cast<const uint8_t *>(p.logits) + t * row_bytes;
    uint8_t *out = static_cast<uint8_t *>(p.dlogits) + t * row_bytes;
    const int64_t slot_step = step * k;
    int64_t slot = t * k + lane;
    const bool slots = p.dtopk_w != nullptr && lane < k;
    float nxt[VPL];
    int nme = -1;
    float ng = 0.0f;
    if (t < p.T) {
        load_logits<VPL, BF16>(row, e0, N, p.vec, nxt);
        if (slots) {
            nme = p.topk_idx[slot];
            ng = p.dtopk_w[slot];
        }
    }
    for (; t < p.T; t += step, row += row_step, out += row_step) {
        // chosen slots, one per lane
        int me = nme;
        float lc = -INFINITY, cm = 0.0f;
        const float g = p.scale * ng;
        if (slots) {
            if (static_cast<uint32_t>(me) >= static_cast<uint32_t>(N)) {
                bad = true;
                me = -1;
            } else {
                lc = clean_logit(load_logit<BF16>(row, me), nan);
                if (p.dp_mean)
                    cm = p.dp_mean[me] * inv_t;
            }
        }
        float l[VPL], mx = -INFINITY, all = 0.0f;
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
            l[i] = nxt[i];
            all += l[i];
        }
        if (__any_sync(kAll, !(all < INFINITY))) {      // a NaN or +inf among them
#pragma unroll
            for (int i = 0; i < VPL; ++i)
                l[i] = clean_logit(l[i], nan);
        }
#pragma unroll
        for (int i = 0; i < VPL; ++i)
            mx = fmaxf(mx, l[i]);
        slot += slot_step;
        if (t + step < p.T) {
            load_logits<VPL, BF16>(row + row_step, e0, N, p.vec, nxt);
            if (slots) {
                nme = p.topk_idx[slot];
                ng = p.dtopk_w[slot];
            }
        }
        mx = warp_max(mx);
        // the shift of the exponentials: none for the logistic function unless it is tiny
        const bool tiny = !SOFTMAX && mx < kTinyScore;
        const float shift = mx == -INFINITY ? 0.0f : mx;
        float s[VPL], om[VPL], z = 0.0f, cz = 0.0f;
        if (SOFTMAX || tiny) {
#pragma unroll
            for (int i = 0; i < VPL; ++i) {
                om[i] = 1.0f;
                s[i] = exp_32(l[i] - shift);
            }
        } else {
#pragma unroll
            for (int i = 0; i < VPL; ++i)
                logistic_pair(l[i], s[i], om[i]);
        }
        float rz = 0.0f;
        if (SOFTMAX || p.dp_mean) {
#pragma unroll
            for (int i = 0; i < VPL; ++i) {
                z += s[i];
                cz = fmaf(c[i], s[i], cz);
            }
            z = warp_sum(z);
            cz = warp_sum(cz);
            rz = z > 0.0f ? __fdividef(1.0f, z) : 0.0f;
        }
        const float cq = cz * rz;
        // chosen: score (up to a factor when renormalised), 1 - s, share of the row's sum
        float sc, oc, share;
        if (SOFTMAX) {
            oc = 1.0f;
            share = expf(lc - shift) * rz;
            sc = share;
        } else {
            logistic(lc, sc, oc);
            share = (tiny ? expf(lc - shift) : sc) * rz;
        }
        float u, gp = 0.0f;
        if (p.renorm) {
            const float mc = slot_max(lc);
            if (SOFTMAX || mc < kTinyScore)
                sc = expf(lc - (mc == -INFINITY ? 0.0f : mc));
            const float d = slot_sum(sc);
            const float r = d > 0.0f ? __fdividef(sc, d) : 0.0f;
            u = r * (g - slot_sum(r * g));
        } else {
            u = sc * g;
            if (SOFTMAX)
                gp = __shfl_sync(kAll, slot_sum(u), 0);
        }
        // the same expert in several slots adds up
        const unsigned twins = __match_any_sync(kAll, me >= 0 ? me : -1 - lane);
        if (__any_sync(kAll, (twins & (twins - 1)) != 0u)) {
            float us = 0.0f;
            for (int j = 0; j < k; ++j) {
                const float uj = __shfl_sync(kAll, u, j);
                us += (twins >> j) & 1u ? uj : 0.0f;
            }
            u = us;
        }
        // every expert without its slots' share, then the chosen ones with it
        const float sub = cq + gp;
        float d[VPL];
#pragma unroll
        for (int i = 0; i < VPL; ++i)
            d[i] = s[i] * rz * (c[i] - sub) * om[i];
        store_logits<VPL, BF16>(out, e0, N, p.vec, d);
        __syncwarp();
        if (me >= 0)
            store_logit<BF16>(out, me, lc == -INFINITY ? 0.0f : oc * (share * (cm - sub) + u));
    }
    if (bad)
        set_status(p.status, DEV_BAD_EXPERT);
    if (nan)
        set_status(p.status, DEV_NAN_LOGIT);
}

// As many blocks as there is work for, at most those that run at once.
int route_grid(int64_t T, int per_sm)
{
    int sms = 148, dev = 0;
    if (cudaGetDevice(&dev) == cudaSuccess)
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    int64_t g = (T + kWarps - 1) / kWarps;
    int64_t cap = static_cast<int64_t>(sms) * per_sm;
    if (cap > kRouteMaxBlocks)
        cap = kRouteMaxBlocks;
    return static_cast<int>(g < cap ? g : cap);
}

// Whether every row of [T, ld] logits starts on a boundary of 16 bytes.
bool rows_on_16(const void *base, int64_t ld, int dtype)
{
    const int64_t es = dtype == MOE_BF16 ? 2 : 4;
    return reinterpret_cast<uintptr_t>(base) % 16 == 0 && (ld * es) % 16 == 0;
}

int lane_values(int N) { return N <= 32 ? 1 : (N <= 64 ? 2 : (N <= 128 ? 4 : 8)); }

// Calls f with the kernel variant's values per lane as a constant.
template <typename F>
void with_vpl(int N, F f)
{
    switch (lane_values(N)) {
    case 1: f(std::integral_constant<int, 1>()); break;
    case 2: f(std::integral_constant<int, 2>()); break;
    case 4: f(std::integral_constant<int, 4>()); break;
    default: f(std::integral_constant<int, 8>()); break;
    }
}

}  // namespace

cudaError_t launch_route(const RouteLaunch &L, cudaStream_t stream)
{
    RouteParams p;
    p.logits = L.logits;
    p.bias = L.bias;
    p.T = L.T;
    p.ld = L.ld;
    p.N = L.N;
    p.k = L.k;
    p.softmax = L.score == MOE_SCORE_SOFTMAX;
    p.renorm = L.renormalize;
    p.n_groups = L.n_groups;
    p.topk_groups = L.topk_groups;
    p.group_top = L.group_top;
    p.scale = L.scale;
    p.topk_idx = L.topk_idx;
    p.topk_w = L.topk_w;
    p.status = L.status;
    p.vec = rows_on_16(L.logits, L.ld, L.dtype);
    p.node_lanes = 1;
    p.node_direct = 0;
    if (L.n_groups > 1) {
        // a node's values lie on whole lanes, a power of two of them, or are
        // gathered onto 32 / n_groups lanes
        const int v = lane_values(L.N), per = L.N / L.n_groups;
        p.per_node = per;
        const int lanes = per / v;
        if (per % v == 0 && (lanes & (lanes - 1)) == 0 && L.group_top <= 4) {
            p.node_lanes = lanes;
            p.node_direct = 1;
        } else {
            int lg = 32;
            while (lg * L.n_groups > 32)
                lg >>= 1;
            p.node_lanes = lg;
        }
    }
    const int grid = route_grid(L.T, lane_values(L.N) == 8 ? 3 : 4);
    p.want_p = L.p_mean != nullptr;
    // one block writes its sums as the result
    p.p_mean = grid == 1 ? L.p_mean : nullptr;
    p.p_part = L.p_mean && grid > 1 ? L.p_part : nullptr;
    with_vpl(L.N, [&](auto v) {
        constexpr int VPL = decltype(v)::value;
        auto kernel = L.dtype == MOE_BF16
                          ? (p.softmax ? route_kernel<VPL, true, true> : route_kernel<VPL, true, false>)
                          : (p.softmax ? route_kernel<VPL, false, true> : route_kernel<VPL, false, false>);
        launch_k(kernel, grid, kThreads, 0, stream, p);
    });
    count_launches(1);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || !p.p_part)
        return e;
    launch_k(route_mean_kernel, dim3((L.N + 7) / 8), dim3(kMeanThreads), 0, stream, L.p_part, grid,
             L.N, 1.0 / static_cast<double>(L.T), L.p_mean);
    count_launches(1);
    return cudaGetLastError();
}

cudaError_t launch_route_grad(const RouteGradLaunch &L, cudaStream_t stream)
{
    RouteGradParams p;
    p.logits = L.logits;
    p.topk_idx = L.topk_idx;
    p.dtopk_w = L.dtopk_w;
    p.dp_mean = L.dp_mean;
    p.dlogits = L.dlogits;
    p.T = L.T;
    p.ld = L.ld;
    p.N = L.N;
    p.k = L.k;
    p.softmax = L.score == MOE_SCORE_SOFTMAX;
    p.renorm = L.renormalize;
    p.scale = L.scale;
    p.status = L.status;
    p.vec = rows_on_16(L.logits, L.ld, L.dtype) && rows_on_16(L.dlogits, L.ld, L.dtype);
    const int grid = route_grid(L.T, 4);
    with_vpl(L.N, [&](auto v) {
        constexpr int VPL = decltype(v)::value;
        auto kernel = L.dtype == MOE_BF16
                          ? (p.softmax ? route_grad_kernel<VPL, true, true> : route_grad_kernel<VPL, true, false>)
                          : (p.softmax ? route_grad_kernel<VPL, false, true> : route_grad_kernel<VPL, false, false>);
        launch_k(kernel, grid, kThreads, 0, stream, p);
    });
    count_launches(1);
    return cudaGetLastError();
}

}  // namespace moe
