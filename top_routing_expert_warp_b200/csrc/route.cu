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
// One warp per token, VPL consecutive experts per lane.
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
// Below this logit the logistic function is e^l to the last bit and its value
// (or a ratio's) may underflow: ratios are formed from e^{l - max} there.
constexpr float kTinyScore = -600.0f;

struct RouteParams {
    const void *logits;
    const float *bias;
    int64_t T, ld;
    int32_t N, k, softmax, renorm, n_groups, topk_groups, group_top;
    float scale;
    int32_t *topk_idx;
    float *topk_w;
    double *p_part;   // [gridDim.x, N] or null
    uint32_t *status;
};

__device__ __forceinline__ double warp_sum(double v)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        v += __shfl_xor_sync(kAll, v, o);
    return v;
}

__device__ __forceinline__ float warp_sum(float v)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        v += __shfl_xor_sync(kAll, v, o);
    return v;
}

__device__ __forceinline__ float warp_max(float v)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        v = fmaxf(v, __shfl_xor_sync(kAll, v, o));
    return v;
}

// Bits that order as the values do (no NaN), all above 1: key 0 marks what
// cannot be chosen, key 1 an expert that is switched off.
__device__ __forceinline__ uint64_t order_key(double v)
{
    const uint64_t b = static_cast<uint64_t>(__double_as_longlong(v + 0.0));   // -0 as +0
    return (b >> 63) ? ~b : (b | 0x8000000000000000ull);
}

__device__ __forceinline__ uint64_t warp_key_max(uint64_t v)
{
    const uint32_t hi = __reduce_max_sync(kAll, static_cast<uint32_t>(v >> 32));
    const uint32_t lo =
        __reduce_max_sync(kAll, static_cast<uint32_t>(v >> 32) == hi ? static_cast<uint32_t>(v) : 0u);
    return (static_cast<uint64_t>(hi) << 32) | lo;
}

// The logit as it counts: NaN as -inf (reported), +inf as the largest finite.
__device__ __forceinline__ float clean_logit(float l, bool &nan)
{
    if (isnan(l)) {
        nan = true;
        return -INFINITY;
    }
    return fminf(l, FLT_MAX);
}

template <bool BF16>
__device__ __forceinline__ float load_logit(const void *row, int e)
{
    if (BF16)
        return __bfloat162float(static_cast<const __nv_bfloat16 *>(row)[e]);
    return static_cast<const float *>(row)[e];
}

template <int VPL, bool BF16>
__global__ void __launch_bounds__(kThreads) route_kernel(RouteParams p)
{
    grid_dep_wait();
    __shared__ double s_val[kWarps][32 * VPL];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int N = p.N, k = p.k;
    const int e0 = lane * VPL;
    const bool nodes = p.n_groups > 1;
    const int per = nodes ? N / p.n_groups : N;

    bool bad = false;
    float b[VPL];
    double acc[VPL];
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
        b[i] = (p.bias && e0 + i < N) ? p.bias[e0 + i] : 0.0f;
        if (isnan(b[i])) {
            bad = true;
            b[i] = -INFINITY;
        }
        acc[i] = 0.0;
    }
    const int64_t esz = BF16 ? 2 : 4;
    const int64_t nwarps = static_cast<int64_t>(gridDim.x) * kWarps;
    for (int64_t t = static_cast<int64_t>(blockIdx.x) * kWarps + warp; t < p.T; t += nwarps) {
        const void *row = static_cast<const uint8_t *>(p.logits) + t * p.ld * esz;
        float l[VPL];
        float mx = -INFINITY;
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
            l[i] = e0 + i < N ? clean_logit(load_logit<BF16>(row, e0 + i), bad) : -INFINITY;
            mx = fmaxf(mx, l[i]);
        }
        mx = warp_max(mx);
        double s[VPL], z = 0.0;
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
            const double li = l[i];
            if (l[i] == -INFINITY)
                s[i] = 0.0;
            else
                s[i] = p.softmax ? exp(li - static_cast<double>(mx)) : 1.0 / (1.0 + exp(-li));
            z += s[i];
        }
        z = warp_sum(z);
        double q[VPL];           // s up to a factor that cancels in s / sum s
#pragma unroll
        for (int i = 0; i < VPL; ++i)
            q[i] = s[i];
        if (!p.softmax && mx < kTinyScore && mx != -INFINITY) {
            z = 0.0;
#pragma unroll
            for (int i = 0; i < VPL; ++i) {
                q[i] = exp(static_cast<double>(l[i]) - static_cast<double>(mx));
                z += q[i];
            }
            z = warp_sum(z);
        }
        const double rz = z > 0.0 ? 1.0 / z : 0.0;
        uint64_t key[VPL];
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
            const double sn = q[i] * rz;
            acc[i] += sn;
            if (p.softmax)
                s[i] = sn;
            const bool off = l[i] == -INFINITY || b[i] == -INFINITY;
            const double v = s[i] + static_cast<double>(b[i]);
            if (nodes)
                s_val[warp][e0 + i] = off ? -INFINITY : v;
            key[i] = e0 + i >= N ? 0ull
                                 : (off ? 1ull : order_key(p.bias ? v : static_cast<double>(l[i])));
        }
        if (nodes) {
            // lane g sums the group_top largest values of node g, largest first
            __syncwarp();
            uint64_t gkey = 0;
            if (lane < p.n_groups) {
                double sum = 0.0, last = INFINITY;
                int taken_at_last = 0;      // how many equal to `last` have been taken
                for (int r = 0; r < p.group_top; ++r) {
                    double best = -INFINITY;
                    int equal = 0;
                    for (int i = 0; i < per; ++i) {
                        const double v = s_val[warp][lane * per + i];
                        if (v == last)
                            ++equal;
                        else if (v < last && v > best)
                            best = v;
                    }
                    if (r > 0 && equal > taken_at_last) {
                        best = last;
                        ++taken_at_last;
                    } else if (r == 0 && equal > 0) {      // values of +inf
                        best = last;
                        taken_at_last = 1;
                    } else {
                        last = best;
                        taken_at_last = 1;
                    }
                    if (best == -INFINITY)
                        break;
                    sum += best;
                }
                gkey = order_key(sum);
            }
            uint32_t chosen = 0;
            for (int r = 0; r < p.topk_groups; ++r) {
                const uint64_t m = warp_key_max(gkey);
                const int g = __ffs(__ballot_sync(kAll, gkey == m)) - 1;
                chosen |= 1u << g;
                if (lane == g)
                    gkey = 0;
            }
#pragma unroll
            for (int i = 0; i < VPL; ++i)
                if (e0 + i < N && !((chosen >> ((e0 + i) / per)) & 1u))
                    key[i] = 0;
            __syncwarp();
        }
        int mine = 0;
        for (int j = 0; j < k; ++j) {
            uint64_t best = 0;
            int bi = 0;
#pragma unroll
            for (int i = 0; i < VPL; ++i)
                if (key[i] > best) {
                    best = key[i];
                    bi = i;
                }
            const uint64_t m = warp_key_max(best);
            const int src = __ffs(__ballot_sync(kAll, best == m)) - 1;
            const int e = __shfl_sync(kAll, e0 + bi, src);
            if (lane == src) {
#pragma unroll
                for (int i = 0; i < VPL; ++i)
                    if (i == bi)
                        key[i] = 0;
            }
            if (lane == j)
                mine = e;
        }
        // weights: lane j has expert e_j; renormalised ones up to a common factor
        bool ignore = false;
        const float le =
            lane < k ? clean_logit(load_logit<BF16>(row, mine), ignore) : -INFINITY;
        const float mc = p.renorm ? warp_max(le) : mx;
        double w = 0.0;
        if (le != -INFINITY) {
            if (p.softmax)
                w = exp(static_cast<double>(le) - static_cast<double>(mc)) * (p.renorm ? 1.0 : rz);
            else if (p.renorm && mc < kTinyScore)
                w = exp(static_cast<double>(le) - static_cast<double>(mc));
            else
                w = 1.0 / (1.0 + exp(-static_cast<double>(le)));
        }
        if (p.renorm) {
            const double d = warp_sum(w);
            w = d > 0.0 ? w / d : 0.0;
        }
        if (lane < k) {
            p.topk_idx[t * k + lane] = mine;
            p.topk_w[t * k + lane] = static_cast<float>(w * static_cast<double>(p.scale));
        }
    }
    if (bad)
        set_status(p.status, DEV_NAN_LOGIT);
    if (p.p_part) {
        // the block's sums, warp by warp in order
        __syncthreads();
#pragma unroll
        for (int i = 0; i < VPL; ++i)
            s_val[warp][e0 + i] = acc[i];
        __syncthreads();
        for (int e = threadIdx.x; e < N; e += kThreads) {
            double sum = 0.0;
            for (int w = 0; w < kWarps; ++w)
                sum += s_val[w][e];
            p.p_part[static_cast<int64_t>(blockIdx.x) * N + e] = sum;
        }
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

// With c = dp_mean / T, q = s / sum s, g = scale * dtopk_w, and over the
// chosen slots r = s / sum s (renormalised):
//   sigmoid: dl_e = (1 - s_e) * (q_e (c_e - sum c q) + [e chosen] u_e),
//            u = r (g - sum g r) renormalised, else s g
//   softmax: dl_e = p_e (c_e - sum c p) + [e chosen] u_e (- p_e sum g p),
//            u = r (g - sum g r) renormalised, else p g (and the last term)
// The sigmoid's ratios are formed from e^{l - m} / (1 + e^l) with m the
// smaller of 0 and the largest logit, so they neither under- nor overflow.
template <int VPL, bool BF16>
__global__ void __launch_bounds__(kThreads) route_grad_kernel(RouteGradParams p)
{
    grid_dep_wait();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int N = p.N, k = p.k;
    const int e0 = lane * VPL;
    const float inv_t = 1.0f / static_cast<float>(p.T);
    float c[VPL];
#pragma unroll
    for (int i = 0; i < VPL; ++i)
        c[i] = (p.dp_mean && e0 + i < N) ? p.dp_mean[e0 + i] * inv_t : 0.0f;
    const int64_t esz = BF16 ? 2 : 4;
    const int64_t nwarps = static_cast<int64_t>(gridDim.x) * kWarps;
    bool bad = false, nan = false;
    for (int64_t t = static_cast<int64_t>(blockIdx.x) * kWarps + warp; t < p.T; t += nwarps) {
        const void *row = static_cast<const uint8_t *>(p.logits) + t * p.ld * esz;
        void *out = static_cast<uint8_t *>(p.dlogits) + t * p.ld * esz;
        // chosen slots, one per lane
        int me = -1;
        float lc = -INFINITY, g = 0.0f;
        if (lane < k && p.dtopk_w) {
            me = p.topk_idx[t * k + lane];
            if (me < 0 || me >= N) {
                bad = true;
                me = -1;
            } else {
                lc = clean_logit(load_logit<BF16>(row, me), nan);
                g = p.scale * p.dtopk_w[t * k + lane];
            }
        }
        float l[VPL], mx = -INFINITY;
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
            l[i] = e0 + i < N ? clean_logit(load_logit<BF16>(row, e0 + i), nan) : -INFINITY;
            mx = fmaxf(mx, l[i]);
        }
        mx = warp_max(mx);
        const float m = p.softmax ? mx : fminf(mx, 0.0f);
        // s up to the factor that cancels in q
        float s[VPL], z = 0.0f, cz = 0.0f;
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
            if (l[i] == -INFINITY)
                s[i] = 0.0f;
            else if (p.softmax)
                s[i] = expf(l[i] - m);
            else
                s[i] = l[i] > 0.0f ? 1.0f / (1.0f + expf(-l[i]))
                                   : expf(l[i] - m) / (1.0f + expf(l[i]));
            z += s[i];
            cz = fmaf(c[i], s[i], cz);
        }
        z = warp_sum(z);
        cz = warp_sum(cz);
        const float rz = z > 0.0f ? 1.0f / z : 0.0f;
        const float cq = cz * rz;
        // chosen: u, and for plain softmax sum g p
        const float mc = warp_max(lc);
        float sc = 0.0f, om = 0.0f;     // score (up to a factor when renormalised), 1 - s
        if (lc != -INFINITY) {
            const float shift = p.renorm ? (p.softmax ? mc : fminf(mc, 0.0f)) : (p.softmax ? mx : 0.0f);
            if (p.softmax) {
                sc = expf(lc - shift) * (p.renorm ? 1.0f : rz);
            } else {
                sc = lc > 0.0f ? 1.0f / (1.0f + expf(-lc)) : expf(lc - shift) / (1.0f + expf(lc));
                om = 1.0f / (1.0f + expf(lc));
            }
        }
        float u, gp = 0.0f;
        if (p.renorm) {
            const float d = warp_sum(sc);
            const float r = d > 0.0f ? sc / d : 0.0f;
            u = r * (g - warp_sum(r * g));
        } else {
            u = sc * g;
            if (p.softmax)
                gp = warp_sum(u);
        }
        if (!p.softmax)
            u *= om;
        // base gradient of every expert
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
            if (e0 + i >= N)
                continue;
            float d = s[i] * rz * (c[i] - cq - gp);
            if (!p.softmax && l[i] != -INFINITY)
                d *= 1.0f / (1.0f + expf(l[i]));
            store_logit<BF16>(out, e0 + i, l[i] == -INFINITY ? 0.0f : d);
        }
        // the chosen experts again, with their slots' share
        float us = 0.0f;
        for (int j = 0; j < k; ++j) {
            const int ej = __shfl_sync(kAll, me, j);
            const float uj = __shfl_sync(kAll, u, j);
            if (ej == me)
                us += uj;
        }
        __syncwarp();
        if (me >= 0) {
            float sb = 0.0f;
            if (lc != -INFINITY)
                sb = p.softmax ? expf(lc - m)
                               : (lc > 0.0f ? 1.0f / (1.0f + expf(-lc)) : expf(lc - m) / (1.0f + expf(lc)));
            const float cm = p.dp_mean ? p.dp_mean[me] * inv_t : 0.0f;
            float d = sb * rz * (cm - cq - gp);
            if (!p.softmax)
                d *= om;
            store_logit<BF16>(out, me, lc == -INFINITY ? 0.0f : d + us);
        }
        __syncwarp();
    }
    if (bad)
        set_status(p.status, DEV_BAD_EXPERT);
    if (nan)
        set_status(p.status, DEV_NAN_LOGIT);
}

int route_grid(int64_t T)
{
    int sms = 148, dev = 0;
    if (cudaGetDevice(&dev) == cudaSuccess)
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    int64_t g = (T + kWarps - 1) / kWarps;
    int64_t cap = static_cast<int64_t>(sms) * 4;
    if (cap > kRouteMaxBlocks)
        cap = kRouteMaxBlocks;
    return static_cast<int>(g < cap ? g : cap);
}

// Calls f with the kernel variant's values per lane as a constant.
template <typename F>
void with_vpl(int N, F f)
{
    if (N <= 32)
        f(std::integral_constant<int, 1>());
    else if (N <= 64)
        f(std::integral_constant<int, 2>());
    else if (N <= 128)
        f(std::integral_constant<int, 4>());
    else
        f(std::integral_constant<int, 8>());
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
    p.p_part = L.p_mean ? L.p_part : nullptr;
    p.status = L.status;
    const int grid = route_grid(L.T);
    with_vpl(L.N, [&](auto v) {
        constexpr int VPL = decltype(v)::value;
        if (L.dtype == MOE_BF16)
            launch_k(route_kernel<VPL, true>, grid, kThreads, 0, stream, p);
        else
            launch_k(route_kernel<VPL, false>, grid, kThreads, 0, stream, p);
    });
    count_launches(1);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || !L.p_mean)
        return e;
    return launch_p_finalize(L.p_part, grid, L.N, L.T, L.p_mean, stream);
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
    const int grid = route_grid(L.T);
    with_vpl(L.N, [&](auto v) {
        constexpr int VPL = decltype(v)::value;
        if (L.dtype == MOE_BF16)
            launch_k(route_grad_kernel<VPL, true>, grid, kThreads, 0, stream, p);
        else
            launch_k(route_grad_kernel<VPL, false>, grid, kThreads, 0, stream, p);
    });
    count_launches(1);
    return cudaGetLastError();
}

}  // namespace moe
