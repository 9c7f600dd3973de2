// Gradient of the combine (combine.cu).
//
//   y[t] = sum over kept slots j of w[t, j] * y_perm[r(t, j)]
//   dy_perm[r(t, j)] = w[t, j] * dy[t],   dw[t, j] = <dy[t], y_perm[r(t, j)]>
//
// Each lane reads its chunks of dy[t] once and uses them for every slot; the
// loads of all slots of a pass are issued before any is used.  fp32 products
// and sums, the order of a sum fixed by the thread count.  Bound by bytes: dy
// and the kept rows of y_perm read once, those of dy_perm written once (bf16,
// 4096 tokens x 4096, top-2: 30 us, 85 % of a plain copy's rate; 4099 x 2048,
// top-8: 47 us, 93 %; a block per token with its barriers took 45 and 64 us).
#include "common.cuh"
#include "kernels.h"
#include "moe.h"

namespace moe {

namespace {

constexpr int kThreads = 256;
constexpr int kMaxK = 8;

template <bool BF16, int V>
__device__ __forceinline__ void unpack(const uint4 q, float (&v)[V])
{
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (BF16) {
            v[2 * i] = __uint_as_float(w[i] << 16);
            v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
        } else {
            v[i] = __uint_as_float(w[i]);
        }
    }
}

// KM: bound on k.  TPT threads per token: a warp, or the block for batches too
// small to fill the GPU with warps.  DW, DY: which outputs are wanted.
template <bool BF16, int KM, int TPT, bool DW, bool DY>
__global__ void __launch_bounds__(kThreads)
    combine_grad_kernel(const uint8_t *__restrict__ dy, const uint8_t *y_perm,
                        const int32_t *__restrict__ inv_row, const float *__restrict__ topk_w,
                        uint8_t *dy_perm, float *__restrict__ dtopk_w, int64_t T, int d, int k,
                        int64_t rows_cap, uint32_t *status)
{
    grid_dep_wait();
    __shared__ float s_dot[kThreads / 32][KM];
    constexpr int V = BF16 ? 8 : 4;
    constexpr int esz = BF16 ? 2 : 4;
    constexpr int U = KM <= 2 ? 4 : (KM <= 4 ? 2 : 1);   // chunks per thread and pass
    constexpr int TPB = kThreads / TPT;                  // tokens per block
    const int chunks = d / V;
    const int64_t row_bytes = static_cast<int64_t>(d) * esz;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int me = threadIdx.x % TPT;
    for (int64_t t = static_cast<int64_t>(blockIdx.x) * TPB + threadIdx.x / TPT; t < T;
         t += static_cast<int64_t>(gridDim.x) * TPB) {
        int32_t my_row = -1;
        float my_w = 0.0f;
        if (lane < k) {
            my_row = inv_row[t * k + lane];
            if (DY)
                my_w = topk_w[t * k + lane];
            if (my_row >= rows_cap || my_row < -1) {
                set_status(status, DEV_BAD_ROW);
                my_row = -1;
            }
        }
        int32_t row[KM];
        float w[KM], dot[KM];
#pragma unroll
        for (int j = 0; j < KM; ++j) {
            row[j] = __shfl_sync(0xffffffffu, my_row, j);
            w[j] = __shfl_sync(0xffffffffu, my_w, j);
            dot[j] = 0.0f;
        }
        const uint4 *src = reinterpret_cast<const uint4 *>(dy + t * row_bytes);
        for (int c0 = me; c0 < chunks; c0 += TPT * U) {
            uint4 a[U], y[DW ? KM : 1][U];
#pragma unroll
            for (int u = 0; u < U; ++u)
                a[u] = c0 + TPT * u < chunks ? __ldg(src + c0 + TPT * u) : make_uint4(0, 0, 0, 0);
            if (DW) {
#pragma unroll
                for (int j = 0; j < KM; ++j)
#pragma unroll
                    for (int u = 0; u < U; ++u)
                        y[DW ? j : 0][u] =
                            (row[j] >= 0 && c0 + TPT * u < chunks)
                                ? reinterpret_cast<const uint4 *>(y_perm + row[j] * row_bytes)[c0 + TPT * u]
                                : make_uint4(0, 0, 0, 0);
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int c = c0 + TPT * u;
                float x[V];
                unpack<BF16, V>(a[u], x);
#pragma unroll
                for (int j = 0; j < KM; ++j) {
                    if (DW) {
                        float v[V];
                        unpack<BF16, V>(y[DW ? j : 0][u], v);
                        if (row[j] >= 0) {       // a dropped slot adds nothing, whatever dy holds
#pragma unroll
                            for (int i = 0; i < V; ++i)
                                dot[j] = fmaf(x[i], v[i], dot[j]);
                        }
                    }
                    if (DY && row[j] >= 0 && c < chunks) {
                        uint4 o;
                        if (BF16) {
                            o.x = pack_bf16x2(w[j] * x[0], w[j] * x[1]);
                            o.y = pack_bf16x2(w[j] * x[2], w[j] * x[3]);
                            o.z = pack_bf16x2(w[j] * x[V - 4], w[j] * x[V - 3]);
                            o.w = pack_bf16x2(w[j] * x[V - 2], w[j] * x[V - 1]);
                        } else {
                            o.x = __float_as_uint(w[j] * x[0]);
                            o.y = __float_as_uint(w[j] * x[1]);
                            o.z = __float_as_uint(w[j] * x[2]);
                            o.w = __float_as_uint(w[j] * x[3]);
                        }
                        reinterpret_cast<uint4 *>(dy_perm + row[j] * row_bytes)[c] = o;
                    }
                }
            }
        }
        if (DW) {
            float mine = 0.0f;
#pragma unroll
            for (int j = 0; j < KM; ++j) {
                float v = dot[j];
#pragma unroll
                for (int o = 16; o > 0; o >>= 1)
                    v += __shfl_xor_sync(0xffffffffu, v, o);
                if (lane == j)
                    mine = v;
            }
            if (TPT == 32) {
                if (lane < k)
                    dtopk_w[t * k + lane] = mine;
            } else {
                if (lane < KM)
                    s_dot[warp][lane] = mine;
                __syncthreads();
                if (threadIdx.x < k) {
                    float v = 0.0f;
#pragma unroll
                    for (int i = 0; i < kThreads / 32; ++i)
                        v += s_dot[i][threadIdx.x];
                    dtopk_w[t * k + threadIdx.x] = v;
                }
                __syncthreads();
            }
        }
    }
}

struct Args {
    const uint8_t *dy, *y_perm;
    const int32_t *inv_row;
    const float *topk_w;
    uint8_t *dy_perm;
    float *dtopk_w;
    int64_t T;
    int32_t d, k, sms;
    uint32_t *status;
    cudaStream_t stream;
};

template <bool BF16, int KM, int TPT>
void run(const Args &a)
{
    constexpr int TPB = kThreads / TPT;
    const int64_t want = (a.T + TPB - 1) / TPB, cap = static_cast<int64_t>(a.sms) * 8;
    auto kernel = a.dtopk_w ? (a.dy_perm ? combine_grad_kernel<BF16, KM, TPT, true, true>
                                         : combine_grad_kernel<BF16, KM, TPT, true, false>)
                            : combine_grad_kernel<BF16, KM, TPT, false, true>;
    launch_k(kernel, static_cast<int>(want < cap ? want : cap), kThreads, 0, a.stream, a.dy, a.y_perm,
             a.inv_row, a.topk_w, a.dy_perm, a.dtopk_w, a.T, a.d, a.k, a.T * a.k, a.status);
    count_launches(1);
}

template <bool BF16, int KM>
void run_km(const Args &a)
{
    // a warp per token once there are more tokens than two blocks per SM
    if (a.T > static_cast<int64_t>(a.sms) * 2)
        run<BF16, KM, 32>(a);
    else
        run<BF16, KM, kThreads>(a);
}

template <bool BF16>
void run_k(const Args &a)
{
    if (a.k <= 1)
        run_km<BF16, 1>(a);
    else if (a.k <= 2)
        run_km<BF16, 2>(a);
    else if (a.k <= 4)
        run_km<BF16, 4>(a);
    else
        run_km<BF16, kMaxK>(a);
}

}  // namespace

cudaError_t launch_combine_grad(int dtype, const void *dy, const void *y_perm,
                                const int32_t *inv_row, const float *topk_w, void *dy_perm,
                                float *dtopk_w, int64_t T, int32_t d, int32_t k,
                                uint32_t *status, cudaStream_t stream)
{
    if (T == 0)
        return cudaSuccess;
    int sms = 148, dev = 0;
    if (cudaGetDevice(&dev) == cudaSuccess)
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    const Args args{static_cast<const uint8_t *>(dy), static_cast<const uint8_t *>(y_perm), inv_row,
                    topk_w, static_cast<uint8_t *>(dy_perm), dtopk_w, T, d, k, sms, status, stream};
    if (dtype == MOE_BF16)
        run_k<true>(args);
    else
        run_k<false>(args);
    return cudaGetLastError();
}

}  // namespace moe
