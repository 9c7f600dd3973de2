// Gradient of the combine (combine.cu).
//
//   y[t] = sum over kept slots j of w[t, j] * y_perm[r(t, j)]
//   dy_perm[r(t, j)] = w[t, j] * dy[t],   dw[t, j] = <dy[t], y_perm[r(t, j)]>
//
// One block per token: each thread reads its chunks of dy[t] once and uses
// them for every slot.  fp32 products and sums, the order of a sum fixed by
// the block's shape.
#include "common.cuh"
#include "kernels.h"
#include "moe.h"

namespace moe {

namespace {

constexpr int kThreads = 256;
constexpr int kMaxK = 8;

template <bool BF16>
__global__ void __launch_bounds__(kThreads)
    combine_grad_kernel(const uint8_t *__restrict__ dy, const uint8_t *y_perm,
                        const int32_t *__restrict__ inv_row, const float *__restrict__ topk_w,
                        uint8_t *dy_perm, float *__restrict__ dtopk_w, int64_t T, int d, int k,
                        int64_t rows_cap, uint32_t *status)
{
    grid_dep_wait();
    __shared__ float s_dot[kMaxK][kThreads / 32];
    constexpr int V = BF16 ? 8 : 4;
    constexpr int esz = BF16 ? 2 : 4;
    const int chunks = d / V;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (int64_t t = blockIdx.x; t < T; t += gridDim.x) {
        int32_t row[kMaxK];
        float w[kMaxK], dot[kMaxK];
#pragma unroll
        for (int j = 0; j < kMaxK; ++j) {
            row[j] = j < k ? inv_row[t * k + j] : -1;
            if (row[j] >= rows_cap || row[j] < -1) {
                if (threadIdx.x == 0)
                    set_status(status, DEV_BAD_ROW);
                row[j] = -1;
            }
            w[j] = (j < k && dy_perm) ? topk_w[t * k + j] : 0.0f;
            dot[j] = 0.0f;
        }
        const uint4 *src = reinterpret_cast<const uint4 *>(dy + t * static_cast<int64_t>(d) * esz);
        for (int c = threadIdx.x; c < chunks; c += kThreads) {
            const uint4 a = src[c];
            const uint32_t aw[4] = {a.x, a.y, a.z, a.w};
            float x[V];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (BF16) {
                    x[2 * i] = __uint_as_float(aw[i] << 16);
                    x[2 * i + 1] = __uint_as_float(aw[i] & 0xFFFF0000u);
                } else {
                    x[i] = __uint_as_float(aw[i]);
                }
            }
#pragma unroll
            for (int j = 0; j < kMaxK; ++j) {
                if (row[j] < 0)
                    continue;
                const int64_t off = static_cast<int64_t>(row[j]) * d * esz;
                if (dtopk_w) {
                    const uint4 v = reinterpret_cast<const uint4 *>(y_perm + off)[c];
                    const uint32_t vw[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        if (BF16) {
                            dot[j] = fmaf(x[2 * i], __uint_as_float(vw[i] << 16), dot[j]);
                            dot[j] = fmaf(x[2 * i + 1], __uint_as_float(vw[i] & 0xFFFF0000u), dot[j]);
                        } else {
                            dot[j] = fmaf(x[i], __uint_as_float(vw[i]), dot[j]);
                        }
                    }
                }
                if (dy_perm) {
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
                    reinterpret_cast<uint4 *>(dy_perm + off)[c] = o;
                }
            }
        }
        if (dtopk_w) {
#pragma unroll
            for (int j = 0; j < kMaxK; ++j) {
                float v = dot[j];
#pragma unroll
                for (int o = 16; o > 0; o >>= 1)
                    v += __shfl_xor_sync(0xffffffffu, v, o);
                if (lane == 0)
                    s_dot[j][warp] = v;
            }
            __syncthreads();
            if (threadIdx.x < k) {
                float v = 0.0f;
                for (int i = 0; i < kThreads / 32; ++i)
                    v += s_dot[threadIdx.x][i];
                dtopk_w[t * k + threadIdx.x] = v;
            }
            __syncthreads();
        }
    }
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
    const int64_t cap = static_cast<int64_t>(sms) * 8;
    const int grid = static_cast<int>(T < cap ? T : cap);
    const int64_t rows_cap = T * k;
    launch_k(dtype == MOE_BF16 ? combine_grad_kernel<true> : combine_grad_kernel<false>, grid,
             kThreads, 0, stream, static_cast<const uint8_t *>(dy),
             static_cast<const uint8_t *>(y_perm), inv_row, topk_w,
             static_cast<uint8_t *>(dy_perm), dtopk_w, T, d, k, rows_cap, status);
    count_launches(1);
    return cudaGetLastError();
}

}  // namespace moe
