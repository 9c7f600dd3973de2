// Dense products on the CUDA cores, for fp32 operands (TF32 would not meet an
// fp32 bound), with the projection's epilogue, and the element-wise half of
// the projection's gradient.
//
//   D[i, j] = sum_k P(i, k) Q(j, k);  out = act(D + bias) + residual
//
// The three products of a projection differ in which index of an operand is
// contiguous:
//   y  = x W^T      P = x  (k contiguous),      Q = W (k contiguous)
//   dx = dz W       P = dz (k contiguous),      Q = W^T (j contiguous)
//   dW = dz^T x     P = dz^T (i contiguous),    Q = x^T (j contiguous)
#include <type_traits>

#include "common.cuh"
#include "kernels.h"
#include "linear.cuh"
#include "moe.h"

namespace moe {

namespace {

constexpr int kThreads = 256;
constexpr int TM = 64, TN = 64, TK = 16;

// One 64 x 64 tile per block, 4 x 4 outputs per thread.
template <typename T, typename TO, int ACT, bool P_K, bool Q_K>
__global__ void __launch_bounds__(kThreads)
    linear_simt_kernel(const T *__restrict__ P, int64_t ldp, const T *__restrict__ Q, int64_t ldq,
                       int64_t I, int J, int64_t K, lin::Epilogue ep)
{
    grid_dep_wait();
    __shared__ float s_p[TK][TM + 4], s_q[TK][TN + 4];
    const int tid = threadIdx.x;
    const int64_t i0 = static_cast<int64_t>(blockIdx.x) * TM;
    const int64_t j0 = static_cast<int64_t>(blockIdx.y) * TN;
    const int ti = (tid >> 4) * 4, tj = (tid & 15) * 4;
    float acc[4][4] = {};
    for (int64_t k0 = 0; k0 < K; k0 += TK) {
        for (int e = tid; e < TM * TK; e += kThreads) {
            const int i = P_K ? e / TK : e % TM, k = P_K ? e % TK : e / TM;
            float v = 0.0f;
            if (i0 + i < I && k0 + k < K)
                v = lin::to_f32(P_K ? P[(i0 + i) * ldp + k0 + k] : P[(k0 + k) * ldp + i0 + i]);
            s_p[k][i] = v;
        }
        for (int e = tid; e < TN * TK; e += kThreads) {
            const int j = Q_K ? e / TK : e % TN, k = Q_K ? e % TK : e / TN;
            float v = 0.0f;
            if (j0 + j < J && k0 + k < K)
                v = lin::to_f32(Q_K ? Q[(j0 + j) * ldq + k0 + k] : Q[(k0 + k) * ldq + j0 + j]);
            s_q[k][j] = v;
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < TK; ++k) {
            float a[4], b[4];
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                a[x] = s_p[k][ti + x];
                b[x] = s_q[k][tj + x];
            }
#pragma unroll
            for (int x = 0; x < 4; ++x)
#pragma unroll
                for (int y = 0; y < 4; ++y)
                    acc[x][y] = fmaf(a[x], b[y], acc[x][y]);
        }
        __syncthreads();
    }
#pragma unroll
    for (int x = 0; x < 4; ++x)
#pragma unroll
        for (int y = 0; y < 4; ++y)
            if (i0 + ti + x < I && j0 + tj + y < J)
                lin::finish<ACT, TO, T>(ep, i0 + ti + x, static_cast<int>(j0) + tj + y, acc[x][y]);
}

// V consecutive values as fp32; vec: they lie on a 16-byte boundary (or V = 1).
template <int V>
__device__ __forceinline__ void load_v(const float *p, float (&v)[V])
{
    if (V % 4 == 0) {
#pragma unroll
        for (int i = 0; i < V / 4; ++i) {
            const float4 w = reinterpret_cast<const float4 *>(p)[i];
            v[4 * i] = w.x;
            v[(4 * i + 1) % V] = w.y;
            v[(4 * i + 2) % V] = w.z;
            v[(4 * i + 3) % V] = w.w;
        }
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i)
            v[i] = p[i];
    }
}

template <int V>
__device__ __forceinline__ void load_v(const __nv_bfloat16 *p, float (&v)[V])
{
    if (V == 8) {
        const uint4 q = *reinterpret_cast<const uint4 *>(p);
        const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[(2 * i) % V] = __uint_as_float(w[i] << 16);
            v[(2 * i + 1) % V] = __uint_as_float(w[i] & 0xFFFF0000u);
        }
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i)
            v[i] = __bfloat162float(p[i]);
    }
}

template <int V>
__device__ __forceinline__ void store_v(float *p, const float (&v)[V])
{
    if (V % 4 == 0) {
#pragma unroll
        for (int i = 0; i < V / 4; ++i)
            reinterpret_cast<float4 *>(p)[i] =
                make_float4(v[4 * i], v[(4 * i + 1) % V], v[(4 * i + 2) % V], v[(4 * i + 3) % V]);
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i)
            p[i] = v[i];
    }
}

template <int V>
__device__ __forceinline__ void store_v(__nv_bfloat16 *p, const float (&v)[V])
{
    if (V == 8) {
        *reinterpret_cast<uint4 *>(p) =
            make_uint4(pack_bf16x2(v[0], v[1 % V]), pack_bf16x2(v[2 % V], v[3 % V]),
                       pack_bf16x2(v[4 % V], v[5 % V]), pack_bf16x2(v[6 % V], v[7 % V]));
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i)
            p[i] = __float2bfloat16_rn(v[i]);
    }
}

// dz = dy * act'(z) in the operand type, and this row block's column sums of
// the unrounded dz, in 32 bits: a warp sums every eighth row of the block's in
// order, then the eight sums are added in order.  A lane holds V columns (16
// bytes of the operand type where rows allow it).  Bound by the bytes of dy, z
// and dz, and for GELU as much by its error function.
template <typename T, typename TO, int ACT, int V>
__global__ void __launch_bounds__(kThreads)
    linear_dz_kernel(const TO *__restrict__ dy, int64_t ldy, const T *__restrict__ z, int64_t M,
                     int n, T *__restrict__ dz, int64_t ldz, float *__restrict__ part,
                     int64_t rows_per_block)
{
    grid_dep_wait();
    __shared__ float s_sum[kThreads / 32][32 * V];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int col = (blockIdx.x * 32 + lane) * V;
    const int64_t r0 = blockIdx.y * rows_per_block;
    const int64_t r1 = r0 + rows_per_block < M ? r0 + rows_per_block : M;
    float sum[V];
#pragma unroll
    for (int i = 0; i < V; ++i)
        sum[i] = 0.0f;
    if (col < n) {
#pragma unroll 4
        for (int64_t r = r0 + warp; r < r1; r += kThreads / 32) {
            float g[V];
            load_v<V>(dy + r * ldy + col, g);
            if (ACT != MOE_LINEAR_NONE) {
                float zz[V];
                load_v<V>(z + r * n + col, zz);
#pragma unroll
                for (int i = 0; i < V; ++i)
                    g[i] *= lin::act_bwd<ACT>(zz[i]);
            }
#pragma unroll
            for (int i = 0; i < V; ++i)
                sum[i] += g[i];
            if (dz)
                store_v<V>(dz + r * ldz + col, g);
        }
    }
    if (part) {
#pragma unroll
        for (int i = 0; i < V; ++i)
            s_sum[warp][lane * V + i] = sum[i];
        __syncthreads();
        for (int c = threadIdx.x; c < 32 * V; c += kThreads) {
            const int at = blockIdx.x * 32 * V + c;
            float v = 0.0f;
#pragma unroll
            for (int w = 0; w < kThreads / 32; ++w)
                v += s_sum[w][c];
            if (at < n)
                part[static_cast<int64_t>(blockIdx.y) * n + at] = v;
        }
    }
}

// db = the row blocks' sums, added in a fixed order: 32 columns per block,
// every eighth row block per warp.
__global__ void __launch_bounds__(kThreads)
    linear_db_kernel(const float *__restrict__ part, int blocks, int n, float *__restrict__ db)
{
    grid_dep_wait();
    __shared__ float s_sum[kThreads / 32][32];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int col = blockIdx.x * 32 + lane;
    float sum = 0.0f;
    if (col < n) {
#pragma unroll 8
        for (int b = warp; b < blocks; b += kThreads / 32)
            sum += part[static_cast<int64_t>(b) * n + col];
    }
    s_sum[warp][lane] = sum;
    __syncthreads();
    if (warp == 0 && col < n) {
        float v = 0.0f;
#pragma unroll
        for (int w = 0; w < kThreads / 32; ++w)
            v += s_sum[w][lane];
        db[col] = v;
    }
}

template <typename T, typename TO>
void run_simt(const LinearGemm &L, cudaStream_t stream)
{
    const dim3 grid(static_cast<unsigned>((L.I + TM - 1) / TM),
                    static_cast<unsigned>((L.J + TN - 1) / TN), 1);
    const T *P = static_cast<const T *>(L.P);
    const T *Q = static_cast<const T *>(L.Q);
    lin::Epilogue ep;
    ep.out = L.out;
    ep.ldo = L.ldo;
    ep.bias = L.bias;
    ep.residual = L.residual;
    ep.ldr = L.ldr;
    ep.preact = L.preact;
    ep.rows = static_cast<int32_t>(L.I);
    ep.cols = L.J;
    if (L.p_kmajor && L.q_kmajor)
        lin::with_act(L.act, [&](auto a) {
            launch_k(linear_simt_kernel<T, TO, decltype(a)::value, true, true>, grid, kThreads, 0,
                     stream, P, L.ldp, Q, L.ldq, L.I, L.J, L.K, ep);
        });
    else if (L.p_kmajor)
        launch_k(linear_simt_kernel<T, TO, MOE_LINEAR_NONE, true, false>, grid, kThreads, 0,
                 stream, P, L.ldp, Q, L.ldq, L.I, L.J, L.K, ep);
    else
        launch_k(linear_simt_kernel<T, TO, MOE_LINEAR_NONE, false, false>, grid, kThreads, 0,
                 stream, P, L.ldp, Q, L.ldq, L.I, L.J, L.K, ep);
    count_launches(1);
}

template <typename T, typename TO>
void run_dz(const LinearDz &L, cudaStream_t stream)
{
    constexpr int VV = 16 / sizeof(T);
    const int64_t per = (L.M + L.row_blocks - 1) / L.row_blocks;
    auto on16 = [](const void *p, int64_t row_bytes) {
        return reinterpret_cast<uintptr_t>(p) % 16 == 0 && row_bytes % 16 == 0;
    };
    const bool vec = L.n % VV == 0 && on16(L.dy, L.ldy * static_cast<int64_t>(sizeof(TO))) &&
                     on16(L.z, L.n * static_cast<int64_t>(sizeof(T))) &&
                     on16(L.dz, L.ldz * static_cast<int64_t>(sizeof(T)));
    const int wide = 32 * (vec ? VV : 1);
    const dim3 grid(static_cast<unsigned>((L.n + wide - 1) / wide),
                    static_cast<unsigned>(L.row_blocks), 1);
    lin::with_act(L.act, [&](auto a) {
        auto kernel = vec ? linear_dz_kernel<T, TO, decltype(a)::value, VV>
                          : linear_dz_kernel<T, TO, decltype(a)::value, 1>;
        launch_k(kernel, grid, kThreads, 0, stream, static_cast<const TO *>(L.dy), L.ldy,
                 static_cast<const T *>(L.z), L.M, L.n, static_cast<T *>(L.dz), L.ldz,
                 L.db ? L.part : nullptr, per);
    });
    count_launches(1);
}

}  // namespace

cudaError_t launch_linear_simt(const LinearGemm &L, cudaStream_t stream)
{
    if (L.dtype == MOE_F32)
        run_simt<float, float>(L, stream);
    else if (L.out_f32)
        run_simt<__nv_bfloat16, float>(L, stream);
    else
        run_simt<__nv_bfloat16, __nv_bfloat16>(L, stream);
    return cudaGetLastError();
}

cudaError_t launch_linear_dz(const LinearDz &L, cudaStream_t stream)
{
    if (L.dtype == MOE_F32)
        run_dz<float, float>(L, stream);
    else if (L.out_f32)
        run_dz<__nv_bfloat16, float>(L, stream);
    else
        run_dz<__nv_bfloat16, __nv_bfloat16>(L, stream);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || !L.db)
        return e;
    launch_k(linear_db_kernel, dim3((L.n + 31) / 32), kThreads, 0, stream,
             static_cast<const float *>(L.part), L.row_blocks, L.n, L.db);
    count_launches(1);
    return cudaGetLastError();
}

}  // namespace moe
