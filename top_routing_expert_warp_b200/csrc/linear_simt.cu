// Dense products on the CUDA cores: for fp32 operands (TF32 would not meet an
// fp32 bound) and, for a few rows of either type, as dot products with the
// weights' rows; with the projection's epilogue.  And the element-wise half of
// the projection's gradient.
//
//   D[i, j] = sum_k P(i, k) Q(j, k);  out = act(D + bias) + residual
//
// The three products of a projection differ in which index of an operand is
// contiguous:
//   y  = x W^T      P = x  (k contiguous),      Q = W (k contiguous)
//   dx = dz W       P = dz (k contiguous),      Q = W^T (j contiguous)
//   dW = dz^T x     P = dz^T (i contiguous),    Q = x^T (j contiguous)
#include <algorithm>
#include <type_traits>

#include "common.cuh"
#include "kernels.h"
#include "linear.cuh"
#include "moe.h"

namespace moe {

namespace {

constexpr int kThreads = 256;
constexpr int TM = 64, TN = 64, TK = 16;
constexpr int kGemmThreads = 128;
constexpr int kPad = 4;                  // floats behind a row of a staged tile

// acc (two floats) += a * (b, b).
__device__ __forceinline__ void fma2(uint64_t &acc, uint64_t a, uint64_t bb)
{
    asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(acc) : "l"(a), "l"(bb));
}

__device__ __forceinline__ uint64_t twice(float b)
{
    uint64_t r;
    asm("mov.b64 %0, {%1, %1};" : "=l"(r) : "f"(b));
    return r;
}

// This thread's 8 elements of a 64 x 16 operand tile, as two runs of 4 along
// the contiguous index: run h starts at (own index, k) = where(h).  Runs that
// do not lie inside the operand are loaded element by element, zero outside.
template <bool K_CONTIG>
struct TileLoad {
    float v[2][4];
    __device__ __forceinline__ static void where(int h, int &own, int &k)
    {
        const int e = (threadIdx.x + h * kGemmThreads) * 4;
        own = K_CONTIG ? e / TK : e % 64;
        k = K_CONTIG ? e % TK : e / 64;
    }
    __device__ __forceinline__ void load(const float *__restrict__ src, int64_t ld, int64_t own0,
                                         int64_t owns, int64_t k0, int64_t k1)
    {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            int o, kk;
            where(h, o, kk);
            const int64_t own = own0 + o, k = k0 + kk;
            const float *at = K_CONTIG ? src + own * ld + k : src + k * ld + own;
            const bool inside = own < owns && k < k1;
            const int64_t left = K_CONTIG ? k1 - k : owns - own;
            if (inside && left >= 4) {
                const float4 q = __ldcg(reinterpret_cast<const float4 *>(at));
                v[h][0] = q.x;
                v[h][1] = q.y;
                v[h][2] = q.z;
                v[h][3] = q.w;
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    v[h][i] = inside && i < left ? __ldcg(at + i) : 0.0f;
            }
        }
    }
    __device__ __forceinline__ void store(float (*dst)[64 + kPad]) const
    {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            int o, kk;
            where(h, o, kk);
            if (K_CONTIG) {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    dst[kk + i][o] = v[h][i];
            } else {
                *reinterpret_cast<float4 *>(&dst[kk][o]) =
                    make_float4(v[h][0], v[h][1], v[h][2], v[h][3]);
            }
        }
    }
};

struct SimtParams {
    const float *P, *Q;
    int64_t ldp, ldq;
    int64_t I, K;
    int32_t J, i_tiles, splits, act;
    int32_t vec;             // output rows start on 16-byte boundaries
    int32_t first_of_two, second_of_two;     // see LinearGemm
    lin::Epilogue ep;
    float *part;             // [units][64][64]
    uint32_t *tickets;       // [tiles], zero between launches
};

__device__ __forceinline__ float act_any(int act, float z)
{
    switch (act) {
    case MOE_LINEAR_RELU: return lin::act_fwd<MOE_LINEAR_RELU>(z);
    case MOE_LINEAR_SILU: return lin::act_fwd<MOE_LINEAR_SILU>(z);
    case MOE_LINEAR_GELU: return lin::act_fwd<MOE_LINEAR_GELU>(z);
    case MOE_LINEAR_GELU_TANH: return lin::act_fwd<MOE_LINEAR_GELU_TANH>(z);
    default: return z;
    }
}

template <int ACT>
__device__ __forceinline__ void act_all(float (&v)[8][4])
{
#pragma unroll
    for (int x = 0; x < 8; ++x)
#pragma unroll
        for (int y = 0; y < 4; ++y)
            v[x][y] = lin::act_fwd<ACT>(v[x][y]);
}

// A 64 x 64 tile (or a slice of its k range) per block, 8 x 4 outputs per
// thread in pairs of rows (fma.rn.f32x2: two products per issue; with single
// products 1024 x 4096 x 4096 took half as long again), the next 16 of k in
// registers while the present ones are multiplied.  Tiles too few to fill the
// GPU are cut along k; the slices' sums go through the workspace and the last
// block to finish adds them in slice order (a ticket per tile, which wraps to
// 0).  Bound by shared memory's read rate (80 % of it) and the fp32 pipes:
// 1024^3 in 64 us, 2048^3 in 403 us = 43 TFLOP/s (a library product takes 47 and
// 309 us).  8 x 8 outputs per thread read half as much but left too few warps:
// 61 and 430 us.
template <bool P_K, bool Q_K>
__device__ __forceinline__ void simt_tile(const SimtParams &p)
{
    __shared__ __align__(16) float s_p[2][TK][TM + kPad];
    __shared__ __align__(16) float s_q[2][TK][TN + kPad];
    __shared__ uint32_t s_last;
    const int tid = threadIdx.x;
    const int64_t unit = blockIdx.x;
    const int64_t tile = unit / p.splits;
    const int slice = static_cast<int>(unit - tile * p.splits);
    const int64_t jt = tile / p.i_tiles;
    const int64_t i0 = (tile - jt * p.i_tiles) * TM, j0 = jt * TN;
    const int64_t steps = (p.K + TK - 1) / TK;
    const int64_t kb = steps * slice / p.splits * TK;
    const int64_t ke = steps * (slice + 1) / p.splits * TK;
    const int64_t k1 = ke < p.K ? ke : p.K;
    const int ti = (tid >> 4) * 8, tj = (tid & 15) * 4;
    uint64_t acc[4][4] = {};                 // [row pair][column]
    TileLoad<P_K> lp;
    TileLoad<Q_K> lq;
    lp.load(p.P, p.ldp, i0, p.I, kb, k1);
    lq.load(p.Q, p.ldq, j0, p.J, kb, k1);
    lp.store(s_p[0]);
    lq.store(s_q[0]);
    __syncthreads();
    int cur = 0;
    for (int64_t k0 = kb; k0 < k1; k0 += TK, cur ^= 1) {
        const bool more = k0 + TK < k1;
        if (more) {
            lp.load(p.P, p.ldp, i0, p.I, k0 + TK, k1);
            lq.load(p.Q, p.ldq, j0, p.J, k0 + TK, k1);
        }
#pragma unroll
        for (int k = 0; k < TK; ++k) {
            const ulonglong2 a0 = *reinterpret_cast<const ulonglong2 *>(&s_p[cur][k][ti]);
            const ulonglong2 a1 = *reinterpret_cast<const ulonglong2 *>(&s_p[cur][k][ti + 4]);
            const float4 b = *reinterpret_cast<const float4 *>(&s_q[cur][k][tj]);
            const uint64_t a[4] = {a0.x, a0.y, a1.x, a1.y};
            const uint64_t bb[4] = {twice(b.x), twice(b.y), twice(b.z), twice(b.w)};
#pragma unroll
            for (int x = 0; x < 4; ++x)
#pragma unroll
                for (int y = 0; y < 4; ++y)
                    fma2(acc[x][y], a[x], bb[y]);
        }
        if (more) {
            lp.store(s_p[cur ^ 1]);
            lq.store(s_q[cur ^ 1]);
        }
        __syncthreads();
    }
    float out[8][4];
#pragma unroll
    for (int x = 0; x < 4; ++x)
#pragma unroll
        for (int y = 0; y < 4; ++y) {
            out[2 * x][y] = __uint_as_float(static_cast<uint32_t>(acc[x][y]));
            out[2 * x + 1][y] = __uint_as_float(static_cast<uint32_t>(acc[x][y] >> 32));
        }
    if (p.splits > 1) {
        float4 *mine = reinterpret_cast<float4 *>(p.part) + unit * (TM * TN / 4) + tid;
#pragma unroll
        for (int x = 0; x < 8; ++x)
            __stcg(mine + x * kGemmThreads, make_float4(out[x][0], out[x][1], out[x][2], out[x][3]));
        __threadfence();
        __syncthreads();
        if (tid == 0) {
            s_last = atomicInc(p.tickets + tile, p.splits - 1) == static_cast<uint32_t>(p.splits - 1);
            __threadfence();
        }
        __syncthreads();
        if (!s_last)
            return;
#pragma unroll
        for (int x = 0; x < 8; ++x)
#pragma unroll
            for (int y = 0; y < 4; ++y)
                out[x][y] = 0.0f;
        const float4 *first = reinterpret_cast<const float4 *>(p.part) +
                              tile * p.splits * (TM * TN / 4) + tid;
        for (int s = 0; s < p.splits; ++s) {
#pragma unroll
            for (int x = 0; x < 8; ++x) {
                const float4 v = __ldcg(first + s * (TM * TN / 4) + x * kGemmThreads);
                out[x][0] += v.x;
                out[x][1] += v.y;
                out[x][2] += v.z;
                out[x][3] += v.w;
            }
        }
    }
    // step by step over all 32 outputs, so that a step's branch is taken once
    const lin::Epilogue &ep = p.ep;
    const int64_t row0 = i0 + ti, col = j0 + tj;
    const int rows = p.I - row0 < 8 ? static_cast<int>(p.I - row0) : 8;
    const int n = p.J - col < 4 ? static_cast<int>(p.J - col) : 4;
    if (ep.bias) {
#pragma unroll
        for (int y = 0; y < 4; ++y) {
            const float b = y < n ? __ldg(ep.bias + col + y) : 0.0f;
#pragma unroll
            for (int x = 0; x < 8; ++x)
                out[x][y] += b;
        }
    }
    if (ep.preact) {
        float *z = static_cast<float *>(ep.preact) + row0 * ep.cols + col;
#pragma unroll
        for (int x = 0; x < 8; ++x)
#pragma unroll
            for (int y = 0; y < 4; ++y)
                if (x < rows && y < n)
                    z[x * static_cast<int64_t>(ep.cols) + y] = out[x][y];
    }
    switch (p.act) {
    case MOE_LINEAR_RELU: act_all<MOE_LINEAR_RELU>(out); break;
    case MOE_LINEAR_SILU: act_all<MOE_LINEAR_SILU>(out); break;
    case MOE_LINEAR_GELU: act_all<MOE_LINEAR_GELU>(out); break;
    case MOE_LINEAR_GELU_TANH: act_all<MOE_LINEAR_GELU_TANH>(out); break;
    default: break;
    }
    if (ep.residual) {
        const float *r = static_cast<const float *>(ep.residual) + row0 * ep.ldr + col;
#pragma unroll
        for (int x = 0; x < 8; ++x)
#pragma unroll
            for (int y = 0; y < 4; ++y)
                if (x < rows && y < n)
                    out[x][y] += r[x * ep.ldr + y];
    }
    float *o = static_cast<float *>(ep.out) + row0 * ep.ldo + col;
    if (p.vec && n == 4) {
#pragma unroll
        for (int x = 0; x < 8; ++x)
            if (x < rows)
                *reinterpret_cast<float4 *>(o + x * ep.ldo) =
                    make_float4(out[x][0], out[x][1], out[x][2], out[x][3]);
    } else {
#pragma unroll
        for (int x = 0; x < 8; ++x)
#pragma unroll
            for (int y = 0; y < 4; ++y)
                if (x < rows && y < n)
                    o[x * ep.ldo + y] = out[x][y];
    }
}

template <bool P_K, bool Q_K>
__global__ void __launch_bounds__(kGemmThreads) linear_simt_kernel(const __grid_constant__ SimtParams p)
{
    if (!p.second_of_two)
        grid_dep_wait();
    if (p.first_of_two)
        grid_dep_launch();
    simt_tile<P_K, Q_K>(p);
    if (p.second_of_two)
        grid_dep_wait();
}

// Few rows (serving): y[m, n] = act(sum_k x[m, k] W[n, k] + bias) + residual.
// WPR warps per output n read its weights once, 16 bytes per lane with 8 loads
// in flight, next to the same places of the rows of x (in L1); the warps' sums
// are added in order.  Bound by the weights' bytes and the launch: one row of
// 7168 -> 2048 bf16 in 8.1 us from HBM, 3.6 TB/s with the launch in it.
template <typename T, typename TO, int MR>
__global__ void __launch_bounds__(kThreads)
    linear_rows_kernel(const T *__restrict__ x, int64_t ldx, const T *__restrict__ W, int M, int K,
                       int N, int wpr, int act, const __grid_constant__ lin::Epilogue ep)
{
    grid_dep_wait();
    constexpr int V = 16 / sizeof(T);
    constexpr int U = 8;
    __shared__ float s_sum[kThreads / 32][MR];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int part = warp % wpr;
    const int n = blockIdx.x * (kThreads / 32 / wpr) + warp / wpr;
    const int chunks = K / V;
    float acc[MR];
#pragma unroll
    for (int m = 0; m < MR; ++m)
        acc[m] = 0.0f;
    if (n < N) {
        const uint4 *w = reinterpret_cast<const uint4 *>(W + static_cast<int64_t>(n) * K);
        const int step = 32 * wpr;
        for (int c0 = part * 32 + lane; c0 < chunks; c0 += step * U) {
            uint4 wq[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int c = c0 + u * step;
                wq[u] = c < chunks ? __ldcs(w + c) : make_uint4(0, 0, 0, 0);
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const uint32_t a[4] = {wq[u].x, wq[u].y, wq[u].z, wq[u].w};
                const int c = c0 + u * step;
                if (c >= chunks)
                    break;
#pragma unroll
                for (int m = 0; m < MR; ++m) {
                    if (m >= M)
                        break;
                    const uint4 xq = __ldg(reinterpret_cast<const uint4 *>(x + m * ldx) + c);
                    const uint32_t b[4] = {xq.x, xq.y, xq.z, xq.w};
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        if (sizeof(T) == 2) {
                            acc[m] = fmaf(__uint_as_float(a[i] << 16), __uint_as_float(b[i] << 16),
                                          acc[m]);
                            acc[m] = fmaf(__uint_as_float(a[i] & 0xFFFF0000u),
                                          __uint_as_float(b[i] & 0xFFFF0000u), acc[m]);
                        } else {
                            acc[m] = fmaf(__uint_as_float(a[i]), __uint_as_float(b[i]), acc[m]);
                        }
                    }
                }
            }
        }
    }
#pragma unroll
    for (int m = 0; m < MR; ++m) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
            acc[m] += __shfl_xor_sync(0xffffffffu, acc[m], o);
        if (lane == 0)
            s_sum[warp][m] = acc[m];
    }
    __syncthreads();
    if (part != 0 || n >= N || lane >= M)
        return;
    float z = 0.0f;
    for (int w = 0; w < wpr; ++w)
        z += s_sum[warp + w][lane];
    if (ep.bias)
        z += ep.bias[n];
    if (ep.preact)
        lin::put(static_cast<T *>(ep.preact) + static_cast<int64_t>(lane) * ep.cols + n, z);
    z = act_any(act, z);
    if (ep.residual)
        z += lin::to_f32(static_cast<const TO *>(ep.residual)[lane * ep.ldr + n]);
    lin::put(static_cast<TO *>(ep.out) + lane * ep.ldo + n, z);
}

// V consecutive values as they lie (on a 16-byte boundary, or V = 1), and as fp32.
template <typename T, int V>
struct Run {
    static constexpr int kWords = V == 1 ? 1 : V * static_cast<int>(sizeof(T)) / 4;
    uint32_t w[kWords];
    __device__ __forceinline__ void load(const T *p)
    {
        if (V == 1) {
            w[0] = sizeof(T) == 4 ? *reinterpret_cast<const uint32_t *>(p)
                                  : *reinterpret_cast<const uint16_t *>(p);
        } else {
#pragma unroll
            for (int i = 0; i < kWords / 4; ++i) {
                const uint4 q = reinterpret_cast<const uint4 *>(p)[i];
                w[(4 * i) % kWords] = q.x;
                w[(4 * i + 1) % kWords] = q.y;
                w[(4 * i + 2) % kWords] = q.z;
                w[(4 * i + 3) % kWords] = q.w;
            }
        }
    }
    __device__ __forceinline__ float at(int i) const
    {
        if (sizeof(T) == 4)
            return __uint_as_float(w[i % kWords]);
        return __uint_as_float((i & 1) ? (w[i / 2 % kWords] & 0xFFFF0000u) : (w[i / 2 % kWords] << 16));
    }
};

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
// and dz for ReLU (4096 x 4096 bf16 in 16 us), by its instructions for the
// others (SiLU 20 us, GELU 26 us, its tanh form 25 us).
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
        // the next two rows' loads are in flight while a row is computed
        constexpr int kAhead = 2, kStep = kThreads / 32;
        Run<TO, V> y[kAhead];
        Run<T, V> zz[kAhead];
        auto fetch = [&](int slot, int64_t r) {
            if (r < r1) {
                y[slot].load(dy + r * ldy + col);
                if (ACT != MOE_LINEAR_NONE)
                    zz[slot].load(z + r * n + col);
            }
        };
#pragma unroll
        for (int a = 0; a < kAhead; ++a)
            fetch(a, r0 + warp + a * kStep);
        for (int64_t r = r0 + warp; r < r1; r += kAhead * kStep) {
#pragma unroll
            for (int a = 0; a < kAhead; ++a) {
                const int64_t row = r + a * kStep;
                if (row >= r1)
                    break;
                float g[V], f[V];
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    g[i] = y[a].at(i);
                    f[i] = ACT != MOE_LINEAR_NONE ? zz[a].at(i) : 0.0f;
                }
                fetch(a, row + kAhead * kStep);
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    if (ACT != MOE_LINEAR_NONE)
                        g[i] *= lin::act_bwd<ACT>(f[i]);
                    sum[i] += g[i];
                }
                if (dz)
                    store_v<V>(dz + row * ldz + col, g);
            }
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
    grid_dep_launch();      // the products need dz, not this
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

lin::Epilogue epilogue_of(const LinearGemm &L)
{
    lin::Epilogue ep;
    ep.out = L.out;
    ep.ldo = L.ldo;
    ep.bias = L.bias;
    ep.residual = L.residual;
    ep.ldr = L.ldr;
    ep.preact = L.preact;
    ep.cols = L.J;
    return ep;
}

template <typename T, typename TO>
void run_rows(const LinearGemm &L, cudaStream_t stream)
{
    // warps per output so that at least 24 warps run on each SM, 40 where more
    // rows make each wait longer (4096 -> 4096: one bf16 row 8.3 us with 24, 9.5
    // with 40; four fp32 rows 36 and 26)
    const int64_t warps = L.I <= 2 ? 148 * 24 : 148 * 40;
    int wpr = 1;
    while (wpr < 8 && static_cast<int64_t>(L.J) * wpr < warps)
        wpr *= 2;
    const int per = kThreads / 32 / wpr;
    auto kernel = L.I == 1 ? linear_rows_kernel<T, TO, 1>
                           : (L.I == 2 ? linear_rows_kernel<T, TO, 2> : linear_rows_kernel<T, TO, 4>);
    launch_k(kernel, dim3((L.J + per - 1) / per), kThreads, 0, stream, static_cast<const T *>(L.P),
             L.ldp, static_cast<const T *>(L.Q), static_cast<int>(L.I), static_cast<int>(L.K), L.J,
             wpr, L.act, epilogue_of(L));
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

SimtPlan simt_plan(int64_t I, int64_t J, int64_t K)
{
    SimtPlan pl;
    pl.tiles = (I + TM - 1) / TM * ((J + TN - 1) / TN);
    // about four blocks per SM, slices of at least 96 of k, at most 16 (the last
    // block of a tile adds them all up): 16 x 4096 x 512 took 37 us in 64 slices
    // and 20 in 16; 64 x 1024 x 64 16 us in slices of 32, 10 of 96, 16 of 256
    int64_t s = std::min<int64_t>(16, 148 * 4 / pl.tiles);
    s = std::min<int64_t>(s, K / 96);
    pl.splits = static_cast<int>(s < 1 ? 1 : s);
    return pl;
}

size_t simt_plan_part_bytes(const SimtPlan &pl)
{
    return pl.splits > 1 ? static_cast<size_t>(pl.tiles) * pl.splits * TM * TN * 4 : 0;
}

cudaError_t launch_linear_simt(const LinearGemm &L, cudaStream_t stream)
{
    const SimtPlan pl = simt_plan(L.I, L.J, L.K);
    const int64_t units = pl.tiles * pl.splits;
    if (units > 0x7FFFFFFF)
        return cudaErrorInvalidValue;
    SimtParams p;
    p.P = static_cast<const float *>(L.P);
    p.Q = static_cast<const float *>(L.Q);
    p.ldp = L.ldp;
    p.ldq = L.ldq;
    p.I = L.I;
    p.K = L.K;
    p.J = L.J;
    p.i_tiles = static_cast<int32_t>((L.I + TM - 1) / TM);
    p.splits = pl.splits;
    p.act = L.act;
    p.vec = reinterpret_cast<uintptr_t>(L.out) % 16 == 0 && L.ldo % 4 == 0;
    p.ep = epilogue_of(L);
    p.part = L.part;
    p.tickets = L.tickets;
    p.first_of_two = L.first_of_two;
    p.second_of_two = L.second_of_two;
    auto kernel = L.p_kmajor ? (L.q_kmajor ? linear_simt_kernel<true, true>
                                           : linear_simt_kernel<true, false>)
                             : linear_simt_kernel<false, false>;
    launch_k(kernel, dim3(static_cast<unsigned>(units)), kGemmThreads, 0, stream, p);
    count_launches(1);
    return cudaGetLastError();
}

cudaError_t launch_linear_rows(const LinearGemm &L, cudaStream_t stream)
{
    if (L.dtype == MOE_F32)
        run_rows<float, float>(L, stream);
    else if (L.out_f32)
        run_rows<__nv_bfloat16, float>(L, stream);
    else
        run_rows<__nv_bfloat16, __nv_bfloat16>(L, stream);
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
