// Dense products on the tensor cores (tcgen05), for bf16 operands, with the
// projection's epilogue.
//
//   D[i, j] = sum_k P(i, k) Q(j, k);  out = act(D + bias) + residual
//
// The three products of a projection (see linear_simt.cu) differ in which
// index of an operand is contiguous; the tensor cores take either: an operand
// with k contiguous is staged as rows of 64 k (128-byte swizzle), one with its
// own index contiguous as blocks of 64 of that index by 64 k.
//
// A tile is
//   CG = 2: 256 x 256 on a CTA pair (cta_group::2, each CTA stages 128 rows of
//           P and 128 of Q), for large products: per SM a 64-wide k block
//           brings 32 KB for 256 cycles of tensor work (narrower tiles, to
//           fill the last round of pairs better, were 3 to 30 % slower);
//   CG = 1: 128 x up to 128 on one CTA, for small ones.
// With few rows (serving) the product is taken transposed: P is the weights
// (128 of them are the MMA's rows) and Q the tokens (rounded up to 16 as the
// MMA's columns), so the weights are read once at the rate of HBM and no MMA
// is spent on absent tokens.
// Tiles too few for the GPU are cut along k into slices, each on its own CTA
// (or pair) of one cluster of at most 8.  The slices' sums meet in shared memory:
// every CTA of the cluster takes a share of the columns, the others send it
// theirs (distributed shared memory, in the space of the finished stages), and
// it adds them in slice order and finishes them.  Through global memory with
// a ticket this took 4-12 us per launch instead of 2.
//
// Roles: warp 0 TMA producer, warp 1 MMA issuer, the others the epilogue: eight
// of them, two per TMEM lane quarter on alternate 32-column steps, or in the
// form with chains sixteen, four per quarter with a quarter of the columns each.
// Two accumulators in TMEM: the epilogue of a tile overlaps the products of the
// next.  Every wait is bounded.
//
// The tensor cores' fp32 sums are cut (not rounded) at every step, an error that
// grows with the length of the chain (1e-9 of the norm per k).  So a slice uses
// both accumulators for the halves of its k range, and fp32 results without
// slices are summed in chains of at most 1280, in the accumulators by turns,
// which 16 epilogue warps add up in registers (CHAINED; 4096^3 in 124 us with
// an error of 1e-6; 102 us in bf16 and one chain; two slices took 186 us).
//
// A lane of the epilogue holds a piece of a row and writes it 16 bytes at a
// time.  Where rows are not 16-byte aligned the warp first turns its 32 x 32
// accumulators over in shared memory, so that its lanes hold consecutive
// columns (element-wise stores of row pieces cost 15 us more at 300 x 300).
//
// What bounds it: large products the tensor cores under the power limit (4096 x
// 4096 -> 14336 back to back 391 us = 1230 TFLOP/s, a library's product 385 to
// 391 us; with bias, GELU, residual and saved pre-activations, 350 MB more of
// traffic, 460 to 475 us); short ones the chain of launch, first loads, slices'
// meeting and stores (16 x 7168 -> 2048 14 us, of it 5 for the weights' bytes;
// 4096 x 7168 -> 256 fp32 27 us, of it 10 for the rows' bytes: the 96 CTAs that
// clusters of 6 leave busy have 18 MB in flight).
#include "common.cuh"
#include "kernels.h"
#include "linear.cuh"
#include "moe.h"

namespace moe {

namespace {

constexpr int BK = 64;
constexpr int A_BYTES = 128 * BK * 2;    // 16 KB: this CTA's 128 rows of P
constexpr int B_BYTES = 128 * BK * 2;    // 16 KB: this CTA's up to 128 rows of Q
constexpr int STAGE_BYTES = A_BYTES + B_BYTES;
// Epilogue warps, threads, stages and shared memory of the kernel's two forms.
template <bool CHAINED>
struct Form {
    static constexpr int kEpiWarps = CHAINED ? 16 : 8;
    static constexpr int kThreads = 64 + 32 * kEpiWarps;
    static constexpr int kStages = CHAINED ? 5 : 6;
    static constexpr int kTurnBytes = kEpiWarps * 32 * 32 * 4;
    static constexpr int kSmem = 1024 + kStages * STAGE_BYTES + kTurnBytes + 8 * (2 * kStages + 5) + 32;
    static_assert(kSmem <= 227 * 1024, "shared memory of a block");
};

struct TcParams {
    int32_t I, J;            // rows and columns of D
    int32_t i_tiles, tiles;
    int32_t slices;
    int32_t chains;          // of sums along k, each in an accumulator of its own (CHAINED)
    int32_t share;           // columns of a tile that a slice's CTA finishes, even
    int32_t kblocks;
    int32_t bn;              // columns of a tile and of the MMA: a multiple of 16 CG
    int32_t b_bytes;         // bytes of Q per CTA and stage
    int32_t act;
    int32_t swap;            // D is the output's transpose
    int32_t out_f32;
    int32_t vec;             // rows of every output start on 16-byte boundaries
    int32_t first_of_two, second_of_two;     // see LinearGemm
    lin::Epilogue ep;        // in terms of the output
    uint32_t *status;
};

// Descriptor of an operand tile whose own index is contiguous, as TMA stages it
// with the 128-byte swizzle: blocks of 64 of that index by 64 k, 8192 bytes
// each (the leading byte offset, from one block to the next); in a block the
// groups of 8 k are 1024 bytes apart (the stride byte offset).
__device__ __forceinline__ uint64_t sdesc_mnmajor_sw128(uint32_t saddr)
{
    uint64_t d = 0;
    d |= static_cast<uint64_t>((saddr >> 4) & 0x3FFFu);
    d |= static_cast<uint64_t>(8192u >> 4) << 16;
    d |= static_cast<uint64_t>(1024u >> 4) << 32;
    d |= static_cast<uint64_t>(1u) << 46;
    d |= static_cast<uint64_t>(2u) << 61;
    return d;
}

// Bits 15 and 16 of the instruction descriptor: A, B with their own index contiguous.
constexpr uint32_t kIdescTransA = 1u << 15, kIdescTransB = 1u << 16;

template <int ACT>
__device__ __forceinline__ void act_all(float (&v)[32])
{
#pragma unroll
    for (int i = 0; i < 32; ++i)
        v[i] = lin::act_fwd<ACT>(v[i]);
}

__device__ __forceinline__ void act32(int act, float (&v)[32])
{
    switch (act) {
    case MOE_LINEAR_RELU: act_all<MOE_LINEAR_RELU>(v); break;
    case MOE_LINEAR_SILU: act_all<MOE_LINEAR_SILU>(v); break;
    case MOE_LINEAR_GELU: act_all<MOE_LINEAR_GELU>(v); break;
    case MOE_LINEAR_GELU_TANH: act_all<MOE_LINEAR_GELU_TANH>(v); break;
    default: break;
    }
}

// n (a multiple of 8, at most 32) consecutive values of a row that starts on a
// 16-byte boundary.
__device__ __forceinline__ void store_run(void *base, int64_t at, bool f32, int n,
                                          const float (&v)[32])
{
#pragma unroll
    for (int i = 0; i < 32; i += 8) {
        if (i >= n)
            continue;
        if (f32) {
            float4 *p = reinterpret_cast<float4 *>(static_cast<float *>(base) + at + i);
            p[0] = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
            p[1] = make_float4(v[i + 4], v[i + 5], v[i + 6], v[i + 7]);
        } else {
            *reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(base) + at + i) =
                make_uint4(pack_bf16x2(v[i], v[i + 1]), pack_bf16x2(v[i + 2], v[i + 3]),
                           pack_bf16x2(v[i + 4], v[i + 5]), pack_bf16x2(v[i + 6], v[i + 7]));
        }
    }
}

// The same run of a row to registers (bf16: the first half of res), and its
// addition to v.
__device__ __forceinline__ void load_run(const void *base, int64_t at, bool f32, int n, uint4 (&res)[8])
{
    if (f32) {
        const uint4 *p = reinterpret_cast<const uint4 *>(static_cast<const float *>(base) + at);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            res[i] = 4 * i < n ? p[i] : make_uint4(0, 0, 0, 0);
    } else {
        const uint4 *p = reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(base) + at);
#pragma unroll
        for (int i = 0; i < 4; ++i)
            res[i] = 8 * i < n ? p[i] : make_uint4(0, 0, 0, 0);
    }
}

__device__ __forceinline__ void add_run(const uint4 (&res)[8], bool f32, int n, float (&v)[32])
{
    if (f32) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            v[4 * i] += __uint_as_float(res[i].x);
            v[4 * i + 1] += __uint_as_float(res[i].y);
            v[4 * i + 2] += __uint_as_float(res[i].z);
            v[4 * i + 3] += __uint_as_float(res[i].w);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t w[4] = {res[i].x, res[i].y, res[i].z, res[i].w};
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                v[8 * i + 2 * x] += __uint_as_float(w[x] << 16);
                v[8 * i + 2 * x + 1] += __uint_as_float(w[x] & 0xFFFF0000u);
            }
        }
    }
}

// v += n bias values, the same for every lane.
__device__ __forceinline__ void add_bias(const float *b, int n, float (&v)[32])
{
    if (n == 32 && reinterpret_cast<uintptr_t>(b) % 16 == 0) {
#pragma unroll
        for (int i = 0; i < 32; i += 4) {
            const float4 q = __ldg(reinterpret_cast<const float4 *>(b + i));
            v[i] += q.x;
            v[i + 1] += q.y;
            v[i + 2] += q.z;
            v[i + 3] += q.w;
        }
    } else {
#pragma unroll
        for (int i = 0; i < 32; ++i)
            if (i < n)
                v[i] += __ldg(b + i);
    }
}

__device__ __forceinline__ float load1(const void *base, int64_t at, bool f32)
{
    return f32 ? static_cast<const float *>(base)[at]
               : __bfloat162float(static_cast<const __nv_bfloat16 *>(base)[at]);
}

__device__ __forceinline__ void store1(void *base, int64_t at, bool f32, float v)
{
    if (f32)
        static_cast<float *>(base)[at] = v;
    else
        static_cast<__nv_bfloat16 *>(base)[at] = __float2bfloat16_rn(v);
}

// 32 values of this lane, as elements at + i * step, n of them: bias added.
__device__ __forceinline__ void finish_run(const TcParams &p, int64_t out, int64_t out_step,
                                           int64_t res, int64_t res_step, int64_t pre,
                                           int64_t pre_step, int n, float (&v)[32])
{
    const lin::Epilogue &ep = p.ep;
    if (ep.preact) {
#pragma unroll
        for (int i = 0; i < 32; ++i)
            if (i < n)
                store1(ep.preact, pre + i * pre_step, false, v[i]);
    }
    act32(p.act, v);
    if (ep.residual) {
#pragma unroll
        for (int i = 0; i < 32; ++i)
            if (i < n)
                v[i] += load1(ep.residual, res + i * res_step, p.out_f32);
    }
#pragma unroll
    for (int i = 0; i < 32; ++i)
        if (i < n)
            store1(ep.out, out + i * out_step, p.out_f32, v[i]);
}

// AHEAD: the residual's loads are on their way while the activation is computed
// (32 registers).
//
// One warp's 32 rows of D from row0 on (one per lane), nc (at most 32) columns
// from c0 on; st: 32 x 32 floats of this warp, an element (column i, row r) at
// 32 i + (r ^ i), so that neither order of access meets a bank twice.
template <bool AHEAD>
__device__ __forceinline__ void finish_block(const TcParams &p, float *st, int64_t row0, int c0,
                                             int nc, float (&v)[32])
{
    const int lane = threadIdx.x & 31;
    const lin::Epilogue &ep = p.ep;
    const int n = p.J - c0 < nc ? p.J - c0 : nc;
    const int64_t r = row0 + lane;
    if (p.swap) {
        // the lanes are consecutive columns of the output, the columns its rows
        if (r < p.I) {
            const float b = ep.bias ? __ldg(ep.bias + r) : 0.0f;
#pragma unroll
            for (int i = 0; i < 32; ++i)
                v[i] += b;
            finish_run(p, c0 * ep.ldo + r, ep.ldo, c0 * ep.ldr + r, ep.ldr,
                       static_cast<int64_t>(c0) * ep.cols + r, ep.cols, n, v);
        }
    } else if (p.vec && n % 8 == 0) {
        // every lane a piece of its own row, 16 bytes at a time
        if (r < p.I) {
            uint4 res[8];
            if (AHEAD && ep.residual)
                load_run(ep.residual, r * ep.ldr + c0, p.out_f32, n, res);
            if (ep.bias)
                add_bias(ep.bias + c0, n, v);
            if (ep.preact)
                store_run(ep.preact, r * ep.cols + c0, false, n, v);
            act32(p.act, v);
            if (!AHEAD && ep.residual)
                load_run(ep.residual, r * ep.ldr + c0, p.out_f32, n, res);
            if (ep.residual)
                add_run(res, p.out_f32, n, v);
            store_run(ep.out, r * ep.ldo + c0, p.out_f32, n, v);
        }
    } else {
        // turned over: the lanes hold consecutive columns, whatever their alignment
#pragma unroll
        for (int i = 0; i < 32; ++i)
            st[i * 32 + (lane ^ i)] = v[i];
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 32; ++i)
            v[i] = st[lane * 32 + (i ^ lane)];
        __syncwarp();
        if (lane < n) {
            const float b = ep.bias ? __ldg(ep.bias + c0 + lane) : 0.0f;
#pragma unroll
            for (int i = 0; i < 32; ++i)
                v[i] += b;
            const int rows = p.I - row0 < 32 ? static_cast<int>(p.I - row0) : 32;
            const int64_t col = c0 + lane;
            finish_run(p, row0 * ep.ldo + col, ep.ldo, row0 * ep.ldr + col, ep.ldr,
                       row0 * ep.cols + col, ep.cols, rows, v);
        }
    }
}

__device__ __forceinline__ void st_cluster_f32(uint32_t addr, float v)
{
    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}

template <int CG, bool P_MN, bool Q_MN, bool SLICED, bool CHAINED>
__global__ void __launch_bounds__(Form<CHAINED>::kThreads, 1)
    linear_tc_kernel(const __grid_constant__ CUtensorMap tmP,
                     const __grid_constant__ CUtensorMap tmQ, const TcParams p)
{
    static_assert(!(SLICED && CHAINED), "");
    constexpr int STAGES = Form<CHAINED>::kStages;
    constexpr int kEpiWarps = Form<CHAINED>::kEpiWarps;
    constexpr int TI = 128 * CG;             // tile rows
    constexpr int ACC = 128 * CG;            // TMEM columns of an accumulator
    constexpr int TMEM_COLS = 2 * ACC;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                                ~static_cast<uintptr_t>(1023));
    float *turn = reinterpret_cast<float *>(smem + STAGES * STAGE_BYTES);
    uint64_t *bars =
        reinterpret_cast<uint64_t *>(smem + STAGES * STAGE_BYTES + Form<CHAINED>::kTurnBytes);
    uint64_t *full = bars;
    uint64_t *empty = bars + STAGES;
    uint64_t *acc_full = bars + 2 * STAGES;
    uint64_t *acc_empty = bars + 2 * STAGES + 2;
    uint64_t *drain = bars + 2 * STAGES + 4;
    uint32_t *s_tmem = reinterpret_cast<uint32_t *>(bars + 2 * STAGES + 5);
    volatile int *s_abort = reinterpret_cast<volatile int *>(s_tmem + 1);

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const uint32_t crank = CG == 2 || SLICED ? cluster_ctarank() : 0u;
    const uint32_t rank = CG == 2 ? (crank & 1u) : 0u;       // in the pair
    const uint32_t lead = crank - rank;                      // the pair's first CTA
    const bool leader = rank == 0;
    const int slice = SLICED ? static_cast<int>(crank) / CG : 0;
    const int worker = blockIdx.x / (SLICED ? CG * p.slices : CG);
    const int workers = gridDim.x / (SLICED ? CG * p.slices : CG);
    const int kb_lo = SLICED ? static_cast<int>(static_cast<int64_t>(p.kblocks) * slice / p.slices) : 0;
    const int kb_hi = SLICED ? static_cast<int>(static_cast<int64_t>(p.kblocks) * (slice + 1) / p.slices)
                             : p.kblocks;
    const int kb_half = SLICED ? (kb_lo + kb_hi + 1) / 2 : kb_hi;   // from here on in accumulator 1
    const int tj = p.bn;                     // tile columns

    if (warp == 0 && lane == 0) {
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        for (int a = 0; a < 2; ++a) {
            mbar_init(&acc_full[a], 1);
            mbar_init(&acc_empty[a], CG * 32 * kEpiWarps);
        }
        mbar_init(drain, 1);
        *s_abort = 0;
        fence_barrier_init();
        tma_prefetch_desc(&tmP);
        tma_prefetch_desc(&tmQ);
    }
    if (warp == 1) {
        if (CG == 2) {
            tmem_alloc_pair(s_tmem, TMEM_COLS);
            tmem_relinquish_pair();
        } else {
            tmem_alloc(s_tmem, TMEM_COLS);
            tmem_relinquish();
        }
    }
    tc_fence_before();
    __syncthreads();
    if (CG == 2)
        cluster_sync_all();      // the peer's barriers exist before any remote arrive
    tc_fence_after();
    const uint32_t tmem_base = *s_tmem;
    if (!p.second_of_two)
        grid_dep_wait();
    if (p.first_of_two)
        grid_dep_launch();

    // consecutive tiles share their columns
    auto tile_at = [&](int u, int &i0, int &j0) {
        const int jt = u / p.i_tiles, it = u - jt * p.i_tiles;
        i0 = it * TI;
        j0 = jt * tj;
    };
    auto wait = [&](uint64_t *bar, uint32_t parity, volatile int *abort) {
        return CG == 2 ? mbar_wait_bounded_cluster(bar, parity, abort)
                       : mbar_wait_bounded(bar, parity, abort);
    };

    if (warp == 0) {
        if (lane == 0) {
            // ================= TMA producer (this CTA's rows of P and Q) =================
            int s = 0;
            uint32_t ph = 0, last_par = 0, used = 0;
            bool ok = true;
            const uint32_t bytes = CG * (A_BYTES + p.b_bytes);
            for (int u = worker; u < p.tiles && ok; u += workers) {
                int i0, j0;
                tile_at(u, i0, j0);
                i0 += static_cast<int>(rank) * 128;
                j0 += static_cast<int>(rank) * (tj / 2);
                for (int kb = kb_lo; kb < kb_hi; ++kb) {
                    if (!wait(&empty[s], ph ^ 1u, s_abort)) {
                        set_status(p.status, DEV_TIMEOUT_PRODUCER);
                        *s_abort = 1;
                        ok = false;
                        break;
                    }
                    uint8_t *sa = smem + s * STAGE_BYTES;
                    uint8_t *sb = sa + A_BYTES;
                    if (leader)
                        mbar_arrive_expect_tx(&full[s], bytes);
                    const uint32_t pbar = CG == 2 ? mapa_shared(smem_u32(&full[s]), lead) : 0u;
                    auto load = [&](uint8_t *dst, const CUtensorMap *m, int c0, int c1) {
                        if (CG == 2)
                            tma_load_2d_pairbar(dst, m, pbar, c0, c1);
                        else
                            tma_load_2d(dst, m, &full[s], c0, c1);
                    };
                    if (P_MN) {
                        load(sa, &tmP, i0, kb * BK);
                        load(sa + 8192, &tmP, i0 + 64, kb * BK);
                    } else {
                        load(sa, &tmP, kb * BK, i0);
                    }
                    if (Q_MN) {
                        for (int b = 0; b < p.b_bytes; b += 8192)
                            load(sb + b, &tmQ, j0 + b / 128, kb * BK);
                    } else {
                        load(sb, &tmQ, kb * BK, j0);
                    }
                    last_par = (last_par & ~(1u << s)) | (ph << s);
                    used |= 1u << s;
                    if (++s == STAGES) {
                        s = 0;
                        ph ^= 1u;
                    }
                }
            }
            // once the barriers that count the copies complete, none is in flight
            for (int i = 0; i < STAGES && leader; ++i) {
                if ((used >> i) & 1u) {
                    volatile int never = 0;
                    if (!wait(&full[i], (last_par >> i) & 1u, &never))
                        set_status(p.status, DEV_TIMEOUT_DRAIN);
                }
            }
        }
    } else if (warp == 1) {
        if (lane == 0 && leader) {
            // ================= MMA issuer =================
            const uint32_t idesc = idesc_bf16_f32(TI, p.bn) |
                                   (P_MN ? kIdescTransA : 0u) | (Q_MN ? kIdescTransB : 0u);
            int s = 0;
            uint32_t ph = 0;
            int it = 0;
            bool ok = true;
            const uint16_t both = static_cast<uint16_t>(0x3u << lead);
            for (int u = worker; u < p.tiles && ok; u += workers) {
                // a tile's k range in one chain of sums, or in p.chains of them, each
                // in the next accumulator
                for (int ch = 0; ch < (CHAINED ? p.chains : 1) && ok; ++ch, ++it) {
                    const int lo = CHAINED ? p.kblocks * ch / p.chains : kb_lo;
                    const int hi = CHAINED ? p.kblocks * (ch + 1) / p.chains : kb_hi;
                    const int a = it & 1;
                    const uint32_t aph = (it >> 1) & 1;
                    if (!wait(&acc_empty[a], aph ^ 1u, s_abort)) {
                        set_status(p.status, DEV_TIMEOUT_MMA);
                        *s_abort = 1;
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t d_tmem = tmem_base + a * ACC;        // a = 0 in a slice
                    for (int kb = lo; kb < hi; ++kb) {
                        if (!wait(&full[s], ph, s_abort)) {
                            set_status(p.status, DEV_TIMEOUT_MMA);
                            *s_abort = 1;
                            ok = false;
                            break;
                        }
                        tc_fence_after();
                        const uint32_t sa = smem_u32(smem + s * STAGE_BYTES);
                        const uint32_t sb = sa + A_BYTES;
#pragma unroll
                        for (int kk = 0; kk < BK / 16; ++kk) {
                            const uint64_t da = P_MN ? sdesc_mnmajor_sw128(sa + kk * 2048)
                                                     : sdesc_kmajor_sw128(sa + kk * 32);
                            const uint64_t db = Q_MN ? sdesc_mnmajor_sw128(sb + kk * 2048)
                                                     : sdesc_kmajor_sw128(sb + kk * 32);
                            const bool second = SLICED && kb >= kb_half;
                            const uint32_t d = second ? d_tmem + ACC : d_tmem;
                            const uint32_t add = (kb > (second ? kb_half : lo) || kk > 0) ? 1u : 0u;
                            if (CG == 2)
                                tc_mma_bf16_pair(d, da, db, idesc, add);
                            else
                                tc_mma_bf16(d, da, db, idesc, add);
                        }
                        if (CG == 2)
                            tc_commit_pair_mc(&empty[s], both);
                        else
                            tc_commit(&empty[s]);
                        if (++s == STAGES) {
                            s = 0;
                            ph ^= 1u;
                        }
                    }
                    if (ok) {
                        if (CG == 2)
                            tc_commit_pair_mc(&acc_full[a], both);
                        else
                            tc_commit(&acc_full[a]);
                    }
                }
            }
        }
    } else {
        // ================= epilogue (this CTA's 128 rows) =================
        const int q = warp & 3;                  // TMEM lanes of this warp
        const int half = (warp - 2) >> 2;
        float *st = turn + (warp - 2) * 32 * 32;
        const uint32_t lead_empty[2] = {
            CG == 2 ? mapa_shared(smem_u32(&acc_empty[0]), lead) : 0u,
            CG == 2 ? mapa_shared(smem_u32(&acc_empty[1]), lead) : 0u};
        int it = 0;
        auto acc_wait = [&](int a, uint32_t aph) {
            const bool got = wait(&acc_full[a], aph, s_abort);
            if (__all_sync(0xffffffffu, got)) {
                tc_fence_after();
                return true;
            }
            if (lane == 0) {
                set_status(p.status, DEV_TIMEOUT_EPILOGUE);
                *s_abort = 1;
            }
            return false;
        };
        auto acc_release = [&](int a) {
            tc_fence_before();
            if (CG == 2 && !leader)
                mbar_arrive_cluster(lead_empty[a]);
            else
                mbar_arrive(&acc_empty[a]);
        };
        const uint32_t lanes = static_cast<uint32_t>(q * 32) << 16;
        if (SLICED) {
            acc_wait(0, 0);                      // one tile; the slices meet below
        } else if (CHAINED) {
            // four warps per row quarter, up to 64 columns each: the chains' sums
            // are added up in registers
            constexpr int CW = CG * 32;
            for (int u = worker; u < p.tiles; u += workers) {
                int i0, j0;
                tile_at(u, i0, j0);
                const int64_t row0 = static_cast<int64_t>(i0) + rank * 128 + q * 32;
                float o[CW / 32][32];
                bool ok = true;
                for (int ch = 0; ch < p.chains && ok; ++ch, ++it) {
                    const int a = it & 1;
                    ok = acc_wait(a, (it >> 1) & 1);
                    if (!ok)
                        break;
#pragma unroll
                    for (int h = 0; h < CW / 16; ++h) {
                        const int c = half * CW + h * 16;
                        uint32_t v[16];
                        tmem_ld16(tmem_base + lanes + a * ACC + (c < tj ? c : 0), v);
                        tmem_wait_ld();
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            float &sum = o[h / 2][h % 2 * 16 + i];
                            sum = ch == 0 ? __uint_as_float(v[i]) : sum + __uint_as_float(v[i]);
                        }
                    }
                    acc_release(a);
                }
                if (!ok)
                    break;
#pragma unroll
                for (int h = 0; h < CW / 32; ++h) {
                    const int c = half * CW + h * 32;
                    if (c < tj && row0 < p.I && j0 + c < p.J)
                        finish_block<false>(p, st, row0, j0 + c, 32, o[h]);
                }
            }
        } else {
            for (int u = worker; u < p.tiles; u += workers, ++it) {
                int i0, j0;
                tile_at(u, i0, j0);
                const int a = it & 1;
                if (!acc_wait(a, (it >> 1) & 1))
                    break;
                const int64_t row0 = static_cast<int64_t>(i0) + rank * 128 + q * 32;
#pragma unroll 1
                for (int c = half * 32; c < tj; c += 64) {
                    if (row0 >= p.I || j0 + c >= p.J)
                        break;
                    uint32_t v[32];
                    float o[32];
                    tmem_ld32(tmem_base + lanes + a * ACC + c, v);
                    tmem_wait_ld();
#pragma unroll
                    for (int i = 0; i < 32; ++i)
                        o[i] = __uint_as_float(v[i]);
                    finish_block<true>(p, st, row0, j0 + c, 32, o);
                }
                acc_release(a);
            }
        }
    }

    if (SLICED) {
        // ================= the slices' sums meet =================
        // Every CTA of the cluster has finished its products, so the stages are
        // free; CTA s of the CTAs with this pair rank takes columns [s w, s w + w).
        // A CTA whose waits gave up takes part in the barriers all the same.
        int i0, j0;
        tile_at(worker, i0, j0);
        const int w = p.share;
        __syncwarp();
        cluster_sync_all();
        tc_fence_after();
        const int q = warp & 3;
        const int half = (warp - 2) >> 2;
        const int r_local = q * 32 + lane;
        const uint32_t recv = smem_u32(smem);    // [slice][w][128 rows] fp32
        const int n = p.J - j0 < tj ? p.J - j0 : tj;
        if (warp >= 2) {
            const uint32_t tacc = tmem_base + (static_cast<uint32_t>(q * 32) << 16);
#pragma unroll 1
            for (int c = half * 32; c < n; c += 64) {
                uint32_t v[32], v2[32];
                tmem_ld32(tacc + c, v);
                tmem_ld32(tacc + ACC + c, v2);
                tmem_wait_ld();
                const bool two = kb_hi > kb_half;
                int owner = c / w, at = c - owner * w;
                uint32_t to = mapa_shared(recv + ((slice * w + at) * 128 + r_local) * 4,
                                          owner * CG + rank);
#pragma unroll
                for (int i = 0; i < 32; ++i) {
                    if (c + i < n)
                        st_cluster_f32(to, __uint_as_float(v[i]) +
                                               (two ? __uint_as_float(v2[i]) : 0.0f));
                    to += 128 * 4;
                    if (++at == w && c + i + 1 < n) {
                        at = 0;
                        ++owner;
                        to = mapa_shared(recv + (slice * w * 128 + r_local) * 4, owner * CG + rank);
                    }
                }
            }
        }
        __syncwarp();
        cluster_sync_all();
        if (warp >= 2) {
            // this CTA's columns, half of them per warp of a row quarter
            const float *sum = reinterpret_cast<const float *>(smem);
            float *st = turn + (warp - 2) * 32 * 32;
            const int wh = w / 2 < 32 ? w / 2 : 32;
            const int64_t row0 = static_cast<int64_t>(i0) + rank * 128 + q * 32;
            for (int c = half * wh; c < w; c += 2 * wh) {
                const int col = slice * w + c;
                if (col >= n || row0 >= p.I)
                    break;
                // the last share may reach past the tile's columns
                int nc = w - c < wh ? w - c : wh;
                nc = n - col < nc ? n - col : nc;
                float o[32];
#pragma unroll
                for (int i = 0; i < 32; ++i)
                    o[i] = 0.0f;
                for (int s = 0; s < p.slices; ++s) {
#pragma unroll
                    for (int i = 0; i < 32; ++i)
                        if (i < nc)
                            o[i] += sum[(s * w + c + i) * 128 + r_local];
                }
                finish_block<true>(p, st, row0, j0 + col, nc, o);
            }
        }
    }

    // ---- teardown: MMAs complete, then TMEM is released
    __syncwarp();
    if (warp == 1 && lane == 0 && leader && *s_abort) {
        if (CG == 2)
            tc_commit_pair_mc(drain, static_cast<uint16_t>(1u << lead));
        else
            tc_commit(drain);
        volatile int never = 0;
        if (!mbar_wait_bounded(drain, 0, &never))
            set_status(p.status, DEV_TIMEOUT_DRAIN);
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (CG == 2)
        cluster_sync_all();
    tc_fence_after();
    if (warp == 1) {
        if (CG == 2)
            tmem_dealloc_pair(tmem_base, TMEM_COLS);
        else
            tmem_dealloc(tmem_base, TMEM_COLS);
    }
    if (p.second_of_two)
        grid_dep_wait();
}

typedef CUresult (*PFN_encode)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *,
                               const cuuint64_t *, const cuuint64_t *, const cuuint32_t *,
                               const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                               CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// Map of `outer` rows of `inner` contiguous bf16 elements, ld elements apart;
// boxes of 64 x box_rows.
bool make_map(CUtensorMap *m, const void *base, int64_t inner, int64_t outer, int64_t ld,
              int box_rows)
{
    static PFN_encode enc = [] {
        void *ptr = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &ptr, cudaEnableDefault, &q) !=
                cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            ptr = nullptr;
        return reinterpret_cast<PFN_encode>(ptr);
    }();
    if (!enc)
        return false;
    cuuint64_t dims[2] = {static_cast<cuuint64_t>(inner), static_cast<cuuint64_t>(outer)};
    cuuint64_t strides[1] = {static_cast<cuuint64_t>(ld) * 2};
    cuuint32_t box[2] = {64, static_cast<cuuint32_t>(box_rows)};
    cuuint32_t estr[2] = {1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void *>(base), dims, strides,
               box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) ==
           CUDA_SUCCESS;
}

template <int CG, bool P_MN, bool Q_MN, bool SLICED, bool CHAINED>
cudaError_t launch_tc(const TcParams &p, const CUtensorMap &mP, const CUtensorMap &mQ, int workers,
                      cudaStream_t stream)
{
    static DeviceOnce once;
    cudaError_t e = device_once(once, nullptr, [](int *) {
        return cudaFuncSetAttribute(linear_tc_kernel<CG, P_MN, Q_MN, SLICED, CHAINED>,
                                    cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    Form<CHAINED>::kSmem);
    });
    if (e != cudaSuccess)
        return e;
    const unsigned cluster = CG * p.slices;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.gridDim = dim3(cluster * static_cast<unsigned>(workers), 1, 1);
    cfg.blockDim = dim3(Form<CHAINED>::kThreads, 1, 1);
    cfg.dynamicSmemBytes = Form<CHAINED>::kSmem;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    e = cudaLaunchKernelEx(&cfg, linear_tc_kernel<CG, P_MN, Q_MN, SLICED, CHAINED>, mP, mQ, p);
    count_launches(1);
    return e;
}

template <int CG, bool P_MN, bool Q_MN>
cudaError_t launch_tc(const TcParams &p, const void *P, int64_t ldp, const void *Q, int64_t ldq,
                      int64_t K, int workers, cudaStream_t stream)
{
    CUtensorMap mP, mQ;
    const bool ok = (P_MN ? make_map(&mP, P, p.I, K, ldp, BK) : make_map(&mP, P, K, p.I, ldp, 128)) &&
                    (Q_MN ? make_map(&mQ, Q, p.J, K, ldq, BK)
                          : make_map(&mQ, Q, K, p.J, ldq, p.bn / CG));
    if (!ok)
        return cudaErrorInvalidValue;
    if (p.slices > 1)
        return launch_tc<CG, P_MN, Q_MN, true, false>(p, mP, mQ, workers, stream);
    if constexpr (!P_MN && !Q_MN)            // fp32 results: forward products only
        if (p.chains > 1)
            return launch_tc<CG, P_MN, Q_MN, false, true>(p, mP, mQ, workers, stream);
    return launch_tc<CG, P_MN, Q_MN, false, false>(p, mP, mQ, workers, stream);
}

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// How a product is cut up; see the file's head.
struct Plan {
    int cg;                  // CTAs per tile
    bool swap;               // the transposed product
    int bn;                  // tile columns
    int slices;              // of k per tile
    int chains;              // of sums along k per tile
    int64_t tiles;
};

Plan plan_of(int64_t I, int64_t J, int64_t K, bool may_swap, bool out_f32)
{
    constexpr int kSms = 148;
    Plan pl{};
    const int64_t kb = ceil_div(K, BK);
    pl.swap = may_swap && I <= 64 && J > I;
    const int64_t rows = pl.swap ? J : I, cols = pl.swap ? I : J;
    const int64_t pairs = ceil_div(rows, 256) * ceil_div(cols, 256);
    if (!pl.swap && rows > 128 && cols > 128 && (pairs >= kSms / 4 || kb * pairs >= kSms * 4)) {
        pl.cg = 2;
        pl.bn = 256;
        pl.tiles = pairs;
    } else {
        pl.cg = 1;
        pl.bn = static_cast<int>(cols >= 128 ? 128 : (cols + 15) / 16 * 16);
        pl.tiles = ceil_div(rows, 128) * ceil_div(cols, pl.bn);
    }
    // idle SMs take slices of k, of at least 2 blocks of 64, as long as all the
    // clusters run at once: the GPU holds this many of each size (with one CTA
    // per SM; not every SM has the neighbours that a cluster needs)
    constexpr int kHeld[9] = {0, 148, 74, 45, 33, 26, 22, 15, 15};
    const int most = 8 / pl.cg;
    pl.slices = 1;
    for (int n = 2; n <= most; ++n)
        if (pl.tiles <= kHeld[n * pl.cg] && kb >= n * 2)
            pl.slices = n;
    // fp32 results without slices: chains of at most 1280 of k
    pl.chains = out_f32 && pl.slices == 1 ? static_cast<int>(ceil_div(kb, 20)) : 1;
    return pl;
}

}  // namespace

cudaError_t launch_linear_tc(const LinearGemm &L, cudaStream_t stream)
{
    int sms = 148, dev = 0;
    if (cudaGetDevice(&dev) == cudaSuccess)
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    const Plan pl = plan_of(L.I, L.J, L.K, L.p_kmajor, L.out_f32);
    const bool sw = pl.swap;
    TcParams p{};
    p.I = static_cast<int32_t>(sw ? L.J : L.I);
    p.J = static_cast<int32_t>(sw ? L.I : L.J);
    p.i_tiles = static_cast<int32_t>(ceil_div(p.I, 128 * pl.cg));
    if (pl.tiles * pl.cg * pl.slices > 0x7FFFFFFF)
        return cudaErrorInvalidValue;
    p.tiles = static_cast<int32_t>(pl.tiles);
    p.slices = pl.slices;
    p.chains = pl.chains;
    // shares in whole 16-byte pieces of a row, twice (two warps); transposed: of any size
    const int unit = sw ? 2 : 16;
    p.share = static_cast<int32_t>(ceil_div(ceil_div(pl.bn, pl.slices), unit) * unit);
    p.kblocks = static_cast<int32_t>(ceil_div(L.K, BK));
    const bool q_mn = sw ? !L.p_kmajor : !L.q_kmajor;
    const bool p_mn = sw ? !L.q_kmajor : !L.p_kmajor;
    p.bn = pl.bn;
    const int bc = p.bn / pl.cg;             // columns per CTA
    p.b_bytes = q_mn ? static_cast<int32_t>(ceil_div(bc, 64)) * 8192 : bc * BK * 2;
    p.act = L.act;
    p.swap = sw;
    p.out_f32 = L.out_f32;
    const int os = L.out_f32 ? 4 : 2;
    auto on16 = [](const void *ptr, int64_t row_bytes) {
        return reinterpret_cast<uintptr_t>(ptr) % 16 == 0 && row_bytes % 16 == 0;
    };
    p.vec = on16(L.out, L.ldo * os) && (!L.residual || on16(L.residual, L.ldr * os)) &&
            (!L.preact || on16(L.preact, L.J * 2ll));
    p.ep.out = L.out;
    p.ep.ldo = L.ldo;
    p.ep.bias = L.bias;
    p.ep.residual = L.residual;
    p.ep.ldr = L.ldr;
    p.ep.preact = L.preact;
    p.ep.cols = L.J;
    p.status = L.status;
    p.first_of_two = L.first_of_two;
    p.second_of_two = L.second_of_two;
    const void *P = sw ? L.Q : L.P, *Q = sw ? L.P : L.Q;
    const int64_t ldp = sw ? L.ldq : L.ldp, ldq = sw ? L.ldp : L.ldq;
    // a cluster of slices takes one tile; without slices the CTAs (pairs) stay
    const int64_t cap = pl.slices > 1 ? pl.tiles : sms / pl.cg;
    const int workers = static_cast<int>(pl.tiles < cap ? pl.tiles : cap);
    if (pl.cg == 2) {
        if (p_mn)
            return q_mn ? launch_tc<2, true, true>(p, P, ldp, Q, ldq, L.K, workers, stream)
                        : cudaErrorInvalidValue;
        return q_mn ? launch_tc<2, false, true>(p, P, ldp, Q, ldq, L.K, workers, stream)
                    : launch_tc<2, false, false>(p, P, ldp, Q, ldq, L.K, workers, stream);
    }
    if (p_mn)
        return q_mn ? launch_tc<1, true, true>(p, P, ldp, Q, ldq, L.K, workers, stream)
                    : launch_tc<1, true, false>(p, P, ldp, Q, ldq, L.K, workers, stream);
    return q_mn ? launch_tc<1, false, true>(p, P, ldp, Q, ldq, L.K, workers, stream)
                : launch_tc<1, false, false>(p, P, ldp, Q, ldq, L.K, workers, stream);
}

}  // namespace moe
