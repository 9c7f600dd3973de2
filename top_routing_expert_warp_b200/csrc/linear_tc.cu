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
// A unit of work is a tile, or one of `splits` slices of a tile's k range:
//   CG = 2: 256 x 256 on a CTA pair (cta_group::2, each CTA stages 128 rows of
//           P and 128 of Q), for large products: per SM a 64-wide k block
//           brings 32 KB for 256 cycles of tensor work;
//   CG = 1: 128 x up to 128 on one CTA, for small ones.
// With few rows (serving) the product is taken transposed: P is the weights
// (128 of them are the MMA's rows) and Q the tokens (rounded up to 16 as the
// MMA's columns), so the weights are read once at the rate of HBM and no MMA
// is spent on absent tokens.
// Slices of one tile leave fp32 partial tiles in the workspace; the last one to
// finish (a ticket per tile, which wraps to 0 by itself) adds them in slice
// order, so the result does not depend on which was last.
//
// Roles: warp 0 TMA producer, warp 1 MMA issuer, warps 2-9 epilogue (two per
// TMEM lane quarter, on alternate 32-column steps).  Two accumulators in TMEM:
// the epilogue of a tile overlaps the products of the next.  Every wait is
// bounded.
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
constexpr int STAGES = 6;
constexpr int kEpiWarps = 8;
constexpr int kThreads = 64 + 32 * kEpiWarps;
constexpr int AUX_BYTES = 8 * (2 * STAGES + 5) + 32;
constexpr int SMEM_BYTES = 1024 + STAGES * STAGE_BYTES + AUX_BYTES;

struct TcParams {
    int32_t I, J;            // rows and columns of D
    int32_t i_tiles, j_tiles;
    int32_t units, splits;
    int32_t kblocks;
    int32_t bn;              // columns of the MMA (CG = 1), multiple of 16
    int32_t b_bytes;         // bytes of Q per CTA and stage
    int32_t act;
    int32_t swap;            // D is the output's transpose
    int32_t out_f32, out_vec, res_vec, pre_vec;
    lin::Epilogue ep;        // in terms of the output
    float *part;             // [units][CG][128 CG columns][128 rows]
    uint32_t *tickets;       // [tiles][CG], zero between launches
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

__device__ __forceinline__ void act32(int act, float (&v)[32])
{
#define MOE_ACT32(A)                          \
    _Pragma("unroll") for (int i = 0; i < 32; ++i) v[i] = lin::act_fwd<A>(v[i]);
    switch (act) {
    case MOE_LINEAR_RELU: MOE_ACT32(MOE_LINEAR_RELU) break;
    case MOE_LINEAR_SILU: MOE_ACT32(MOE_LINEAR_SILU) break;
    case MOE_LINEAR_GELU: MOE_ACT32(MOE_LINEAR_GELU) break;
    case MOE_LINEAR_GELU_TANH: MOE_ACT32(MOE_LINEAR_GELU_TANH) break;
    default: break;
    }
#undef MOE_ACT32
}

// 32 consecutive values of a row to bf16 or fp32.
__device__ __forceinline__ void store32(void *base, int64_t at, bool f32, bool vec, int n,
                                        const float (&v)[32])
{
    if (f32) {
        float *p = static_cast<float *>(base) + at;
        if (vec && n == 32) {
#pragma unroll
            for (int i = 0; i < 32; i += 4)
                *reinterpret_cast<float4 *>(p + i) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
        } else {
#pragma unroll
            for (int i = 0; i < 32; ++i)
                if (i < n)
                    p[i] = v[i];
        }
    } else {
        __nv_bfloat16 *p = static_cast<__nv_bfloat16 *>(base) + at;
        if (vec && n == 32) {
#pragma unroll
            for (int i = 0; i < 32; i += 8) {
                uint4 w;
                w.x = pack_bf16x2(v[i], v[i + 1]);
                w.y = pack_bf16x2(v[i + 2], v[i + 3]);
                w.z = pack_bf16x2(v[i + 4], v[i + 5]);
                w.w = pack_bf16x2(v[i + 6], v[i + 7]);
                *reinterpret_cast<uint4 *>(p + i) = w;
            }
        } else {
#pragma unroll
            for (int i = 0; i < 32; ++i)
                if (i < n)
                    p[i] = __float2bfloat16_rn(v[i]);
        }
    }
}

// v += 32 consecutive values of a row.
__device__ __forceinline__ void add32(const void *base, int64_t at, bool f32, bool vec, int n,
                                      float (&v)[32])
{
    if (f32) {
        const float *p = static_cast<const float *>(base) + at;
        if (vec && n == 32) {
#pragma unroll
            for (int i = 0; i < 32; i += 4) {
                const float4 w = *reinterpret_cast<const float4 *>(p + i);
                v[i] += w.x;
                v[i + 1] += w.y;
                v[i + 2] += w.z;
                v[i + 3] += w.w;
            }
        } else {
#pragma unroll
            for (int i = 0; i < 32; ++i)
                if (i < n)
                    v[i] += p[i];
        }
    } else {
        const __nv_bfloat16 *p = static_cast<const __nv_bfloat16 *>(base) + at;
        if (vec && n == 32) {
#pragma unroll
            for (int i = 0; i < 32; i += 8) {
                const uint4 q = *reinterpret_cast<const uint4 *>(p + i);
                const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    v[i + 2 * x] += __uint_as_float(w[x] << 16);
                    v[i + 2 * x + 1] += __uint_as_float(w[x] & 0xFFFF0000u);
                }
            }
        } else {
#pragma unroll
            for (int i = 0; i < 32; ++i)
                if (i < n)
                    v[i] += __bfloat162float(p[i]);
        }
    }
}

// One thread's 32 accumulators (row r of D, columns c0..) to the output.
__device__ __forceinline__ void finish32(const TcParams &p, int64_t r, int c0, float (&v)[32])
{
    const lin::Epilogue &ep = p.ep;
    if (r >= p.I || c0 >= p.J)
        return;
    const int n = p.J - c0 < 32 ? p.J - c0 : 32;
    if (!p.swap) {
        if (ep.bias) {
#pragma unroll
            for (int i = 0; i < 32; ++i)
                if (i < n)
                    v[i] += __ldg(ep.bias + c0 + i);
        }
        if (ep.preact)
            store32(ep.preact, r * ep.cols + c0, false, p.pre_vec, n, v);
        act32(p.act, v);
        if (ep.residual)
            add32(ep.residual, r * ep.ldr + c0, p.out_f32, p.res_vec, n, v);
        store32(ep.out, r * ep.ldo + c0, p.out_f32, p.out_vec, n, v);
    } else {
        // r is the output's column (consecutive over the lanes), c0 + i its row
        const float b = ep.bias ? __ldg(ep.bias + r) : 0.0f;
#pragma unroll
        for (int i = 0; i < 32; ++i)
            v[i] += b;
        if (ep.preact) {
#pragma unroll
            for (int i = 0; i < 32; ++i)
                if (i < n)
                    static_cast<__nv_bfloat16 *>(ep.preact)[static_cast<int64_t>(c0 + i) * ep.cols + r] =
                        __float2bfloat16_rn(v[i]);
        }
        act32(p.act, v);
#pragma unroll
        for (int i = 0; i < 32; ++i) {
            if (i >= n)
                continue;
            const int64_t row = c0 + i;
            if (p.out_f32) {
                if (ep.residual)
                    v[i] += static_cast<const float *>(ep.residual)[row * ep.ldr + r];
                static_cast<float *>(ep.out)[row * ep.ldo + r] = v[i];
            } else {
                if (ep.residual)
                    v[i] += __bfloat162float(
                        static_cast<const __nv_bfloat16 *>(ep.residual)[row * ep.ldr + r]);
                static_cast<__nv_bfloat16 *>(ep.out)[row * ep.ldo + r] = __float2bfloat16_rn(v[i]);
            }
        }
    }
}

__device__ __forceinline__ void epi_barrier()
{
    asm volatile("bar.sync 1, %0;" ::"n"(32 * kEpiWarps) : "memory");
}

template <int CG, bool P_MN, bool Q_MN>
__global__ void __launch_bounds__(kThreads, 1)
    linear_tc_kernel(const __grid_constant__ CUtensorMap tmP,
                     const __grid_constant__ CUtensorMap tmQ, const TcParams p)
{
    constexpr int TI = 128 * CG;             // tile rows
    constexpr int ACC = 128 * CG;            // TMEM columns of an accumulator
    constexpr int TMEM_COLS = 2 * ACC;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                                ~static_cast<uintptr_t>(1023));
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + STAGES * STAGE_BYTES);
    uint64_t *full = bars;
    uint64_t *empty = bars + STAGES;
    uint64_t *acc_full = bars + 2 * STAGES;
    uint64_t *acc_empty = bars + 2 * STAGES + 2;
    uint64_t *drain = bars + 2 * STAGES + 4;
    uint32_t *s_tmem = reinterpret_cast<uint32_t *>(bars + 2 * STAGES + 5);
    volatile int *s_abort = reinterpret_cast<volatile int *>(s_tmem + 1);
    volatile uint32_t *s_last = reinterpret_cast<volatile uint32_t *>(s_tmem + 2);

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const uint32_t rank = CG == 2 ? cluster_ctarank() : 0u;
    const bool leader = rank == 0;
    const int worker = blockIdx.x / CG;
    const int workers = gridDim.x / CG;
    const int tj = CG == 2 ? 256 : p.bn;     // tile columns

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
    grid_dep_wait();

    // unit u: slice u % splits of tile u / splits; consecutive tiles share their columns
    auto unit_at = [&](int u, int &i0, int &j0, int &kb0, int &kb1) {
        const int tile = u / p.splits, s = u - tile * p.splits;
        const int jt = tile / p.i_tiles, it = tile - jt * p.i_tiles;
        i0 = it * TI;
        j0 = jt * tj;
        kb0 = static_cast<int>(static_cast<int64_t>(p.kblocks) * s / p.splits);
        kb1 = static_cast<int>(static_cast<int64_t>(p.kblocks) * (s + 1) / p.splits);
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
            for (int u = worker; u < p.units && ok; u += workers) {
                int i0, j0, kb0, kb1;
                unit_at(u, i0, j0, kb0, kb1);
                i0 += static_cast<int>(rank) * 128;
                j0 += static_cast<int>(rank) * 128;
                for (int kb = kb0; kb < kb1; ++kb) {
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
                    const uint32_t pbar = CG == 2 ? mapa_shared(smem_u32(&full[s]), 0) : 0u;
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
            const uint32_t idesc = idesc_bf16_f32(TI, CG == 2 ? 256 : p.bn) |
                                   (P_MN ? kIdescTransA : 0u) | (Q_MN ? kIdescTransB : 0u);
            int s = 0;
            uint32_t ph = 0;
            int it = 0;
            bool ok = true;
            for (int u = worker; u < p.units && ok; u += workers, ++it) {
                int i0, j0, kb0, kb1;
                unit_at(u, i0, j0, kb0, kb1);
                const int a = it & 1;
                const uint32_t aph = (it >> 1) & 1;
                if (!wait(&acc_empty[a], aph ^ 1u, s_abort)) {
                    set_status(p.status, DEV_TIMEOUT_MMA);
                    *s_abort = 1;
                    break;
                }
                tc_fence_after();
                const uint32_t d_tmem = tmem_base + a * ACC;
                for (int kb = kb0; kb < kb1; ++kb) {
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
                        const uint32_t add = (kb > kb0 || kk > 0) ? 1u : 0u;
                        if (CG == 2)
                            tc_mma_bf16_pair(d_tmem, da, db, idesc, add);
                        else
                            tc_mma_bf16(d_tmem, da, db, idesc, add);
                    }
                    if (CG == 2)
                        tc_commit_pair_mc(&empty[s], 0x3);
                    else
                        tc_commit(&empty[s]);
                    if (++s == STAGES) {
                        s = 0;
                        ph ^= 1u;
                    }
                }
                if (ok) {
                    if (CG == 2)
                        tc_commit_pair_mc(&acc_full[a], 0x3);
                    else
                        tc_commit(&acc_full[a]);
                }
            }
        }
    } else {
        // ================= epilogue (this CTA's 128 rows) =================
        const int q = warp & 3;                  // TMEM lanes of this warp
        const int half = (warp - 2) >> 2;
        const int r_local = q * 32 + lane;
        const uint32_t leader_empty[2] = {
            CG == 2 ? mapa_shared(smem_u32(&acc_empty[0]), 0) : 0u,
            CG == 2 ? mapa_shared(smem_u32(&acc_empty[1]), 0) : 0u};
        int it = 0;
        for (int u = worker; u < p.units; u += workers, ++it) {
            int i0, j0, kb0, kb1;
            unit_at(u, i0, j0, kb0, kb1);
            const int a = it & 1;
            const uint32_t aph = (it >> 1) & 1;
            bool got = wait(&acc_full[a], aph, s_abort);
            got = __all_sync(0xffffffffu, got);
            if (!got && lane == 0) {
                set_status(p.status, DEV_TIMEOUT_EPILOGUE);
                *s_abort = 1;
            }
            if (!got && p.splits == 1)
                break;
            tc_fence_after();
            const uint32_t tacc = tmem_base + (static_cast<uint32_t>(q * 32) << 16) + a * ACC;
            const int64_t row = static_cast<int64_t>(i0) + rank * 128 + r_local;
            if (p.splits == 1) {
#pragma unroll 1
                for (int c = half * 32; c < tj; c += 64) {
                    uint32_t v[32];
                    float o[32];
                    tmem_ld32(tacc + c, v);
                    tmem_wait_ld();
#pragma unroll
                    for (int i = 0; i < 32; ++i)
                        o[i] = __uint_as_float(v[i]);
                    finish32(p, row, j0 + c, o);
                }
            } else {
                // leave the partial tile; the last slice adds them up
                float *mine = p.part + (static_cast<int64_t>(u) * CG + rank) * (ACC * 128);
#pragma unroll 1
                for (int c = half * 32; c < tj && got; c += 64) {
                    uint32_t v[32];
                    tmem_ld32(tacc + c, v);
                    tmem_wait_ld();
                    const int n = p.J - (j0 + c);        // columns that exist
                    if (n >= 32) {
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            __stcg(mine + (c + i) * 128 + r_local, __uint_as_float(v[i]));
                    } else {
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            if (i < n)
                                __stcg(mine + (c + i) * 128 + r_local, __uint_as_float(v[i]));
                    }
                }
                const int tile = u / p.splits;
                __threadfence();
                epi_barrier();
                if (threadIdx.x == 64) {
                    // every slice arrives, after a wait that gave up too, so the
                    // ticket always comes back to 0
                    *s_last = atomicInc(p.tickets + tile * CG + rank, p.splits - 1) ==
                              static_cast<uint32_t>(p.splits - 1);
                    __threadfence();
                }
                epi_barrier();
                if (*s_last && got) {
                    const float *first = p.part + (static_cast<int64_t>(tile) * p.splits * CG + rank) *
                                                      (ACC * 128);
#pragma unroll 1
                    for (int c = half * 32; c < tj; c += 64) {
                        float o[32];
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            o[i] = 0.0f;
                        const int n = p.J - (j0 + c);
                        const float *src = first + c * 128 + r_local;
                        if (n >= 32) {
                            for (int s = 0; s < p.splits; ++s, src += CG * (ACC * 128)) {
#pragma unroll
                                for (int i = 0; i < 32; ++i)
                                    o[i] += __ldcg(src + i * 128);
                            }
                        } else {
                            // few columns: the loads of the slices in flight together
#pragma unroll
                            for (int i = 0; i < 32; ++i)
                                if (i < n) {
#pragma unroll 8
                                    for (int s = 0; s < p.splits; ++s)
                                        o[i] += __ldcg(src + i * 128 + s * (CG * (ACC * 128)));
                                }
                        }
                        finish32(p, row, j0 + c, o);
                    }
                }
                if (!got)
                    break;
            }
            tc_fence_before();
            if (CG == 2 && !leader)
                mbar_arrive_cluster(leader_empty[a]);
            else
                mbar_arrive(&acc_empty[a]);
        }
    }

    // ---- teardown: MMAs complete, then TMEM is released
    __syncwarp();
    if (warp == 1 && lane == 0 && leader && *s_abort) {
        if (CG == 2)
            tc_commit_pair_mc(drain, 0x1);
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

template <int CG, bool P_MN, bool Q_MN>
cudaError_t launch_tc(const TcParams &p, const void *P, int64_t ldp, const void *Q, int64_t ldq,
                      int64_t K, int workers, cudaStream_t stream)
{
    CUtensorMap mP, mQ;
    const bool ok = (P_MN ? make_map(&mP, P, p.I, K, ldp, BK) : make_map(&mP, P, K, p.I, ldp, 128)) &&
                    (Q_MN ? make_map(&mQ, Q, p.J, K, ldq, BK)
                          : make_map(&mQ, Q, K, p.J, ldq, CG == 2 ? 128 : p.bn));
    if (!ok)
        return cudaErrorInvalidValue;
    static DeviceOnce once;
    cudaError_t e = device_once(once, nullptr, [](int *) {
        return cudaFuncSetAttribute(linear_tc_kernel<CG, P_MN, Q_MN>,
                                    cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM_BYTES);
    });
    if (e != cudaSuccess)
        return e;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = CG;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.gridDim = dim3(static_cast<unsigned>(CG * workers), 1, 1);
    cfg.blockDim = dim3(kThreads, 1, 1);
    cfg.dynamicSmemBytes = SMEM_BYTES;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = CG == 2 ? 2 : 1;
    e = cudaLaunchKernelEx(&cfg, linear_tc_kernel<CG, P_MN, Q_MN>, mP, mQ, p);
    count_launches(1);
    return e;
}

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

}  // namespace

// How a product is cut up; see the file's head.
LinearPlan linear_plan(int64_t I, int64_t J, int64_t K, bool may_swap)
{
    constexpr int kSms = 148;
    LinearPlan pl{};
    const int64_t kb = ceil_div(K, BK);
    pl.swap = may_swap && I <= 64 && J > I;
    const int64_t rows = pl.swap ? J : I, cols = pl.swap ? I : J;
    int64_t tiles;
    const int64_t pairs = ceil_div(rows, 256) * ceil_div(cols, 256);
    if (!pl.swap && rows > 128 && cols > 128 && (pairs >= kSms / 4 || kb * pairs >= kSms * 4)) {
        pl.cg = 2;
        pl.bn = 256;
        tiles = pairs;
    } else {
        pl.cg = 1;
        pl.bn = static_cast<int>(cols >= 128 ? 128 : (cols + 15) / 16 * 16);
        tiles = ceil_div(rows, 128) * ceil_div(cols, pl.bn);
    }
    // idle SMs take slices of k, of at least 4 blocks of 64
    int64_t s = kSms / (tiles * pl.cg);
    if (s > kb / 4)
        s = kb / 4;
    pl.splits = static_cast<int>(s < 1 ? 1 : s);
    pl.tiles = tiles;
    return pl;
}

size_t linear_plan_part_bytes(const LinearPlan &pl)
{
    return pl.splits > 1 ? static_cast<size_t>(pl.tiles) * pl.splits * pl.cg * (128 * pl.cg) * 128 * 4
                         : 0;
}

cudaError_t launch_linear_tc(const LinearGemm &L, cudaStream_t stream)
{
    int sms = 148, dev = 0;
    if (cudaGetDevice(&dev) == cudaSuccess)
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    const LinearPlan pl = linear_plan(L.I, L.J, L.K, L.p_kmajor);
    const bool sw = pl.swap;
    TcParams p{};
    p.I = static_cast<int32_t>(sw ? L.J : L.I);
    p.J = static_cast<int32_t>(sw ? L.I : L.J);
    p.i_tiles = static_cast<int32_t>(ceil_div(p.I, 128 * pl.cg));
    p.j_tiles = static_cast<int32_t>(ceil_div(p.J, pl.bn));
    p.splits = pl.splits;
    const int64_t units = static_cast<int64_t>(p.i_tiles) * p.j_tiles * p.splits;
    if (units > 0x7FFFFFFF)
        return cudaErrorInvalidValue;
    p.units = static_cast<int32_t>(units);
    p.kblocks = static_cast<int32_t>(ceil_div(L.K, BK));
    const bool q_mn = sw ? !L.p_kmajor : !L.q_kmajor;
    const bool p_mn = sw ? !L.q_kmajor : !L.p_kmajor;
    p.bn = pl.bn;
    if (q_mn && pl.cg == 1)
        p.bn = pl.bn;
    p.b_bytes = pl.cg == 2 ? B_BYTES : (q_mn ? static_cast<int32_t>(ceil_div(p.bn, 64)) * 8192
                                             : p.bn * BK * 2);
    p.act = L.act;
    p.swap = sw;
    p.out_f32 = L.out_f32;
    const int os = L.out_f32 ? 4 : 2;
    auto vec = [](const void *ptr, int64_t ld, int es) {
        return reinterpret_cast<uintptr_t>(ptr) % 16 == 0 && (ld * es) % 16 == 0;
    };
    p.out_vec = vec(L.out, L.ldo, os);
    p.res_vec = vec(L.residual, L.ldr, os);
    p.pre_vec = vec(L.preact, L.J, 2);
    p.ep.out = L.out;
    p.ep.ldo = L.ldo;
    p.ep.bias = L.bias;
    p.ep.residual = L.residual;
    p.ep.ldr = L.ldr;
    p.ep.preact = L.preact;
    p.ep.rows = static_cast<int32_t>(L.I);
    p.ep.cols = L.J;
    p.part = L.part;
    p.tickets = L.tickets;
    p.status = L.status;
    const void *P = sw ? L.Q : L.P, *Q = sw ? L.P : L.Q;
    const int64_t ldp = sw ? L.ldq : L.ldp, ldq = sw ? L.ldp : L.ldq;
    // slices: one unit per worker, so that a launch that gave up leaves no ticket behind
    const int64_t cap = p.splits > 1 ? units : sms / pl.cg;
    const int workers = static_cast<int>(units < cap ? units : cap);
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
