// sq_mx4_gemm.cuh -- the microscaled 4-bit product for many tokens on CTA pairs
// (tcgen05.mma cta_group::2, kind::mxf4).
//
//   y[m, n] = sum_k x[m, k] w[n, k], x and w the values that codes and scales
//   stand for; fp32 accumulation, one rounding to y's type
//
// An output tile is 256 tokens x BN channels.  CTA r of a pair loads rows
// [m0 + 128 r, +128) of x and rows [n0 + r BN/2, +BN/2) of w with plain TMA,
// and the scale tiles of its own x rows and of all BN rows of w (each SM's
// tensor core applies the scales of every column of its 128 rows).  The pair's
// first CTA copies both CTAs' scale tiles into TMEM columns that belong to the
// stage and issues the MMAs.  No scale is left for the epilogue: it rounds and
// stores.
//
// TMEM (512 columns): the accumulators and 8 + 16 columns of scales a stage.
// BN = 192 and 128 fit two accumulators, so the epilogue of one tile overlaps
// the main loop of the next.  BN = 256 (a quarter less operand traffic a
// product than 192) fits one; its epilogue hands the columns back in eight
// parts and the next tile's main loop starts when all are read.
#pragma once

#include <cstdint>
#include <cuda.h>
#include <cuda_bf16.h>

#include "sq_gemm_pair.cuh"
#include "sq_mx4_stream.cuh"
#include "sq_ptx.cuh"

namespace sq {

template <int BN>
struct Mx4PairCfg {
    static constexpr int A_BYTES = 128 * 128;
    static constexpr int B_BYTES = (BN / 2) * 128;
    static constexpr int SA_BYTES = 2 * kMx4TileBytes;                    // 128 rows
    static constexpr int RT_B = BN > 128 ? 2 : 1;                         // row tiles that BN rows touch
    static constexpr int SB_BYTES = RT_B * 2 * kMx4TileBytes;
    static constexpr int STAGE_BYTES = A_BYTES + B_BYTES + SA_BYTES + SB_BYTES;
    static constexpr int SCALE_COLS = 8 + 8 * RT_B;
    static constexpr int NACC = BN == 256 ? 1 : 2;
    static constexpr int FIT_TMEM = (512 - NACC * BN) / SCALE_COLS;
    static constexpr int FIT_SMEM = (232448 - 1024 - 256) / STAGE_BYTES;
    static constexpr int STAGES = FIT_TMEM < FIT_SMEM ? FIT_TMEM : FIT_SMEM;
    static constexpr int TMEM_COLS = 512;
    static constexpr int NUM_BARS = 2 * STAGES + 5;  // full, empty, tfull[2], tempty[2], drain
    static constexpr int SMEM_BYTES = 1024 + STAGES * STAGE_BYTES + NUM_BARS * 8 + 16;
    static_assert(BN == 128 || BN == 192 || BN == 256, "tile width");
    static_assert(STAGES >= 4 && SMEM_BYTES <= 232448, "ring");
    static_assert(NACC * BN + STAGES * SCALE_COLS <= TMEM_COLS, "TMEM");
};

// 32 consecutive outputs of one row (16 where N ends)
template <int OUT>
__device__ __forceinline__ void mx4_store_row(const uint32_t (&r)[32], int n0, int N, void *__restrict__ y, int64_t m)
{
    const int valid = min(32, N - n0);  // 32 or 16 (N % 16 == 0)
    if constexpr (OUT == OUT_F32) {
        uint4 *dst = reinterpret_cast<uint4 *>(reinterpret_cast<float *>(y) + m * N + n0);
#pragma unroll
        for (int v = 0; v < 8; ++v)
            if (v * 4 < valid)
                dst[v] = make_uint4(r[4 * v], r[4 * v + 1], r[4 * v + 2], r[4 * v + 3]);
    } else {
        uint4 *dst = reinterpret_cast<uint4 *>(reinterpret_cast<__nv_bfloat16 *>(y) + m * N + n0);
        uint32_t p[16];
#pragma unroll
        for (int j = 0; j < 16; ++j) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(__uint_as_float(r[2 * j]), __uint_as_float(r[2 * j + 1]));
            p[j] = *reinterpret_cast<const uint32_t *>(&h);
        }
#pragma unroll
        for (int v = 0; v < 4; ++v)
            if (v * 8 < valid)
                dst[v] = make_uint4(p[4 * v], p[4 * v + 1], p[4 * v + 2], p[4 * v + 3]);
    }
}

template <int BN, int OUT>
__global__ void __launch_bounds__(kPairThreads, 1)
    mx4_pair_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmSA,
                    const __grid_constant__ CUtensorMap tmB, const __grid_constant__ CUtensorMap tmSB,
                    void *__restrict__ y, int M, int N, int K, int group_m)
{
    using Cfg = Mx4PairCfg<BN>;
    constexpr int STAGES = Cfg::STAGES;
    if (threadIdx.x == 0) {
        tma_prefetch_desc(&tmA);
        tma_prefetch_desc(&tmSA);
        tma_prefetch_desc(&tmB);
        tma_prefetch_desc(&tmSB);
    }
    pdl_prologue();
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    uint8_t *gbase = smem_raw + (base - raw);
    const uint32_t sA = base;
    const uint32_t sB = sA + STAGES * Cfg::A_BYTES;
    const uint32_t sSA = sB + STAGES * Cfg::B_BYTES;
    const uint32_t sSB = sSA + STAGES * Cfg::SA_BYTES;
    const uint32_t sBar = sSB + STAGES * Cfg::SB_BYTES;
    auto full_bar = [&](int s) { return sBar + 8u * s; };
    auto empty_bar = [&](int s) { return sBar + 8u * (STAGES + s); };
    auto tfull_bar = [&](int b) { return sBar + 8u * (2 * STAGES + b); };
    auto tempty_bar = [&](int b) { return sBar + 8u * (2 * STAGES + 2 + b); };
    const uint32_t drain_bar = sBar + 8u * (2 * STAGES + 4);
    const uint32_t slot_off = (sBar - base) + 8u * Cfg::NUM_BARS;
    volatile uint32_t *tmem_slot = reinterpret_cast<volatile uint32_t *>(gbase + slot_off);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(gbase + slot_off + 4);

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const uint32_t rank = cluster_ctarank();  // 0: the pair's first CTA (issues the MMAs)
    const int pair = static_cast<int>(blockIdx.x >> 1);
    const int pairs = static_cast<int>(gridDim.x >> 1);

    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(full_bar(s), 1);
            mbar_init(empty_bar(s), 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(tfull_bar(b), 1);
            mbar_init(tempty_bar(b), 8);  // 4 epilogue warps in each CTA
        }
        mbar_init(drain_bar, 1);
        *abort_flag = 0;
        fence_barrier_init();
    }
    if (warp == 1) {
        tmem_alloc_pair(smem_u32(const_cast<uint32_t *>(tmem_slot)), Cfg::TMEM_COLS);
        tmem_relinquish_pair();
    }
    tc_fence_before_sync();
    __syncthreads();
    cluster_arrive();  // both CTAs' barriers and TMEM exist before any cross-CTA use
    cluster_wait();
    tc_fence_after_sync();
    const uint32_t tmem_base = *tmem_slot;

    const int m_tiles = (M + kPairBM - 1) / kPairBM;
    const int n_tiles = (N + BN - 1) / BN;
    const int tiles = m_tiles * n_tiles;
    const int k_blocks = (K + kMx4KB - 1) / kMx4KB;

    uint32_t issued_mask = 0, issued_parity = 0;
    bool mma_issued_any = false;

    if (warp == 0) {
        if (lane == 0) {
            int stage = 0;
            uint32_t phase = 0;
            bool ok = true;
            for (int t = pair; t < tiles && ok; t += pairs) {
                int m_blk, n_blk;
                pair_tile_mn(t, m_tiles, n_tiles, group_m, m_blk, n_blk);
                const int a_row = m_blk * kPairBM + static_cast<int>(rank) * 128;
                const int b_row = n_blk * BN + static_cast<int>(rank) * (BN / 2);
                const int b_rt = n_blk * BN / 128;
                for (int kb = 0; kb < k_blocks; ++kb) {
                    if (!bounded_wait(empty_bar(stage), phase ^ 1u, kErrWaitProducer, abort_flag)) {
                        ok = false;
                        break;
                    }
                    if (rank == 0)
                        mbar_arrive_expect_tx(full_bar(stage), 2u * Cfg::STAGE_BYTES);
                    const uint32_t fb = map_shared_rank(full_bar(stage), 0);
                    tma_load_2d_pair(sA + stage * Cfg::A_BYTES, &tmA, fb, kb * 128, a_row);
                    tma_load_2d_pair(sB + stage * Cfg::B_BYTES, &tmB, fb, kb * 128, b_row);
                    tma_load_3d_pair(sSA + stage * Cfg::SA_BYTES, &tmSA, fb, 0, kb * 2, a_row / 128);
                    tma_load_3d_pair(sSB + stage * Cfg::SB_BYTES, &tmSB, fb, 0, kb * 2, b_rt);
                    issued_mask |= 1u << stage;
                    issued_parity = (issued_parity & ~(1u << stage)) | (phase << stage);
                    if (++stage == STAGES) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
            }
            // every commit that frees a stage of this CTA has arrived before
            // the CTA may leave (they are multicast from the first CTA)
            for (int s = 0; s < STAGES && ok; ++s)
                if (issued_mask & (1u << s))
                    ok = bounded_wait(empty_bar(s), (issued_parity >> s) & 1u, kErrWaitDrain, abort_flag);
        }
    } else if (warp == 1) {
        if (lane == 0 && rank == 0) {
            const uint32_t tS = tmem_base + Cfg::NACC * BN;
            int stage = 0;
            uint32_t phase = 0;
            int acc = 0;
            uint32_t acc_phase = 0;
            bool ok = true;
            for (int t = pair; t < tiles && ok; t += pairs) {
                if (!bounded_wait_cluster(tempty_bar(acc), acc_phase ^ 1u, kErrWaitAccEmpty, abort_flag))
                    break;
                tc_fence_after_sync();
                const uint32_t d = tmem_base + static_cast<uint32_t>(acc * BN);
                int m_blk, n_blk;
                pair_tile_mn(t, m_tiles, n_tiles, group_m, m_blk, n_blk);
                // a tile that starts in the middle of a scale tile (BN = 192)
                // starts that many columns in, 32 rows a column
                const uint32_t shift = static_cast<uint32_t>(n_blk * BN % 128 / 32);
                for (int kb = 0; kb < k_blocks; ++kb) {
                    if (!bounded_wait(full_bar(stage), phase, kErrWaitMma, abort_flag)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after_sync();
                    const uint32_t a0 = sA + stage * Cfg::A_BYTES;
                    const uint32_t b0 = sB + stage * Cfg::B_BYTES;
                    const uint32_t ta = tS + static_cast<uint32_t>(Cfg::SCALE_COLS * stage), tb = ta + 8;
                    const int steps = min(4, (K - kb * kMx4KB + 63) >> 6);
                    // the scale tiles in TMEM: x [k tile], w [k tile][row tile], 4 columns each
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        if (2 * i >= steps)
                            break;
                        tmem_cp_scales_pair(ta + 4 * i,
                                            smem_desc_scales(sSA + stage * Cfg::SA_BYTES + i * kMx4TileBytes));
#pragma unroll
                        for (int rt = 0; rt < Cfg::RT_B; ++rt)
                            tmem_cp_scales_pair(tb + 4 * (i * Cfg::RT_B + rt),
                                                smem_desc_scales(sSB + stage * Cfg::SB_BYTES +
                                                                 (rt * 2 + i) * kMx4TileBytes));
                    }
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        if (k < steps)
                            mma_mx4_pair(d, smem_desc_k_sw128(a0 + 32 * k), smem_desc_k_sw128(b0 + 32 * k),
                                         (k & 1) ? idesc_mx4(kPairBM, BN, 2) : idesc_mx4(kPairBM, BN, 0),
                                         ta + 4 * (k >> 1), tb + 4 * Cfg::RT_B * (k >> 1) + shift,
                                         (kb > 0 || k != 0) ? 1u : 0u);
                    mma_issued_any = true;
                    mma_commit_pair(empty_bar(stage), 0x3);
                    if (++stage == STAGES) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
                if (!ok)
                    break;
                mma_commit_pair(tfull_bar(acc), 0x3);
                if (++acc == Cfg::NACC) {
                    acc = 0;
                    acc_phase ^= 1u;
                }
            }
        }
    } else {
        // epilogue warps 2..5: warp w reads TMEM lanes 32 (w % 4) .. +31
        const int quarter = warp & 3;
        const int row = quarter * 32 + lane;
        const uint32_t tempty_first = map_shared_rank(tempty_bar(0), 0);
        int acc = 0;
        uint32_t acc_phase = 0;
        for (int t = pair; t < tiles; t += pairs) {
            int m_blk, n_blk;
            pair_tile_mn(t, m_tiles, n_tiles, group_m, m_blk, n_blk);
            const bool ok = bounded_wait(tfull_bar(acc), acc_phase, kErrWaitAccFull, abort_flag);
            if (!__all_sync(0xFFFFFFFFu, ok))
                break;
            tc_fence_after_sync();
            const int64_t m = static_cast<int64_t>(m_blk) * kPairBM + rank * 128 + row;
            const uint32_t tbase =
                tmem_base + (static_cast<uint32_t>(quarter * 32) << 16) + static_cast<uint32_t>(acc * BN);
#pragma unroll 1
            for (int c = 0; c < BN / 32; ++c) {
                const int n0 = n_blk * BN + c * 32;
                if (n0 >= N)
                    break;
                uint32_t r[32];
                tmem_ld_32x32b_x32(tbase + c * 32, r);
                tmem_ld_wait();
                if (m < M)
                    mx4_store_row<OUT>(r, n0, N, y, m);
                __syncwarp();
            }
            tc_fence_before_sync();
            __syncwarp();
            if (lane == 0)
                mbar_arrive_remote_release(tempty_first + 8u * acc);
            if (++acc == Cfg::NACC) {
                acc = 0;
                acc_phase ^= 1u;
            }
        }
    }

    // ---- teardown ----------------------------------------------------------
    if (warp == 1 && lane == 0 && rank == 0 && *abort_flag && mma_issued_any) {
        // every MMA of the pair finishes before either CTA releases TMEM
        mma_commit_pair_local(drain_bar);
        bounded_wait(drain_bar, 0, kErrWaitDrain, nullptr, kWaitTimeoutNs / 4);
    }
    if (warp == 0 && lane == 0 && rank == 0 && *abort_flag) {
        // copies still in flight complete on the first CTA's full barriers
        for (int s = 0; s < STAGES; ++s)
            if (issued_mask & (1u << s))
                bounded_wait(full_bar(s), (issued_parity >> s) & 1u, kErrWaitDrain, nullptr, kWaitTimeoutNs / 4);
    }
    tc_fence_before_sync();
    __syncthreads();
    cluster_arrive();  // neither CTA leaves while the other may still touch its memory
    cluster_wait();
    if (warp == 1) {
        __syncwarp();
        tc_fence_after_sync();
        tmem_dealloc_pair(tmem_base, Cfg::TMEM_COLS);
    }
}

}  // namespace sq
