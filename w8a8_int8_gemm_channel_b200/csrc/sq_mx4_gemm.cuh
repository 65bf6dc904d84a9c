// sq_mx4_gemm.cuh -- the microscaled 4-bit product for many tokens on CTA pairs
// (tcgen05.mma cta_group::2, kind::mxf4).
//
//   y[m, n] = sum_k x[m, k] w[n, k], x and w the values that codes and scales
//   stand for; fp32 accumulation, one rounding to y's type
//
// An output tile is 256 tokens x BN channels.  CTA r of a pair loads rows
// [m0 + 128 r, +128) of x and rows [n0 + r BN/2, +BN/2) of w with plain TMA,
// and the scale tiles of its own x rows and of all BN rows of w (each SM's
// tensor core applies the scales of every column of its 128 rows).  In the
// pair's first CTA one warp copies both CTAs' scale tiles into TMEM columns that
// belong to the stage (tcgen05.cp) and another issues the MMAs.  Issued by the
// MMA thread itself the copies and the MMAs took turns (8192 x 8192 x 28672: 1025
// us against 755); from a warp of their own they run stages ahead.  No scale is
// left for the epilogue: it rounds and stores.
//
// TMEM (512 columns): the accumulators and 8 + 16 columns of scales a stage.
// BN = 192 and 128 fit two accumulators, 256 one.  The epilogue therefore first
// takes the whole accumulator into registers (eight warps, half the columns
// each) and frees it, and stores while the next tile multiplies.
//
// Bound: the operands' way from L2 (11 TB/s at 256 wide) and, held, the 1 kW power
// cap.  8192 x 8192 x 28672 runs at 4.8 PFLOP/s held (1.44 GHz) and 5.5 in a burst,
// 4096 x 6144 x 4096 at 4.2; without its operand loads the same loop makes 6.5 at
// 1.85 GHz, without the scale copies as well 8.3.  An MMA of N = 128 takes as long
// as one of 256 (some 130 cycles), so narrow tiles are for few rounds only.
// Groups of 8 m blocks (4, 16, 32: 811, 811, 895 us against 786).
#pragma once

#include <cstdint>
#include <cuda.h>
#include <cuda_bf16.h>

#include "sq_gemm_pair.cuh"
#include "sq_mx4_stream.cuh"
#include "sq_ptx.cuh"

namespace sq {

constexpr int kMx4PairThreads = 352;  // producer, MMA, scale copies, 8 epilogue warps

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
    static constexpr int NUM_BARS = 3 * STAGES + 5;  // full, empty, tfull[2], tempty[2], drain, scales
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
__global__ void __launch_bounds__(kMx4PairThreads, 1)
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
    auto scale_bar = [&](int s) { return sBar + 8u * (2 * STAGES + 5 + s); };
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
            mbar_init(scale_bar(s), 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(tfull_bar(b), 1);
            mbar_init(tempty_bar(b), 16);  // 8 epilogue warps in each CTA
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
        if (rank == 0) {
            const uint32_t leader = elect_one();
            const uint32_t tS = tmem_base + Cfg::NACC * BN;
            auto steps_of = [&](int kb) { return min(4, (K - kb * kMx4KB + 63) >> 6); };
            const uint64_t a_desc = smem_desc_k_sw128(sA), b_desc = smem_desc_k_sw128(sB);  // + 2 a 32-byte step
            int stage = 0;
            uint32_t phase = 0;
            int acc = 0;
            uint32_t acc_phase = 0;
            bool ok = true;
            for (int t = pair; t < tiles && ok; t += pairs) {
                if (!__all_sync(0xFFFFFFFFu, bounded_wait_cluster(tempty_bar(acc), acc_phase ^ 1u, kErrWaitAccEmpty, abort_flag)))
                    break;
                tc_fence_after_sync();
                const uint32_t d = tmem_base + static_cast<uint32_t>(acc * BN);
                int m_blk, n_blk;
                pair_tile_mn(t, m_tiles, n_tiles, group_m, m_blk, n_blk);
                // a tile that starts in the middle of a scale tile (BN = 192)
                // starts that many columns in, 32 rows a column
                const uint32_t shift = static_cast<uint32_t>(n_blk * BN % 128 / 32);
                for (int kb = 0; kb < k_blocks; ++kb) {
                    const int next = stage + 1 == STAGES ? 0 : stage + 1;
                    if (!warp_wait2(full_bar(stage), scale_bar(stage), phase, kErrWaitMma, abort_flag)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after_sync();
                    const uint64_t a0 = a_desc + static_cast<uint32_t>(stage * (Cfg::A_BYTES >> 4));
                    const uint64_t b0 = b_desc + static_cast<uint32_t>(stage * (Cfg::B_BYTES >> 4));
                    const uint32_t ta = tS + static_cast<uint32_t>(Cfg::SCALE_COLS * stage), tb = ta + 8;
                    const int steps = steps_of(kb);
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        if (k < steps)
                            mma_mx4_pair_warp(leader, d, a0 + 2 * k, b0 + 2 * k,
                                         (k & 1) ? idesc_mx4(kPairBM, BN, 2) : idesc_mx4(kPairBM, BN, 0),
                                         ta + 4 * (k >> 1), tb + 4 * Cfg::RT_B * (k >> 1) + shift,
                                         (kb > 0 || k != 0) ? 1u : 0u);
                    mma_issued_any = true;
                    mma_commit_pair_warp(leader, empty_bar(stage), 0x3);
                    stage = next;
                    phase ^= next == 0 ? 1u : 0u;
                }
                if (!ok)
                    break;
                mma_commit_pair_warp(leader, tfull_bar(acc), 0x3);
                if (++acc == Cfg::NACC) {
                    acc = 0;
                    acc_phase ^= 1u;
                }
            }
        }
    } else if (warp == 2) {
        if (lane == 0 && rank == 0) {
            const uint32_t tS = tmem_base + Cfg::NACC * BN;
            auto steps_of = [&](int kb) { return min(4, (K - kb * kMx4KB + 63) >> 6); };
            // scale tiles of a filled stage into its TMEM columns: x [k tile],
            // w [k tile][row tile], 4 columns each
            auto copy_scales = [&](int stage, int steps) {
                const uint32_t ta = tS + static_cast<uint32_t>(Cfg::SCALE_COLS * stage), tb = ta + 8;
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    if (2 * i >= steps)
                        break;
                    tmem_cp_scales_pair(ta + 4 * i, smem_desc_scales(sSA + stage * Cfg::SA_BYTES + i * kMx4TileBytes));
#pragma unroll
                    for (int rt = 0; rt < Cfg::RT_B; ++rt)
                        tmem_cp_scales_pair(tb + 4 * (i * Cfg::RT_B + rt),
                                            smem_desc_scales(sSB + stage * Cfg::SB_BYTES + (rt * 2 + i) * kMx4TileBytes));
                }
            };
            int stage = 0;
            uint32_t phase = 0;
            bool ok = true;
            int last = -1;
            uint32_t last_phase = 0;
            for (int t = pair; t < tiles && ok; t += pairs)
                for (int kb = 0; kb < k_blocks; ++kb) {
                    if (!bounded_wait(full_bar(stage), phase, kErrWaitMma, abort_flag)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after_sync();
                    copy_scales(stage, steps_of(kb));
                    mma_commit_pair_local(scale_bar(stage));
                    last = stage;
                    last_phase = phase;
                    if (++stage == STAGES) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
            // the last copies have landed before the CTA may release TMEM
            if (last >= 0)
                bounded_wait(scale_bar(last), last_phase, kErrWaitDrain, nullptr, kWaitTimeoutNs / 4);
        }
    } else {
        // epilogue warps 3..10: warp w reads TMEM lanes 32 (w % 4) .. +31, half
        // of the tile's columns, all into registers; then the accumulator is
        // free for the next tile while the stores run
        constexpr int NC = BN / 64;  // chunks of 32 columns a warp
        const int quarter = warp & 3;
        const int half = (warp - 3) >> 2;
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
            const uint32_t tbase = tmem_base + (static_cast<uint32_t>(quarter * 32) << 16) +
                                   static_cast<uint32_t>(acc * BN + half * (BN / 2));
            uint32_t r[NC][32];
#pragma unroll
            for (int c = 0; c < NC; ++c)
                tmem_ld_32x32b_x32(tbase + c * 32, r[c]);
            tmem_ld_wait();
            tc_fence_before_sync();
            __syncwarp();
            if (lane == 0)
                mbar_arrive_remote_release(tempty_first + 8u * acc);
            if (++acc == Cfg::NACC) {
                acc = 0;
                acc_phase ^= 1u;
            }
            if (m < M) {
#pragma unroll
                for (int c = 0; c < NC; ++c) {
                    const int n0 = n_blk * BN + half * (BN / 2) + c * 32;
                    if (n0 < N)
                        mx4_store_row<OUT>(r[c], n0, N, y, m);
                }
            }
            __syncwarp();
        }
    }

    // ---- teardown ----------------------------------------------------------
    if (warp == 1 && rank == 0 && *abort_flag && mma_issued_any) {
        // every MMA of the pair finishes before either CTA releases TMEM
        // (by the lane that issued them)
        __syncwarp();
        if (elect_one())
            mma_commit_pair_local(drain_bar);
        __syncwarp();
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
