// sq_mx4_moe.cuh -- first half of the experts layer for few tokens: every
// chosen expert's gate and up projections, the gated activation and its
// quantisation, in one kernel.
//
//   h[g, m, j] = silu(sum_k x[m, k] wg[e_g, j, k]) * sum_k x[m, k] wu[e_g, j, k]
//   silu(v) = v / (1 + e^-v), in fp32; then 32 values of j share a scale
//
// for every expert e_g that any token chose and the tokens m that chose it.  The
// second half (the down projection and the weighted sum over a token's choices)
// is mx4_stream_kernel with MOE.
//
// All tokens ride along as the N side of every expert's product, so nothing is
// gathered or sorted: the weights' bytes bound the layer, and the tensor cores
// have time to spare for columns that are not kept (a 128-row k block of
// weights takes an SM about 700 cycles to stream and the MMAs of 64 columns
// some 260).  Only the chosen (expert, token) pairs are activated and stored.
//
// Work.  A unit is 32 channels of one expert, which is one block of the
// quantised h, so every unit's scale is made by one warp and no CTA needs
// another's sums.  The units are cut into equal contiguous ranges, one a CTA; a
// CTA takes up to four units that lie in one 128-row tile at a time and loads
// just their rows (the other rows of the MMA tile hold whatever was there: they
// reach only their own, unread, accumulator rows).
//
// Roles as in mx4_stream_kernel.  The gate and the up product of a unit are two
// accumulators in the same lanes, so a thread holds both values of its channel.
#pragma once

#include <cstdint>
#include <cuda.h>

#include "sq_mx4_stream.cuh"

namespace sq {

template <int BNX>
struct Mx4UpCfg {
    static constexpr int W_BYTES = 128 * 128;  // of gate and of up
    static constexpr int X_BYTES = BNX * 128;
    static constexpr int S_BYTES = 2 * kMx4TileBytes;
    static constexpr int STAGE_BYTES = 2 * W_BYTES + X_BYTES + 3 * S_BYTES;
    static constexpr int STAGES = BNX == 128 ? 4 : 5;
    static constexpr int NACC = BNX == 128 ? 1 : 2;  // sets of (gate, up) accumulators
    static constexpr int SCALE_COLS = 24;
    static constexpr int TMEM_COLS = pow2_at_least(NACC * 2 * BNX + STAGES * SCALE_COLS, 32);
    static constexpr int NUM_BARS = 3 * STAGES + 5;
    static constexpr int SMEM_BYTES = 1024 + STAGES * STAGE_BYTES + NUM_BARS * 8 + 24 + 2 * 16 +
                                      (kMx4MaxExperts / 32) * 4 + kMx4MaxExperts * 2;
    static_assert(TMEM_COLS <= 512 && SMEM_BYTES <= 232448, "limits");
};

// The E2M1 code of one scaled value (bits 0-3).
__device__ __forceinline__ uint32_t mx4_code1(float v)
{
    uint32_t d;
    asm("{\n\t.reg .b8 b;\n\t.reg .b16 t;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b, %2, %1;\n\t"
        "mov.b16 t, {b, b};\n\t"
        "cvt.u32.u16 %0, t;\n\t}"
        : "=r"(d)
        : "f"(v), "f"(0.0f));
    return d & 0xFu;
}

template <int BNX>
__global__ void __launch_bounds__(kMx4StreamThreads, 1)
    mx4_moe_up_kernel(const __grid_constant__ CUtensorMap tmG, const __grid_constant__ CUtensorMap tmSG,
                      const __grid_constant__ CUtensorMap tmU, const __grid_constant__ CUtensorMap tmSU,
                      const __grid_constant__ CUtensorMap tmX, const __grid_constant__ CUtensorMap tmSX,
                      uint8_t *__restrict__ hq, uint8_t *__restrict__ hs, int *__restrict__ cnt, int ncnt, int M, int H,
                      int I, Mx4MoeArgs moe)
{
    using Cfg = Mx4UpCfg<BNX>;
    constexpr int STAGES = Cfg::STAGES;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    uint8_t *gb = smem_raw + (base - raw);
    const uint32_t sG = base;
    const uint32_t sU = sG + STAGES * Cfg::W_BYTES;
    const uint32_t sX = sU + STAGES * Cfg::W_BYTES;
    const uint32_t sS = sX + STAGES * Cfg::X_BYTES;  // scales of a stage: gate, up, x
    const uint32_t bars = sS + STAGES * 3 * Cfg::S_BYTES;
    auto full_bar = [&](int i) { return bars + 8u * i; };
    auto empty_bar = [&](int i) { return bars + 8u * (STAGES + i); };
    auto tfull_bar = [&](int b) { return bars + 8u * (2 * STAGES + b); };
    auto tempty_bar = [&](int b) { return bars + 8u * (2 * STAGES + 2 + b); };
    const uint32_t drain_bar = bars + 8u * (2 * STAGES + 4);
    auto scale_bar = [&](int i) { return bars + 8u * (2 * STAGES + 5 + i); };
    const uint32_t misc_off = (bars - base) + 8u * Cfg::NUM_BARS;
    volatile uint32_t *tmem_slot = reinterpret_cast<volatile uint32_t *>(gb + misc_off);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(gb + misc_off + 4);
    volatile int *n_groups = reinterpret_cast<volatile int *>(gb + misc_off + 8);
    uint32_t *tok_mask = reinterpret_cast<uint32_t *>(gb + misc_off + 24);  // [2][4]
    uint32_t *e_mask = tok_mask + 8;
    uint16_t *e_list = reinterpret_cast<uint16_t *>(e_mask + kMx4MaxExperts / 32);

    if (threadIdx.x == 32) {
        for (int i = 0; i < STAGES; ++i) {
            mbar_init(full_bar(i), 1);
            mbar_init(empty_bar(i), 1);
            mbar_init(scale_bar(i), 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(tfull_bar(b), 1);
            mbar_init(tempty_bar(b), 4);  // the 4 epilogue warps
        }
        mbar_init(drain_bar, 1);
        *abort_flag = 0;
        fence_barrier_init();
    }
    if (threadIdx.x == 0) {
        tma_prefetch_desc(&tmG);
        tma_prefetch_desc(&tmSG);
        tma_prefetch_desc(&tmU);
        tma_prefetch_desc(&tmSU);
        tma_prefetch_desc(&tmX);
        tma_prefetch_desc(&tmSX);
    }
    if (warp == 1) {
        tmem_alloc(smem_u32(const_cast<uint32_t *>(tmem_slot)), Cfg::TMEM_COLS);
        tmem_relinquish();
    }
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem_base = *tmem_slot;
    pdl_prologue();
    const int G = mx4_active_experts(moe.ids, M * moe.topk, moe.E, e_mask, e_list, n_groups);
    // the second half's tile counters
    for (int i = blockIdx.x * blockDim.x + threadIdx.x; i < ncnt; i += gridDim.x * blockDim.x)
        cnt[i] = 0;

    const int IU = I / 32, RT = (I + 127) / 128, KB = (H + kMx4KB - 1) / kMx4KB;
    const int64_t V = static_cast<int64_t>(G) * IU;
    const int64_t v0 = dec_start(blockIdx.x, V, gridDim.x), v1 = dec_start(blockIdx.x + 1, V, gridDim.x);
    // item at unit v: up to four units of one expert's 128-row tile
    struct Item {
        int g, tile, sub, nu;
    };
    auto item_at = [&](int64_t v) {
        Item it;
        it.g = static_cast<int>(v / IU);
        const int q = static_cast<int>(v - static_cast<int64_t>(it.g) * IU);
        it.tile = q >> 2;
        it.sub = q & 3;
        it.nu = static_cast<int>(min(static_cast<int64_t>(min(4 - it.sub, IU - q)), v1 - v));
        return it;
    };

    auto steps_of = [&](int kb) { return min(4, (H - kb * kMx4KB + 63) >> 6); };
    uint32_t issued_mask = 0, issued_parity = 0;
    bool mma_issued_any = false;

    if (warp == 0) {
        if (lane == 0) {
            int stage = 0;
            uint32_t phase = 0;
            bool ok = true;
            for (int64_t v = v0; v < v1 && ok;) {
                const Item it = item_at(v);
                v += it.nu;
                const int e = e_list[it.g];
                for (int kb = 0; kb < KB; ++kb) {
                    if (!bounded_wait(empty_bar(stage), phase ^ 1u, kErrWaitProducer, abort_flag)) {
                        ok = false;
                        break;
                    }
                    const uint32_t fb = full_bar(stage);
                    mbar_arrive_expect_tx(fb, static_cast<uint32_t>(it.nu * 2 * 4096 + Cfg::X_BYTES + 3 * Cfg::S_BYTES));
                    const uint32_t s0 = sS + stage * 3 * Cfg::S_BYTES;
                    for (int q = it.sub; q < it.sub + it.nu; ++q) {
                        const int r = e * I + it.tile * 128 + q * 32;
                        tma_load_2d(sG + stage * Cfg::W_BYTES + q * 4096, &tmG, fb, kb * 128, r);
                        tma_load_2d(sU + stage * Cfg::W_BYTES + q * 4096, &tmU, fb, kb * 128, r);
                    }
                    tma_load_3d(s0, &tmSG, fb, 0, kb * 2, e * RT + it.tile);
                    tma_load_3d(s0 + Cfg::S_BYTES, &tmSU, fb, 0, kb * 2, e * RT + it.tile);
                    tma_load_2d(sX + stage * Cfg::X_BYTES, &tmX, fb, kb * 128, 0);
                    tma_load_3d(s0 + 2 * Cfg::S_BYTES, &tmSX, fb, 0, kb * 2, 0);
                    issued_mask |= 1u << stage;
                    issued_parity = (issued_parity & ~(1u << stage)) | (phase << stage);
                    if (++stage == STAGES) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
            }
        }
    } else if (warp == 1) {
        const uint32_t leader = elect_one();
        const uint32_t tS = tmem_base + Cfg::NACC * 2 * BNX;
        const uint64_t g_desc = smem_desc_k_sw128(sG), u_desc = smem_desc_k_sw128(sU), x_desc = smem_desc_k_sw128(sX);
        int stage = 0;
        uint32_t phase = 0;
        int acc = 0;
        uint32_t acc_phase = 0;
        bool ok = true;
        for (int64_t v = v0; v < v1 && ok;) {
            v += item_at(v).nu;
            if (!bounded_wait(tempty_bar(acc), acc_phase ^ 1u, kErrWaitAccEmpty, abort_flag))
                break;
            tc_fence_after_sync();
            const uint32_t d = tmem_base + static_cast<uint32_t>(acc * 2 * BNX);
            for (int kb = 0; kb < KB; ++kb) {
                if (!bounded_wait(full_bar(stage), phase, kErrWaitMma, abort_flag) ||
                    !bounded_wait(scale_bar(stage), phase, kErrWaitMma, abort_flag)) {
                    ok = false;
                    break;
                }
                __syncwarp();
                tc_fence_after_sync();
                const uint32_t t0 = tS + static_cast<uint32_t>(Cfg::SCALE_COLS * stage);
                const uint32_t w_at = static_cast<uint32_t>(stage * (Cfg::W_BYTES >> 4));
                const uint64_t x = x_desc + static_cast<uint32_t>(stage * (Cfg::X_BYTES >> 4));
                mx4_stage_mma<BNX, 1>(leader, d, g_desc + w_at, x, t0, t0 + 16, steps_of(kb), kb == 0);
                mx4_stage_mma<BNX, 1>(leader, d + BNX, u_desc + w_at, x, t0 + 8, t0 + 16, steps_of(kb), kb == 0);
                mma_issued_any = true;
                mma_commit_warp(leader, empty_bar(stage));
                if (++stage == STAGES) {
                    stage = 0;
                    phase ^= 1u;
                }
            }
            if (!ok)
                break;
            mma_commit_warp(leader, tfull_bar(acc));
            if (++acc == Cfg::NACC) {
                acc = 0;
                acc_phase ^= 1u;
            }
        }
    } else if (warp == 2) {
        if (lane == 0) {
            const uint32_t tS = tmem_base + Cfg::NACC * 2 * BNX;
            int stage = 0, last = -1;
            uint32_t phase = 0, last_phase = 0;
            bool ok = true;
            for (int64_t v = v0; v < v1 && ok;) {
                v += item_at(v).nu;
                for (int kb = 0; kb < KB; ++kb) {
                    if (!bounded_wait(full_bar(stage), phase, kErrWaitMma, abort_flag)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after_sync();
                    const uint32_t t0 = tS + static_cast<uint32_t>(Cfg::SCALE_COLS * stage);
                    const uint32_t s0 = sS + stage * 3 * Cfg::S_BYTES;
                    mx4_copy_scales(t0, s0, steps_of(kb));
                    mx4_copy_scales(t0 + 8, s0 + Cfg::S_BYTES, steps_of(kb));
                    mx4_copy_scales(t0 + 16, s0 + 2 * Cfg::S_BYTES, steps_of(kb));
                    mma_commit(scale_bar(stage));
                    last = stage;
                    last_phase = phase;
                    if (++stage == STAGES) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
            }
            // the last copies have landed before the CTA may release TMEM
            if (last >= 0)
                bounded_wait(scale_bar(last), last_phase, kErrWaitDrain, nullptr, kWaitTimeoutNs / 4);
        }
    } else {
        // epilogue warps 3..6: warp w holds unit w % 4 of the tile, a channel a lane
        const int quarter = warp & 3;
        const int et = threadIdx.x - 96;
        int acc = 0, wb = 0;
        uint32_t acc_phase = 0;
        for (int64_t v = v0; v < v1;) {
            const Item it = item_at(v);
            v += it.nu;
            {
                // the tokens that chose this expert
                const int e = e_list[it.g];
                bool has = false;
                if (et < M)
                    for (int k = 0; k < moe.topk; ++k)
                        has = has || __ldg(moe.ids + et * moe.topk + k) == e;
                const uint32_t m = __ballot_sync(0xFFFFFFFFu, has);
                if (lane == 0)
                    tok_mask[wb * 4 + (et >> 5)] = m;
                dec_bar_sync();
            }
            // as in mx4_stream_kernel, a wait that gives up lets the warps go on
            bounded_wait(tfull_bar(acc), acc_phase, kErrWaitAccFull, abort_flag);
            __syncwarp();
            tc_fence_after_sync();
            if (quarter >= it.sub && quarter < it.sub + it.nu) {
                const int unit = it.tile * 4 + quarter;
                const uint32_t lane_addr =
                    tmem_base + (static_cast<uint32_t>(quarter * 32) << 16) + static_cast<uint32_t>(acc * 2 * BNX);
                uint8_t *srow = hs + (static_cast<int64_t>(it.g) * RT + it.tile) * kMx4TileBytes + quarter;
#pragma unroll 1
                for (int cc = 0; cc < BNX / 32; ++cc) {
                    const uint32_t m = tok_mask[wb * 4 + cc];
                    if (m == 0u)
                        continue;
                    uint32_t a[32], b[32];
                    tmem_ld_32x32b_x32(lane_addr + cc * 32, a);
                    tmem_ld_32x32b_x32(lane_addr + BNX + cc * 32, b);
                    tmem_ld_wait();
#pragma unroll
                    for (int j = 0; j < 32; ++j) {
                        if (!(m & (1u << j)))
                            continue;
                        const float gv = __uint_as_float(a[j]);
                        const float h = __fmul_rn(__fdiv_rn(gv, __fadd_rn(1.0f, expf(-gv))), __uint_as_float(b[j]));
                        const uint32_t top = __reduce_max_sync(0xFFFFFFFFu, __float_as_uint(h) & 0x7FFFFFFFu);
                        const uint32_t byte = mx4_scale_byte(__uint_as_float(top));
                        uint32_t c = byte == 255u ? 0u : mx4_code1(h * mx4_inv_scale(byte)) << (4 * (lane & 7));
                        c |= __shfl_xor_sync(0xFFFFFFFFu, c, 1);
                        c |= __shfl_xor_sync(0xFFFFFFFFu, c, 2);
                        c |= __shfl_xor_sync(0xFFFFFFFFu, c, 4);
                        const int64_t t = static_cast<int64_t>(it.g) * M + cc * 32 + j;
                        if ((lane & 7) == 0)
                            *reinterpret_cast<uint32_t *>(hq + t * (I / 2) + unit * 16 + (lane >> 3) * 4) = c;
                        if (lane == 0) {
                            uint8_t *s = srow + j * 16 + cc * 4;
                            *s = static_cast<uint8_t>(byte);
                            if (unit == IU - 1)  // the blocks behind the last one hold 0
                                for (int p = 1; p < 4 - quarter; ++p)
                                    s[p] = 0;
                        }
                    }
                }
            }
            wb ^= 1;
            tc_fence_before_sync();
            __syncwarp();
            if (lane == 0)
                mbar_arrive(tempty_bar(acc));
            if (++acc == Cfg::NACC) {
                acc = 0;
                acc_phase ^= 1u;
            }
        }
    }

    // ---- teardown ------------------------------------------------------------
    if (warp == 1 && *abort_flag && mma_issued_any) {
        __syncwarp();
        mma_commit_warp(elect_one(), drain_bar);
        bounded_wait(drain_bar, 0, kErrWaitDrain, nullptr, kWaitTimeoutNs / 4);
    }
    if (warp == 0 && lane == 0 && *abort_flag) {
        for (int i = 0; i < STAGES; ++i)
            if (issued_mask & (1u << i))
                bounded_wait(full_bar(i), (issued_parity >> i) & 1u, kErrWaitDrain, nullptr, kWaitTimeoutNs / 4);
    }
    tc_fence_before_sync();
    __syncthreads();
    if (warp == 1) {
        __syncwarp();
        tc_fence_after_sync();
        tmem_dealloc(tmem_base, Cfg::TMEM_COLS);
    }
}

}  // namespace sq
