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
// Work.  A unit is one 256-value k block of one 128-channel tile of one expert,
// gate and up together: 32 KB of codes and 2 KB of scales.  The units, tile by
// tile and expert by expert, are cut into equal contiguous ranges, one a CTA.  (An
// earlier cut into whole-K items of 32 to 128 channels needed no sums across CTAs
// but left the CTAs with the narrow items behind: their rings held too few bytes
// to hide the loaded memory's latency; two experts of 4096 x 14336 took 38 us.)
//
// A tile that several CTAs share is summed through the workspace; the last of
// them (mx4_last_of) adds the partials in the contributors' order, activates and
// stores.  A look at the count while its part still streams spares it writing and
// counting its own partial where the others are done already, as they are when a
// tile has fewer k blocks than a CTA units (64 tokens, 48 of 64 experts of 2048 x
// 1408: 80 -> 78 us the layer).
//
// Measured (B200, calls one after another, this kernel and the second half): one
// token, 2 experts of 4096 x 14336, 46 us; 16 tokens, 80 experts of 2048 x 768, 54
// us; 64 tokens, 64 experts of 2048 x 1408, 72 us; the weights alone take 29, 32 and
// 45 us at the copy rate.  This kernel streams at 5 to 6 TB/s once it runs; what
// is left is fixed: finding the experts (1.3 us), the first loads (2 to 6 us),
// the boundary between the halves (4 us) and the shared tiles at the ends (3 to 8
// us).  Prefetching the second half's weights into L2 from here, two warps
// issuing the MMAs, and four instead of two partials in flight changed nothing.
//
// Roles as in mx4_stream_kernel, with 16 epilogue warps (kMx4UpSets).  The gate and the up product are two
// accumulators in the same lanes, so a thread holds both values of its channel,
// and a warp the 32 channels of one block of the quantised h.
#pragma once

#include <cstdint>
#include <cuda.h>

#include "sq_div.cuh"
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
                                      (kMx4MaxExperts / 32) * 4 + kMx4MaxExperts * 2 + kMx4MaxSlots * 2;
    static_assert(TMEM_COLS <= 512 && SMEM_BYTES <= 232448, "limits");
};

// Counts this CTA in at a shared tile's word and tells whether it is the last of
// `total`.  Nothing runs before this kernel to clear the words, and the workspace
// may hold anything.  So a word carries a tag in its upper 48 bits, and the lower
// 16 count: the second half leaves every word at (tag, 0), and one add is enough
// then.  A word without the tag (the workspace's first call) is replaced: whoever
// finds it swaps in (tag, 1), or (tag, n + 1) where another one was faster; what
// was added to it before that is lost with it.  Release and acquire: the partials
// written before (ordered by the caller's barrier) are visible to the last one.
// (Contents that become the tag by an add are no exception: whoever finds the tag
// counts from what stands there, and everyone else swaps.)
__device__ __forceinline__ bool mx4_last_of(unsigned long long *word, int total)
{
    unsigned long long seen = atom_add_acq_rel_gpu_u64(word, 1ull), count;
    if ((seen & ~0xFFFFull) == kMx4Tag) {
        count = (seen & 0xFFFFu) + 1;
    } else {
        ++seen;     // as the add left it
        for (;;) {  // a failed swap means that another contributor added or swapped in between: at most 2 * total times
            count = (seen & ~0xFFFFull) == kMx4Tag ? (seen & 0xFFFFu) + 1 : 1;
            const unsigned long long old = atom_cas_acq_rel_gpu(word, seen, kMx4Tag | count);
            if (old == seen)
                break;
            seen = old;
        }
    }
    return count == static_cast<unsigned long long>(total);
}

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

// v / (1 + e^-v), as n / d with t = e^-|v|, d = 1 + t in [1, 2] and n = v or v t:
// d needs no guards, so one Newton step on the quotient from the approximate
// reciprocal stands in for the IEEE division, a long sequence (46 tokens, 40
// experts of 384 x 6112: 93 -> 86 us).  In units of 2^-24: 2 from e^x, 1 each from
// n and d, a little over 1 from the step; below v = -87 e^x is subnormal and has
// fewer bits (|v e^v| < 2^-118 there).  An infinite v gives a NaN and so a NaN
// block, as the formula's infinity or NaN does.
__device__ __forceinline__ float mx4_silu(float v)
{
    const float t = expf(-fabsf(v));
    const float n = v < 0.0f ? v * t : v;
    const float d = 1.0f + t;
    const float r = rcp_approx(d);
    const float q = n * r;
    return fmaf(fmaf(-q, d, n), r, q);
}

// Epilogue warps of the first half: sets of four.  A token's channels of one block
// are a chain of a maximum, a quantisation and three shuffles, mostly latency: one
// set with four tokens at a time took 46 tokens, 40 experts of 384 x 6112 in 87 us
// and 128 tokens, 16 experts of 2048 x 1024 in 57, two sets 81 and 51, four sets 77
// and 49, and four with two tokens at a time 72 and 48.
constexpr int kMx4UpSets = 4;
constexpr int kMx4UpThreads = 96 + kMx4UpSets * 128;

// the epilogue warps' barrier
__device__ __forceinline__ void up_bar_sync() { asm volatile("bar.sync 2, %0;" ::"n"(kMx4UpSets * 128) : "memory"); }

// Two tokens (t < 0: none) of every lane's channel: activates, quantises over the
// 32 lanes and stores codes and scale byte.  Written once and looped over the
// chosen tokens: unrolled over all of a tile's columns, the instruction fetches
// took longer than the work.
__device__ __forceinline__ void mx4_store_h2(const int (&t)[2], const float (&g)[2], const float (&u)[2], uint8_t *codes,
                                             int row_bytes, uint8_t *scale, int zero_behind)
{
    const int lane = threadIdx.x & 31;
    float h[2];
    uint32_t byte[2], c[2];
#pragma unroll
    for (int i = 0; i < 2; ++i)
        h[i] = mx4_silu(g[i]) * u[i];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        byte[i] = mx4_scale_byte(__uint_as_float(__reduce_max_sync(0xFFFFFFFFu, __float_as_uint(h[i]) & 0x7FFFFFFFu)));
        c[i] = byte[i] == 255u ? 0u : mx4_code1(h[i] * mx4_inv_scale(byte[i])) << (4 * (lane & 7));
    }
#pragma unroll
    for (int d = 1; d < 8; d <<= 1)
#pragma unroll
        for (int i = 0; i < 2; ++i)
            c[i] |= __shfl_xor_sync(0xFFFFFFFFu, c[i], d);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        if (t[i] < 0)
            continue;
        if ((lane & 7) == 0)
            *reinterpret_cast<uint32_t *>(codes + static_cast<int64_t>(t[i]) * row_bytes + (lane >> 3) * 4) = c[i];
        if (lane == 0) {
            uint8_t *s = scale + (t[i] & 31) * 16 + (t[i] >> 5) * 4;
            *s = static_cast<uint8_t>(byte[i]);
            for (int p = 1; p <= zero_behind; ++p)
                s[p] = 0;
        }
    }
}

template <int BNX>
__global__ void __launch_bounds__(kMx4UpThreads, 1)
    mx4_moe_up_kernel(const __grid_constant__ CUtensorMap tmG, const __grid_constant__ CUtensorMap tmSG,
                      const __grid_constant__ CUtensorMap tmU, const __grid_constant__ CUtensorMap tmSU,
                      const __grid_constant__ CUtensorMap tmX, const __grid_constant__ CUtensorMap tmSX,
                      uint8_t *__restrict__ hq, uint8_t *__restrict__ hs, float *__restrict__ ws,
                      unsigned long long *__restrict__ words, int *__restrict__ cnt, int M, int H, int I,
                      Mx4MoeArgs moe)
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
    volatile int *last_flag = reinterpret_cast<volatile int *>(gb + misc_off + 12);
    volatile int *early_flag = reinterpret_cast<volatile int *>(gb + misc_off + 16);  // [2]
    uint32_t *tok_mask = reinterpret_cast<uint32_t *>(gb + misc_off + 24);  // [2][4]
    uint32_t *e_mask = tok_mask + 8;
    uint16_t *e_list = reinterpret_cast<uint16_t *>(e_mask + kMx4MaxExperts / 32);
    uint16_t *chosen = e_list + kMx4MaxExperts;

    if (threadIdx.x == 32) {
        for (int i = 0; i < STAGES; ++i) {
            mbar_init(full_bar(i), 1);
            mbar_init(empty_bar(i), 1);
            mbar_init(scale_bar(i), 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(tfull_bar(b), 1);
            mbar_init(tempty_bar(b), 4 * kMx4UpSets);  // the 16 epilogue warps
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
    const int G = mx4_active_experts(moe.ids, M * moe.topk, moe.E, e_mask, e_list, chosen, n_groups);
    // the second half's tile counts
    if (threadIdx.x == 0 && blockIdx.x < kMx4MaxCtas)
        cnt[blockIdx.x] = 0;
    const int RT = (I + 127) / 128, KB = (H + kMx4KB - 1) / kMx4KB;
    const int64_t U = static_cast<int64_t>(G) * RT * KB;
    const int64_t C = mx4_share(G * RT, KB, static_cast<int>(gridDim.x), mx4_up_cost(M, moe.topk, G));  // CTAs with work
    const int64_t c = blockIdx.x;
    const bool works = c < C;
    const int64_t u0 = works ? dec_start(c, U, C) : 0;
    const int nu = works ? static_cast<int>(dec_start(c + 1, U, C) - u0) : 0;
    const Mx4Unit first(u0, static_cast<int64_t>(RT) * KB, KB);  // t: expert's place in the list, g: its tile
    auto steps_of = [&](int kb) { return min(4, (H - kb * kMx4KB + 63) >> 6); };
    uint32_t issued_mask = 0, issued_parity = 0;
    bool mma_issued_any = false;

    if (warp == 0) {
        if (lane == 0) {
            int stage = 0;
            uint32_t phase = 0;
            Mx4Unit w = first;
            for (int i = 0; i < nu; ++i) {
                if (!bounded_wait(empty_bar(stage), phase ^ 1u, kErrWaitProducer, abort_flag))
                    break;
                const uint32_t fb = full_bar(stage);
                mbar_arrive_expect_tx(fb, Cfg::STAGE_BYTES);
                const int e = e_list[w.t];
                const uint32_t s0 = sS + stage * 3 * Cfg::S_BYTES;
                tma_load_2d(sG + stage * Cfg::W_BYTES, &tmG, fb, w.kb * 128, e * I + w.g * 128);
                tma_load_2d(sU + stage * Cfg::W_BYTES, &tmU, fb, w.kb * 128, e * I + w.g * 128);
                tma_load_3d(s0, &tmSG, fb, 0, w.kb * 2, e * RT + w.g);
                tma_load_3d(s0 + Cfg::S_BYTES, &tmSU, fb, 0, w.kb * 2, e * RT + w.g);
                tma_load_2d(sX + stage * Cfg::X_BYTES, &tmX, fb, w.kb * 128, 0);
                tma_load_3d(s0 + 2 * Cfg::S_BYTES, &tmSX, fb, 0, w.kb * 2, 0);
                w.next(KB, RT);
                issued_mask |= 1u << stage;
                issued_parity = (issued_parity & ~(1u << stage)) | (phase << stage);
                if (++stage == STAGES) {
                    stage = 0;
                    phase ^= 1u;
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
        int left = nu;
        for (int kb0 = first.kb; left > 0 && ok; kb0 = 0) {
            const int kb1 = min(KB, kb0 + left);
            left -= kb1 - kb0;
            if (!warp_wait(tempty_bar(acc), acc_phase ^ 1u, kErrWaitAccEmpty, abort_flag))
                break;
            tc_fence_after_sync();
            const uint32_t d = tmem_base + static_cast<uint32_t>(acc * 2 * BNX);
            for (int kb = kb0; kb < kb1; ++kb) {
                if (!warp_wait2(full_bar(stage), scale_bar(stage), phase, kErrWaitMma, abort_flag)) {
                    ok = false;
                    break;
                }
                __syncwarp();
                tc_fence_after_sync();
                const uint32_t t0 = tS + static_cast<uint32_t>(Cfg::SCALE_COLS * stage);
                const uint32_t w_at = static_cast<uint32_t>(stage * (Cfg::W_BYTES >> 4));
                const uint64_t x = x_desc + static_cast<uint32_t>(stage * (Cfg::X_BYTES >> 4));
                mx4_stage_mma<BNX, 1>(leader, d, g_desc + w_at, x, t0, t0 + 16, steps_of(kb), kb == kb0);
                mx4_stage_mma<BNX, 1>(leader, d + BNX, u_desc + w_at, x, t0 + 8, t0 + 16, steps_of(kb), kb == kb0);
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
            int kb = first.kb;
            for (int left = nu; left > 0; --left) {
                if (!bounded_wait(full_bar(stage), phase, kErrWaitMma, abort_flag))
                    break;
                tc_fence_after_sync();
                const uint32_t t0 = tS + static_cast<uint32_t>(Cfg::SCALE_COLS * stage);
                const uint32_t s0 = sS + stage * 3 * Cfg::S_BYTES;
                const int steps = steps_of(kb);
                if (++kb == KB)
                    kb = 0;
                mx4_copy_scales(t0, s0, steps);
                mx4_copy_scales(t0 + 8, s0 + Cfg::S_BYTES, steps);
                mx4_copy_scales(t0 + 16, s0 + 2 * Cfg::S_BYTES, steps);
                mma_commit(scale_bar(stage));
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
        // epilogue warps 3..18: warp w holds block w % 4 of the tile, a channel a lane;
        // the four sets of four warps take the tile's chosen tokens in turn, two at a time
        const int quarter = warp & 3;
        const int row = quarter * 32 + lane;
        const int et = threadIdx.x - 96;
        const int set = et >> 7;
        constexpr int SLOT = 2 * BNX * 128;  // floats of a partial tile: [gate, up][token][row]
        int acc = 0, wb = 0;
        uint32_t acc_phase = 0;
        Mx4Unit w = first;
        for (int left = nu; left > 0;) {
            const int g = w.t, tile = w.g, kb0 = w.kb, kb1 = min(KB, kb0 + left);
            const bool whole = kb0 == 0 && kb1 == KB;
            left -= kb1 - kb0;
            w.kb = KB - 1;
            w.next(KB, RT);
            // a shared tile's contributors (worked out while the tile streams);
            // only the first one's range may begin in an earlier tile
            const int64_t ut = (static_cast<int64_t>(g) * RT + tile) * KB;
            const int64_t cf = whole ? 0 : dec_owner(ut, U, C), cl = whole ? 0 : dec_owner(ut + KB - 1, U, C);
            const int cf_slot = !whole && dec_start(cf, U, C) < ut;
            {
                // the tokens that chose this expert
                if (set == 0) {
                    const int e = e_list[g];
                    bool has = false;
                    if (et < M)
                        for (int k = 0; k < moe.topk; ++k)
                            has = has || chosen[et * moe.topk + k] == e;
                    const uint32_t m = __ballot_sync(0xFFFFFFFFu, has);
                    if (lane == 0)
                        tok_mask[wb * 4 + (et >> 5)] = m;
                }
                if (et == 0)
                    early_flag[wb] = !whole && ld_acquire_gpu_u64(words + cf) == (kMx4Tag | static_cast<unsigned long long>(cl - cf));
                up_bar_sync();
            }
            const uint32_t *mask = tok_mask + wb * 4;
            const bool early = early_flag[wb];  // every other part of this tile is in the workspace
            wb ^= 1;
            // as in mx4_stream_kernel, a wait that gives up lets the warps go on
            bounded_wait(tfull_bar(acc), acc_phase, kErrWaitAccFull, abort_flag);
            __syncwarp();
            tc_fence_after_sync();
            const int unit = tile * 4 + quarter;
            const bool inside = unit * 32 < I;
            const int zero_behind = (unit + 1) * 32 == I ? 3 - quarter : 0;  // padding blocks of the last tile
            uint8_t *codes = hq + static_cast<int64_t>(g) * M * (I / 2) + unit * 16;
            uint8_t *scale = hs + (static_cast<int64_t>(g) * RT + tile) * kMx4TileBytes + quarter;
            float *mine = ws + (c * 2 + (g == first.t && tile == first.g ? 0 : 1)) * SLOT;
            const uint32_t lane_addr =
                tmem_base + (static_cast<uint32_t>(quarter * 32) << 16) + static_cast<uint32_t>(acc * 2 * BNX);
            // two chosen tokens at a time
            auto take2 = [](uint32_t &m, int cc, int (&t)[2]) {
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    t[i] = m != 0u ? cc * 32 + __ffs(m) - 1 : -1;
                    m &= m - 1;
                }
            };
            // sums over the contributors in their order, two partials in flight at a
            // time; `own` (-1: none) is the one whose values gv, uv hold already
            auto sum2 = [&](const int (&t)[2], int64_t own, float (&gv)[2], float (&uv)[2]) {
                float sg[2] = {}, su[2] = {};
                for (int64_t c2 = cf; c2 <= cl; c2 += 2) {
                    float a[2][2], b[2][2];
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        const int64_t cs = min(c2 + k, cl);
                        const float *p = ws + (cs * 2 + (cs == cf ? cf_slot : 0)) * SLOT + row;
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const bool on = t[i] >= 0 && c2 + k <= cl && cs != own;
                            a[k][i] = on ? __ldcg(p + t[i] * 128) : 0.0f;
                            b[k][i] = on ? __ldcg(p + (BNX + t[i]) * 128) : 0.0f;
                        }
                    }
#pragma unroll
                    for (int k = 0; k < 2; ++k)
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            sg[i] += c2 + k == own ? gv[i] : a[k][i];
                            su[i] += c2 + k == own ? uv[i] : b[k][i];
                        }
                }
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    gv[i] = sg[i];
                    uv[i] = su[i];
                }
            };
            if (inside) {
                int turn = kMx4UpSets - set;
#pragma unroll 1
                for (int cc = 0; cc < BNX / 32; ++cc)
#pragma unroll 1
                    for (uint32_t m = mask[cc]; m != 0u;) {
                        int t[2];
                        float gv[2], uv[2];
                        take2(m, cc, t);
                        if (turn++ % kMx4UpSets != 0)
                            continue;
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const uint32_t col = lane_addr + static_cast<uint32_t>(max(t[i], 0));
                            gv[i] = __uint_as_float(tmem_ld_32x32b_x1(col));
                            uv[i] = __uint_as_float(tmem_ld_32x32b_x1(col + BNX));
                        }
                        tmem_ld_wait();
                        if (whole || early) {
                            if (early)
                                sum2(t, c, gv, uv);
                            mx4_store_h2(t, gv, uv, codes, I / 2, scale, zero_behind);
                        } else {
#pragma unroll
                            for (int i = 0; i < 2; ++i)
                                if (t[i] >= 0) {
                                    mine[t[i] * 128 + row] = gv[i];
                                    mine[(BNX + t[i]) * 128 + row] = uv[i];
                                }
                        }
                    }
            }
            tc_fence_before_sync();
            __syncwarp();
            if (lane == 0)
                mbar_arrive(tempty_bar(acc));
            if (++acc == Cfg::NACC) {
                acc = 0;
                acc_phase ^= 1u;
            }
            if (whole || early)
                continue;
            up_bar_sync();  // this CTA's partial is written
            if (et == 0)
                *last_flag = mx4_last_of(words + cf, static_cast<int>(cl - cf + 1));
            up_bar_sync();
            if (*last_flag && inside) {
                int turn = kMx4UpSets - set;
#pragma unroll 1
                for (int cc = 0; cc < BNX / 32; ++cc)
#pragma unroll 1
                    for (uint32_t m = mask[cc]; m != 0u;) {
                        int t[2];
                        float gv[2], uv[2];
                        take2(m, cc, t);
                        if (turn++ % kMx4UpSets != 0)
                            continue;
                        sum2(t, -1, gv, uv);
                        mx4_store_h2(t, gv, uv, codes, I / 2, scale, zero_behind);
                    }
            }
            up_bar_sync();  // last_flag is rewritten by the next shared tile
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
