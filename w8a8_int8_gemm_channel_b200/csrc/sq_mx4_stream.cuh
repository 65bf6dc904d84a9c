// sq_mx4_stream.cuh -- the microscaled 4-bit product for few tokens (at most
// 128): a stream over the weight, split evenly over every SM.
//
//   linear  y[m, n] = sum_k x[m, k] w[n, k]
//   experts y[m, n] = sum_g v[g, m] sum_k h[g, m, k] w[e_g, n, k]
//
// (x, h, w the values that codes and scales stand for; e_g the g-th expert that
// any token chose, v[g, m] token m's routing weight for it.)
//
// The tensor cores take the codes as they are (tcgen05.mma kind::mxf4) and
// apply the scales of both sides to every 32 values of K, so nothing is
// unpacked; the product accumulates in fp32.  The weight takes the 128-row MMA
// side (a tile = 128 output channels), the tokens its N (BNX padded rows).  A
// unit is one 128-byte k block (256 values) of one tile: 16 KB of codes and
// 1 KB of scales.  The units, tile by tile (and within a tile expert by
// expert), are cut into equal contiguous ranges, one per CTA and at most one CTA per
// SM: the bound is the weight's bytes, and every SM streams the same number of
// them whatever N, K and the experts are.  A tile that several CTAs share is
// summed through the workspace: each contributor writes its fp32 partial and
// counts itself in, and the one that completes the count adds the partials in
// the contributors' order, so the sum's order is fixed by the sizes alone.  The
// kernel right before clears the counts.
//
// Scales.  A stage's scale tiles go from shared memory to TMEM columns that
// belong to the stage (tcgen05.cp), so they are rewritten only after the
// commit that freed the stage.  A warp of its own copies them, stages ahead of
// the MMAs: issued by the MMA thread, the copies and the MMAs took turns.
//
// Roles (224 threads): warp 0 TMA producer, warp 1 TMEM and MMA issue, warp 2
// scale copies, warps 3..6 epilogue.  Two accumulators, so a range's next tile (or expert)
// accumulates while the epilogue drains one.
//
// Measured (B200, with the quantiser before it, calls in a graph): 1 x 6144 x 4096
// 10.9 us, 32 x 28672 x 4096 16.3 us (3.8 TB/s of weights; the weights' floor is
// 10 us), 128 x 28672 x 4096 20.3 us.  A unit takes 320 ns once the stream runs;
// the rest is the quantiser and its boundary (5 us), the first loads (2.7 us) and
// a shared tile's sum (3 us).  As many CTAs as SMs with tiles shared unevenly
// (21 us), and weight loads before the wait for the quantiser (20.8 us) were
// slower at 32 x 28672 x 4096, when it took 20, than the plan stream_ctas picks.
// The experts' second half streams slower, 2.5 TB/s (27.6 us for 69 MB, 16 tokens,
// 8 of 128 experts of 2048 x 768, cold): for every tile and expert its four epilogue
// warps read the choices again, wait for one another and drain 32 columns of four
// accumulators for the one or two tokens that chose it.
#pragma once

#include <cstdint>
#include <cuda.h>
#include <cuda_bf16.h>

#include "sq_decode.cuh"
#include "sq_mx4.cuh"
#include "sq_ptx.cuh"

namespace sq {

constexpr int kMx4KB = 256;          // values of K a stage holds (128 bytes of codes a row)
constexpr int kMx4MaxTokens = 128;   // of the streaming kernels
constexpr int kMx4MaxSlots = 1024;   // tokens x choices of the experts layer
constexpr int kMx4MaxExperts = 1024;
constexpr int kMx4StreamThreads = 224;
constexpr unsigned long long kMx4Tag = 0x9E3779B97F4Aull << 16;  // of a tile word (see mx4_last_of)
constexpr int kMx4MaxCtas = 160;  // of a streaming kernel: at least the SM count of every sm_100 part

template <int BNX>
struct Mx4StreamCfg {
    static constexpr int W_BYTES = 128 * 128;
    static constexpr int X_BYTES = BNX * 128;
    static constexpr int S_BYTES = 2 * kMx4TileBytes;  // scale tiles of one operand's stage
    static constexpr int STAGE_BYTES = W_BYTES + X_BYTES + 2 * S_BYTES;
    static constexpr int MAX_STAGES = BNX == 128 ? 6 : 8;
    static constexpr int NACC = BNX == 32 ? 4 : (BNX == 64 ? 2 : 1);  // accumulators a tile rotates over
    static constexpr int SCALE_COL = 2 * NACC * BNX;                 // two sets of them, then the scales
    static constexpr int TMEM_COLS = pow2_at_least(SCALE_COL + 16 * MAX_STAGES, 32);
    static_assert(TMEM_COLS <= 512, "TMEM");
};

// ring, barriers (full, empty, tfull[2], tempty[2], drain, scales), TMEM slot and two
// flags, routing weights of a group [128] and its mask [4], expert mask and list
__host__ __device__ constexpr int mx4_stream_smem(int stage_bytes, int stages, bool moe)
{
    return 1024 + stages * stage_bytes + (3 * stages + 5) * 8 + 24 +
           (moe ? 2 * 512 + 2 * 16 + (kMx4MaxExperts / 32) * 4 + kMx4MaxExperts * 2 + kMx4MaxSlots * 2 : 0);
}

// The experts that any of the S choices names, ascending, into `list`; returns
// their number.  Choices outside [0, E) name none.  The whole block calls it.
// `chosen` [S] keeps the choices themselves, 0xFFFF for none.
__device__ __forceinline__ int mx4_active_experts(const int *__restrict__ ids, int S, int E, uint32_t *mask,
                                                  uint16_t *list, uint16_t *chosen, volatile int *count)
{
    for (int i = threadIdx.x; i < kMx4MaxExperts / 32; i += blockDim.x)
        mask[i] = 0u;
    __syncthreads();
    for (int i = threadIdx.x; i < S; i += blockDim.x) {
        const int e = __ldg(ids + i);
        const bool here = e >= 0 && e < E;
        chosen[i] = here ? static_cast<uint16_t>(e) : 0xFFFFu;
        if (here)
            atomicOr(mask + (e >> 5), 1u << (e & 31));
    }
    __syncthreads();
    // word w's first place in the list is the number of experts in the words
    // before it: every warp scans the 32 words and lists the bits of some
    const int lane = threadIdx.x & 31;
    const uint32_t m = mask[lane];
    int before = __popc(m);
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int o = __shfl_up_sync(0xFFFFFFFFu, before, d);
        if (lane >= d)
            before += o;
    }
    const int total = __shfl_sync(0xFFFFFFFFu, before, 31);
    before -= __popc(m);
    for (int w = threadIdx.x >> 5; w < (E + 31) / 32; w += blockDim.x >> 5) {
        const uint32_t bits = __shfl_sync(0xFFFFFFFFu, m, w);
        const int at = __shfl_sync(0xFFFFFFFFu, before, w);
        if (bits & (1u << lane))
            list[at + __popc(bits & ((1u << lane) - 1))] = static_cast<uint16_t>(w * 32 + lane);
    }
    if (threadIdx.x == 0)
        *count = total;
    __syncthreads();
    return *count;
}

// How many of `grid` CTAs share the work of `tiles` tiles of `per_tile` units: all
// of them, the units cut evenly wherever that falls, or S for each tile (S = 1:
// nothing is summed), whichever the estimate says is done first.  Times in ns: a
// unit's, a shared tile's fixed part, and what each contributor adds to its sum.
// (54 tokens, 4 experts of 2656 x 320, cut into ranges of one unit whatever the sums
// cost: 92 us.)
struct Mx4Cost {
    int unit, fixed, each;
};

// the first half: a contributor costs 400 ns for every four tokens of a tile, which
// has M * topk / G on average
__host__ __device__ __forceinline__ Mx4Cost mx4_up_cost(int M, int topk, int G)
{
    return {850, 2500, 400 * ((M * topk / (G > 1 ? G : 1) + 3) / 4)};
}

__host__ __device__ __forceinline__ Mx4Cost mx4_down_cost(int M) { return {320, 2500, M > 32 ? 500 : 150}; }

// the estimate of S CTAs a tile and S itself in one number (~0: there are not as many)
__host__ __device__ __forceinline__ unsigned mx4_split_key(int s, int tiles, int per_tile, int grid, Mx4Cost t)
{
    if (s > per_tile || static_cast<int64_t>(s) * tiles > grid)
        return ~0u;
    const int split = (per_tile + s - 1) / s * t.unit + (s > 1 ? t.fixed + t.each * s : 0);
    return static_cast<unsigned>(split < 1 << 25 ? split : 1 << 25) << 6 | static_cast<unsigned>(s);
}

// the choice, `best` the least of the keys
__host__ __device__ __forceinline__ int mx4_share_of(unsigned best, int tiles, int per_tile, int grid, Mx4Cost t)
{
    const int64_t units = static_cast<int64_t>(tiles) * per_tile;
    const int64_t range = (units + grid - 1) / grid;
    const int64_t even = range * t.unit + t.fixed + t.each * (per_tile / (range > 1 ? range : 1) + 2);
    return best == ~0u || even <= static_cast<int64_t>(best >> 6) ? static_cast<int>(grid < units ? grid : units)
                                                                  : static_cast<int>(best & 63u) * tiles;
}

// All lanes of a converged warp call it; lane S - 1 looks at S.
__device__ __forceinline__ int mx4_share(int tiles, int per_tile, int grid, Mx4Cost t)
{
    const int s = (threadIdx.x & 31) + 1;
    return mx4_share_of(__reduce_min_sync(0xFFFFFFFFu, mx4_split_key(s, tiles, per_tile, grid, t)), tiles, per_tile, grid, t);
}

// The same on the host, for the printed plan.
inline int mx4_share_on_host(int tiles, int per_tile, int grid, Mx4Cost t)
{
    unsigned best = ~0u;
    for (int s = 1; s <= 32; ++s) {
        const unsigned key = mx4_split_key(s, tiles, per_tile, grid, t);
        best = key < best ? key : best;
    }
    return mx4_share_of(best, tiles, per_tile, grid, t);
}

// The scale tiles of one operand's stage into its 8 TMEM columns; `steps` MMAs
// of 64 values are inside K, two a tile.
__device__ __forceinline__ void mx4_copy_scales(uint32_t taddr, uint32_t saddr, int steps)
{
    tmem_cp_scales(taddr, smem_desc_scales(saddr));
    if (steps > 2)
        tmem_cp_scales(taddr + 4, smem_desc_scales(saddr + kMx4TileBytes));
}

// The MMAs of one stage (a whole warp calls; a, b: descriptors of the stage's
// operands, ta, tb: their scales in TMEM), over NACC accumulators `stride`
// columns apart in turn: an MMA of few columns is over long before its sum may be
// added to again.
template <int N, int NACC>
__device__ __forceinline__ void mx4_stage_mma(uint32_t leader, uint32_t d, uint64_t a, uint64_t b, uint32_t ta,
                                              uint32_t tb, int steps, bool first, uint32_t stride = N)
{
#pragma unroll
    for (int k = 0; k < 4; ++k)
        if (k < steps)
            mma_mx4_warp(leader, d + (k % NACC) * stride, a + 2 * k, b + 2 * k,
                         (k & 1) ? idesc_mx4(128, N, 2) : idesc_mx4(128, N, 0), ta + 4 * (k >> 1), tb + 4 * (k >> 1),
                         (first && k < NACC) ? 0u : 1u);
}

template <int V>
struct Mx4Int {
    static constexpr int value = V;
};

// Where a unit lies: tile, expert (its place in the list) and k block.  Made
// once for the first unit of a range and stepped from there: dividing 64-bit
// unit numbers in the producer's loop took it longer than the loads (32 x 28672
// x 4096: 350 ns a unit with nothing else in the loops).
struct Mx4Unit {
    int t, g, kb;
    __device__ __forceinline__ Mx4Unit(int64_t u, int64_t per_tile, int KB)
    {
        t = static_cast<int>(u / per_tile);
        const int r = static_cast<int>(u - t * per_tile);
        g = r / KB;
        kb = r - g * KB;
    }
    __device__ __forceinline__ void next(int KB, int G)
    {
        if (++kb == KB) {
            kb = 0;
            if (++g == G) {
                g = 0;
                ++t;
            }
        }
    }
};

// The weight side of a launch.  Linear: G = 1, one matrix.  Experts: the group
// list is made in the kernel from ids.
struct Mx4MoeArgs {
    const int *ids;        // [T, topk]
    const float *weights;  // [T, topk]
    int topk, E;
    unsigned long long *words;  // the first half's tile words, set back here for the next call
};

template <int BNX, int OUT, bool MOE>
__global__ void __launch_bounds__(kMx4StreamThreads, 1)
    mx4_stream_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmSW,
                      const __grid_constant__ CUtensorMap tmX, const __grid_constant__ CUtensorMap tmSX,
                      void *__restrict__ y, float *__restrict__ ws, int *__restrict__ cnt, int M, int N, int K, int ctas, int stages, int pre_wait, Mx4MoeArgs moe)
{
    using Cfg = Mx4StreamCfg<BNX>;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const bool producer = warp == 0 && lane == 0;

    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    uint8_t *gb = smem_raw + (base - raw);
    const uint32_t sW = base;
    const uint32_t sX = sW + stages * Cfg::W_BYTES;
    const uint32_t sSW = sX + stages * Cfg::X_BYTES;
    const uint32_t sSX = sSW + stages * Cfg::S_BYTES;
    const uint32_t bars = sSX + stages * Cfg::S_BYTES;
    auto full_bar = [&](int i) { return bars + 8u * i; };
    auto empty_bar = [&](int i) { return bars + 8u * (stages + i); };
    auto tfull_bar = [&](int b) { return bars + 8u * (2 * stages + b); };
    auto tempty_bar = [&](int b) { return bars + 8u * (2 * stages + 2 + b); };
    const uint32_t drain_bar = bars + 8u * (2 * stages + 4);
    auto scale_bar = [&](int i) { return bars + 8u * (2 * stages + 5 + i); };
    const uint32_t misc_off = (bars - base) + 8u * (3 * stages + 5);
    volatile uint32_t *tmem_slot = reinterpret_cast<volatile uint32_t *>(gb + misc_off);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(gb + misc_off + 4);
    volatile int *last_flag = reinterpret_cast<volatile int *>(gb + misc_off + 8);
    volatile int *n_groups = reinterpret_cast<volatile int *>(gb + misc_off + 12);
    float *wt_s = reinterpret_cast<float *>(gb + misc_off + 24);             // [2][128]
    uint32_t *wt_mask = reinterpret_cast<uint32_t *>(gb + misc_off + 24 + 1024);  // [2][4]
    uint32_t *e_mask = wt_mask + 8;
    uint16_t *e_list = reinterpret_cast<uint16_t *>(e_mask + kMx4MaxExperts / 32);
    uint16_t *chosen = e_list + kMx4MaxExperts;

    if (threadIdx.x == 32) {
        for (int i = 0; i < stages; ++i) {
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
    if (producer) {
        tma_prefetch_desc(&tmW);
        tma_prefetch_desc(&tmSW);
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

    // With pre_wait the grid before is a kernel of this library that let this
    // one start only after every earlier grid had completed: what that kernel
    // does not write (the weight, the choices) may be read before the wait.
    if (!pre_wait)
        asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    int G = 1;
    if constexpr (MOE)
        G = mx4_active_experts(moe.ids, M * moe.topk, moe.E, e_mask, e_list, chosen, n_groups);
    if (pre_wait && !producer)
        asm volatile("griddepcontrol.wait;" ::: "memory");
    if constexpr (MOE) {
        if (threadIdx.x == 64 && blockIdx.x < kMx4MaxCtas)
            moe.words[blockIdx.x] = kMx4Tag;
    }

    const int T = (N + 127) / 128;
    const int KB = (K + kMx4KB - 1) / kMx4KB;
    const int64_t per_tile = static_cast<int64_t>(G) * KB;  // units of a tile
    const int64_t U = T * per_tile;
    const int64_t C = MOE ? mx4_share(T, G * KB, ctas, mx4_down_cost(M))
                          : min(static_cast<int64_t>(ctas), U);  // CTAs with work
    const int64_t c = blockIdx.x;
    const bool works = c < C;
    const int64_t u0 = works ? dec_start(c, U, C) : 0, u1 = works ? dec_start(c + 1, U, C) : 0;
    const int64_t first_tile = works ? u0 / per_tile : 0;
    auto steps_of = [&](int kb) { return min(4, (K - kb * kMx4KB + 63) >> 6); };

    uint32_t issued_mask = 0, issued_parity = 0;
    bool mma_issued_any = false;

    if (warp == 0) {
        if (lane == 0) {
            auto load_w = [&](const Mx4Unit &c, int stage) {
                const int e = MOE ? e_list[c.g] : 0;
                tma_load_2d(sW + stage * Cfg::W_BYTES, &tmW, full_bar(stage), c.kb * 128, e * N + c.t * 128);
                tma_load_3d(sSW + stage * Cfg::S_BYTES, &tmSW, full_bar(stage), 0, c.kb * 2, e * T + c.t);
            };
            auto load_x = [&](const Mx4Unit &c, int stage) {
                tma_load_2d(sX + stage * Cfg::X_BYTES, &tmX, full_bar(stage), c.kb * 128, MOE ? c.g * M : 0);
                tma_load_3d(sSX + stage * Cfg::S_BYTES, &tmSX, full_bar(stage), 0, c.kb * 2, c.g);
            };
            Mx4Unit w(works ? u0 : 0, max(per_tile, int64_t{1}), KB), x = w;
            const int nu = static_cast<int>(u1 - u0);
            const int pre = pre_wait ? min(nu, stages) : 0;
            for (int i = 0; i < pre; ++i) {
                mbar_arrive_expect_tx(full_bar(i), Cfg::STAGE_BYTES);
                load_w(w, i);
                w.next(KB, G);
                issued_mask |= 1u << i;
            }
            if (pre_wait)
                asm volatile("griddepcontrol.wait;" ::: "memory");
            for (int i = 0; i < pre; ++i) {
                load_x(x, i);
                x.next(KB, G);
            }
            int stage = pre == stages ? 0 : pre;
            uint32_t phase = (pre == stages) ? 1u : 0u;
            for (int i = pre; i < nu; ++i) {
                if (!bounded_wait(empty_bar(stage), phase ^ 1u, kErrWaitProducer, abort_flag))
                    break;
                mbar_arrive_expect_tx(full_bar(stage), Cfg::STAGE_BYTES);
                load_w(w, stage);
                load_x(w, stage);
                w.next(KB, G);
                issued_mask |= 1u << stage;
                issued_parity = (issued_parity & ~(1u << stage)) | (phase << stage);
                if (++stage == stages) {
                    stage = 0;
                    phase ^= 1u;
                }
            }
        }
    } else if (warp == 1) {
        const uint32_t leader = elect_one();
        const uint32_t tS = tmem_base + Cfg::SCALE_COL;  // scales: 16 columns a stage
        const uint64_t w_desc = smem_desc_k_sw128(sW), x_desc = smem_desc_k_sw128(sX);
        int stage = 0;
        uint32_t phase = 0;
        int acc = 0;
        uint32_t acc_phase = 0;
        bool ok = true;
        int left = static_cast<int>(u1 - u0);
        for (int kb0 = static_cast<int>(u0 % KB); left > 0 && ok; kb0 = 0) {
            // one accumulator: the k blocks of one tile and expert
            const int kb1 = min(KB, kb0 + left);
            left -= kb1 - kb0;
            if (!warp_wait(tempty_bar(acc), acc_phase ^ 1u, kErrWaitAccEmpty, abort_flag))
                break;
            tc_fence_after_sync();
            const uint32_t d = tmem_base + static_cast<uint32_t>(acc * Cfg::NACC * BNX);
            for (int kb = kb0; kb < kb1; ++kb) {
                if (!warp_wait2(full_bar(stage), scale_bar(stage), phase, kErrWaitMma, abort_flag)) {
                    ok = false;
                    break;
                }
                __syncwarp();
                tc_fence_after_sync();
                const uint32_t t0 = tS + 16u * stage;
                mx4_stage_mma<BNX, Cfg::NACC>(leader, d, w_desc + static_cast<uint32_t>(stage * (Cfg::W_BYTES >> 4)),
                                   x_desc + static_cast<uint32_t>(stage * (Cfg::X_BYTES >> 4)), t0, t0 + 8, steps_of(kb),
                                   kb == kb0);
                mma_issued_any = true;
                mma_commit_warp(leader, empty_bar(stage));
                if (++stage == stages) {
                    stage = 0;
                    phase ^= 1u;
                }
            }
            if (!ok)
                break;
            mma_commit_warp(leader, tfull_bar(acc));
            acc ^= 1;
            if (acc == 0)
                acc_phase ^= 1u;
        }
    } else if (warp == 2) {
        if (lane == 0) {
            const uint32_t tS = tmem_base + Cfg::SCALE_COL;
            int stage = 0, last = -1;
            uint32_t phase = 0, last_phase = 0;
            int kb = static_cast<int>(u0 % KB);
            for (int left = static_cast<int>(u1 - u0); left > 0; --left) {
                if (!bounded_wait(full_bar(stage), phase, kErrWaitMma, abort_flag))
                    break;
                tc_fence_after_sync();
                const uint32_t t0 = tS + 16u * stage;
                const int steps = steps_of(kb);
                if (++kb == KB)
                    kb = 0;
                mx4_copy_scales(t0, sSW + stage * Cfg::S_BYTES, steps);
                mx4_copy_scales(t0 + 8, sSX + stage * Cfg::S_BYTES, steps);
                mma_commit(scale_bar(stage));
                last = stage;
                last_phase = phase;
                if (++stage == stages) {
                    stage = 0;
                    phase ^= 1u;
                }
            }
            // the last copies have landed before the CTA may release TMEM
            if (last >= 0)
                bounded_wait(scale_bar(last), last_phase, kErrWaitDrain, nullptr, kWaitTimeoutNs / 4);
        }
    } else {
        // epilogue warps 3..6: warp w reads TMEM lanes 32 (w % 4) .. +31
        const int quarter = warp & 3;
        const int row = quarter * 32 + lane;  // weight row within the tile
        const int et = threadIdx.x - 96;      // 0..127
        int acc = 0, wb = 0;
        uint32_t acc_phase = 0;
        auto store = [&](const float (&o)[BNX], int64_t n) {
#pragma unroll
            for (int j = 0; j < BNX; ++j)
                if (j < M) {
                    if constexpr (OUT == OUT_F32)
                        reinterpret_cast<float *>(y)[static_cast<int64_t>(j) * N + n] = o[j];
                    else
                        reinterpret_cast<__nv_bfloat16 *>(y)[static_cast<int64_t>(j) * N + n] = __float2bfloat16_rn(o[j]);
                }
        };
        if constexpr (MOE) {
            if (U == 0) {  // no token chose an expert: zeros
                const int64_t n = static_cast<int64_t>(M) * N;
                for (int64_t i = c * 128 + et; i < n; i += static_cast<int64_t>(gridDim.x) * 128) {
                    if constexpr (OUT == OUT_F32)
                        reinterpret_cast<float *>(y)[i] = 0.0f;
                    else
                        reinterpret_cast<__nv_bfloat16 *>(y)[i] = __float2bfloat16_rn(0.0f);
                }
            }
        }
        for (int64_t u = u0; u < u1;) {
            const int64_t t = u / per_tile;
            const int64_t seg_begin = u;
            const int64_t seg_end = min(u1, (t + 1) * per_tile);
            const bool whole = seg_begin == t * per_tile && seg_end == (t + 1) * per_tile;
            const int64_t n = t * 128 + row;
            // a shared tile's contributors (worked out while the tile streams)
            const int64_t cf = whole ? 0 : dec_owner(t * per_tile, U, C);
            const int64_t cl = whole ? 0 : dec_owner((t + 1) * per_tile - 1, U, C);
            const int cf_slot = !whole && dec_start(cf, U, C) < t * per_tile;
            float o[BNX];
#pragma unroll
            for (int j = 0; j < BNX; ++j)
                o[j] = 0.0f;
            while (u < seg_end) {
                const int r0 = static_cast<int>(u - t * per_tile);
                const int g = r0 / KB, kb0 = r0 - g * KB;
                u = min(seg_end, u + (KB - kb0));
                if constexpr (MOE) {
                    // this group's routing weights: thread i sums token i's
                    // choices of the expert (two buffers, as the accumulators)
                    const int e = e_list[g];
                    float w = 0.0f;
                    bool has = false;
                    if (et < M)
                        for (int k = 0; k < moe.topk; ++k)
                            if (chosen[et * moe.topk + k] == e) {
                                w += __ldg(moe.weights + et * moe.topk + k);
                                has = true;
                            }
                    wt_s[wb * 128 + et] = w;
                    const uint32_t m = __ballot_sync(0xFFFFFFFFu, has);
                    if (lane == 0)
                        wt_mask[wb * 4 + (et >> 5)] = m;
                    dec_bar_sync();
                }
                // a wait that gives up has set the error word and the abort
                // flag: the warps go on (every later wait returns at once), so
                // that their barriers stay matched
                bounded_wait(tfull_bar(acc), acc_phase, kErrWaitAccFull, abort_flag);
                __syncwarp();
                tc_fence_after_sync();
                const uint32_t lane_addr =
                    tmem_base + (static_cast<uint32_t>(quarter * 32) << 16) + static_cast<uint32_t>(acc * Cfg::NACC * BNX);
                const int parts = min(Cfg::NACC, steps_of(kb0));  // accumulators the first k block set
#pragma unroll
                for (int cc = 0; cc < BNX / 32; ++cc) {
                    const uint32_t m = MOE ? wt_mask[wb * 4 + cc] : 0u;
                    if (MOE ? m == 0u : cc * 32 >= M)
                        continue;
                    uint32_t r[32];
                    tmem_ld_32x32b_x32(lane_addr + cc * 32, r);
                    tmem_ld_wait();
#pragma unroll 1
                    for (int a = 1; a < parts; ++a) {
                        uint32_t q[32];
                        tmem_ld_32x32b_x32(lane_addr + static_cast<uint32_t>(a * BNX) + cc * 32, q);
                        tmem_ld_wait();
#pragma unroll
                        for (int j = 0; j < 32; ++j)
                            r[j] = __float_as_uint(__uint_as_float(r[j]) + __uint_as_float(q[j]));
                    }
#pragma unroll
                    for (int j = 0; j < 32; ++j) {
                        if constexpr (MOE) {
                            if (m & (1u << j))
                                o[cc * 32 + j] += wt_s[wb * 128 + cc * 32 + j] * __uint_as_float(r[j]);
                        } else {
                            o[cc * 32 + j] = __uint_as_float(r[j]);
                        }
                    }
                }
                wb ^= 1;
                tc_fence_before_sync();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(tempty_bar(acc));
                acc ^= 1;
                if (acc == 0)
                    acc_phase ^= 1u;
            }
            if (whole) {
                if (n < N)
                    store(o, n);
                continue;
            }
            // this range's part of a shared tile: 4 tokens x 128 rows at a time
            const int nv = (M + 3) >> 2;
            // only the first contributor's range may begin in an earlier tile
            auto slot_of = [&](int64_t c2) {
                return reinterpret_cast<float4 *>(ws) + (c2 * 2 + (c2 == cf ? cf_slot : 0)) * (BNX / 4 * 128);
            };
            {
                float4 *mine = reinterpret_cast<float4 *>(ws) + (c * 2 + (t == first_tile ? 0 : 1)) * (BNX / 4 * 128);
#pragma unroll
                for (int v = 0; v < BNX / 4; ++v)
                    if (v < nv)
                        mine[v * 128 + row] = make_float4(o[4 * v], o[4 * v + 1], o[4 * v + 2], o[4 * v + 3]);
            }
            dec_bar_sync();
            // release: this CTA's partial (ordered before it by the barrier)
            // precedes the count; acquire: the others' partials precede the
            // reads that follow.  A CTA is the first of at most one shared
            // tile: its number is the count's.
            if (et == 0)
                *last_flag = atom_add_acq_rel_gpu(cnt + cf, 1) == static_cast<int>(cl - cf);
            dec_bar_sync();
            if (*last_flag) {
#pragma unroll
                for (int j = 0; j < BNX; ++j)
                    o[j] = 0.0f;
                // CB contributors' loads in flight at a time (few tokens have few each)
                auto reduce = [&](auto quads, auto contributors) {
                    constexpr int Q = decltype(quads)::value, CB = decltype(contributors)::value;
                    for (int64_t c2 = cf; c2 <= cl; c2 += CB) {
                        float4 a[CB][Q];
#pragma unroll
                        for (int i = 0; i < CB; ++i) {
                            const float4 *p = slot_of(min(c2 + i, cl)) + row;
#pragma unroll
                            for (int v = 0; v < Q; ++v)
                                a[i][v] = c2 + i <= cl && v < nv ? __ldcg(p + v * 128) : make_float4(0.f, 0.f, 0.f, 0.f);
                        }
#pragma unroll
                        for (int i = 0; i < CB; ++i)
#pragma unroll
                            for (int v = 0; v < Q; ++v) {
                                o[4 * v] += a[i][v].x;
                                o[4 * v + 1] += a[i][v].y;
                                o[4 * v + 2] += a[i][v].z;
                                o[4 * v + 3] += a[i][v].w;
                            }
                    }
                };
                if (nv <= 1)
                    reduce(Mx4Int<1>{}, Mx4Int<8>{});
                else if (nv <= 4)
                    reduce(Mx4Int<4>{}, Mx4Int<4>{});
                else if constexpr (BNX <= 64)
                    reduce(Mx4Int<BNX / 4>{}, Mx4Int<BNX == 32 ? 2 : 1>{});
                else
                    reduce(Mx4Int<BNX / 4>{}, Mx4Int<1>{});
                if (n < N)
                    store(o, n);
            }
            dec_bar_sync();  // last_flag is rewritten by the next shared tile
        }
    }

    // ---- teardown ------------------------------------------------------------
    if (warp == 1 && *abort_flag && mma_issued_any) {
        __syncwarp();
        mma_commit_warp(elect_one(), drain_bar);
        bounded_wait(drain_bar, 0, kErrWaitDrain, nullptr, kWaitTimeoutNs / 4);
    }
    if (warp == 0 && lane == 0 && *abort_flag) {
        for (int i = 0; i < stages; ++i)
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
