// sq_mx4_api.cu -- the microscaled 4-bit entry points of the C ABI (declared
// in include/sq.h): argument validation on the host, tensor maps and launches.
// No entry point allocates memory; no C++ exception crosses the interface.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstdio>

#include "sq.h"
#include "sq_host.cuh"
#include "sq_mx4.cuh"
#include "sq_mx4_gemm.cuh"
#include "sq_mx4_moe.cuh"
#include "sq_mx4_stream.cuh"
#include "sq_resnorm.cuh"

namespace sq {

cudaError_t mx4_read_device_error(unsigned int *code)
{
    return cudaMemcpyFromSymbol(code, g_sq_device_error, sizeof *code);
}

cudaError_t mx4_clear_device_error()
{
    const unsigned int zero = 0;
    return cudaMemcpyToSymbol(g_sq_device_error, &zero, sizeof zero);
}

}  // namespace sq

namespace {

using sq::OUT_BF16;
using sq::OUT_F32;

inline size_t round256(size_t v) { return (v + 255) / 256 * 256; }

inline bool ok_ptr(const void *p) { return p != nullptr && aligned16(p); }

constexpr int64_t kMx4MaxDim = int64_t{1} << 24;  // rows and columns: TMA coordinates and the kernels' int sizes

inline bool mx4_dims(int64_t rows, int64_t K) { return rows >= 1 && K >= 32 && K % 32 == 0; }

inline size_t scale_bytes(int64_t rows, int64_t K)
{
    return static_cast<size_t>((rows + 127) / 128) * static_cast<size_t>((K + 127) / 128) * sq::kMx4TileBytes;
}

// ---- quantiser and read-back ---------------------------------------------------
// The CTA covers 2^log2tx chunks of 8 columns; the row bands fill every SM
// about eight times over.
struct Mx4Walk {
    int log2tx, band;
    unsigned gx, gy;
};

inline Mx4Walk mx4_walk(int64_t rows, int64_t K, int64_t sms)
{
    Mx4Walk w;
    const int64_t chunks = (K + 127) / 128 * 16;
    w.log2tx = chunks <= 16 ? 4 : 5;
    const int64_t TX = int64_t{1} << w.log2tx, step = sq::kMx4Threads / TX * 4;
    const int64_t gx = (chunks + TX - 1) / TX;
    const int64_t want = std::max<int64_t>(1, sms * 8 / gx);
    int64_t band = std::max<int64_t>(step, ((rows + want - 1) / want + step - 1) / step * step);
    while ((rows + band - 1) / band > 65535)
        band *= 2;
    w.band = static_cast<int>(band);
    w.gx = static_cast<unsigned>(gx);
    w.gy = static_cast<unsigned>((rows + band - 1) / band);
    return w;
}

template <typename T>
sq_status launch_mx4_quant(const T *x, int64_t rows, int64_t K, const float *s, int op, uint8_t *q, uint8_t *sc,
                           cudaStream_t st, int *zero, int nzero)
{
    DeviceInfo di;
    if (!device_info(di))
        return SQ_ERR_CUDA;
    const Mx4Walk w = mx4_walk(rows, K, di.sms);
    auto kernel = s == nullptr ? sq::mx4_quant_kernel<T, sq::MX4_PLAIN>
                               : (op == sq::MX4_TIMES ? sq::mx4_quant_kernel<T, sq::MX4_TIMES>
                                                      : sq::mx4_quant_kernel<T, sq::MX4_OVER>);
    return launch_kernel(kernel, dim3(w.gx, w.gy), dim3(sq::kMx4Threads), 0, st, 0, 0, x, static_cast<int>(rows),
                         static_cast<int>(K), s, q, sc, w.log2tx,
                         w.band, zero, nzero);
}

sq_status mx4_quant(const void *x, sq_dtype dt, int64_t rows, int64_t K, const float *s, int op, uint8_t *q, uint8_t *sc,
                    cudaStream_t st, int *zero = nullptr, int nzero = 0)
{
    return dt == SQ_BF16
               ? launch_mx4_quant(static_cast<const __nv_bfloat16 *>(x), rows, K, s, op, q, sc, st, zero, nzero)
               : launch_mx4_quant(static_cast<const float *>(x), rows, K, s, op, q, sc, st, zero, nzero);
}

sq_status check_mx4_quant(const void *x, sq_dtype dt, int64_t rows, int64_t K, const float *s, const void *q,
                          const void *sc)
{
    if (!ok_ptr(x) || !valid_dtype(dt) || !mx4_dims(rows, K) || !aligned16(s) || !ok_ptr(q) || !ok_ptr(sc))
        return SQ_ERR_INVALID_ARG;
    if (rows > kMx4MaxDim || K > kMx4MaxDim)
        return SQ_ERR_UNSUPPORTED;
    return SQ_OK;
}

// ---- products ------------------------------------------------------------------
// codes [rows, K / 2]: box of 128 bytes x box_rows rows, 128-byte swizzle
bool make_tmap_mx4(CUtensorMap *map, const uint8_t *codes, int64_t rows, int64_t K, int box_rows)
{
    return make_tmap_i8(map, codes, rows, K / 2, box_rows);
}

// scale tiles [row tiles, k tiles, 512 bytes]: box of box_rt row tiles x 2 k
// tiles, a tile's 512 bytes contiguous; zeros outside
bool make_tmap_scales(CUtensorMap *map, const uint8_t *scales, int64_t row_tiles, int64_t K, int box_rt)
{
    auto fn = encode_fn();
    if (fn == nullptr)
        return false;
    const int64_t KT = (K + 127) / 128;
    cuuint64_t dims[3] = {128, static_cast<cuuint64_t>(KT), static_cast<cuuint64_t>(row_tiles)};
    cuuint64_t strides[2] = {512, static_cast<cuuint64_t>(KT * 512)};
    cuuint32_t box[3] = {128, 2, static_cast<cuuint32_t>(box_rt)};
    cuuint32_t estr[3] = {1, 1, 1};
    CUresult r = fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT32, 3, const_cast<uint8_t *>(scales), dims, strides, box, estr,
                    CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                    CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS;
}

using sq::kMx4MaxCtas;

inline int mx4_bnx(int64_t M) { return M <= 32 ? 32 : (M <= 64 ? 64 : 128); }

constexpr size_t kMx4Words = kMx4MaxCtas * sizeof(unsigned long long);  // a tagged tile count for each CTA
constexpr size_t kMx4Counts = kMx4MaxCtas * sizeof(int);                // a plain one

// Workspace of the product for few tokens: the tile counts, then two partial
// tiles a CTA.  More tokens need none.
struct Mx4Ws {
    size_t cnt = 0, slots = 0, total = 0;
    bool few = false;
};

inline Mx4Ws mx4_ws(int64_t M, size_t base)
{
    Mx4Ws w;
    w.total = base;
    if (M > sq::kMx4MaxTokens)
        return w;
    w.few = true;
    w.cnt = base;
    w.slots = base + round256(kMx4Counts);
    w.total = w.slots + static_cast<size_t>(kMx4MaxCtas) * 2 * mx4_bnx(M) * 128 * sizeof(float);
    return w;
}

template <int BNX, int OUT>
sq_status launch_mx4_stream(const uint8_t *xq, const uint8_t *sx, const uint8_t *wq, const uint8_t *sw, int64_t M,
                            int64_t N, int64_t K, void *y, int *cnt, float *slots, cudaStream_t st)
{
    using Cfg = sq::Mx4StreamCfg<BNX>;
    DeviceInfo di;
    if (!device_info(di))
        return SQ_ERR_CUDA;
    auto kernel = sq::mx4_stream_kernel<BNX, OUT, false>;
    static std::atomic<uint64_t> attr_done{0};
    if (!ensure_smem_attr(kernel, kMaxDynSmem, attr_done))
        return SQ_ERR_CUDA;
    CUtensorMap tw, tsw, tx, tsx;
    if (!make_tmap_mx4(&tw, wq, N, K, 128) || !make_tmap_scales(&tsw, sw, (N + 127) / 128, K, 1) ||
        !make_tmap_mx4(&tx, xq, M, K, BNX) || !make_tmap_scales(&tsx, sx, 1, K, 1))
        return SQ_ERR_CUDA;
    const int64_t T = (N + 127) / 128, KB = (K + sq::kMx4KB - 1) / sq::kMx4KB;
    const int64_t G = stream_ctas(M, T, KB, std::min<int64_t>(di.sms, kMx4MaxCtas));
    const int stages = Cfg::MAX_STAGES;
    const int smem = sq::mx4_stream_smem(Cfg::STAGE_BYTES, stages, false);
    static_assert(sq::mx4_stream_smem(Cfg::STAGE_BYTES, Cfg::MAX_STAGES, false) <= kMaxDynSmem, "shared memory");
    if (debug_plan())
        std::fprintf(stderr, "sq mx4 stream M=%lld N=%lld K=%lld: BNX=%d ctas=%lld stages=%d\n", (long long)M,
                     (long long)N, (long long)K, BNX, (long long)G, stages);
    return launch_kernel(kernel, dim3(static_cast<unsigned>(G)), dim3(sq::kMx4StreamThreads), smem, st, 0, 0, tw, tsw, tx,
                         tsx, y, slots, cnt, static_cast<int>(M), static_cast<int>(N),
                         static_cast<int>(K), static_cast<int>(G), stages, 0, sq::Mx4MoeArgs{});
}

template <int BN, int OUT>
sq_status launch_mx4_pair_cfg(const uint8_t *xq, const uint8_t *sx, const uint8_t *wq, const uint8_t *sw, int64_t M,
                              int64_t N, int64_t K, void *y, cudaStream_t st)
{
    using Cfg = sq::Mx4PairCfg<BN>;
    auto kernel = sq::mx4_pair_kernel<BN, OUT>;
    static std::atomic<uint64_t> attr_done{0};
    if (!ensure_smem_attr(kernel, Cfg::SMEM_BYTES, attr_done))
        return SQ_ERR_CUDA;
    const int active = active_clusters(kernel, 2, Cfg::SMEM_BYTES, sq::kMx4PairThreads);
    if (active <= 0)
        return SQ_ERR_CUDA;
    const int64_t tiles = ((M + sq::kPairBM - 1) / sq::kPairBM) * ((N + BN - 1) / BN);
    if (tiles > INT_MAX / 2)
        return SQ_ERR_UNSUPPORTED;
    CUtensorMap ta, tsa, tb, tsb;
    if (!make_tmap_mx4(&ta, xq, M, K, 128) || !make_tmap_scales(&tsa, sx, (M + 127) / 128, K, 1) ||
        !make_tmap_mx4(&tb, wq, N, K, BN / 2) || !make_tmap_scales(&tsb, sw, (N + 127) / 128, K, Cfg::RT_B))
        return SQ_ERR_CUDA;
    const int64_t pairs = std::min<int64_t>(tiles, active);
    if (debug_plan())
        std::fprintf(stderr, "sq mx4 pair M=%lld N=%lld K=%lld: BN=%d stages=%d tiles=%lld pairs=%lld\n", (long long)M,
                     (long long)N, (long long)K, BN, Cfg::STAGES, (long long)tiles, (long long)pairs);
    return launch_kernel(kernel, dim3(static_cast<unsigned>(2 * pairs)), dim3(sq::kMx4PairThreads), Cfg::SMEM_BYTES, st, 2,
                         1, ta, tsa, tb, tsb, y, static_cast<int>(M), static_cast<int>(N), static_cast<int>(K), 8);
}

// Tile width: the fewest rounds of tiles over the pairs, a round costing one
// tile's time.  A tile's time is far from proportional to its width (an MMA of
// N = 128 takes as long as one of 256): at 8192 x 8192 x 28672 a 256 / 192 /
// 128-wide tile took 50.1 / 43.2 / 34.1 us, which gives the weights below.
inline int pick_mx4_bn(int64_t M, int64_t N, int64_t pairs)
{
    constexpr int cand[3] = {256, 192, 128};
    constexpr int64_t tile_time[3] = {100, 86, 68};
    const int64_t mt = (M + sq::kPairBM - 1) / sq::kPairBM;
    int best = 256;
    int64_t best_cost = INT64_MAX;
    for (int i = 0; i < 3; ++i) {
        const int64_t tiles = mt * ((N + cand[i] - 1) / cand[i]);
        const int64_t cost = (tiles + pairs - 1) / pairs * tile_time[i];
        if (cost < best_cost) {
            best_cost = cost;
            best = cand[i];
        }
    }
    return best;
}

template <int OUT>
sq_status launch_mx4_pair(const uint8_t *xq, const uint8_t *sx, const uint8_t *wq, const uint8_t *sw, int64_t M,
                          int64_t N, int64_t K, void *y, cudaStream_t st)
{
    DeviceInfo di;
    if (!device_info(di))
        return SQ_ERR_CUDA;
    switch (pick_mx4_bn(M, N, std::max(di.sms / 2, 1))) {
    case 256: return launch_mx4_pair_cfg<256, OUT>(xq, sx, wq, sw, M, N, K, y, st);
    case 192: return launch_mx4_pair_cfg<192, OUT>(xq, sx, wq, sw, M, N, K, y, st);
    default: return launch_mx4_pair_cfg<128, OUT>(xq, sx, wq, sw, M, N, K, y, st);
    }
}

// cnt: the tile counts, cleared by the kernel right before on the stream
template <int OUT>
sq_status launch_mx4_gemm(const uint8_t *xq, const uint8_t *sx, const uint8_t *wq, const uint8_t *sw, int64_t M,
                          int64_t N, int64_t K, void *y, int *cnt, float *slots, cudaStream_t st)
{
    if (M > sq::kMx4MaxTokens)
        return launch_mx4_pair<OUT>(xq, sx, wq, sw, M, N, K, y, st);
    switch (mx4_bnx(M)) {
    case 32: return launch_mx4_stream<32, OUT>(xq, sx, wq, sw, M, N, K, y, cnt, slots, st);
    case 64: return launch_mx4_stream<64, OUT>(xq, sx, wq, sw, M, N, K, y, cnt, slots, st);
    default: return launch_mx4_stream<128, OUT>(xq, sx, wq, sw, M, N, K, y, cnt, slots, st);
    }
}

sq_status check_mx4_gemm_dims(int64_t M, int64_t N, int64_t K)
{
    if (!mx4_dims(M, K) || N < 16 || N % 16 != 0)
        return SQ_ERR_INVALID_ARG;
    if (M > kMx4MaxDim || N > kMx4MaxDim || K > kMx4MaxDim)
        return SQ_ERR_UNSUPPORTED;
    return SQ_OK;
}

__global__ void mx4_clear_kernel(int *p, int n)
{
    sq::pdl_prologue();
    for (int i = threadIdx.x; i < n; i += blockDim.x)
        p[i] = 0;
}

// Workspace of sq_mx4_linear: codes and scales of x, then the product's.
struct Mx4LinearWs {
    size_t sx = 0;
    Mx4Ws g;
};

inline Mx4LinearWs mx4_linear_ws(int64_t M, int64_t N, int64_t K)
{
    Mx4LinearWs w;
    w.sx = round256(static_cast<size_t>(M) * static_cast<size_t>(K / 2));
    w.g = mx4_ws(M, w.sx + scale_bytes(M, K));
    return w;
}

// ---- experts layer for few tokens ------------------------------------------------
// Workspace: h's codes and scale tiles (a tile per expert in use and 128
// values), the two halves' tile counts, and partial tiles (the first half's, two
// accumulators each; the second half's are fewer).
struct Mx4MoeWs {
    size_t hs = 0, words = 0, cnt = 0, slots = 0, total = 0;
    int64_t groups = 0;  // experts that can be in use at once
};

inline Mx4MoeWs mx4_moe_ws(int64_t T, int64_t topk, int64_t E, int64_t I)
{
    Mx4MoeWs w;
    w.groups = std::min(E, T * topk);
    w.hs = round256(static_cast<size_t>(w.groups * T) * static_cast<size_t>(I / 2));
    w.words = w.hs + static_cast<size_t>(w.groups) * scale_bytes(1, I);
    w.cnt = w.words + round256(kMx4Words);
    w.slots = w.cnt + round256(kMx4Counts);
    w.total = w.slots + static_cast<size_t>(kMx4MaxCtas) * 2 * 2 * mx4_bnx(T) * 128 * sizeof(float);
    return w;
}

sq_status check_mx4_moe_dims(int64_t T, int64_t topk, int64_t E, int64_t H, int64_t I)
{
    if (T < 1 || topk < 1 || E < 1 || !mx4_dims(1, H) || !mx4_dims(1, I))
        return SQ_ERR_INVALID_ARG;
    if (T > sq::kMx4MaxTokens || topk > sq::kMx4MaxSlots || T * topk > sq::kMx4MaxSlots || E > sq::kMx4MaxExperts ||
        H > kMx4MaxDim || I > kMx4MaxDim || E * std::max(H, I) > (int64_t{1} << 30))
        return SQ_ERR_UNSUPPORTED;
    return SQ_OK;
}

struct Mx4MoeCall {
    const uint8_t *xq, *sx, *wg, *sg, *wu, *su, *wd, *sd;
    sq::Mx4MoeArgs route;
    int64_t T, H, I;
    void *y;
    uint8_t *ws;
    Mx4MoeWs L;
};

template <int BNX, int OUT>
sq_status launch_mx4_moe(const Mx4MoeCall &c, cudaStream_t st)
{
    using Up = sq::Mx4UpCfg<BNX>;
    using Cfg = sq::Mx4StreamCfg<BNX>;
    DeviceInfo di;
    if (!device_info(di))
        return SQ_ERR_CUDA;
    auto up = sq::mx4_moe_up_kernel<BNX>;
    auto down = sq::mx4_stream_kernel<BNX, OUT, true>;
    static std::atomic<uint64_t> up_done{0}, down_done{0};
    if (!ensure_smem_attr(up, Up::SMEM_BYTES, up_done) || !ensure_smem_attr(down, kMaxDynSmem, down_done))
        return SQ_ERR_CUDA;
    uint8_t *hq = c.ws, *hs = c.ws + c.L.hs;
    int *cnt = reinterpret_cast<int *>(c.ws + c.L.cnt);
    float *slots = reinterpret_cast<float *>(c.ws + c.L.slots);
    const int64_t E = c.route.E, RI = (c.I + 127) / 128, RH = (c.H + 127) / 128;
    CUtensorMap tg, tsg, tu, tsu, tx, tsx, td, tsd, th, tsh;
    if (!make_tmap_mx4(&tg, c.wg, E * c.I, c.H, 128) || !make_tmap_scales(&tsg, c.sg, E * RI, c.H, 1) ||
        !make_tmap_mx4(&tu, c.wu, E * c.I, c.H, 128) || !make_tmap_scales(&tsu, c.su, E * RI, c.H, 1) ||
        !make_tmap_mx4(&tx, c.xq, c.T, c.H, BNX) || !make_tmap_scales(&tsx, c.sx, 1, c.H, 1) ||
        !make_tmap_mx4(&td, c.wd, E * c.H, c.I, 128) || !make_tmap_scales(&tsd, c.sd, E * RH, c.I, 1) ||
        !make_tmap_mx4(&th, hq, c.L.groups * c.T, c.I, BNX) || !make_tmap_scales(&tsh, hs, c.L.groups, c.I, 1))
        return SQ_ERR_CUDA;
    const int ctas = static_cast<int>(std::min<int64_t>(di.sms, kMx4MaxCtas));
    if (debug_plan()) {  // with as many experts in use as there can be (the kernels know how many there are)
        const int G = static_cast<int>(c.L.groups), T = static_cast<int>(c.T), topk = c.route.topk;
        const int ut = G * static_cast<int>(RI), un = static_cast<int>((c.H + sq::kMx4KB - 1) / sq::kMx4KB);
        const int dt = static_cast<int>(RH), dn = G * static_cast<int>((c.I + sq::kMx4KB - 1) / sq::kMx4KB);
        std::fprintf(stderr, "sq mx4 moe T=%d topk=%d E=%lld H=%lld I=%lld: BNX=%d experts=%d up tiles=%d units=%d ctas=%d "
                     "down tiles=%d units=%d ctas=%d\n", T, topk, (long long)E, (long long)c.H, (long long)c.I, BNX, G, ut, un,
                     sq::mx4_share_on_host(ut, un, ctas, sq::mx4_up_cost(T, topk, G)), dt, dn,
                     sq::mx4_share_on_host(dt, dn, ctas, sq::mx4_down_cost(T)));
    }
    sq_status r = launch_kernel(up, dim3(static_cast<unsigned>(ctas)), dim3(sq::kMx4UpThreads), Up::SMEM_BYTES, st, 0, 0,
                                tg, tsg, tu, tsu, tx, tsx, hq, hs, slots, c.route.words, cnt, static_cast<int>(c.T),
                                static_cast<int>(c.H), static_cast<int>(c.I), c.route);
    // what the first half counts is set back by the second; without that one the
    // next call on this workspace would go by it
    auto uncounted = [&](sq_status err) {
        launch_kernel(mx4_clear_kernel, dim3(1), dim3(kMx4MaxCtas), 0, st, 0, 0, reinterpret_cast<int *>(c.route.words),
                      static_cast<int>(kMx4Words / sizeof(int)));
        return err;
    };
    if (r != SQ_OK)
        return uncounted(r);
    constexpr int stages = BNX == 128 ? 6 : 8;
    constexpr int smem = sq::mx4_stream_smem(Cfg::STAGE_BYTES, stages, true);
    static_assert(smem <= kMaxDynSmem && stages <= Cfg::MAX_STAGES, "shared memory");
    r = launch_kernel(down, dim3(static_cast<unsigned>(ctas)), dim3(sq::kMx4StreamThreads), smem, st, 0, 0, td, tsd, th, tsh,
                      c.y, slots, cnt, static_cast<int>(c.T), static_cast<int>(c.H), static_cast<int>(c.I), ctas,
                      stages, 1, c.route);
    return r == SQ_OK ? r : uncounted(r);
}

template <int OUT>
sq_status launch_mx4_moe_bnx(const Mx4MoeCall &c, cudaStream_t st)
{
    switch (mx4_bnx(c.T)) {
    case 32: return launch_mx4_moe<32, OUT>(c, st);
    case 64: return launch_mx4_moe<64, OUT>(c, st);
    default: return launch_mx4_moe<128, OUT>(c, st);
    }
}

// ---- norms around a block --------------------------------------------------------
template <typename T, bool MX4, int CH, int THREADS, bool CACHE, int BLOCKS>
sq_status launch_res_norm_cfg(const sq::ResArgs &p, int64_t sms, cudaStream_t st)
{
    auto kernel = sq::res_norm_kernel<T, MX4, CH, THREADS, CACHE, BLOCKS>;
    const int smem = CACHE ? static_cast<int>(2 * p.K * sizeof(float)) : 0;
    static std::atomic<uint64_t> attr_done{0};
    if (CACHE && !ensure_smem_attr(kernel, kMaxDynSmem - 2048, attr_done))
        return SQ_ERR_CUDA;
    const int64_t blocks = CACHE ? std::min<int64_t>(p.M, BLOCKS * sms) : p.M;  // with CACHE one wave
    return launch_kernel(kernel, dim3(static_cast<unsigned>(blocks)), dim3(THREADS), smem, st, 0, 0, p);
}

// Few rows: every row spread over 512 threads.  Enough rows for several a CTA:
// the factors staged in shared memory, as many warps on an SM as the registers
// of a row's chunks allow.
template <typename T, bool MX4>
sq_status launch_res_norm(const sq::ResArgs &p, cudaStream_t st)
{
    DeviceInfo di;
    if (!device_info(di))
        return SQ_ERR_CUDA;
    const int64_t chunks = p.K / 8, sms = di.sms;
    constexpr bool W = sizeof(T) == 2;
    if (p.M < 4 * sms) {
        if (chunks <= 512)
            return launch_res_norm_cfg<T, MX4, 1, 512, false, 2>(p, sms, st);
        if (chunks <= 1024)
            return launch_res_norm_cfg<T, MX4, 2, 512, false, 2>(p, sms, st);
    } else {
        if (chunks <= 256)
            return launch_res_norm_cfg<T, MX4, 1, 256, true, 4>(p, sms, st);
        if (chunks <= 512)
            return launch_res_norm_cfg<T, MX4, 2, 256, true, W ? 4 : 2>(p, sms, st);
        if (chunks <= 1024 && MX4)
            return launch_res_norm_cfg<T, MX4, 4, 256, true, 2>(p, sms, st);
        if (chunks <= 1024)  // the int8 codes' second pass over the row: more threads (88 against 96 us)
            return launch_res_norm_cfg<T, MX4, 2, 512, true, W ? 2 : 1>(p, sms, st);
    }
    if constexpr (W)
        if (chunks > 2048)
            return launch_res_norm_cfg<T, MX4, 8, 512, false, 1>(p, sms, st);
    return launch_res_norm_cfg<T, MX4, 4, 512, false, 1>(p, sms, st);
}

// gate_tokens: tokens that share a gate row; gate and gamma may be NULL
sq_status residual_norm(const void *b, sq_dtype dt, int64_t M, int64_t K, const float *gamma, const void *gate,
                        int64_t gate_tokens, float c, const void *r, void *r_out, const float *g, float eps, uint8_t *q,
                        void *sx, bool mx4, sq_stream_t stream)
{
    if (!ok_ptr(b) || !valid_dtype(dt) || M < 1 || K < 16 || K % (mx4 ? 32 : 16) != 0 || !aligned16(gamma) ||
        !aligned16(gate) || (gate != nullptr && gate_tokens < 1) || !std::isfinite(c) || !ok_ptr(r) || !ok_ptr(r_out) ||
        b == r_out || !ok_ptr(g) || !(eps >= 0.0f) || !std::isfinite(eps) || !ok_ptr(q) || !ok_ptr(sx))
        return SQ_ERR_INVALID_ARG;
    if (K > (dt == SQ_BF16 ? 32768 : 16384) || M > kMx4MaxDim)
        return SQ_ERR_UNSUPPORTED;
    const sq::ResArgs p{b, r, gate, gamma, g, r_out, q, sx, M, K, gate == nullptr ? 1 : gate_tokens, c, eps};
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (dt == SQ_BF16)
        return mx4 ? launch_res_norm<__nv_bfloat16, true>(p, st) : launch_res_norm<__nv_bfloat16, false>(p, st);
    return mx4 ? launch_res_norm<float, true>(p, st) : launch_res_norm<float, false>(p, st);
}

}  // namespace

extern "C" {

size_t sq_mx4_scale_size(int64_t rows, int64_t K) { return mx4_dims(rows, K) ? scale_bytes(rows, K) : 0; }

sq_status sq_mx4_quant_act(const void *x, sq_dtype dt, int64_t M, int64_t K, const float *s, uint8_t *xq, uint8_t *sx,
                           sq_stream_t stream)
{
    const sq_status r = check_mx4_quant(x, dt, M, K, s, xq, sx);
    return r != SQ_OK ? r : mx4_quant(x, dt, M, K, s, sq::MX4_OVER, xq, sx, reinterpret_cast<cudaStream_t>(stream));
}

sq_status sq_mx4_quant_weight(const void *w, sq_dtype dt, int64_t N, int64_t K, const float *s, uint8_t *wq,
                              uint8_t *sw, sq_stream_t stream)
{
    const sq_status r = check_mx4_quant(w, dt, N, K, s, wq, sw);
    return r != SQ_OK ? r : mx4_quant(w, dt, N, K, s, sq::MX4_TIMES, wq, sw, reinterpret_cast<cudaStream_t>(stream));
}

sq_status sq_mx4_dequant(const uint8_t *q, const uint8_t *sc, int64_t rows, int64_t K, void *out, sq_dtype out_dt,
                         sq_stream_t stream)
{
    const sq_status r = check_mx4_quant(out, out_dt, rows, K, nullptr, q, sc);
    if (r != SQ_OK)
        return r;
    DeviceInfo di;
    if (!device_info(di))
        return SQ_ERR_CUDA;
    const Mx4Walk w = mx4_walk(rows, K, di.sms);
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (out_dt == SQ_BF16)
        return launch_kernel(sq::mx4_dequant_kernel<__nv_bfloat16>, dim3(w.gx, w.gy), dim3(sq::kMx4Threads), 0, st, 0, 0,
                             q, sc, static_cast<int>(rows), static_cast<int>(K), static_cast<__nv_bfloat16 *>(out), w.log2tx, w.band);
    return launch_kernel(sq::mx4_dequant_kernel<float>, dim3(w.gx, w.gy), dim3(sq::kMx4Threads), 0, st, 0, 0, q, sc,
                         static_cast<int>(rows), static_cast<int>(K), static_cast<float *>(out), w.log2tx, w.band);
}

size_t sq_mx4_gemm_workspace_size(int64_t M, int64_t N, int64_t K)
{
    return check_mx4_gemm_dims(M, N, K) == SQ_OK ? mx4_ws(M, 0).total : 0;
}

sq_status sq_mx4_gemm(const uint8_t *xq, const uint8_t *sx, const uint8_t *wq, const uint8_t *sw, int64_t M, int64_t N,
                      int64_t K, void *y, sq_dtype out_dt, void *workspace, size_t ws_bytes, sq_stream_t stream)
{
    if (!ok_ptr(xq) || !ok_ptr(sx) || !ok_ptr(wq) || !ok_ptr(sw) || !ok_ptr(y) || !valid_dtype(out_dt))
        return SQ_ERR_INVALID_ARG;
    sq_status r = check_mx4_gemm_dims(M, N, K);
    if (r != SQ_OK)
        return r;
    const Mx4Ws w = mx4_ws(M, 0);
    if (w.total > 0 && (!ok_ptr(workspace) || ws_bytes < w.total))
        return SQ_ERR_INVALID_ARG;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    int *cnt = w.few ? reinterpret_cast<int *>(static_cast<uint8_t *>(workspace) + w.cnt) : nullptr;
    float *slots = w.few ? reinterpret_cast<float *>(static_cast<uint8_t *>(workspace) + w.slots) : nullptr;
    if (w.few) {
        r = launch_kernel(mx4_clear_kernel, dim3(1), dim3(kMx4MaxCtas), 0, st, 0, 0, cnt, static_cast<int>(kMx4MaxCtas));
        if (r != SQ_OK)
            return r;
    }
    return out_dt == SQ_BF16 ? launch_mx4_gemm<OUT_BF16>(xq, sx, wq, sw, M, N, K, y, cnt, slots, st)
                             : launch_mx4_gemm<OUT_F32>(xq, sx, wq, sw, M, N, K, y, cnt, slots, st);
}

size_t sq_mx4_linear_workspace_size(int64_t M, int64_t N, int64_t K)
{
    return check_mx4_gemm_dims(M, N, K) == SQ_OK ? mx4_linear_ws(M, N, K).g.total : 0;
}

sq_status sq_mx4_linear(const void *x, sq_dtype in_dt, const float *s, const uint8_t *wq, const uint8_t *sw, int64_t M,
                        int64_t N, int64_t K, void *y, sq_dtype out_dt, void *workspace, size_t ws_bytes,
                        sq_stream_t stream)
{
    if (!ok_ptr(x) || !valid_dtype(in_dt) || !aligned16(s) || !ok_ptr(wq) || !ok_ptr(sw) || !ok_ptr(y) ||
        !valid_dtype(out_dt))
        return SQ_ERR_INVALID_ARG;
    sq_status r = check_mx4_gemm_dims(M, N, K);
    if (r != SQ_OK)
        return r;
    const Mx4LinearWs L = mx4_linear_ws(M, N, K);
    if (!ok_ptr(workspace) || ws_bytes < L.g.total)
        return SQ_ERR_INVALID_ARG;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    uint8_t *xq = static_cast<uint8_t *>(workspace), *sx = xq + L.sx;
    int *cnt = L.g.few ? reinterpret_cast<int *>(xq + L.g.cnt) : nullptr;
    float *slots = L.g.few ? reinterpret_cast<float *>(xq + L.g.slots) : nullptr;
    r = mx4_quant(x, in_dt, M, K, s, sq::MX4_OVER, xq, sx, st, cnt, L.g.few ? static_cast<int>(kMx4MaxCtas) : 0);
    if (r != SQ_OK)
        return r;
    return out_dt == SQ_BF16 ? launch_mx4_gemm<OUT_BF16>(xq, sx, wq, sw, M, N, K, y, cnt, slots, st)
                             : launch_mx4_gemm<OUT_F32>(xq, sx, wq, sw, M, N, K, y, cnt, slots, st);
}

size_t sq_mx4_moe_workspace_size(int64_t T, int64_t topk, int64_t E, int64_t H, int64_t I)
{
    return check_mx4_moe_dims(T, topk, E, H, I) == SQ_OK ? mx4_moe_ws(T, topk, E, I).total : 0;
}

sq_status sq_mx4_moe(const uint8_t *xq, const uint8_t *sx, const int32_t *ids, const float *weights, int64_t T,
                     int64_t topk, int64_t E, int64_t H, int64_t I, const uint8_t *wg, const uint8_t *sg,
                     const uint8_t *wu, const uint8_t *su, const uint8_t *wd, const uint8_t *sd, void *y,
                     sq_dtype out_dt, void *workspace, size_t ws_bytes, sq_stream_t stream)
{
    if (!ok_ptr(xq) || !ok_ptr(sx) || !ok_ptr(ids) || !ok_ptr(weights) || !ok_ptr(wg) || !ok_ptr(sg) || !ok_ptr(wu) ||
        !ok_ptr(su) || !ok_ptr(wd) || !ok_ptr(sd) || !ok_ptr(y) || !valid_dtype(out_dt))
        return SQ_ERR_INVALID_ARG;
    const sq_status r = check_mx4_moe_dims(T, topk, E, H, I);
    if (r != SQ_OK)
        return r;
    const Mx4MoeWs L = mx4_moe_ws(T, topk, E, I);
    if (!ok_ptr(workspace) || ws_bytes < L.total)
        return SQ_ERR_INVALID_ARG;
    const Mx4MoeCall c{xq, sx, wg, sg, wu, su, wd, sd, {ids, weights, static_cast<int>(topk), static_cast<int>(E),
                        reinterpret_cast<unsigned long long *>(static_cast<uint8_t *>(workspace) + L.words)},
                       T,  H,  I,  y,  static_cast<uint8_t *>(workspace), L};
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    return out_dt == SQ_BF16 ? launch_mx4_moe_bnx<OUT_BF16>(c, st) : launch_mx4_moe_bnx<OUT_F32>(c, st);
}

sq_status sq_residual_norm_quant(const void *b, sq_dtype dt, int64_t M, int64_t K, const float *gamma,
                                 const void *gate, int64_t gate_tokens, float c, const void *r, void *r_out,
                                 const float *g, float eps, int8_t *xq, float *sx, sq_stream_t stream)
{
    return residual_norm(b, dt, M, K, gamma, gate, gate_tokens, c, r, r_out, g, eps, reinterpret_cast<uint8_t *>(xq), sx,
                         false, stream);
}

sq_status sq_residual_norm_quant_mx4(const void *b, sq_dtype dt, int64_t M, int64_t K, const float *gamma,
                                     const void *gate, int64_t gate_tokens, float c, const void *r, void *r_out,
                                     const float *g, float eps, uint8_t *xq, uint8_t *sx, sq_stream_t stream)
{
    return residual_norm(b, dt, M, K, gamma, gate, gate_tokens, c, r, r_out, g, eps, xq, sx, true, stream);
}

}  // extern "C"
