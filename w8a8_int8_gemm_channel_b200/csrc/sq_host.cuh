// sq_host.cuh -- host-side helpers shared by the library's translation units:
// argument predicates, cached device facts, the launch wrapper (programmatic
// dependent launch, cluster shape), tensor maps and per-kernel attributes.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include <algorithm>
#include <atomic>
#include <climits>
#include <cstdint>
#include <cstdlib>
#include <mutex>
#include <utility>

#include "sq.h"
#include "sq_ptx.cuh"

namespace sq {

// Read and clear the error word of the other translation unit (sq_mx4_api.cu).
cudaError_t mx4_read_device_error(unsigned int *code);
cudaError_t mx4_clear_device_error();

}  // namespace sq

namespace {

constexpr int kMaxDevices = 64;
constexpr int kMaxDynSmem = 232448;  // 227 KB of dynamic shared memory per CTA on sm_100
constexpr int kSmSmemBytes = 233472;  // shared memory of one SM (228 KB)

inline bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

inline bool valid_dtype(sq_dtype dt) { return dt == SQ_F32 || dt == SQ_BF16; }

inline size_t dtype_size(sq_dtype dt) { return dt == SQ_F32 ? 4 : 2; }

// Whether a call of the runtime succeeded; its error is taken from the runtime,
// so that no later call is told of it.
inline bool cuda_ok(cudaError_t e)
{
    if (e == cudaSuccess)
        return true;
    cudaGetLastError();
    return false;
}

struct DeviceInfo {
    int sms = 0;
    bool ok = false;
};

bool device_info(DeviceInfo &info)
{
    static DeviceInfo cache[kMaxDevices];
    static std::mutex mu;
    int dev = 0;
    if (!cuda_ok(cudaGetDevice(&dev)) || dev < 0 || dev >= kMaxDevices)
        return false;
    std::lock_guard<std::mutex> lk(mu);
    if (!cache[dev].ok) {
        int sms = 0;
        if (!cuda_ok(cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)))
            return false;
        cache[dev].sms = sms;
        cache[dev].ok = true;
    }
    info = cache[dev];
    return true;
}

// Launch plans are printed to stderr when SQ_DEBUG_PLAN is set (diagnostics).
bool debug_plan()
{
    static const bool on = std::getenv("SQ_DEBUG_PLAN") != nullptr;
    return on;
}

// Programmatic dependent launch for every kernel of the library (each one
// begins with griddepcontrol.wait, so it sees all work before it on the
// stream); SQ_PDL=0 turns the attribute off.
bool pdl_enabled()
{
    static const bool on = !(std::getenv("SQ_PDL") && std::atoi(std::getenv("SQ_PDL")) == 0);
    return on;
}

// Launch `kernel` on `st`.  Kernels that use cluster features (distributed
// shared memory, cluster barriers, remote mbarrier arrivals) pass their
// cluster shape cx x cy, which is set even when it is 1 x 1; other kernels
// pass cx = 0.
template <typename... KArgs, typename... Args>
sq_status launch_kernel(void (*kernel)(KArgs...), dim3 grid, dim3 block, int smem, cudaStream_t st, int cx,
                        int cy, Args &&...args)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = static_cast<size_t>(smem);
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    unsigned n = 0;
    if (cx > 0) {
        attr[n].id = cudaLaunchAttributeClusterDimension;
        attr[n].val.clusterDim.x = static_cast<unsigned>(cx);
        attr[n].val.clusterDim.y = static_cast<unsigned>(cy);
        attr[n].val.clusterDim.z = 1;
        ++n;
    }
    if (pdl_enabled()) {
        attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[n].val.programmaticStreamSerializationAllowed = 1;
        ++n;
    }
    cfg.attrs = attr;
    cfg.numAttrs = n;
    return cuda_ok(cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...)) ? SQ_OK : SQ_ERR_CUDA;
}

// ---- tensor maps -----------------------------------------------------------
PFN_cuTensorMapEncodeTiled_v12000 encode_fn()
{
    static std::atomic<PFN_cuTensorMapEncodeTiled_v12000> fn{nullptr};
    auto f = fn.load(std::memory_order_acquire);
    if (f == nullptr) {  // the first call, and every one after a failure
        void *p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cuda_ok(cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q)) &&
            q == cudaDriverEntryPointSuccess) {
            f = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
            fn.store(f, std::memory_order_release);
        }
    }
    return f;
}

// int8 matrix [rows, cols] (cols contiguous, row pitch = cols bytes); box of
// 128 bytes x box_rows rows, 128-byte swizzle, zero fill out of bounds.
bool make_tmap_i8(CUtensorMap *map, const void *base, int64_t rows, int64_t cols, int box_rows)
{
    auto fn = encode_fn();
    if (fn == nullptr)
        return false;
    cuuint64_t dims[2] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows)};
    cuuint64_t strides[1] = {static_cast<cuuint64_t>(cols)};
    cuuint32_t box[2] = {128u, static_cast<cuuint32_t>(box_rows)};
    cuuint32_t estr[2] = {1, 1};
    CUresult r = fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void *>(base), dims, strides,
                    box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                    CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS;
}

// ---- per-kernel one-time attribute setup ----------------------------------
// `done_mask` must be distinct for every kernel instantiation (all GEMM
// instantiations share one function-pointer type), so each caller owns it.
template <typename KernelT>
bool ensure_smem_attr(KernelT kernel, int bytes, std::atomic<uint64_t> &done_mask)
{
    int dev = 0;
    if (!cuda_ok(cudaGetDevice(&dev)) || dev < 0 || dev >= kMaxDevices)
        return false;
    const uint64_t bit = 1ull << dev;
    if (done_mask.load(std::memory_order_acquire) & bit)
        return true;
    if (!cuda_ok(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes)))
        return false;
    done_mask.fetch_or(bit, std::memory_order_release);
    return true;
}

// Answers of queries, kept by what was asked.  A fixed table: no allocation, so
// nothing throws; what it has no room for is asked again.
template <typename Key, int N>
class Answers {
    std::mutex mu_;
    Key keys_[N];
    int values_[N];
    int n_ = 0;

public:
    bool find(const Key &k, int &value)
    {
        std::lock_guard<std::mutex> lk(mu_);
        for (int i = 0; i < n_; ++i)
            if (keys_[i] == k) {
                value = values_[i];
                return true;
            }
        return false;
    }
    void keep(const Key &k, int value)
    {
        std::lock_guard<std::mutex> lk(mu_);
        if (n_ < N) {
            keys_[n_] = k;
            values_[n_++] = value;
        }
    }
};

// Clusters of `csize` CTAs of `threads` threads and `smem` bytes each that the
// device can hold at once (cudaOccupancyMaxActiveClusters), cached per kernel
// and shape; 0 where the query fails.
template <typename KernelT>
int active_clusters(KernelT kernel, int csize, int smem, int threads)
{
    struct Asked {
        const void *fn;
        int dev, csize, smem, threads;
        bool operator==(const Asked &o) const
        {
            return fn == o.fn && dev == o.dev && csize == o.csize && smem == o.smem && threads == o.threads;
        }
    };
    static Answers<Asked, 256> cache;
    int dev = 0, n = 0;
    if (!cuda_ok(cudaGetDevice(&dev)))
        return 0;
    const Asked asked{reinterpret_cast<const void *>(kernel), dev, csize, smem, threads};
    if (cache.find(asked, n))
        return n;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(csize * 64));
    cfg.blockDim = dim3(static_cast<unsigned>(threads));
    cfg.dynamicSmemBytes = smem;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = csize;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (!cuda_ok(cudaOccupancyMaxActiveClusters(&n, kernel, &cfg)))
        return 0;  // of this call alone: the next one asks again
    cache.keep(asked, n);
    return n;
}

// CTAs of the weight-streaming GEMM.  The units are cut into G equal
// ranges: with G = S * T (T tiles, S <= KB) every range lies inside one tile,
// so a CTA has one partial tile to sum through the workspace instead of up
// to two; with G = T / D (D dividing T, for T above the SM count) every range
// is D whole tiles and nothing is summed.  A shared tile's epilogue (stores,
// a release, a count, the reduction) costs, in units of streaming, a fixed
// kDecodeEpiUnits plus, per contributor, a part that grows with the tokens
// (its partial's bytes); G is the choice with the fewest units per CTA plus
// that cost.  Fitted to sq_linear calls on B200 (one call, L2 flushed): at
// 1 to 16 tokens three or four CTAs a 4096-long tile were best, at 32 two,
// from 64 one; with K = 14336 four at every token count; at 64 to 128
// tokens and N = 28672, two whole tiles a CTA (42 -> 36 us, 52 -> 40 us).
// Small layers, whose units number at most the SMs, were once cut one unit
// a CTA at no modelled reduction cost; costed like the rest they take fewer,
// longer ranges (64 x 1024 x 2048: 44 -> 19 us; 1 x 1040 x 3088: 21.5 ->
// 17.4 us; 128 x 2048 x 8192: 54 -> 40 us).
// The MXFP4 product takes the same rule with its own units (256 values of K, 16 KB
// too).  Its costs were not fitted; the choice was measured at one shape only
// (sq_mx4_stream.cuh).
constexpr int64_t kDecodeEpiUnits = 4;
inline int64_t decode_epi_units(int64_t M, int64_t S) { return kDecodeEpiUnits + (1 + std::min<int64_t>(M, 64) / 8) * S; }

// The plan for T tiles of KB units each and M tokens.
inline int64_t stream_ctas(int64_t M, int64_t T, int64_t KB, int64_t sms)
{
    const int64_t U = T * KB;
    int64_t best = 0, best_cost = INT64_MAX;
    if (U > sms) {
        // the stream cut over every SM: ranges of `per` units may span two
        // tiles, each tile shared by about KB / per + 1 CTAs; the first
        // partial tile's reduction overlaps the rest of the range, so the
        // second's costs in full and the first's its fixed part
        const int64_t per = (U + sms - 1) / sms;
        const int64_t shared = std::max<int64_t>(2, (KB + per - 1) / per + 1);
        best = sms;
        best_cost = per + decode_epi_units(M, shared) + kDecodeEpiUnits;
    }
    for (int64_t S = 1; S <= KB && S * T <= sms; ++S) {
        const int64_t cost = (KB + S - 1) / S + (S > 1 ? decode_epi_units(M, S) : 0);
        if (cost < best_cost) {
            best_cost = cost;
            best = S * T;
        }
    }
    for (int64_t D = 2; D <= T && T > sms; ++D) {
        if (T % D != 0 || T / D > sms)
            continue;
        const int64_t cost = D * KB;
        if (cost < best_cost) {
            best_cost = cost;
            best = T / D;
        }
    }
    return best > 0 ? best : std::min(U, sms);
}

}  // namespace
