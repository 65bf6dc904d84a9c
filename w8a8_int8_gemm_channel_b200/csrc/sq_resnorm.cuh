// sq_resnorm.cuh -- the norms on both sides of a residual addition, fused with
// the gate, the residual scale and the next linear's quantiser.
//
//   n  = (b * rb) * gamma        rb = RN(1 / sqrt(mean(b^2) + eps))   (gamma given; else n = b)
//   u  = n * gate                                                     (gate given; else u = n)
//   r' = RN_dt(r + u * c)
//   a  = (r' * ra) * g           ra = RN(1 / sqrt(mean(r'^2) + eps))
//   then a's int8 codes with one scale a token, or its MXFP4 codes and scales
//
// every step one fp32 operation, rounded to nearest; the mean squares are sums
// of exact squares in fp64, so codes do not hang on the order of a fp32 sum.
//
// A token is read once and r' written once: a CTA holds a row's b and r in
// registers (CH chunks of 8 values a thread) from the load to the codes, across
// the two or three block-wide reductions the definition needs.  The per-channel
// factors gamma and g, 8 bytes a value against the 6.6 a bf16 value moves, would
// make L2 the bound if every row fetched them; with several rows a CTA they are
// staged in shared memory once, and the next row's loads are in flight while the
// present row is reduced.
//
// Bound: latency.  At 4096 x 8192 bf16 (MXFP4, 64 us, 3.4 TB/s) 53 % of the issue
// slots are taken (33 instructions a value) and no pipe is busy (ALU 33 %, XU 29 %,
// fp64 10 %), with 16 warps an SM, as many as registers and shared memory allow.
// The warps wait for short-scoreboard results and fixed latencies: unpacking, fp64
// squares and two reductions are a serial chain a row, and half of the factors'
// shared-memory wavefronts are bank conflicts (a lane's two float4 lie 32 bytes
// from the next lane's).  Two CTAs of 256 threads with the next row in flight,
// against 71 us for three without and 68 for two of 512.  The int8 form takes 87 us:
// it forms a row's values twice, for the maximum and for the codes.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>

#include "sq_mx4.cuh"
#include "sq_ptx.cuh"

namespace sq {

// rounds to T and stores; `r` keeps what was stored
__device__ __forceinline__ void res_store(Raw8<__nv_bfloat16> &r, __nv_bfloat16 *p, const float (&v)[8])
{
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t *>(&h);
    }
    r.a = make_uint4(w[0], w[1], w[2], w[3]);
    *reinterpret_cast<uint4 *>(p) = r.a;
}
__device__ __forceinline__ void res_store(Raw8<float> &r, float *p, const float (&v)[8])
{
    r.a = make_float4(v[0], v[1], v[2], v[3]);
    r.b = make_float4(v[4], v[5], v[6], v[7]);
    reinterpret_cast<float4 *>(p)[0] = r.a;
    reinterpret_cast<float4 *>(p)[1] = r.b;
}

__device__ __forceinline__ double res_squares(const float (&v)[8])
{
    double s = 0.0;
#pragma unroll
    for (int i = 0; i < 8; ++i)
        s = fma(static_cast<double>(v[i]), static_cast<double>(v[i]), s);
    return s;
}

// 1 / RMS from a row's sum of squares: every thread's `s` summed over the
// block.  One barrier: each warp adds the warps' sums from `buf` [32] by itself.
// buf is written again at the earliest two calls later (the caller alternates).
template <int THREADS>
__device__ __forceinline__ float res_rinv(double s, double inv_k, float eps, double *buf)
{
#pragma unroll
    for (int d = 16; d > 0; d >>= 1)
        s += __shfl_xor_sync(0xFFFFFFFFu, s, d);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (lane == 0)
        buf[warp] = s;
    __syncthreads();
    double t = buf[lane & (THREADS / 32 - 1)];
#pragma unroll
    for (int d = THREADS / 64; d > 0; d >>= 1)
        t += __shfl_xor_sync(0xFFFFFFFFu, t, d);
    const double ms = t * inv_k + static_cast<double>(eps);
    return ms > 0.0 ? static_cast<float>(rsqrt(ms)) : (ms == 0.0 ? 0.0f : static_cast<float>(ms));
}

template <int THREADS>
__device__ __forceinline__ float res_max(float m, float *buf)
{
    uint32_t u = __reduce_max_sync(0xFFFFFFFFu, __float_as_uint(m));  // m >= 0
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (lane == 0)
        buf[warp] = __uint_as_float(u);
    __syncthreads();
    u = __reduce_max_sync(0xFFFFFFFFu, lane < THREADS / 32 ? __float_as_uint(buf[lane]) : 0u);
    return __uint_as_float(u);
}

// clamp(round_half_even(RN(a / sx)), -127, 127) of 8 values.  a * RN(1 / sx) is
// within 127 * 2^-23 + 127 * 2^-24 < 2.5e-5 of RN(a / sx), so only a product
// that near to a half-integer (or a scale too small for a normal reciprocal)
// needs the division.
__device__ __forceinline__ uint2 res_int8(const float (&a)[8], float sx, float inv, bool exact)
{
    uint32_t w[2] = {0u, 0u};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        float t = __fmul_rn(a[i], inv);
        const float q = rintf(t);
        if (exact || fabsf(fabsf(t - q) - 0.5f) < 2.5e-5f)
            t = sx > 0.0f ? __fdiv_rn(a[i], sx) : 0.0f;
        const int c = max(-127, min(127, __float2int_rn(t)));
        w[i >> 2] |= (static_cast<uint32_t>(c) & 0xFFu) << (8 * (i & 3));
    }
    return make_uint2(w[0], w[1]);
}

struct ResArgs {
    const void *b, *r, *gate;
    const float *gamma, *g;
    void *r_out;
    uint8_t *q;   // int8 [M, K] or MXFP4 codes [M, K / 2]
    void *sx;     // float [M] or scale tiles
    int64_t M, K, gate_tokens;
    float c, eps;
};

// CH: chunks of 8 values a thread holds (K <= 8 * CH * THREADS); CACHE: gamma and
// g in shared memory, BLOCKS: CTAs an SM holds.
template <typename T, bool MX4, int CH, int THREADS, bool CACHE, int BLOCKS>
__global__ void __launch_bounds__(THREADS, BLOCKS) res_norm_kernel(const ResArgs p)
{
    pdl_prologue();
    extern __shared__ float factors[];  // [2][K] with CACHE
    __shared__ double sums[2][2][32];   // [row parity][norm][warp]
    __shared__ float top_s[32];
    constexpr bool AHEAD = CACHE && CH * sizeof(T) <= (BLOCKS <= 2 ? 8 : 4);  // the next row's loads in flight (registers allow)
    const int K = static_cast<int>(p.K), KT = (K + 127) >> 7;
    const double inv_k = 1.0 / static_cast<double>(K);
    const T *b = static_cast<const T *>(p.b), *r = static_cast<const T *>(p.r), *gate = static_cast<const T *>(p.gate);
    T *r_out = static_cast<T *>(p.r_out);
    const bool post = p.gamma != nullptr;
    int col[CH];
#pragma unroll
    for (int i = 0; i < CH; ++i)
        col[i] = (i * THREADS + static_cast<int>(threadIdx.x)) * 8;

    if constexpr (CACHE) {
        for (int k = threadIdx.x * 4; k < K; k += THREADS * 4) {
            if (post)
                *reinterpret_cast<float4 *>(factors + k) = __ldg(reinterpret_cast<const float4 *>(p.gamma + k));
            *reinterpret_cast<float4 *>(factors + K + k) = __ldg(reinterpret_cast<const float4 *>(p.g + k));
        }
        __syncthreads();
    }
    auto factor = [&](const float *global, int at, int c, float (&f)[8]) {
        if constexpr (CACHE) {
            const float4 x = *reinterpret_cast<const float4 *>(factors + at + c);
            const float4 y = *reinterpret_cast<const float4 *>(factors + at + c + 4);
            f[0] = x.x, f[1] = x.y, f[2] = x.z, f[3] = x.w, f[4] = y.x, f[5] = y.y, f[6] = y.z, f[7] = y.w;
        } else {
            load8<float>(global + c, f);
        }
    };
    Raw8<T> bv[CH], rv[CH], bn[AHEAD ? CH : 1], rn[AHEAD ? CH : 1];
    auto fetch = [&](int64_t m, Raw8<T> *x, Raw8<T> *y) {
        const T *pb = b + m * K, *pr = r + m * K;
#pragma unroll
        for (int i = 0; i < CH; ++i) {
            if (col[i] < K && m < p.M) {
                raw_load(x[i], pb + col[i]);
                raw_load(y[i], pr + col[i]);
            } else {
                raw_zero(x[i]);
                raw_zero(y[i]);
            }
        }
    };
    if constexpr (AHEAD)
        fetch(blockIdx.x, bn, rn);
    int parity = 0;
    for (int64_t m = blockIdx.x; m < p.M; m += gridDim.x, parity ^= 1) {
        if constexpr (AHEAD) {
#pragma unroll
            for (int i = 0; i < CH; ++i) {
                bv[i] = bn[i];
                rv[i] = rn[i];
            }
            fetch(m + gridDim.x, bn, rn);
        } else {
            fetch(m, bv, rv);
        }
        float rb = 0.0f;
        if (post) {
            double s = 0.0;
#pragma unroll
            for (int i = 0; i < CH; ++i) {
                float v[8];
                raw_values(bv[i], v);
                s += res_squares(v);
            }
            rb = res_rinv<THREADS>(s, inv_k, p.eps, sums[parity][0]);
        }
        const T *gr = gate == nullptr ? nullptr : gate + (m / p.gate_tokens) * K;
        T *po = r_out + m * K;
        double s = 0.0;
#pragma unroll
        for (int i = 0; i < CH; ++i) {
            if (col[i] >= K)
                continue;
            float u[8], f[8], o[8];
            raw_values(bv[i], u);
            if (post) {
                factor(p.gamma, 0, col[i], f);
                mul8(u, rb);
                mul8(u, f);
            }
            if (gr != nullptr) {
                load8<T>(gr + col[i], f);
                mul8(u, f);
            }
            raw_values(rv[i], o);
            // scalar: a packed product and sum would be fused into one rounding
#pragma unroll
            for (int j = 0; j < 8; ++j)
                o[j] = __fadd_rn(o[j], __fmul_rn(u[j], p.c));
            res_store(rv[i], po + col[i], o);
            raw_values(rv[i], o);
            s += res_squares(o);
        }
        const float ra = res_rinv<THREADS>(s, inv_k, p.eps, sums[parity][1]);
        auto scaled = [&](int i, float (&a)[8]) {
            float f[8];
            raw_values(rv[i], a);
            factor(p.g, K, col[i], f);
            mul8(a, ra);
            mul8(a, f);
        };
        if constexpr (MX4) {
            uint8_t *pq = p.q + m * (K / 2);
            uint8_t *ps = static_cast<uint8_t *>(p.sx) + mx4_scale_word(m, 0, KT);
#pragma unroll
            for (int i = 0; i < CH; ++i) {
                const int kt = col[i] >> 7;
                if (__ballot_sync(0xFFFFFFFFu, kt < KT) == 0u)  // a whole warp behind the last scale tile has nothing to do
                    continue;
                const bool in_k = col[i] < K;
                float a[8];
                if (in_k) {
                    scaled(i, a);
                } else {
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        a[j] = 0.0f;
                }
                mx4_store_chunk(a, in_k, reinterpret_cast<uint32_t *>(pq + col[i] / 2),
                                (threadIdx.x & 15) == 0 && kt < KT
                                    ? reinterpret_cast<uint32_t *>(ps + static_cast<int64_t>(kt) * kMx4TileBytes)
                                    : nullptr);
            }
        } else {
            float top = 0.0f;
#pragma unroll
            for (int i = 0; i < CH; ++i)
                if (col[i] < K) {
                    float a[8];
                    scaled(i, a);
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        top = fmaxf(top, fabsf(a[j]));
                }
            top = res_max<THREADS>(top, top_s);
            const float sx = __fdiv_rn(top, 127.0f);
            const bool exact = sx < 1e-30f;
            const float inv = exact ? 0.0f : __frcp_rn(sx);
            if (threadIdx.x == 0)
                static_cast<float *>(p.sx)[m] = sx;
            uint8_t *pq = p.q + m * K;
#pragma unroll
            for (int i = 0; i < CH; ++i)
                if (col[i] < K) {
                    float a[8];
                    scaled(i, a);
                    *reinterpret_cast<uint2 *>(pq + col[i]) = res_int8(a, sx, inv, exact);
                }
        }
    }
    if constexpr (MX4)
        mx4_zero_pad(static_cast<uint8_t *>(p.sx), static_cast<int>(p.M), KT, blockIdx.x * THREADS + threadIdx.x,
                     gridDim.x * THREADS);
}

}  // namespace sq
