// sq_mx4.cuh -- the microscaled 4-bit format (OCP MXFP4): quantiser and
// read-back.
//
// A block of 32 consecutive values along K shares one scale 2^(b - 127) (b a
// byte, E8M0) and each value is an E2M1 code: sign, then 0, .5, 1, 1.5, 2, 3,
// 4, 6.  For a block with largest magnitude a
//   b    = max(e - 2, 0), e the biased fp32 exponent of a, so a / scale is in [4, 8)
//   code = the nearest E2M1 value of v / scale, ties to the even code, at most 6
// and a block that holds a NaN or an infinity gets b = 255 (NaN) and zero codes.
// 1 / scale is a normal power of two, so v / scale is exact (or underflows to a
// value that rounds to 0 anyway): the only rounding is the code's.
//
// Layout.  Codes [rows, K / 2] bytes, the even one of a pair in the low half.
// Scale bytes in tiles of 128 rows x 4 blocks, 512 bytes a tile, the tiles of
// one row tile contiguous along K: byte (r % 32) * 16 + (r % 128 / 32) * 4 +
// block % 4 of tile (r / 128, block / 4).  Padding rows and blocks hold 0.
// That is the order in which one tcgen05.cp moves a tile into tensor memory for
// the block-scaled MMA, so no kernel reorders a scale.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "sq_ptx.cuh"

namespace sq {

constexpr int kMx4Block = 32;        // values that share a scale
constexpr int kMx4TileBytes = 512;   // scale bytes of 128 rows x 4 blocks
constexpr int kMx4Threads = 256;

enum : int { MX4_PLAIN = 0, MX4_TIMES = 1, MX4_OVER = 2 };  // v, v * s, v * RN(1 / s)

__device__ __forceinline__ float max_nan(float a, float b)
{
    float d;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
    return d;
}

// max(a, |b|, |c|), NaN if any is
__device__ __forceinline__ float max3_abs(float a, float b, float c)
{
    float d;
    asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

// 8 consecutive values of dtype T as fp32
template <typename T>
__device__ __forceinline__ void load8(const T *p, float (&v)[8]);
template <>
__device__ __forceinline__ void load8<float>(const float *p, float (&v)[8])
{
    const float4 a = __ldg(reinterpret_cast<const float4 *>(p)), b = __ldg(reinterpret_cast<const float4 *>(p) + 1);
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
}
__device__ __forceinline__ void bf16x8_to_f32(const uint4 &u, float (&v)[8])
{
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(w[i] << 16);
        v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
}
template <>
__device__ __forceinline__ void load8<__nv_bfloat16>(const __nv_bfloat16 *p, float (&v)[8])
{
    bf16x8_to_f32(__ldg(reinterpret_cast<const uint4 *>(p)), v);
}

template <typename T>
struct Raw8;  // 8 values as loaded
template <>
struct Raw8<__nv_bfloat16> {
    uint4 a;
};
template <>
struct Raw8<float> {
    float4 a, b;
};

__device__ __forceinline__ void raw_load(Raw8<__nv_bfloat16> &r, const __nv_bfloat16 *p)
{
    r.a = *reinterpret_cast<const uint4 *>(p);
}
__device__ __forceinline__ void raw_load(Raw8<float> &r, const float *p)
{
    r.a = reinterpret_cast<const float4 *>(p)[0];
    r.b = reinterpret_cast<const float4 *>(p)[1];
}
// through the read-only path
__device__ __forceinline__ void raw_load_nc(Raw8<__nv_bfloat16> &r, const __nv_bfloat16 *p)
{
    r.a = __ldg(reinterpret_cast<const uint4 *>(p));
}
__device__ __forceinline__ void raw_load_nc(Raw8<float> &r, const float *p)
{
    r.a = __ldg(reinterpret_cast<const float4 *>(p));
    r.b = __ldg(reinterpret_cast<const float4 *>(p) + 1);
}
__device__ __forceinline__ void raw_zero(Raw8<__nv_bfloat16> &r) { r.a = make_uint4(0, 0, 0, 0); }
__device__ __forceinline__ void raw_zero(Raw8<float> &r) { r.a = r.b = make_float4(0, 0, 0, 0); }
__device__ __forceinline__ void raw_values(const Raw8<__nv_bfloat16> &r, float (&v)[8]) { bf16x8_to_f32(r.a, v); }
__device__ __forceinline__ void raw_values(const Raw8<float> &r, float (&v)[8])
{
    v[0] = r.a.x, v[1] = r.a.y, v[2] = r.a.z, v[3] = r.a.w, v[4] = r.b.x, v[5] = r.b.y, v[6] = r.b.z, v[7] = r.b.w;
}

// v[i] * f[i] and v[i] * f, two at a time (packed fp32, rounded like the scalar)
__device__ __forceinline__ void mul8(float (&v)[8], const float (&f)[8])
{
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
        const float2 t = f2_mul(make_float2(v[i], v[i + 1]), make_float2(f[i], f[i + 1]));
        v[i] = t.x;
        v[i + 1] = t.y;
    }
}
__device__ __forceinline__ void mul8(float (&v)[8], float f)
{
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
        const float2 t = f2_mul(make_float2(v[i], v[i + 1]), make_float2(f, f));
        v[i] = t.x;
        v[i + 1] = t.y;
    }
}

// Eight values scaled by `inv` as E2M1 codes, value i in bits 4i..4i+3.
__device__ __forceinline__ uint32_t mx4_codes8(const float (&x)[8], float inv)
{
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
        v[i] = x[i];
    mul8(v, inv);
    uint32_t d;
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
        "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
        : "=r"(d)
        : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
    return d;
}

// Scale byte of a block whose largest magnitude is `top` (NaN or infinity: 255).
__device__ __forceinline__ uint32_t mx4_scale_byte(float top)
{
    const uint32_t e = __float_as_uint(top) >> 23;
    return e == 255u ? 255u : (e > 2u ? e - 2u : 0u);
}

// 1 / scale of a finite block's byte: a normal power of two (byte <= 252)
__device__ __forceinline__ float mx4_inv_scale(uint32_t byte) { return __uint_as_float((254u - byte) << 23); }

// The scale a byte stands for (byte 0 is subnormal in fp32, 255 a NaN).
__device__ __forceinline__ float mx4_scale(uint32_t byte)
{
    return __uint_as_float(byte == 255u ? 0x7FFFFFFFu : (byte == 0u ? 0x00400000u : byte << 23));
}

// Offset of the word that holds the four scale bytes of row r in tile (r / 128, kt).
__host__ __device__ __forceinline__ int64_t mx4_scale_word(int64_t r, int64_t kt, int64_t KT)
{
    return ((r >> 7) * KT + kt) * kMx4TileBytes + (r & 31) * 16 + ((r >> 5) & 3) * 4;
}

// One row's 8 values in each of 16 neighbouring lanes (128 values, 4 blocks;
// all 32 lanes take part): writes the codes and, from the first of the 16, the
// word of scale bytes.  A block is the 8 values of each of 4 lanes.
__device__ __forceinline__ void mx4_store_chunk(const float (&v)[8], bool in_k, uint32_t *codes, uint32_t *word)
{
    float top = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; i += 2)
        top = max3_abs(top, v[i], v[i + 1]);
    top = max_nan(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
    top = max_nan(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
    uint32_t byte = mx4_scale_byte(top);
    const uint32_t c = byte == 255u ? 0u : mx4_codes8(v, mx4_inv_scale(byte));
    if (in_k)
        *codes = c;
    else
        byte = 0u;
    byte |= __shfl_down_sync(0xFFFFFFFFu, byte, 4) << 8;
    byte |= __shfl_down_sync(0xFFFFFFFFu, byte, 8) << 16;
    if (word != nullptr)
        *word = byte;
}

// Zero scale bytes of the padding rows behind row `rows` (at most 127 rows of KT
// words, so 32-bit numbers hold them): word i of them for this thread and every
// `step`-th after it.
__device__ __forceinline__ void mx4_zero_pad(uint8_t *scales, int rows, int KT, unsigned i, unsigned step)
{
    const unsigned n = static_cast<unsigned>(((rows + 127) & ~127) - rows) * static_cast<unsigned>(KT);
    for (; i < n; i += step) {
        const unsigned r = i / static_cast<unsigned>(KT);
        *reinterpret_cast<uint32_t *>(scales + mx4_scale_word(rows + static_cast<int>(r), i - r * KT, KT)) = 0u;
    }
}

// Quantiser.  A thread owns 8 columns (its factors stay in registers) and walks
// down the rows of its band, U rows in flight; 16 neighbouring threads make one
// word of scale bytes.  A CTA covers TX * 8 columns, TX a multiple of 16, and 256
// / TX rows at a time.  Memory-bound for fp32 (4096 x 8192 at 5.3 TB/s); with
// bf16's 2.5 bytes a value the instructions count too (69 % of the issue slots and
// 66 % of the ALU pipe taken), so the maximum takes three operands an instruction
// and the products are packed: 28672 x 4096 in 64 us, 4.6 TB/s.  (16 columns a
// thread halve the shuffles but spread each load over twice the lines: 94 us.)  The
// smoothing divides by multiplying with RN(1 / s), one division a column and band
// instead of one a value.
// `zero`: tile counts of the product after it, cleared on the side.
template <typename T, int OP>
__global__ void __launch_bounds__(kMx4Threads) mx4_quant_kernel(const T *__restrict__ x, int rows, int K,
                                                                const float *__restrict__ s,
                                                                uint8_t *__restrict__ codes,
                                                                uint8_t *__restrict__ scales, int log2tx, int band,
                                                                int *__restrict__ zero, int nzero)
{
    pdl_prologue();
    constexpr int U = 4;
    const int tx = threadIdx.x & ((1 << log2tx) - 1), ty = threadIdx.x >> log2tx;
    const int TY = kMx4Threads >> log2tx;
    const int KT = (K + 127) >> 7;
    const int c = (static_cast<int>(blockIdx.x) << log2tx) + tx;  // chunk of 8 columns
    const int kt = c >> 4;
    const bool in_k = c * 8 < K;
    const bool word_lane = (threadIdx.x & 15) == 0 && kt < KT;
    float f[8];
    if constexpr (OP != MX4_PLAIN) {
        if (in_k)
            load8<float>(s + c * 8, f);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            f[i] = !in_k ? 1.0f : (OP == MX4_OVER ? __frcp_rn(f[i]) : f[i]);
    }
    const int r0 = static_cast<int>(blockIdx.y) * band, r1 = min(rows, r0 + band);
    const T *px = x + (static_cast<int64_t>(r0) + ty) * K + c * 8;
    uint8_t *pq = codes + (static_cast<int64_t>(r0) + ty) * (K / 2) + c * 4;
    uint8_t *ps = scales + static_cast<int64_t>(kt) * kMx4TileBytes;
    const int64_t xstep = static_cast<int64_t>(TY) * K, row_tile = static_cast<int64_t>(KT) * kMx4TileBytes;
    // every lane of a warp takes the same trips (rows behind the end are neither
    // loaded nor stored), so the shuffles are whole
    for (int rb = r0; rb < r1; rb += TY * U) {
        Raw8<T> raw[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (in_k && rb + ty + u * TY < r1)
                raw_load_nc(raw[u], px + u * xstep);
            else
                raw_zero(raw[u]);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int r = rb + ty + u * TY;
            const bool live = r < r1;
            float v[8];
            raw_values(raw[u], v);
            if constexpr (OP != MX4_PLAIN)
                mul8(v, f);
            mx4_store_chunk(v, in_k && live, reinterpret_cast<uint32_t *>(pq + u * (xstep / 2)),
                            word_lane && live ? reinterpret_cast<uint32_t *>(ps + (r >> 7) * row_tile + (r & 31) * 16 +
                                                                            ((r >> 5) & 3) * 4)
                                              : nullptr);
        }
        px += xstep * U;
        pq += xstep / 2 * U;
    }
    // (a grid has at most 2^24 threads: 8 CTAs an SM, or one CTA for each 256 columns of at most 2^24)
    const unsigned nt = gridDim.x * gridDim.y * kMx4Threads;
    const unsigned me = (blockIdx.y * gridDim.x + blockIdx.x) * kMx4Threads + threadIdx.x;
    mx4_zero_pad(scales, rows, KT, me, nt);
    for (int i = static_cast<int>(me); i < nzero; i += static_cast<int>(nt))
        zero[i] = 0;
}

// E2M1 pairs of one byte as two halves (exact)
__device__ __forceinline__ __half2 e2m1x2_to_half2(uint32_t byte)
{
    uint32_t d;
    asm("{\n\t.reg .b8 b;\n\t.reg .b16 t;\n\tcvt.u16.u32 t, %1;\n\tmov.b16 {b, _}, t;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, b;\n\t}"
        : "=r"(d)
        : "r"(byte));
    return *reinterpret_cast<__half2 *>(&d);
}

// The values the codes stand for: 8 codes (4 bytes) a thread, U rows in flight,
// the same walk as the quantiser (28672 x 4096 to bf16 in 61 us, 4.9 TB/s).  E2M1 times a power of two is exact in fp32
// and in bf16 (subnormal ones included).
template <typename T>
__global__ void __launch_bounds__(kMx4Threads) mx4_dequant_kernel(const uint8_t *__restrict__ codes,
                                                                  const uint8_t *__restrict__ scales, int rows, int K,
                                                                  T *__restrict__ out, int log2tx, int band)
{
    pdl_prologue();
    constexpr int U = 4;
    const int tx = threadIdx.x & ((1 << log2tx) - 1), ty = threadIdx.x >> log2tx;
    const int TY = kMx4Threads >> log2tx;
    const int KT = (K + 127) >> 7;
    const int c = (static_cast<int>(blockIdx.x) << log2tx) + tx;
    if (c * 8 >= K)
        return;
    const int r0 = static_cast<int>(blockIdx.y) * band, r1 = min(rows, r0 + band);
    const uint8_t *pq = codes + (static_cast<int64_t>(r0) + ty) * (K / 2) + c * 4;
    const uint8_t *ps = scales + static_cast<int64_t>(c >> 4) * kMx4TileBytes + ((c >> 2) & 3);
    T *po = out + (static_cast<int64_t>(r0) + ty) * K + c * 8;
    const int64_t step = static_cast<int64_t>(TY) * K, row_tile = static_cast<int64_t>(KT) * kMx4TileBytes;
    for (int rb = r0 + ty; rb < r1; rb += TY * U) {
        uint32_t q[U], b[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int r = rb + u * TY;
            if (r < r1) {
                q[u] = __ldg(reinterpret_cast<const uint32_t *>(pq + u * (step / 2)));
                b[u] = __ldg(ps + (r >> 7) * row_tile + (r & 31) * 16 + ((r >> 5) & 3) * 4);
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (rb + u * TY >= r1)
                break;
            float v[8];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 p = __half22float2(e2m1x2_to_half2((q[u] >> (8 * i)) & 0xFFu));
                v[2 * i] = p.x;
                v[2 * i + 1] = p.y;
            }
            mul8(v, mx4_scale(b[u]));
            T *dst = po + u * step;
            if constexpr (sizeof(T) == 4) {
                reinterpret_cast<float4 *>(dst)[0] = make_float4(v[0], v[1], v[2], v[3]);
                reinterpret_cast<float4 *>(dst)[1] = make_float4(v[4], v[5], v[6], v[7]);
            } else {
                uint32_t o[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const __nv_bfloat162 x2 = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
                    o[i] = *reinterpret_cast<const uint32_t *>(&x2);
                }
                *reinterpret_cast<uint4 *>(dst) = make_uint4(o[0], o[1], o[2], o[3]);
            }
        }
        pq += step / 2 * U;
        po += step * U;
    }
}

}  // namespace sq
