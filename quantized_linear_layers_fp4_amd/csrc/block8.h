// Block-scaled E4M3 operands and the 4-bit key/value cache: host-side launchers and the device
// helpers their kernels share (internal; the C ABI is include/fp4lin.h).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "fp4_common.h"

namespace fp4 {

// One E4M3 operand of a product, contraction-contiguous: codes R x ld bytes (ld = the contraction
// length rounded up to 128, the pad zero) and one E8M0 byte per block of 128 along the contraction,
// four consecutive blocks of one scale row in a dword: byte kb % 4 of dword (kb / 4) * srows +
// (row >> sshift).  sshift is 0 (vector blocks) or 7 (square blocks: 128 rows share a byte).
struct Op8 {
    const uint8_t *codes;
    const uint32_t *scales;
    int64_t ld;
    int srows, sshift;
};

hipError_t launch_block8_quant(const void *X, int dt, int64_t R, int64_t C, int64_t ld, bool square, uint8_t *rc,
                               uint8_t *rs, uint8_t *cc, uint8_t *cs, hipStream_t s);
hipError_t launch_block8_dequant(const uint8_t *codes, const uint8_t *scales, int64_t R, int64_t C, bool square,
                                 void *Y, int y_dt, hipStream_t s);
// Y (M x N, rows ldy apart) = A . B^T
hipError_t launch_block8_gemm(const Op8 &A, const Op8 &B, int64_t M, int64_t N, int64_t K, void *Y, int y_dt, int cus,
                              hipStream_t s);

// The same for few rows of A, and with A (X, rows ldx apart) quantized on the way.
// Where: measured on a bf16 layer with the weight out of the caches, few rows' kernel | tiles of 64 x 64,
// us, at (K, N) = (4096, 22016): 24.3 | 25.8 for 16 rows, 31.3 | 26.7 for 32; (4096, 12288): 14.1 | 14.6 for
// 16, 20.3 | 14.7 for 32; (2048, 6144): 9.9 | 9.3 for 32, 13.5 | 9.7 for 64; (4096, 4096): 11.4 | 13.7 for 48, 12.9 | 13.8 for 64;
// (11008, 4096): 12.0 | 27.6 for one, 18.5 | 28.9 for 48, 21.8 | 29.3 for 64.  Its work grows with the rows, in steps of 16;
// the tiles' is a chain of K / 128 loads until they fill the device.
inline bool block8_few(int64_t M, int64_t N) {
    return M <= 64 && (N + 15) / 16 * ((M + 15) / 16) <= 1024;
}
// Quantizing in every workgroup instead of once: 20.4 | 26.9 us for one row at (4096, 22016), where four
// rows are 27.0 | 26.8; with a workgroup or two a CU it is the shorter way up to 128 blocks (8.8 | 9.5 for four
// rows at (4096, 4096)), which is also what fits beside the patches.
inline bool block8_few_direct(int64_t M, int64_t N, int64_t K) {
    return M * ((K + 127) / 128) <= 128 && M <= ((N + 15) / 16 <= 512 ? 16 : 2);
}
hipError_t launch_block8_few(const Op8 &A, const Op8 &B, int64_t M, int64_t N, int64_t K, void *Y, int y_dt, hipStream_t s);
hipError_t launch_block8_few_direct(const void *X, int x_dt, int64_t ldx, const Op8 &B, int64_t M, int64_t N, int64_t K,
                                    void *Y, int y_dt, hipStream_t s);

typedef int v8i __attribute__((ext_vector_type(8)));
typedef float v4f __attribute__((ext_vector_type(4)));
typedef __bf16 v8bf __attribute__((ext_vector_type(8)));
typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));

// Loads and stores at the element's own alignment (global memory takes any on gfx950).
typedef unsigned int ua_u32x4 __attribute__((ext_vector_type(4), aligned(2)));

// E8M0 byte of the smallest e >= -127 with amax <= 1.75 * 2^(lg + e) (limits 448 = 1.75 * 2^8 and
// 7 = 1.75 * 2^2), from amax's bits; 255 when they are an infinity's or a NaN's.  Adding 0x1FFFFF
// carries into the exponent field exactly when the mantissa is above 1.75's.
__device__ __forceinline__ uint32_t e8m0_of(uint32_t amax_bits, int lg) {
    const int b = (int)((amax_bits + 0x1FFFFFu) >> 23) - lg;
    return amax_bits >= 0x7F800000u ? 255u : (uint32_t)max(b, 0);
}
// 2^-e of an E8M0 byte (exact: e lies in [-127, 126]); NaN for 255, so every code of such a block
// is the format's NaN.
__device__ __forceinline__ float e8m0_inv(uint32_t b) {
    return b == 255u ? __uint_as_float(0x7FC00000u) : __uint_as_float((254u - b) << 23);
}
// 2^e of an E8M0 byte; byte 0 (2^-127) is a subnormal float, 255 a NaN.
__device__ __forceinline__ float e8m0_value(uint32_t b) {
    return __uint_as_float(b == 0 ? 0x00400000u : (b == 255u ? 0x7FC00000u : b << 23));
}
// Eight E4M3 codes (nearest, ties to even) of v * m.
__device__ __forceinline__ uint2 e4m3_pack8(const float v[8], float m) {
    int lo = 0, hi = 0;
    lo = __builtin_amdgcn_cvt_pk_fp8_f32(v[0] * m, v[1] * m, lo, false);
    lo = __builtin_amdgcn_cvt_pk_fp8_f32(v[2] * m, v[3] * m, lo, true);
    hi = __builtin_amdgcn_cvt_pk_fp8_f32(v[4] * m, v[5] * m, hi, false);
    hi = __builtin_amdgcn_cvt_pk_fp8_f32(v[6] * m, v[7] * m, hi, true);
    return make_uint2((uint32_t)lo, (uint32_t)hi);
}

// Eight consecutive elements from any element-aligned address as fp32 (n: how many lie inside).
template <int DT>
__device__ __forceinline__ void load8_any(const void *__restrict__ X, int64_t elem, int n, float v[8]) {
    if constexpr (DT == DT_BF16) {
        const uint16_t *p = static_cast<const uint16_t *>(X) + elem;
        if (n >= 8) {
            const ua_u32x4 q = *reinterpret_cast<const ua_u32x4 *>(p);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                v[2 * i] = __uint_as_float(q[i] << 16);
                v[2 * i + 1] = __uint_as_float(q[i] & 0xFFFF0000u);
            }
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = i < n ? __uint_as_float((uint32_t)p[i] << 16) : 0.0f;
        }
    } else {
        const float *p = static_cast<const float *>(X) + elem;
        if (n >= 8) {
            const ua_u32x4 q0 = *reinterpret_cast<const ua_u32x4 *>(p), q1 = *reinterpret_cast<const ua_u32x4 *>(p + 4);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                v[i] = __uint_as_float(q0[i]);
                v[4 + i] = __uint_as_float(q1[i]);
            }
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = i < n ? p[i] : 0.0f;
        }
    }
}

// fp32 -> bf16 bits, nearest even, a NaN staying one (v_cvt_pk_bf16_f32's own rounding).
__device__ __forceinline__ uint32_t bf16_pack2(float lo, float hi) {
    typedef __bf16 bf2 __attribute__((ext_vector_type(2)));
    const bf2 v = {(__bf16)lo, (__bf16)hi};
    return __builtin_bit_cast(uint32_t, v);
}

__device__ __forceinline__ uint32_t amax8(const float v[8]) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(v[i]) & 0x7FFFFFFFu);
    return m;
}

// Operands of a product with fp32 output, on the bf16 instruction at half the rate.  The scaled E4M3
// instruction aligns its products in groups of eight to the largest and drops what lies 14 or more
// binary places below (measured: 1.4e-5 of the result on normal data, 5e-5 with outlier channels),
// which a bf16 output (2^-8) does not see and an fp32 one does.  E4M3 values times their power of two
// are exact in bf16 but at the ends of the range (below 2^-126, and 256 * 2^120), and the conversion
// applies the scale.
template <int KK>
__device__ __forceinline__ void to_bf16(const v8i &x, uint32_t s, v8bf (&f)[4]) {
    const float sc = __uint_as_float(((s >> (8 * KK)) & 255u) << 23);
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        u32x4 w;
        w[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(x[2 * q], sc, false));
        w[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(x[2 * q], sc, true));
        w[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(x[2 * q + 1], sc, false));
        w[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(x[2 * q + 1], sc, true));
        f[q] = __builtin_bit_cast(v8bf, w);
    }
}
}  // namespace fp4
