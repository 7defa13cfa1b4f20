// E4M3 quantization in blocks of 128 (1 x 128 along the contraction, or 128 x 128) with
// power-of-two scales, for the block-scaled products of block8_gemm.hip.
//
// A matrix X (R x C) can be an operand in two ways: with its rows kept (contraction along C, codes
// R x Cp) or transposed (contraction along R, codes C x Rp).  A training step needs X both ways
// (the forward contracts the features, the weight gradient the tokens), so one pass over a
// 128 x 128 tile makes both: the tile stays in registers (8 rows x 8 columns a thread), row maxima
// are taken across 16 lanes, column maxima through LDS, and the transposed codes are turned in LDS
// so that both outputs are written in whole 128-byte lines.  Bound by memory: es + 2 bytes an
// element for both outputs.
#include <algorithm>

#include "block8.h"

namespace fp4 {

template <int DT, bool SQ, bool ROWS, bool COLS>
__global__ __launch_bounds__(256) void k_block8_tile(const void *__restrict__ X, int64_t R, int64_t C, int64_t ld,
                                                     int tilesC, uint8_t *__restrict__ rc, uint8_t *__restrict__ rs,
                                                     uint8_t *__restrict__ cc, uint8_t *__restrict__ cs) {
    __shared__ __attribute__((aligned(16))) uint32_t cmax[COLS && !SQ ? 16 * 128 : 4];
    __shared__ __attribute__((aligned(16))) float cinv[128];
    __shared__ __attribute__((aligned(16))) uint8_t turn[COLS ? 128 * 128 : 16];
    const int tid = threadIdx.x, rb = tid >> 4, cg = tid & 15;
    const int64_t tr = blockIdx.x / tilesC, tc = blockIdx.x % tilesC;
    const int64_t r0 = tr * 128 + rb * 8, c0 = tc * 128 + cg * 8;
    const int cn = (int)min((int64_t)8, C - c0);  // columns inside (may be <= 0)

    float v[8][8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        if (r0 + i < R && cn > 0) {
            load8_any<DT>(X, (r0 + i) * ld + c0, cn, v[i]);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) v[i][j] = 0.0f;
        }
    }
    float inv = 0.0f;  // square blocks: the tile's 2^-e
    if constexpr (SQ) {
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) m = max(m, amax8(v[i]));
        m = wave_max_u32(m);
        if ((tid & 63) == 0) cmax[tid >> 6] = m;
        __syncthreads();
        m = max(max(cmax[0], cmax[1]), max(cmax[2], cmax[3]));
        const uint32_t b = e8m0_of(m, 8);
        inv = e8m0_inv(b);
        if (tid == 0) {
            if constexpr (ROWS) rs[((tc >> 2) * ((R + 127) / 128) + tr) * 4 + (tc & 3)] = (uint8_t)b;
            if constexpr (COLS) cs[((tr >> 2) * ((C + 127) / 128) + tc) * 4 + (tr & 3)] = (uint8_t)b;
        }
    }
    if constexpr (COLS && !SQ) {
        uint32_t m[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            m[j] = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) m[j] = max(m[j], __float_as_uint(v[i][j]) & 0x7FFFFFFFu);
        }
        *reinterpret_cast<uint4 *>(&cmax[rb * 128 + cg * 8]) = make_uint4(m[0], m[1], m[2], m[3]);
        *reinterpret_cast<uint4 *>(&cmax[rb * 128 + cg * 8 + 4]) = make_uint4(m[4], m[5], m[6], m[7]);
    }
    if constexpr (ROWS) {
        const int64_t rld = (int64_t)tilesC * 128;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            float f = inv;
            if constexpr (!SQ) {
                uint32_t m = amax8(v[i]);
#pragma unroll
                for (int off = 8; off > 0; off >>= 1) m = max(m, (uint32_t)__shfl_xor((int)m, off, 64));
                const uint32_t b = e8m0_of(m, 8);
                f = e8m0_inv(b);
                if (cg == 0 && r0 + i < R) rs[((tc >> 2) * R + r0 + i) * 4 + (tc & 3)] = (uint8_t)b;
            }
            if (r0 + i < R) *reinterpret_cast<uint2 *>(rc + (r0 + i) * rld + c0) = e4m3_pack8(v[i], f);
        }
    }
    if constexpr (COLS) {
        float f[8];
        if constexpr (!SQ) {
            __syncthreads();
            if (tid < 128) {
                uint32_t m = 0;
#pragma unroll
                for (int i = 0; i < 16; ++i) m = max(m, cmax[i * 128 + tid]);
                const uint32_t b = e8m0_of(m, 8);
                cinv[tid] = e8m0_inv(b);
                if (tc * 128 + tid < C) cs[((tr >> 2) * C + tc * 128 + tid) * 4 + (tr & 3)] = (uint8_t)b;
            }
            __syncthreads();
            const float4 f0 = *reinterpret_cast<const float4 *>(&cinv[cg * 8]);
            const float4 f1 = *reinterpret_cast<const float4 *>(&cinv[cg * 8 + 4]);
            f[0] = f0.x; f[1] = f0.y; f[2] = f0.z; f[3] = f0.w;
            f[4] = f1.x; f[5] = f1.y; f[6] = f1.z; f[7] = f1.w;
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) f[j] = inv;
        }
        // column c = 8 cg + j of the tile is LDS row c; its 8-byte piece of rows 8 rb.. lies at
        // piece rb ^ cg, so the 16 lanes that write one rb at once hit 16 different pieces
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            float t[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) t[i] = v[i][j];
            *reinterpret_cast<uint2 *>(&turn[(cg * 8 + j) * 128 + ((rb ^ cg) << 3)]) = e4m3_pack8(t, f[j]);
        }
        __syncthreads();
        const int64_t cld = (R + 127) / 128 * 128;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int c = k * 32 + (tid >> 3), h = tid & 7, x = c >> 3;  // pieces 2h and 2h + 1 of column c
            const uint2 a = *reinterpret_cast<const uint2 *>(&turn[c * 128 + (((2 * h) ^ x) << 3)]);
            const uint2 b = *reinterpret_cast<const uint2 *>(&turn[c * 128 + (((2 * h + 1) ^ x) << 3)]);
            const int64_t col = tc * 128 + c;
            if (col < C) *reinterpret_cast<uint4 *>(cc + col * cld + tr * 128 + h * 16) = make_uint4(a.x, a.y, b.x, b.y);
        }
    }
}

// Rows kept, vector blocks: 16 lanes take one block of 128, so a few tokens spread over many
// workgroups (a decode batch) as well as a long prompt does.
template <int DT>
__global__ __launch_bounds__(256) void k_block8_rows(const void *__restrict__ X, int64_t R, int64_t C, int64_t ld,
                                                     int64_t KB, uint8_t *__restrict__ rc, uint8_t *__restrict__ rs) {
    const int lane16 = threadIdx.x & 15;
    const int64_t item = (int64_t)blockIdx.x * 16 + (threadIdx.x >> 4);
    if (item >= R * KB) return;  // whole groups of 16 lanes leave together
    const int64_t r = item / KB, kb = item % KB, c0 = kb * 128 + lane16 * 8;
    const int cn = (int)min((int64_t)8, C - c0);
    float v[8];
    if (cn > 0) {
        load8_any<DT>(X, r * ld + c0, cn, v);
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = 0.0f;
    }
    uint32_t m = amax8(v);
#pragma unroll
    for (int off = 8; off > 0; off >>= 1) m = max(m, (uint32_t)__shfl_xor((int)m, off, 64));
    const uint32_t b = e8m0_of(m, 8);
    *reinterpret_cast<uint2 *>(rc + r * KB * 128 + c0) = e4m3_pack8(v, e8m0_inv(b));
    if (lane16 == 0) rs[((kb >> 2) * R + r) * 4 + (kb & 3)] = (uint8_t)b;
}

template <int DT>
static hipError_t quant_dt(const void *X, int64_t R, int64_t C, int64_t ld, bool sq, uint8_t *rc, uint8_t *rs,
                           uint8_t *cc, uint8_t *cs, hipStream_t s) {
    const int64_t tr = (R + 127) / 128, tc = (C + 127) / 128;
    if (!sq && !cc) {
        const int64_t blocks = (R * tc + 15) / 16;
        hipLaunchKernelGGL(k_block8_rows<DT>, dim3((unsigned)blocks), dim3(256), 0, s, X, R, C, ld, tc, rc, rs);
        return hipGetLastError();
    }
    const dim3 g((unsigned)(tr * tc)), b(256);
#define Q(SQ, RO, CO) \
    hipLaunchKernelGGL((k_block8_tile<DT, SQ, RO, CO>), g, b, 0, s, X, R, C, ld, (int)tc, rc, rs, cc, cs)
    if (sq) {
        if (rc && cc) Q(true, true, true);
        else if (rc) Q(true, true, false);
        else Q(true, false, true);
    } else {
        if (rc) Q(false, true, true);
        else Q(false, false, true);
    }
#undef Q
    return hipGetLastError();
}

hipError_t launch_block8_quant(const void *X, int dt, int64_t R, int64_t C, int64_t ld, bool square, uint8_t *rc,
                               uint8_t *rs, uint8_t *cc, uint8_t *cs, hipStream_t s) {
    return dt == DT_BF16 ? quant_dt<DT_BF16>(X, R, C, ld, square, rc, rs, cc, cs, s)
                         : quant_dt<DT_F32>(X, R, C, ld, square, rc, rs, cc, cs, s);
}

// Values of an operand (R x C): value(code) * 2^e, exact in fp32 (bf16 too: four significant bits).
template <int YDT>
__global__ __launch_bounds__(256) void k_block8_dequant(const uint8_t *__restrict__ codes,
                                                        const uint8_t *__restrict__ scales, int64_t R, int64_t C,
                                                        int64_t ld, int64_t srows, int sshift, void *__restrict__ Y) {
    const int64_t quads = ld / 4;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < R * quads; i += (int64_t)gridDim.x * 256) {
        const int64_t r = i / quads, c = i % quads * 4;
        const int64_t kb = c >> 7;
        const uint32_t b = scales[((kb >> 2) * srows + (r >> sshift)) * 4 + (kb & 3)];
        const int w = *reinterpret_cast<const int *>(codes + r * ld + c);
        const float s = e8m0_value(b);
        const float v[4] = {__builtin_amdgcn_cvt_f32_fp8(w, 0) * s, __builtin_amdgcn_cvt_f32_fp8(w, 1) * s,
                            __builtin_amdgcn_cvt_f32_fp8(w, 2) * s, __builtin_amdgcn_cvt_f32_fp8(w, 3) * s};
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (c + j < C) {
                if constexpr (YDT == DT_F32) static_cast<float *>(Y)[r * C + c + j] = v[j];
                else static_cast<uint16_t *>(Y)[r * C + c + j] = (uint16_t)(b == 255u ? 0x7FC0u : f32_to_bf16_bits(v[j]));
            }
    }
}

hipError_t launch_block8_dequant(const uint8_t *codes, const uint8_t *scales, int64_t R, int64_t C, bool square,
                                 void *Y, int y_dt, hipStream_t s) {
    const int64_t ld = (C + 127) / 128 * 128, n = R * (ld / 4);
    // the largest matrix would take 2^32 threads, one more than a launch may have: from half of it on, a second turn
    const dim3 g((unsigned)std::min<int64_t>((n + 255) / 256, (int64_t)1 << 23)), b(256);
    const int64_t srows = square ? (R + 127) / 128 : R;
    if (y_dt == DT_BF16)
        hipLaunchKernelGGL(k_block8_dequant<DT_BF16>, g, b, 0, s, codes, scales, R, C, ld, srows, square ? 7 : 0, Y);
    else
        hipLaunchKernelGGL(k_block8_dequant<DT_F32>, g, b, 0, s, codes, scales, R, C, ld, srows, square ? 7 : 0, Y);
    return hipGetLastError();
}

}  // namespace fp4
