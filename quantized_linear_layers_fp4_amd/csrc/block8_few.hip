// Y = A . B^T for few rows of A (a decode batch), operands as in block8_gemm.hip.
//
// The weight's bytes bound it: every one is read once, by one wave, with eight lanes to a cache line, and
// turned in the wave's own patch of LDS into the matrix instruction's operand, whose neighbouring lanes are
// rows (V_MFMA_SCALE_F32_16X16X128_F8F6F4: a step is one block of 128).  Loaded in that layout each
// quarter of a wave touches 16 lines and takes as many cycles: 27 instead of 17 us for 48 x 11008 x 4096.
// A workgroup owns 16 weight rows (columns of Y) and all rows of A; its waves take the blocks along K in
// turn, each with the loads of several blocks in flight all the time, and join in LDS in wave order, so the
// call fills the device whatever N is, with no partial results in memory.  A's codes are read by every workgroup: for
// 48 x 11008 x 4096 that is 135 of the 183 MB that the call reads through the L2s.
//
// For a few rows A comes as it is, and every workgroup quantizes it into LDS while its first weights are on
// their way: a launch less.
#include <algorithm>

#include "block8.h"

namespace fp4 {

namespace {

constexpr int CODES = 2;  // A is quantized already (DT_F32 = 0, DT_BF16 = 1: it comes in that type)

struct FewArgs {
    Op8 A, B;
    const void *X;
    int64_t ldx;
    int64_t M, N, K;
    int KB;
    void *Y;
};

typedef int v4i __attribute__((ext_vector_type(4)));
__device__ __forceinline__ v8i two(const u32x4 &x, const u32x4 &y) {
    return v8i{(int)x.x, (int)x.y, (int)x.z, (int)x.w, (int)y.x, (int)y.y, (int)y.z, (int)y.w};
}
// Block kb of 16 rows from row0 on (rows past the last are the last): lane l has 16-byte chunk l % 8 of rows
// l / 8 and 8 + l / 8.
__device__ __forceinline__ v8i codes_at(const Op8 &o, int64_t row0, int64_t rows, int kb, int lane) {
    const uint8_t *c = o.codes + kb * 128 + (lane & 7) * 16;
    return two(*reinterpret_cast<const u32x4 *>(c + min(row0 + (lane >> 3), rows - 1) * o.ld),
               *reinterpret_cast<const u32x4 *>(c + min(row0 + 8 + (lane >> 3), rows - 1) * o.ld));
}
// 16-byte piece c of a row of 128, turned so that 16 consecutive rows' lie on distinct banks
__device__ __forceinline__ int piece(int row, int c) { return row * 128 + ((c ^ ((row >> 1) & 7)) << 4); }
// What codes_at loaded, through the wave's patch: lane l gets 32 values of row l % 16.
__device__ __forceinline__ v8i turned(const v8i &x, uint8_t *patch, int lane) {
    const int r = lane >> 3, c = lane & 7, n = lane & 15, q = lane >> 4;
    *reinterpret_cast<v4i *>(patch + piece(r, c)) = v4i{x[0], x[1], x[2], x[3]};
    *reinterpret_cast<v4i *>(patch + piece(r + 8, c)) = v4i{x[4], x[5], x[6], x[7]};
    const v4i a = *reinterpret_cast<const v4i *>(patch + piece(n, 2 * q)), b = *reinterpret_cast<const v4i *>(patch + piece(n, 2 * q + 1));
    return v8i{a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
}
__device__ __forceinline__ uint32_t scale_at(const Op8 &o, int64_t row, int kb) {
    return reinterpret_cast<const uint8_t *>(o.scales + (int64_t)(kb >> 2) * o.srows + (row >> o.sshift))[kb & 3];
}

}  // namespace

// waves of a workgroup, at most: 16 leave a lane 128 registers, too few for more than 16 rows
// (nor does LDS hold more than 8 waves' patches beside the quantized rows)
constexpr int most_waves(int src, int mt) { return src == 2 && mt == 1 ? 16 : 8; }

template <int SRC, int YDT, int MT>
__global__ __launch_bounds__(64 * most_waves(SRC, MT)) void k_block8_few(FewArgs p) {
    constexpr bool DIRECT = SRC != CODES;
    constexpr int U = DIRECT ? 6 : MT == 1 ? 4 : 3;  // blocks whose loads a wave has in flight
    // the waves' patches (B's and A's of 2 KiB each) and, DIRECT, A's codes [KB][M][128] and scales [KB][M]; when
    // those are done with, the waves' sums [waves][MT * 16 rows][16 columns]
    extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
    const int lane = threadIdx.x & 63, n = lane & 15, q = lane >> 4, waves = blockDim.x >> 6;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t n0 = (int64_t)blockIdx.x * 16, brow = min(n0 + n, p.N - 1);
    const int M = (int)p.M;
    v4f acc[MT];
#pragma unroll
    for (int i = 0; i < MT; ++i) acc[i] = v4f{0, 0, 0, 0};

    v8i a[U][MT], b[U];
    uint32_t sa[U][MT], sb[U];
    auto load = [&](int kb, v8i(&x)[MT], v8i &y, uint32_t(&sx)[MT], uint32_t &sy) {
        y = codes_at(p.B, n0, p.N, kb, lane);
        sy = scale_at(p.B, brow, kb);
        if constexpr (!DIRECT) {
#pragma unroll
            for (int i = 0; i < MT; ++i) {
                x[i] = codes_at(p.A, 16 * i, M, kb, lane);
                sx[i] = scale_at(p.A, min(16 * i + n, M - 1), kb);
            }
        }
    };
#pragma unroll
    for (int u = 0; u < U; ++u)
        if (wave + u * waves < p.KB) load(wave + u * waves, a[u], b[u], sa[u], sb[u]);

    uint8_t *patch = lds + wave * 4096, *lc = lds + waves * 4096, *ls = lc + M * p.KB * 128;
    if constexpr (DIRECT) {  // 16 lanes a block
        for (int i = threadIdx.x >> 4; i < M * p.KB; i += blockDim.x >> 4) {
            const int kb = i / M, row = i % M;
            const int64_t c0 = (int64_t)kb * 128 + n * 8;
            const int cn = (int)min(p.K - c0, (int64_t)8);
            float v[8];
            if (cn > 0) {
                load8_any<SRC>(p.X, row * p.ldx + c0, cn, v);
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j) v[j] = 0.0f;
            }
            uint32_t m = amax8(v);
#pragma unroll
            for (int off = 8; off > 0; off >>= 1) m = max(m, (uint32_t)__shfl_xor((int)m, off, 64));
            const uint32_t e = e8m0_of(m, 8);
            *reinterpret_cast<uint2 *>(lc + kb * M * 128 + piece(row, n >> 1) + (n & 1) * 8) = e4m3_pack8(v, e8m0_inv(e));
            if (n == 0) ls[i] = (uint8_t)e;
        }
        __syncthreads();
    }

    for (int k0 = wave; k0 < p.KB; k0 += waves * U) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int kb = k0 + u * waves;
            if (kb >= p.KB) break;
            const v8i bt = turned(b[u], patch, lane);
            v8i at[MT];
            if constexpr (DIRECT) {
                const int row = min(n, M - 1);
                const uint8_t *c = lc + kb * M * 128;
                at[0] = two(*reinterpret_cast<const u32x4 *>(c + piece(row, 2 * q)),
                            *reinterpret_cast<const u32x4 *>(c + piece(row, 2 * q + 1)));
                sa[u][0] = ls[kb * M + row];
            } else {
#pragma unroll
                for (int i = 0; i < MT; ++i) at[i] = turned(a[u][i], patch + 2048, lane);
            }
            if constexpr (YDT == DT_F32) {
                v8bf bf[4];
                to_bf16<0>(bt, sb[u], bf);
#pragma unroll
                for (int i = 0; i < MT; ++i) {
                    v8bf af[4];
                    to_bf16<0>(at[i], sa[u][i], af);
#pragma unroll
                    for (int t = 0; t < 4; ++t) acc[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(bf[t], af[t], acc[i], 0, 0, 0);
                }
            } else {
#pragma unroll
                for (int i = 0; i < MT; ++i)
                    acc[i] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(bt, at[i], acc[i], 0, 0, 0, (int)sb[u], 0,
                                                                              (int)sa[u][i]);
            }
            if (kb + waves * U < p.KB) load(kb + waves * U, a[u], b[u], sa[u], sb[u]);
        }
    }
    __syncthreads();
    float *part = reinterpret_cast<float *>(lds);
    // lane: row 16 i + n of Y, columns 4 q + r of the workgroup's
#pragma unroll
    for (int i = 0; i < MT; ++i)
        *reinterpret_cast<v4f *>(&part[((wave * MT + i) * 16 + n) * 16 + 4 * q]) = acc[i];
    __syncthreads();
    for (int e = threadIdx.x; e < MT * 256; e += blockDim.x) {
        const int64_t row = e >> 4, col = n0 + (e & 15);
        if (row >= p.M || col >= p.N) continue;
        float y = part[e];
        for (int w = 1; w < waves; ++w) y += part[w * MT * 256 + e];
        if constexpr (YDT == DT_BF16)
            static_cast<uint16_t *>(p.Y)[row * p.N + col] = (uint16_t)bf16_pack2(y, 0.0f);
        else
            static_cast<float *>(p.Y)[row * p.N + col] = y;
    }
}

template <int SRC, int YDT, int MT>
static hipError_t launch_few(const FewArgs &p, hipStream_t s) {
    // waves a workgroup: about 4096 in the call, at most one a block of K
    const int64_t groups = (p.N + 15) / 16;
    int waves = 4;
    while (waves < most_waves(SRC, MT) && groups * waves < 4096 && waves < p.KB) waves *= 2;
    const int64_t sums = waves * MT * 1024, held = waves * 4096 + (SRC == CODES ? 0 : p.M * p.KB * 129);
    hipLaunchKernelGGL((k_block8_few<SRC, YDT, MT>), dim3((unsigned)groups), dim3(64 * waves),
                       (unsigned)std::max(sums, held), s, p);
    return hipGetLastError();
}

hipError_t launch_block8_few(const Op8 &A, const Op8 &B, int64_t M, int64_t N, int64_t K, void *Y, int y_dt, hipStream_t s) {
    const FewArgs p{A, B, nullptr, 0, M, N, K, (int)((K + 127) / 128), Y};
    if (y_dt == DT_BF16)
        return M <= 16 ? launch_few<CODES, DT_BF16, 1>(p, s) : M <= 32 ? launch_few<CODES, DT_BF16, 2>(p, s) : M <= 48 ? launch_few<CODES, DT_BF16, 3>(p, s) : launch_few<CODES, DT_BF16, 4>(p, s);
    return M <= 16 ? launch_few<CODES, DT_F32, 1>(p, s) : M <= 32 ? launch_few<CODES, DT_F32, 2>(p, s) : M <= 48 ? launch_few<CODES, DT_F32, 3>(p, s) : launch_few<CODES, DT_F32, 4>(p, s);
}

hipError_t launch_block8_few_direct(const void *X, int x_dt, int64_t ldx, const Op8 &B, int64_t M, int64_t N, int64_t K,
                                    void *Y, int y_dt, hipStream_t s) {
    const FewArgs p{B, B, X, ldx, M, N, K, (int)((K + 127) / 128), Y};
    if (x_dt == DT_BF16)
        return y_dt == DT_BF16 ? launch_few<DT_BF16, DT_BF16, 1>(p, s) : launch_few<DT_BF16, DT_F32, 1>(p, s);
    return y_dt == DT_BF16 ? launch_few<DT_F32, DT_BF16, 1>(p, s) : launch_few<DT_F32, DT_F32, 1>(p, s);
}

}  // namespace fp4
