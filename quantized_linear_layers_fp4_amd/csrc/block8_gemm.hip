// Y = A . B^T for E4M3 operands with a power-of-two scale per block of 128 along the contraction
// (block8.hip writes them; both operands are contraction-contiguous).
//
//      Y[m][n] = sum over blocks kb of 2^(ea[m,kb] + eb[n,kb]) * sum over k in kb of a[m][k] b[n][k]
//
// The scales are E8M0 bytes, which the CDNA4 scaled matrix instruction takes beside its operands
// (one byte per row and 32 values), so the block scaling costs no vector work and the sum stays in
// one fp32 accumulator.  A lane keeps the four bytes of four consecutive blocks of its row in one
// register and the instruction selects the byte.
//
// Workgroup: 4 waves as 2 x 2, each WI x WJ tiles of 32 x 32 (V_MFMA_SCALE_F32_32X32X64_F8F6F4); a
// stage is one block of 128 along K (128 bytes a row) for both operands, loaded straight to LDS into
// one of two buffers while the other is multiplied.  The product is formed transposed, so a lane
// holds four consecutive columns of one row; the tiles are turned to row order through LDS and
// stored 16 bytes a lane.
#include <type_traits>

#include "block8.h"

namespace fp4 {

typedef int v8i __attribute__((ext_vector_type(8)));
typedef float v16f __attribute__((ext_vector_type(16)));
typedef __bf16 v8bf __attribute__((ext_vector_type(8)));
typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));
#define LDS_PTR(p) ((__attribute__((address_space(3))) void *)(p))

namespace {

constexpr int BUF_FLAGS = 0x00020000;  // raw buffer descriptor word 3 (gfx9 family)

struct Args8 {
    Op8 A, B;
    int64_t M, N;
    int KB;  // blocks of 128 along the contraction
    void *Y;
    int tilesM, tilesN, group;
};

// 16-byte piece of (row, chunk) in a tile of 8 chunks a row: 16 consecutive rows of one chunk lie on
// 16 distinct pieces modulo 16.
__device__ __forceinline__ int piece(int row, int chunk) { return row * 8 + (chunk ^ ((row >> 1) & 7)); }

// The scale dwords of quad kq for the lane's row of each of the NT tiles from row0 on.
template <int NT>
__device__ __forceinline__ void scale_load(const Op8 &o, int64_t row0, int64_t rows, int kq, uint32_t (&s)[NT]) {
#pragma unroll
    for (int i = 0; i < NT; ++i) {
        const int64_t r = min(row0 + i * 32 + (int)(threadIdx.x & 31), rows - 1);
        s[i] = o.scales[(int64_t)kq * o.srows + (r >> o.sshift)];
    }
}

// fp32 outputs: the same product on the bf16 instruction, at half the rate.  The scaled E4M3
// instruction aligns its products in groups of eight to the largest and drops what lies 14 or more
// binary places below (measured: 1.4e-5 of the result on normal data, 5e-5 with outlier channels),
// which a bf16 output (2^-9) does not see and an fp32 one does.  E4M3 values times their power of two
// are exact in bf16, and the conversion applies the scale.
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
template <int KK, int WI, int WJ>
__device__ __forceinline__ void mma_exact(v16f (&acc)[WI][WJ], const v8i (&a)[WI], const v8i (&b)[WJ],
                                          const uint32_t (&sa)[WI], const uint32_t (&sb)[WJ]) {
    v8bf bf[WJ][4];
#pragma unroll
    for (int j = 0; j < WJ; ++j) to_bf16<KK>(b[j], sb[j], bf[j]);
#pragma unroll
    for (int i = 0; i < WI; ++i) {
        v8bf af[4];
        to_bf16<KK>(a[i], sa[i], af);
#pragma unroll
        for (int q = 0; q < 4; ++q)
#pragma unroll
            for (int j = 0; j < WJ; ++j)
                acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(bf[j][q], af[q], acc[i][j], 0, 0, 0);
    }
}

template <int KK, int WI, int WJ>
__device__ __forceinline__ void mma(v16f (&acc)[WI][WJ], const v8i (&a)[WI], const v8i (&b)[WJ],
                                    const uint32_t (&sa)[WI], const uint32_t (&sb)[WJ]) {
#pragma unroll
    for (int i = 0; i < WI; ++i)
#pragma unroll
        for (int j = 0; j < WJ; ++j)
            acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(b[j], a[i], acc[i][j], 0, 0, KK, (int)sb[j], KK,
                                                                        (int)sa[i]);
}

}  // namespace

template <int YDT, int WI, int WJ>
__global__ __launch_bounds__(256) void k_block8_gemm(Args8 p) {
    constexpr int TM = 64 * WI, TN = 64 * WJ, STAGE = (TM + TN) * 128;
    __shared__ __attribute__((aligned(1024))) uint8_t sm[2][STAGE];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave >> 1, wn = wave & 1;

    // each XCD (consecutive workgroups go to different ones) takes a contiguous range of tiles;
    // within it `group` tile rows sweep the columns together
    const int tiles = p.tilesM * p.tilesN, per = gridDim.x / 8;
    const int lg = (blockIdx.x & 7) * per + (blockIdx.x >> 3);
    if (lg >= tiles) return;
    const int grp = lg / (p.group * p.tilesN), first = grp * p.group, gm = min(p.group, p.tilesM - first);
    const int in = lg - grp * p.group * p.tilesN;
    const int64_t m0 = (int64_t)(first + in % gm) * TM, n0 = (int64_t)(in / gm) * TN;

    // descriptors start at the tile's first row: offsets stay small whatever the operand's size, and
    // rows past the matrix read zeros
    const int ldA = (int)p.A.ld, ldB = (int)p.B.ld;
    const int rowsA = (int)min((int64_t)TM, p.M - m0), rowsB = (int)min((int64_t)TN, p.N - n0);
    const __amdgpu_buffer_rsrc_t ra = __builtin_amdgcn_make_buffer_rsrc(
        const_cast<uint8_t *>(p.A.codes + m0 * p.A.ld), 0, rowsA * ldA, BUF_FLAGS);
    const __amdgpu_buffer_rsrc_t rb = __builtin_amdgcn_make_buffer_rsrc(
        const_cast<uint8_t *>(p.B.codes + n0 * p.B.ld), 0, rowsB * ldB, BUF_FLAGS);
    auto stage = [&](int buf, int kb) {
        // 1 KiB (8 rows) a load; lane l fills piece l of it: row l / 8 at swizzled chunk l % 8
#pragma unroll
        for (int j = 0; j < TM / 32; ++j) {
            const int blk = wave * (TM / 32) + j, row = blk * 8 + (lane >> 3);
            const int off = row * ldA + (((lane & 7) ^ ((row >> 1) & 7)) << 4);
            __builtin_amdgcn_raw_ptr_buffer_load_lds(ra, LDS_PTR(&sm[buf][blk * 1024]), 16, off, kb * 128, 0, 0);
        }
#pragma unroll
        for (int j = 0; j < TN / 32; ++j) {
            const int blk = wave * (TN / 32) + j, row = blk * 8 + (lane >> 3);
            const int off = row * ldB + (((lane & 7) ^ ((row >> 1) & 7)) << 4);
            __builtin_amdgcn_raw_ptr_buffer_load_lds(rb, LDS_PTR(&sm[buf][TM * 128 + blk * 1024]), 16, off, kb * 128, 0,
                                                     0);
        }
    };
    // lane l: row l % 32 of the tile, 32 consecutive values from 64 h + 32 (l / 32)
    auto frag = [&](const uint8_t *op, int row, int h) {
        const int c = 4 * h + 2 * (lane >> 5);
        const u32x4 x = *reinterpret_cast<const u32x4 *>(op + piece(row, c) * 16);
        const u32x4 y = *reinterpret_cast<const u32x4 *>(op + piece(row, c + 1) * 16);
        return v8i{(int)x.x, (int)x.y, (int)x.z, (int)x.w, (int)y.x, (int)y.y, (int)y.z, (int)y.w};
    };

    v16f acc[WI][WJ];
#pragma unroll
    for (int i = 0; i < WI; ++i)
#pragma unroll
        for (int j = 0; j < WJ; ++j)
#pragma unroll
            for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.0f;

    stage(0, 0);
    uint32_t sa[WI], sb[WJ];
    auto step = [&](int kb, auto kk) {
        constexpr int KK = decltype(kk)::value;
        // stage kb has landed (this wave's loads by the wait, the others' by the barrier) and
        // everyone is done with the other buffer
        __builtin_amdgcn_s_waitcnt(0x0F70);  // vmcnt(0)
        __syncthreads();
        if (kb + 1 < p.KB) stage((kb + 1) & 1, kb + 1);
        const uint8_t *cur = sm[kb & 1];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            v8i a[WI], b[WJ];
#pragma unroll
            for (int i = 0; i < WI; ++i) a[i] = frag(cur, (wm * WI + i) * 32 + (lane & 31), h);
#pragma unroll
            for (int j = 0; j < WJ; ++j) b[j] = frag(cur + TM * 128, (wn * WJ + j) * 32 + (lane & 31), h);
            if constexpr (YDT == DT_F32) mma_exact<KK, WI, WJ>(acc, a, b, sa, sb);
            else mma<KK, WI, WJ>(acc, a, b, sa, sb);
        }
    };
    for (int kb = 0; kb < p.KB; kb += 4) {
        scale_load<WI>(p.A, m0 + wm * WI * 32, p.M, kb >> 2, sa);
        scale_load<WJ>(p.B, n0 + wn * WJ * 32, p.N, kb >> 2, sb);
        step(kb, std::integral_constant<int, 0>{});
        if (kb + 1 < p.KB) step(kb + 1, std::integral_constant<int, 1>{});
        if (kb + 2 < p.KB) step(kb + 2, std::integral_constant<int, 2>{});
        if (kb + 3 < p.KB) step(kb + 3, std::integral_constant<int, 3>{});
    }
    __syncthreads();

    // transposed 32 x 32 result: lane l holds row l % 32, columns 8 (r / 4) + 4 (l / 32) + r % 4.
    // Patch of the wave: 32 rows of 128 bytes (64 bf16 or 32 fp32 columns), 144 bytes apart, so that
    // 16 rows' 16-byte pieces lie on distinct banks.
    constexpr int PJ = YDT == DT_BF16 && WJ > 1 ? 2 : 1;  // tiles side by side in the patch
    constexpr int ES = YDT == DT_BF16 ? 2 : 4, CHUNKS = PJ * 32 * ES / 16, EL = 16 / ES;
    uint8_t *P = &sm[0][wave * 32 * 144];
#pragma unroll
    for (int i = 0; i < WI; ++i)
#pragma unroll
        for (int j0 = 0; j0 < WJ; j0 += PJ) {
#pragma unroll
            for (int t = 0; t < PJ; ++t)
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const v16f &x = acc[i][j0 + t];
                    uint8_t *d = P + (lane & 31) * 144 + (t * 32 + 8 * q + 4 * (lane >> 5)) * ES;
                    if constexpr (YDT == DT_BF16) {
                        *reinterpret_cast<uint2 *>(d) =
                            make_uint2(bf16_pack2(x[4 * q], x[4 * q + 1]), bf16_pack2(x[4 * q + 2], x[4 * q + 3]));
                    } else {
                        *reinterpret_cast<float4 *>(d) = make_float4(x[4 * q], x[4 * q + 1], x[4 * q + 2], x[4 * q + 3]);
                    }
                }
            __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
            __builtin_amdgcn_wave_barrier();
            __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
#pragma unroll
            for (int k = 0; k < 32 * CHUNKS / 64; ++k) {
                const int c = k * 64 + lane, lr = c / CHUNKS, ch = c % CHUNKS;
                const u32x4 o = *reinterpret_cast<const u32x4 *>(P + lr * 144 + ch * 16);
                const int64_t row = m0 + (wm * WI + i) * 32 + lr, col = n0 + (wn * WJ + j0) * 32 + ch * EL;
                if (row < p.M && col < p.N) {
                    uint8_t *y = static_cast<uint8_t *>(p.Y) + (row * p.N + col) * ES;
                    if (col + EL <= p.N) {
                        *reinterpret_cast<ua_u32x4 *>(y) = o;
                    } else {
                        const int n = (int)(p.N - col);
                        for (int e = 0; e < n; ++e) {
                            if constexpr (YDT == DT_BF16)
                                reinterpret_cast<uint16_t *>(y)[e] = (uint16_t)(o[e >> 1] >> (16 * (e & 1)));
                            else
                                reinterpret_cast<uint32_t *>(y)[e] = o[e];
                        }
                    }
                }
            }
            __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
            __builtin_amdgcn_wave_barrier();
            __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
        }
}

template <int YDT, int W>
static hipError_t launch_tiles(Args8 p, hipStream_t s) {
    const int64_t T = 64 * W, tm = (p.M + T - 1) / T, tn = (p.N + T - 1) / T;
    p.tilesM = (int)tm;
    p.tilesN = (int)tn;
    p.group = (int)(tm < 4 ? tm : 4);
    hipLaunchKernelGGL((k_block8_gemm<YDT, W, W>), dim3((unsigned)((tm * tn + 7) / 8 * 8)), dim3(256), 0, s, p);
    return hipGetLastError();
}

hipError_t launch_block8_gemm(const Op8 &A, const Op8 &B, int64_t M, int64_t N, int64_t K, void *Y, int y_dt, int cus,
                              hipStream_t s) {
    Args8 p;
    p.A = A;
    p.B = B;
    p.M = M;
    p.N = N;
    p.KB = (int)((K + 127) / 128);
    p.Y = Y;
    p.tilesM = p.tilesN = p.group = 0;
    // the largest tile that still gives every CU a workgroup
    auto count = [&](int64_t t) { return ((M + t - 1) / t) * ((N + t - 1) / t); };
    const int w = count(256) >= cus ? 4 : (count(128) >= cus ? 2 : 1);
    if (y_dt == DT_BF16)
        return w == 4 ? launch_tiles<DT_BF16, 4>(p, s) : w == 2 ? launch_tiles<DT_BF16, 2>(p, s) : launch_tiles<DT_BF16, 1>(p, s);
    return w == 4 ? launch_tiles<DT_F32, 4>(p, s) : w == 2 ? launch_tiles<DT_F32, 2>(p, s) : launch_tiles<DT_F32, 1>(p, s);
}

}  // namespace fp4
