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
// Workgroup: 4 waves as 2 x 2, each W x W tiles of 32 x 32 (V_MFMA_SCALE_F32_32X32X64_F8F6F4), so
// 64 W rows and columns.  K advances in slices of 64 (one step of the instruction), which travel
// straight to one of four LDS buffers, three slices ahead; the fragments of a slice are read under the
// matrix work of the one before it, so one barrier a slice is all that the waves wait for.  W = 4 is
// persistent (one workgroup a CU): the next tile's first slices are on their way while a tile's results
// are stored, and its stores drain under the next tile's products.  The product is formed
// transposed, so a lane holds four consecutive columns of one row; the tiles are turned to row order
// through LDS and stored 16 bytes a lane.
#include <type_traits>

#include "block8.h"

namespace fp4 {

typedef int v8i __attribute__((ext_vector_type(8)));
typedef float v16f __attribute__((ext_vector_type(16)));
typedef __bf16 v8bf __attribute__((ext_vector_type(8)));
typedef unsigned int u32x2 __attribute__((ext_vector_type(2)));
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

// s_waitcnt vmcnt(n), other counters untouched (gfx9 encoding)
template <int N>
__device__ __forceinline__ void wait_vm() {
    __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | 0x0F70);
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

// One wave's share of a slice of an operand: W loads of 1 KiB, straight to LDS.
template <int W>
__device__ __forceinline__ void rows_to_lds(const uint8_t *base, int bytes, uint8_t *buf, const int *off, int koff) {
    const __amdgpu_buffer_rsrc_t r = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t *>(base), 0, bytes, BUF_FLAGS);
#pragma unroll
    for (int j = 0; j < W; ++j)
        __builtin_amdgcn_raw_ptr_buffer_load_lds(r, LDS_PTR(buf + j * 1024), 16, off[j], koff, 0, 0);
}

// A choice by value: as a conditional expression it would be one of two variables, which then live in memory.
template <typename T>
__device__ __forceinline__ T pick(bool c, T x, T y) {
    return c ? x : y;
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

template <int YDT, int W>
__global__ __launch_bounds__(256, W == 4 ? 1 : W == 2 ? 2 : 4) void k_block8_gemm(Args8 p) {
    constexpr int T = 64 * W, OP = T * 64, SLICE = 2 * OP;
    constexpr bool WALK = W == 4;       // persistent
    constexpr int D = 2 * W;            // loads to LDS a wave issues a slice, and scale loads a pair of blocks
    constexpr int PATCH = 32 * 144;
    __shared__ __attribute__((aligned(1024))) uint8_t sb0[SLICE < 4 * PATCH && !WALK ? 4 * PATCH : SLICE];
    __shared__ __attribute__((aligned(1024))) uint8_t sb1[SLICE];
    __shared__ __attribute__((aligned(1024))) uint8_t sb2[SLICE];
    __shared__ __attribute__((aligned(1024))) uint8_t sb3[SLICE];
    __shared__ __attribute__((aligned(16))) uint8_t own_patch[WALK ? 4 * PATCH : 16];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave >> 1, wn = wave & 1;

    // each XCD (consecutive workgroups go to different ones) takes a contiguous range of tiles;
    // within it `group` tile rows sweep the columns together
    const int tiles = p.tilesM * p.tilesN, per = gridDim.x / 8, tpx = (tiles + 7) / 8;
    const int last = min(((int)(blockIdx.x & 7) + 1) * tpx, tiles);
    int lg = (blockIdx.x & 7) * tpx + (blockIdx.x >> 3);
    if (lg >= last) return;
    auto origin = [&](int l, int64_t &m0, int64_t &n0) {
        const int grp = l / (p.group * p.tilesN), first = grp * p.group, gm = min(p.group, p.tilesM - first);
        const int in = l - grp * p.group * p.tilesN;
        m0 = (int64_t)(first + in % gm) * T;
        n0 = (int64_t)(in / gm) * T;
    };
    int64_t m0, n0;
    origin(lg, m0, n0);

    // Descriptors start at a tile's first row: offsets stay small whatever the operand's size, and rows
    // past the matrix read zeros.  A slice past the contraction's end (or past the last tile) has an
    // empty descriptor and reads zeros.  1 KiB (16 rows of 64 bytes) a load: lane l fills 16-byte place l of
    // it, row l / 4 at place l % 4, whose chunk is turned by the row's bits 2 and 3, so that 16
    // consecutive rows of one chunk lie on 16 distinct places modulo 16.
    const int ldA = (int)p.A.ld, ldB = (int)p.B.ld;
    int offA[W], offB[W];
#pragma unroll
    for (int j = 0; j < W; ++j) {
        const int row = (wave * W + j) * 16 + (lane >> 2), ch = ((lane & 3) ^ ((lane >> 4) & 3)) * 16;
        offA[j] = row * ldA + ch;
        offB[j] = row * ldB + ch;
    }
    struct Src {
        const uint8_t *a, *b;
        int na, nb;
    };
    auto source = [&](int64_t m, int64_t n) {
        return Src{p.A.codes + m * p.A.ld, p.B.codes + n * p.B.ld, (int)min((int64_t)T, p.M - m) * ldA,
                   (int)min((int64_t)T, p.N - n) * ldB};
    };
    auto dma = [&](uint8_t *buf, Src s, int koff, bool in) {
        rows_to_lds<W>(s.a, in ? s.na : 0, buf + wave * W * 1024, offA, koff);
        rows_to_lds<W>(s.b, in ? s.nb : 0, buf + OP + wave * W * 1024, offB, koff);
    };
    // lane l: row l % 32 of a tile, 32 consecutive values from 32 (l / 32)
    const int at0 = (lane & 31) * 64 + (((2 * (lane >> 5)) ^ ((lane >> 2) & 3)) << 4), at1 = at0 ^ 16;
    auto frags = [&](const uint8_t *buf, v8i (&a)[W], v8i (&b)[W]) {
#pragma unroll
        for (int i = 0; i < W; ++i) {
            const uint8_t *t = buf + (wm * W + i) * 2048;
            const u32x4 x = *reinterpret_cast<const u32x4 *>(t + at0), y = *reinterpret_cast<const u32x4 *>(t + at1);
            a[i] = v8i{(int)x.x, (int)x.y, (int)x.z, (int)x.w, (int)y.x, (int)y.y, (int)y.z, (int)y.w};
        }
#pragma unroll
        for (int j = 0; j < W; ++j) {
            const uint8_t *t = buf + OP + (wn * W + j) * 2048;
            const u32x4 x = *reinterpret_cast<const u32x4 *>(t + at0), y = *reinterpret_cast<const u32x4 *>(t + at1);
            b[j] = v8i{(int)x.x, (int)x.y, (int)x.z, (int)x.w, (int)y.x, (int)y.y, (int)y.z, (int)y.w};
        }
    };
    // scale bytes of blocks 2 it and 2 it + 1 of the lane's rows
    const int iters = (p.KB + 1) / 2;
    auto scales = [&](int64_t m, int64_t n, int it, uint32_t (&sa)[W], uint32_t (&sb)[W]) {
        const int sel = (it >> 1), half = it & 1;
#pragma unroll
        for (int i = 0; i < W; ++i) {
            const int64_t r = min(m + (wm * W + i) * 32 + (lane & 31), p.M - 1);
            sa[i] = reinterpret_cast<const uint16_t *>(p.A.scales + (int64_t)sel * p.A.srows + (r >> p.A.sshift))[half];
        }
#pragma unroll
        for (int j = 0; j < W; ++j) {
            const int64_t r = min(n + (wn * W + j) * 32 + (lane & 31), p.N - 1);
            sb[j] = reinterpret_cast<const uint16_t *>(p.B.scales + (int64_t)sel * p.B.srows + (r >> p.B.sshift))[half];
        }
    };

    v16f acc[W][W];
    v8i a0[W], b0[W], a1[W], b1[W];
    uint32_t sa[W], sb[W], ta[W], tb[W];
    Src cur = source(m0, n0);
    // slices 0..3 of the first tile, and its first scales, in the order of the loop
    dma(sb0, cur, 0, true);
    dma(sb1, cur, 64, true);
    __builtin_amdgcn_sched_barrier(0);
    scales(m0, n0, 0, ta, tb);
    __builtin_amdgcn_sched_barrier(0);
    dma(sb2, cur, 128, 1 < p.KB);
    dma(sb3, cur, 192, 1 < p.KB);
    __builtin_amdgcn_sched_barrier(0);
    wait_vm<4 * D>();  // slice 0 has landed: slices 1..3 and the scales came after it
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_sched_barrier(0);
    frags(sb0, a0, b0);

    // One slice: (a, b) hold its fragments.  The wait leaves NW loads in flight, those issued after
    // the next slice's; then everyone's part of the next slice has landed and everyone holds its
    // fragments of this one, whose buffer takes the slice four further on.
    auto slice = [&](auto nw, auto kk, uint8_t *buf, const uint8_t *nbuf, const v8i (&a)[W], const v8i (&b)[W],
                     v8i (&na)[W], v8i (&nb)[W], Src src, int koff, bool in, auto &&before) {
        __builtin_amdgcn_sched_barrier(0);
        wait_vm<decltype(nw)::value>();
        __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0)
        __builtin_amdgcn_s_barrier();
        __builtin_amdgcn_sched_barrier(0);
        before();
        dma(buf, src, koff, in);
        frags(nbuf, na, nb);
        constexpr int KK = decltype(kk)::value;
        if constexpr (YDT == DT_F32) {
            mma_exact<KK, W, W>(acc, a, b, sa, sb);
        } else {
            mma<KK, W, W>(acc, a, b, sa, sb);
            if constexpr (W == 4) {
#pragma unroll
                for (int q = 0; q < 8; ++q) {
                    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);  // matrix instruction
                    __builtin_amdgcn_sched_group_barrier(0x100, 2, 0);  // LDS read
                    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
                    __builtin_amdgcn_sched_group_barrier(0x020, 1, 0);  // load to LDS
                }
            }
        }
        __builtin_amdgcn_sched_barrier(0);
    };
    // Two blocks: four slices.  The scales of the next pair (tile (sm, sn), pair sit) are fetched between
    // slice 1's loads and slice 2's, so a wait sees, of the loads issued after those it is for, two
    // slices' and, in slices 3 and 0, the scales' too.  FRESH: the STORES stores of the tile before lie
    // behind slice 3's loads, and the first three waits leave them in flight.
    constexpr int STORES = W == 4 ? 32 : 0;
    using I0 = std::integral_constant<int, 0>;
    using I1 = std::integral_constant<int, 1>;
    auto pair = [&](auto fresh, int it, Src src, int koff, bool in, bool in2, int64_t sm, int64_t sn, int sit) {
        constexpr int E = decltype(fresh)::value ? STORES : 0;
        // a block past the end gets 2^0: its codes are zeros, but its scale byte is not written
        const bool whole = 2 * it + 1 < p.KB;
        const uint32_t keep = whole ? 0xFFFFu : 0xFFu, fill = whole ? 0u : 0x7F00u;
#pragma unroll
        for (int i = 0; i < W; ++i) {
            sa[i] = (ta[i] & keep) | fill;
            sb[i] = (tb[i] & keep) | fill;
        }
        auto none = [] {};
        slice(std::integral_constant<int, 3 * D + E>{}, I0{}, sb0, sb1, a0, b0, a1, b1, src, koff, in, none);
        slice(std::integral_constant<int, 2 * D + E>{}, I0{}, sb1, sb2, a1, b1, a0, b0, src, koff + 64, in, none);
        slice(std::integral_constant<int, 2 * D + E>{}, I1{}, sb2, sb3, a0, b0, a1, b1, src, koff + 128, in2, [&] {
            scales(sm, sn, sit, ta, tb);
            __builtin_amdgcn_sched_barrier(0);
        });
        slice(std::integral_constant<int, 3 * D>{}, I1{}, sb3, sb0, a1, b1, a0, b0, src, koff + 192, in2, none);
    };

    bool fresh = false;
    for (;;) {
        const int nlg = lg + per;
        const bool more = WALK && nlg < last;
        int64_t nm0 = m0, nn0 = n0;
        if (more) origin(nlg, nm0, nn0);
        const Src nxt = source(nm0, nn0);
#pragma unroll
        for (int i = 0; i < W; ++i)
#pragma unroll
            for (int j = 0; j < W; ++j)
#pragma unroll
                for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.0f;
        // pair `it` is multiplied while pair it + 1, or the next tile's first, is fetched
        auto run = [&](auto f, int it) {
            const bool end = it + 1 == iters;
            const int kb = end ? 0 : 2 * it + 2;  // first block fetched
            const Src src{pick(end, nxt.a, cur.a), pick(end, nxt.b, cur.b), pick(end, nxt.na, cur.na), pick(end, nxt.nb, cur.nb)};
            pair(f, it, src, kb * 128, !end || more, end ? more && p.KB > 1 : kb + 1 < p.KB, pick(end, nm0, m0),
                 pick(end, nn0, n0), end ? 0 : it + 1);
        };
        int it = 0;
        if constexpr (WALK) {
            if (fresh) {
                run(std::true_type{}, 0);
                it = 1;
            }
        }
        for (; it < iters; ++it) run(std::false_type{}, it);
        if constexpr (!WALK) {  // the patches lie in slice buffers: nothing may land there any more
            wait_vm<0>();
            __builtin_amdgcn_s_waitcnt(0xC07F);
            __builtin_amdgcn_s_barrier();
        }
        // pin the accumulators here: keeps the last matrix instructions out of the epilogue's blocks
        if constexpr (W == 4) {
#pragma unroll
            for (int i = 0; i < W; ++i)
#pragma unroll
                for (int j = 0; j < W; ++j) asm volatile("" : "+a"(acc[i][j]));
        }

        // transposed 32 x 32 result: lane l holds row l % 32, columns 8 (r / 4) + 4 (l / 32) + r % 4.
        // Patch of the wave: 32 rows of 128 bytes (64 bf16 or 32 fp32 columns), 144 bytes apart, so that
        // 16 rows' 16-byte pieces lie on distinct banks.
        constexpr int PJ = YDT == DT_BF16 && W > 1 ? 2 : 1;  // tiles side by side in the patch
        constexpr int ES = YDT == DT_BF16 ? 2 : 4, CHUNKS = PJ * 32 * ES / 16, EL = 16 / ES;
        static_assert(W < 4 || W * W / PJ * (32 * CHUNKS / 64) >= STORES, "a whole tile's stores");
        const uint32_t loff = (uint32_t)(lane / CHUNKS) * (uint32_t)p.N * ES + lane % CHUNKS * 16;  // below 2^30
        // A wave's LDS accesses execute in order, and the patch is its own: no barrier.
        auto store = [&](auto whole) {
#pragma unroll
            for (int i = 0; i < W; ++i)
#pragma unroll
                for (int j0 = 0; j0 < W; j0 += PJ) {
                    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                    for (int t = 0; t < PJ; ++t)
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            const v16f &x = acc[i][j0 + t];
                            const int at = wave * PATCH + (lane & 31) * 144 + (t * 32 + 8 * q + 4 * (lane >> 5)) * ES;
                            uint8_t *d = (WALK ? own_patch : sb0) + at;
                            if constexpr (YDT == DT_BF16)
                                *reinterpret_cast<u32x2 *>(d) =
                                    u32x2{bf16_pack2(x[4 * q], x[4 * q + 1]), bf16_pack2(x[4 * q + 2], x[4 * q + 3])};
                            else
                                *reinterpret_cast<u32x4 *>(d) =
                                    u32x4{__float_as_uint(x[4 * q]), __float_as_uint(x[4 * q + 1]),
                                          __float_as_uint(x[4 * q + 2]), __float_as_uint(x[4 * q + 3])};
                        }
                    // rows lr = k RK + lane / CHUNKS of the patch: a uniform base and the lane's offset
                    constexpr int RK = 64 / CHUNKS;
                    const int64_t row = m0 + (wm * W + i) * 32, col = n0 + (wn * W + j0) * 32;
                    uint8_t *base = static_cast<uint8_t *>(p.Y) + (row * p.N + col) * ES;
#pragma unroll
                    for (int k = 0; k < 32 / RK; ++k) {
                        const u32x4 o = *reinterpret_cast<const u32x4 *>((WALK ? own_patch : sb0) + wave * PATCH +
                                                                         (k * RK + lane / CHUNKS) * 144 + lane % CHUNKS * 16);
                        uint8_t *y = base + k * RK * p.N * ES + loff;
                        const int rows = (int)min(p.M - row - k * RK, (int64_t)RK);  // may be <= 0, as cols
                        const int cols = (int)min(p.N - col, (int64_t)(PJ * 32)) - lane % CHUNKS * EL;
                        if (decltype(whole)::value || (lane / CHUNKS < rows && cols >= EL)) {
                            *reinterpret_cast<ua_u32x4 *>(y) = o;
                        } else if (lane / CHUNKS < rows) {
#pragma unroll
                            for (int e = 0; e < EL; ++e) {
                                if (e >= cols) break;
                                if constexpr (YDT == DT_BF16)
                                    reinterpret_cast<uint16_t *>(y)[e] = (uint16_t)(o[e >> 1] >> (16 * (e & 1)));
                                else
                                    reinterpret_cast<uint32_t *>(y)[e] = o[e];
                            }
                        }
                    }
                }
        };
        const bool full = m0 + T <= p.M && n0 + T <= p.N;
        if (full) store(std::true_type{});
        else store(std::false_type{});
        if (!more) break;
        if (!full) wait_vm<0>();  // fewer stores than the next waits count
        fresh = true;
        lg = nlg;
        m0 = nm0;
        n0 = nn0;
        cur = nxt;
    }
    wait_vm<0>();  // no load to LDS outlives the workgroup
}

template <int YDT, int W>
static hipError_t launch_tiles(Args8 p, int cus, hipStream_t s) {
    const int64_t T = 64 * W, tm = (p.M + T - 1) / T, tn = (p.N + T - 1) / T, tiles = (tm * tn + 7) / 8 * 8;
    p.tilesM = (int)tm;
    p.tilesN = (int)tn;
    p.group = (int)(tm < 4 ? tm : 4);
    const int64_t grid = W == 4 ? (tiles < cus / 8 * 8 ? tiles : cus / 8 * 8) : tiles;
    hipLaunchKernelGGL((k_block8_gemm<YDT, W>), dim3((unsigned)grid), dim3(256), 0, s, p);
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
        return w == 4 ? launch_tiles<DT_BF16, 4>(p, cus, s)
                      : w == 2 ? launch_tiles<DT_BF16, 2>(p, cus, s) : launch_tiles<DT_BF16, 1>(p, cus, s);
    return w == 4 ? launch_tiles<DT_F32, 4>(p, cus, s)
                  : w == 2 ? launch_tiles<DT_F32, 2>(p, cus, s) : launch_tiles<DT_F32, 1>(p, cus, s);
}

}  // namespace fp4
