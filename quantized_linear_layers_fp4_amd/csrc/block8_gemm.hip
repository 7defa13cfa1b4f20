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
// 64 W rows and columns.  A stage is one block of 128 along K (a whole cache line a row) of both
// operands, loaded straight to LDS; the fragments of a step of 64 are read under the matrix work of the
// one before it, and a stage's buffer is refilled as soon as its second step's fragments are read, so a
// stage has one barrier.  W = 4 is persistent (one workgroup a CU): the next tile's first stages are on
// their way while a tile's results are stored, and its stores drain under the next tile's products.
// The product is formed transposed, so a lane holds four consecutive columns of one row; the tiles are
// turned to row order through LDS and stored 16 bytes a lane.
#include <algorithm>
#include <cmath>
#include <type_traits>

#include "block8.h"

namespace fp4 {

typedef float v16f __attribute__((ext_vector_type(16)));
typedef unsigned int u32x2 __attribute__((ext_vector_type(2)));
#define LDS_PTR(p) ((__attribute__((address_space(3))) void *)(p))

namespace {

constexpr int BUF_FLAGS = 0x00020000;  // raw buffer descriptor word 3 (gfx9 family)

struct Args8 {
    Op8 A, B;
    int M, N;  // below 2^23
    int KB;  // blocks of 128 along the contraction
    void *Y;
    int tilesM, tilesN, group;
};

// s_waitcnt vmcnt(n), other counters untouched (gfx9 encoding)
template <int N>
__device__ __forceinline__ void wait_vm() {
    __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | 0x0F70);
}

// fp32 outputs: the product on the bf16 instruction (to_bf16).
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

// One wave's share of a stage of an operand: L loads of 1 KiB, straight to LDS.
template <int L>
__device__ __forceinline__ void rows_to_lds(const uint8_t *base, int bytes, uint8_t *buf, const int *off, int koff) {
    const __amdgpu_buffer_rsrc_t r = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t *>(base), 0, bytes, BUF_FLAGS);
#pragma unroll
    for (int j = 0; j < L; ++j)
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
__global__ __launch_bounds__(256, W == 4 ? 1 : 2) void k_block8_gemm(Args8 p) {
    constexpr int T = 64 * W, OP = T * 128, STAGE = 2 * OP;
    constexpr bool WALK = W == 4;             // persistent
    constexpr int NST = W == 1 ? 4 : 2;       // stage buffers
    constexpr int D = 4 * W, S = 2 * W;       // a wave's loads to LDS a stage, and its scale loads a pair of blocks
    constexpr int PATCH = 32 * 144;
    // arrays of their own: the compiler would make a read wait for every load on its way into the same one
    __shared__ __attribute__((aligned(1024))) uint8_t sm0[STAGE < 4 * PATCH && !WALK ? 4 * PATCH : STAGE];
    __shared__ __attribute__((aligned(1024))) uint8_t sm1[STAGE];
    __shared__ __attribute__((aligned(1024))) uint8_t sm2[NST > 2 ? STAGE : 16];
    __shared__ __attribute__((aligned(1024))) uint8_t sm3[NST > 2 ? STAGE : 16];
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
    auto origin = [&](int l, int &m0, int &n0) {
        const int grp = l / (p.group * p.tilesN), first = grp * p.group, gm = min(p.group, p.tilesM - first);
        const int in = l - grp * p.group * p.tilesN;
        m0 = (first + in % gm) * T;
        n0 = in / gm * T;
    };
    int m0, n0;
    origin(lg, m0, n0);

    // Descriptors start at a tile's first row: offsets stay small whatever the operand's size, and rows
    // past the matrix read zeros.  A stage past the contraction's end (or past the last tile) has an
    // empty descriptor and reads zeros.  1 KiB (8 rows of 128 bytes) a load: lane l fills 16-byte place l of
    // it, row l / 8 at place l % 8, whose chunk is turned by the row's bits 1 to 3, so that 16
    // consecutive rows of one chunk lie on 16 distinct places modulo 16.
    const int ldA = (int)p.A.ld, ldB = (int)p.B.ld;
    int offA[2 * W], offB[2 * W];
#pragma unroll
    for (int j = 0; j < 2 * W; ++j) {
        const int row = (wave * 2 * W + j) * 8 + (lane >> 3), ch = ((lane & 7) ^ ((row >> 1) & 7)) * 16;
        offA[j] = row * ldA + ch;
        offB[j] = row * ldB + ch;
    }
    struct Src {
        const uint8_t *a, *b;
        int na, nb;
    };
    auto source = [&](int m, int n) {
        return Src{p.A.codes + m * p.A.ld, p.B.codes + n * p.B.ld, min(T, p.M - m) * ldA, min(T, p.N - n) * ldB};
    };
    auto dma = [&](uint8_t *buf, Src s, int koff, bool in) {
        rows_to_lds<2 * W>(s.a, in ? s.na : 0, buf + wave * W * 2048, offA, koff);
        rows_to_lds<2 * W>(s.b, in ? s.nb : 0, buf + OP + wave * W * 2048, offB, koff);
    };
    // step h of a stage; lane l: row l % 32 of a tile, 32 consecutive values from 64 h + 32 (l / 32)
    const int at = (lane & 31) * 128 + (((2 * (lane >> 5)) ^ ((lane >> 1) & 7)) << 4);
    auto frags = [&](const uint8_t *buf, int h, v8i (&a)[W], v8i (&b)[W]) {
        const uint8_t *sa_ = buf + wm * W * 4096, *sb_ = buf + OP + wn * W * 4096;
        const int x0 = at ^ (h * 64), x1 = x0 ^ 16;
#pragma unroll
        for (int i = 0; i < W; ++i) {
            const u32x4 x = *reinterpret_cast<const u32x4 *>(sa_ + i * 4096 + x0), y = *reinterpret_cast<const u32x4 *>(sa_ + i * 4096 + x1);
            a[i] = v8i{(int)x.x, (int)x.y, (int)x.z, (int)x.w, (int)y.x, (int)y.y, (int)y.z, (int)y.w};
        }
#pragma unroll
        for (int j = 0; j < W; ++j) {
            const u32x4 x = *reinterpret_cast<const u32x4 *>(sb_ + j * 4096 + x0), y = *reinterpret_cast<const u32x4 *>(sb_ + j * 4096 + x1);
            b[j] = v8i{(int)x.x, (int)x.y, (int)x.z, (int)x.w, (int)y.x, (int)y.y, (int)y.z, (int)y.w};
        }
    };
    // scale bytes of blocks 2 it and 2 it + 1 of the lane's rows
    const int iters = (p.KB + 1) / 2;
    auto scales = [&](int m, int n, int it, uint32_t (&sa)[W], uint32_t (&sb)[W]) {
        const uint8_t *pa = reinterpret_cast<const uint8_t *>(p.A.scales + (int64_t)(it >> 1) * p.A.srows) + (it & 1) * 2;
        const uint8_t *pb = reinterpret_cast<const uint8_t *>(p.B.scales + (int64_t)(it >> 1) * p.B.srows) + (it & 1) * 2;
#pragma unroll
        for (int i = 0; i < W; ++i) {
            const uint32_t r = (uint32_t)min(m + (wm * W + i) * 32 + (lane & 31), p.M - 1) >> p.A.sshift;
            sa[i] = *reinterpret_cast<const uint16_t *>(pa + r * 4);
        }
#pragma unroll
        for (int j = 0; j < W; ++j) {
            const uint32_t r = (uint32_t)min(n + (wn * W + j) * 32 + (lane & 31), p.N - 1) >> p.B.sshift;
            sb[j] = *reinterpret_cast<const uint16_t *>(pb + r * 4);
        }
    };

    v16f acc[W][W];
    v8i a0[W], b0[W], a1[W], b1[W];
    uint32_t sa[W], sb[W], ta[W], tb[W];
    Src cur = source(m0, n0);
    // the first stages and scales, in the order of the loop
    dma(sm0, cur, 0, true);
    __builtin_amdgcn_sched_barrier(0);
    scales(m0, n0, 0, ta, tb);
    __builtin_amdgcn_sched_barrier(0);
    dma(sm1, cur, 128, 1 < p.KB);
    if constexpr (NST > 2) {
        dma(sm2, cur, 256, 2 < p.KB);
        dma(sm3, cur, 384, 3 < p.KB);
    }
    __builtin_amdgcn_sched_barrier(0);
    wait_vm<(NST - 1) * D + S>();  // stage 0 has landed: the others and the scales came after it
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_sched_barrier(0);
    frags(sm0, 0, a0, b0);

    // One block: (a0, b0) hold its first step's fragments.  At the barrier everyone holds the second step's,
    // so the buffer takes the stage NST further on, and the wait, which leaves NW loads in flight (those
    // issued after the next stage's), has made everyone's part of the next stage land.
    auto block = [&](auto nw, auto kk, uint8_t *buf, const uint8_t *nbuf, Src src, int koff, bool in, auto &&before) {
        constexpr int KK = decltype(kk)::value;
        __builtin_amdgcn_sched_barrier(0);
        before();
        frags(buf, 1, a1, b1);
        if constexpr (YDT == DT_F32) mma_exact<KK, W, W>(acc, a0, b0, sa, sb);
        else mma<KK, W, W>(acc, a0, b0, sa, sb);
        if constexpr (W == 4 && YDT == DT_BF16) {
#pragma unroll
            for (int q = 0; q < 8; ++q) {
                __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);  // matrix instruction
                __builtin_amdgcn_sched_group_barrier(0x100, 2, 0);  // LDS read
            }
            __builtin_amdgcn_sched_group_barrier(0x008, 8, 0);
        }
        __builtin_amdgcn_sched_barrier(0);
        wait_vm<decltype(nw)::value>();
        __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0)
        __builtin_amdgcn_s_barrier();
        __builtin_amdgcn_sched_barrier(0);
        dma(buf, src, koff, in);
        frags(nbuf, 0, a0, b0);
        if constexpr (YDT == DT_F32) mma_exact<KK, W, W>(acc, a1, b1, sa, sb);
        else mma<KK, W, W>(acc, a1, b1, sa, sb);
        if constexpr (W == 4 && YDT == DT_BF16) {
#pragma unroll
            for (int q = 0; q < 16; ++q) {
                __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
                if (q < 8) __builtin_amdgcn_sched_group_barrier(0x100, 2, 0);
                __builtin_amdgcn_sched_group_barrier(0x020, 1, 0);  // load to LDS
            }
        }
        __builtin_amdgcn_sched_barrier(0);
    };
    // Two blocks.  The scales of the next pair (tile (sm, sn), pair sit) are fetched at the second's start.
    // What was issued after the next block's stage: NST - 2 stages, and the scales of the pairs begun
    // since; in a workgroup's first pair (FIRST) not even those.  FRESH: the STORES stores of the tile
    // before lie behind its last loads.
    constexpr int STORES = W == 4 ? 32 : 0;
    constexpr int NORMAL = 0, FIRST = 1, FRESH = 2;
    auto pair = [&](auto mode, uint8_t *u0, uint8_t *u1, const uint8_t *u2, int it, Src src, int koff, bool in, bool in2, int sm_, int sn, int sit) {
        constexpr int MODE = decltype(mode)::value;
        constexpr int W0 = (NST - 2) * D + (MODE == FIRST ? 0 : (NST - 2) / 2 * S) + (MODE == FRESH ? STORES : 0);
        constexpr int W1 = (NST - 2) * D + (MODE == FIRST && NST > 2 ? 0 : NST / 2 * S);
        // a block past the end gets 2^0: its codes are zeros, but its scale byte is not written
        const bool both = 2 * it + 1 < p.KB;
        const uint32_t keep = both ? 0xFFFFu : 0xFFu, fill = both ? 0u : 0x7F00u;
#pragma unroll
        for (int i = 0; i < W; ++i) {
            sa[i] = (ta[i] & keep) | fill;
            sb[i] = (tb[i] & keep) | fill;
        }
        block(std::integral_constant<int, W0>{}, std::integral_constant<int, 0>{}, u0, u1, src, koff, in, [] {});
        block(std::integral_constant<int, W1>{}, std::integral_constant<int, 1>{}, u1, u2, src, koff + 128, in2, [&] {
            scales(sm_, sn, sit, ta, tb);
            __builtin_amdgcn_sched_barrier(0);
        });
    };

    bool fresh = false;
    for (;;) {
        const int nlg = lg + per;
        const bool more = WALK && nlg < last;
        int nm0 = m0, nn0 = n0;
        if (more) origin(nlg, nm0, nn0);
        const Src nxt = source(nm0, nn0);
#pragma unroll
        for (int i = 0; i < W; ++i)
#pragma unroll
            for (int j = 0; j < W; ++j)
#pragma unroll
                for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.0f;
        // pair `it` is multiplied while the stages NST blocks on, or the next tile's first, are fetched
        auto run = [&](auto mode, uint8_t *u0, uint8_t *u1, const uint8_t *u2, int it) {
            const bool end = it + 1 == iters, far = 2 * it + NST >= 2 * iters;  // far: past this tile
            const int kb = far ? 2 * it + NST - 2 * iters : 2 * it + NST;       // first block fetched
            const Src src{pick(far, nxt.a, cur.a), pick(far, nxt.b, cur.b), pick(far, nxt.na, cur.na), pick(far, nxt.nb, cur.nb)};
            pair(mode, u0, u1, u2, it, src, kb * 128, (!far || more) && kb < p.KB, (!far || more) && kb + 1 < p.KB, pick(end, nm0, m0),
                 pick(end, nn0, n0), end ? 0 : it + 1);
        };
        using Normal = std::integral_constant<int, NORMAL>;
        int it = 0;
        if constexpr (NST > 2) {
            run(std::integral_constant<int, FIRST>{}, sm0, sm1, sm2, 0);
            for (it = 1; it < iters; it += 2) {
                run(Normal{}, sm2, sm3, sm0, it);
                if (it + 1 < iters) run(Normal{}, sm0, sm1, sm2, it + 1);
            }
        } else {
            if (WALK && fresh) {
                run(std::integral_constant<int, FRESH>{}, sm0, sm1, sm0, 0);
                it = 1;
            }
            for (; it < iters; ++it) run(Normal{}, sm0, sm1, sm0, it);
        }
        if constexpr (!WALK) {  // the patches lie in stage buffers: nothing may land there any more
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
                            uint8_t *d = (WALK ? own_patch : sm0) + at;
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
                    const int row = m0 + (wm * W + i) * 32, col = n0 + (wn * W + j0) * 32;
                    uint8_t *base = static_cast<uint8_t *>(p.Y) + ((int64_t)row * p.N + col) * ES;
#pragma unroll
                    for (int k = 0; k < 32 / RK; ++k) {
                        const u32x4 o = *reinterpret_cast<const u32x4 *>((WALK ? own_patch : sm0) + wave * PATCH +
                                                                         (k * RK + lane / CHUNKS) * 144 + lane % CHUNKS * 16);
                        uint8_t *y = base + (int64_t)(k * RK) * p.N * ES + loff;
                        const int rows = min(p.M - row - k * RK, RK);  // may be <= 0, as cols
                        const int cols = min(p.N - col, PJ * 32) - lane % CHUNKS * EL;
                        if (decltype(whole)::value || (lane / CHUNKS < rows && cols >= EL)) {
                            __builtin_nontemporal_store((ua_u32x4)o, reinterpret_cast<ua_u32x4 *>(y));
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
    p.M = (int)M;
    p.N = (int)N;
    p.KB = (int)((K + 127) / 128);
    p.Y = Y;
    p.tilesM = p.tilesN = p.group = 0;
    if (block8_few(M, N)) return launch_block8_few(A, B, M, N, K, Y, y_dt, s);
    // The tile with the least expected time: rounds of the device (tiles of 256 one a CU, the others two a CU, a
    // last round of those counting by its part) times a round's, which is a K-proportional part and a fixed one,
    // fitted in us to thirteen shapes of up to 6000 x 6000 x 4096.  Measured, tiles of 64 | 128 | 256, bf16 output at
    // K = 4096: 512 x 4096 17.3 | 21.6 | 40.6, 2048 x 4096 63 | 35 | 45, 3000 x 4096 100 | 57 | 49, 4096 x 4096
    // 123 | 76 | 55, 4600 x 4600 152 | 105 | 109; fp32 output 23 | 35 | 84, 82 | 59 | 95, 126 | 90 | 101, 169 | 120 | 108,
    // 214 | 165 | 209.
    auto count = [&](int64_t t) { return (double)(((M + t - 1) / t) * ((N + t - 1) / t)); };
    const bool f32 = y_dt != DT_BF16;
    const double k = (double)K / 4096;
    const double t4 = std::ceil(count(256) / cus) * (k * (f32 ? 92 : 46) + (f32 ? 12 : 8));
    const double t2 = std::max(count(128) / (2 * cus), 0.67) * (k * (f32 ? 54 : 33) + (f32 ? 5 : 3));
    const double t1 = std::max(count(64) / (2 * cus), 0.7) * (k * (f32 ? 19 : 14) + 2);
    const int w = t4 <= t2 && t4 <= t1 ? 4 : t2 <= t1 ? 2 : 1;
    if (y_dt == DT_BF16)
        return w == 4 ? launch_tiles<DT_BF16, 4>(p, cus, s)
                      : w == 2 ? launch_tiles<DT_BF16, 2>(p, cus, s) : launch_tiles<DT_BF16, 1>(p, cus, s);
    return w == 4 ? launch_tiles<DT_F32, 4>(p, cus, s)
                  : w == 2 ? launch_tiles<DT_F32, 2>(p, cus, s) : launch_tiles<DT_F32, 1>(p, cus, s);
}

}  // namespace fp4
