// Attention of packed queries over the 4-bit paged cache (layout: kv4.h).
//
//      s = scale * q . k   over the visible tokens: j <= p, and j > p - window if there is a window
//      o = sum softmax(s) v,   lse = log sum exp s
//
// Query i of a sequence with len tokens in the cache and qlen queries stands at p = len - qlen + i.
// Query heads hq = hkv * g share key/value heads; the rows of one key/value head are (query, head of
// the group) pairs, row r = i * g + head.
//
// Scores.  K is unpacked in registers to bf16, where every scaled E2M1 value is exact, and multiplied
// with q on the bf16 matrix instructions.  (The scaled instruction would take the FP4 codes and E8M0 bytes as
// they lie, beside q split into two E4M3 terms, at the same matrix time; but its adder drops what lies
// below 2^-13 of the largest of eight products, which left scores 1e-5..5e-5 off.)
// Softmax.  Base 2, running maximum and sum in fp32, tokens in the accumulator's rows and query rows
// in its columns, so a lane holds one query row: rescaling is one factor a lane.
// Values.  O^T += V^T . P^T in bf16: a lane's eight P values are where the instruction wants them
// (the token order of a tile is chosen for that), and V is unpacked in registers from 32 contiguous
// bytes (8 tokens x 8 columns) with the scale in the converting instruction.  Unpacked V is exact in
// bf16; P is rounded to bf16 (2^-9 of each term, as the output itself is), the sum of P is taken
// before that rounding.
#include <algorithm>

#include "block8.h"
#include "kv4.h"

namespace fp4 {

typedef float v4f __attribute__((ext_vector_type(4)));
typedef __bf16 v8bf __attribute__((ext_vector_type(8)));
typedef __bf16 v2bf __attribute__((ext_vector_type(2)));
typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));

namespace {

constexpr int NW = 4;        // waves of a decode workgroup
constexpr int TT = 32;       // tokens a wave takes at once
constexpr float LN2 = 0.69314718055994530942f;
constexpr float LOG2E = 1.44269504088896340736f;

struct DecArgs {
    Kv4Attn a;
    int g, rt;        // heads a group; row tiles of 16 a (sequence, head)
    int splits;       // workgroups along the tokens
    int chunk;        // tokens each takes (a multiple of NW * TT)
    float c;          // scale * log2(e)
};

// What one workgroup's rows see: rows of sequence `seq`, tile rt.
struct Span {
    int len, qlen, qbeg;
    int rows;         // qlen * g
    int lo, hi;       // tokens any of the tile's rows sees: [lo, hi), lo a multiple of TT
    int full_lo, full_hi;  // tokens that all of its rows see
};

__device__ __forceinline__ Span span_of(const Kv4Attn &a, int g, int seq, int row0, int nrows) {
    Span s;
    s.len = a.lens[seq];
    s.qbeg = a.q_start ? max(a.q_start[seq], 0) : seq;
    s.qlen = a.q_start ? min(a.q_start[seq + 1], a.nq) - s.qbeg : 1;
    s.rows = max(s.qlen, 0) * g;
    const int cap = min(s.len, a.width << a.geo.page_log2);
    if (row0 >= s.rows) {
        s.lo = s.hi = s.full_lo = s.full_hi = 0;
        return s;
    }
    const int j0 = row0 / g, j1 = min(row0 + nrows - 1, s.rows - 1) / g;
    const int p0 = s.len - s.qlen + j0, p1 = s.len - s.qlen + j1;
    s.hi = max(min(p1 + 1, cap), 0);
    s.full_hi = min(p0 + 1, cap);
    s.lo = a.window ? max(p0 - a.window + 1, 0) & ~(TT - 1) : 0;
    s.full_lo = a.window ? max(p1 - a.window + 1, 0) : 0;
    return s;
}

// E8M0 byte I of a dword as a scale: its exponent field.
template <int I>
__device__ __forceinline__ float scale_of(uint32_t w) {
    if constexpr (I == 3) return __uint_as_float((w >> 1) & 0x7F800000u);
    else return __uint_as_float((w << (23 - 8 * I)) & 0x7F800000u);
}

// N dwords of a token (8 values each) times the group's scale -> N operands of 8 bf16
// values; a poisoned token (scale byte 255) becomes NaN.
template <int N>
__device__ __forceinline__ void unpack_row(const uint32_t (&w)[N], uint32_t b, v8bf (&f)[N]) {
    const float sc = __uint_as_float(b << 23);
#pragma unroll
    for (int i = 0; i < N; ++i) {
        u32x4 x;
        x[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w[i], sc, 0));
        x[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w[i], sc, 1));
        x[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w[i], sc, 2));
        x[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w[i], sc, 3));
        if (i == 0) x[0] = b == 255u ? 0x7FC07FC0u : x[0];
        f[i] = __builtin_bit_cast(v8bf, x);
    }
}

// Byte B (two columns) of the eight tokens' dwords w -> the two columns' eight bf16 values, sc[t]
// token t's scale.
template <int B>
__device__ __forceinline__ void unpack_cols(const uint32_t (&w)[8], const float (&sc)[8], v8bf &c0, v8bf &c1) {
    uint32_t lo[4], hi[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
        const uint32_t x = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w[2 * u], sc[2 * u], B));
        const uint32_t y = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w[2 * u + 1], sc[2 * u + 1], B));
        lo[u] = __builtin_amdgcn_perm(y, x, 0x05040100u);
        hi[u] = __builtin_amdgcn_perm(y, x, 0x07060302u);
    }
    c0 = __builtin_bit_cast(v8bf, u32x4{lo[0], lo[1], lo[2], lo[3]});
    c1 = __builtin_bit_cast(v8bf, u32x4{hi[0], hi[1], hi[2], hi[3]});
}

}  // namespace

// Few rows (single tokens, drafts): 16 rows of one (sequence, key/value head) a workgroup, its four
// waves taking tiles of 32 tokens in turn and joining in LDS; `splits` workgroups share the tokens.
// Bound by the cache's bytes.
template <int D>
__global__ __launch_bounds__(64 * NW) void k_kv4_decode(DecArgs p) {
    constexpr int J = D / 16;   // columns a lane owns in the O^T tiles: J n + j
    constexpr int KS = D / 32;  // contraction steps of the scores
    const Kv4Attn &a = p.a;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, n = lane & 15, h = lane >> 4;
    int id = blockIdx.x;
    const int split = id % p.splits; id /= p.splits;
    const int head = id % a.geo.hkv; id /= a.geo.hkv;
    const int rt = id % p.rt, seq = id / p.rt;
    const int row0 = rt * 16;
    const Span sp = span_of(a, p.g, seq, row0, 16);
    if (row0 >= sp.rows) return;
    const int beg = sp.lo + split * p.chunk, end = min(sp.hi, beg + p.chunk);
    if (p.splits > 1 && beg >= end) return;  // the joining kernel counts the splits the same way

    // this lane's row
    const int row = row0 + n;
    const bool live = row < sp.rows;
    const int qi = live ? row / p.g : 0, qh = live ? head * p.g + row % p.g : 0;
    const int pos = sp.len - sp.qlen + qi;
    const int vhi = live ? pos + 1 : 0, vlo = a.window ? pos - a.window + 1 : 0;
    // q: lane h owns D/4 consecutive columns, KS operands of 8
    v8bf qf[KS];
#pragma unroll
    for (int i = 0; i < KS; ++i) {
        u32x4 x = {0, 0, 0, 0};
        if (live)
            x = *reinterpret_cast<const ua_u32x4 *>(a.q + (int64_t)(sp.qbeg + qi) * a.q_ts + (int64_t)qh * a.q_hs +
                                                    h * (D / 4) + 8 * i);
        qf[i] = __builtin_bit_cast(v8bf, x);
    }

    const int P = 1 << a.geo.page_log2;
    const int64_t region = a.geo.region();
    const int32_t *table = a.pages + (int64_t)seq * a.page_rs;
    v4f acc[J];
#pragma unroll
    for (int j = 0; j < J; ++j) acc[j] = v4f{0, 0, 0, 0};
    float m = -INFINITY, l = 0.0f;

    for (int t0 = beg + wave * TT; t0 < end; t0 += NW * TT) {
        // tokens of the scores' row n in half s: 8 (n / 4) + 4 s + n % 4; of V's step: 8 h + 0..7.
        // A page that the table does not hold (outside the cache) is as if its tokens were masked.
        const int tk = t0 + 8 * (n >> 2), tv = t0 + 8 * h;
        const int pk = tk < end ? table[tk >> a.geo.page_log2] : -1;
        const int pv = tv < end ? table[tv >> a.geo.page_log2] : -1;
        const bool okk = (uint32_t)pk < (uint64_t)a.geo.pages, okv = (uint32_t)pv < (uint64_t)a.geo.pages;
        uint32_t kw[2][KS], ks[2];
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            ks[s] = 0;
#pragma unroll
            for (int i = 0; i < KS; ++i) kw[s][i] = 0;
            if (okk) {
                const int tok = (tk & (P - 1)) + 4 * s + (n & 3);
                const uint8_t *base = a.cache + ((int64_t)pk * a.geo.hkv + head) * region;
                const uint32_t *src = reinterpret_cast<const uint32_t *>(base + tok * (D / 2) + h * (D / 8));
#pragma unroll
                for (int i = 0; i < KS; ++i) kw[s][i] = src[i];
                ks[s] = base[a.geo.ks_off() + (h * D / 128) * P + tok];
            }
        }
        uint32_t vw[8];
        uint2 vs = make_uint2(0, 0);
#pragma unroll
        for (int i = 0; i < 8; ++i) vw[i] = 0;
        if (okv) {
            const int tok = tv & (P - 1);
            const uint8_t *base = a.cache + ((int64_t)pv * a.geo.hkv + head) * region;
            const int dw = D == 128 ? n : n >> 1;
            const u32x4 *src = reinterpret_cast<const u32x4 *>(base + a.geo.v_off() + ((tok >> 3) * (D / 8) + dw) * 32);
            const u32x4 x = src[0], y = src[1];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                vw[i] = x[i];
                vw[4 + i] = y[i];
            }
            vs = *reinterpret_cast<const uint2 *>(base + a.geo.vs_off() + (n * J / 32) * P + tok);
        }
        if constexpr (D == 64) {
#pragma unroll
            for (int i = 0; i < 8; ++i) vw[i] >>= 16 * (n & 1);
        }

        // scores: element r of half s is token t0 + 8 h + 4 s + r, row n
        float x[8];
        const bool okp = __shfl((int)okk, 4 * h, 64) != 0;  // of the lane's score tokens' page
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            v4f d = v4f{0, 0, 0, 0};
            v8bf kf[KS];
            unpack_row<KS>(kw[s], ks[s], kf);
#pragma unroll
            for (int i = 0; i < KS; ++i) d = __builtin_amdgcn_mfma_f32_16x16x32_bf16(kf[i], qf[i], d, 0, 0, 0);
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int tok = t0 + 8 * h + 4 * s + r;
                x[4 * s + r] = okp && tok < min(vhi, end) && tok >= vlo ? d[r] * p.c : -INFINITY;
            }
        }
        float mx = m;
#pragma unroll
        for (int i = 0; i < 8; ++i) mx = fmaxf(mx, x[i]);
        mx = fmaxf(mx, __shfl_xor(mx, 16, 64));
        mx = fmaxf(mx, __shfl_xor(mx, 32, 64));
        const float mu = mx == -INFINITY ? 0.0f : mx;
        const float alpha = __builtin_amdgcn_exp2f(m - mu);
        m = mx;
        l *= alpha;
#pragma unroll
        for (int j = 0; j < J; ++j) acc[j] *= alpha;
        float e[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            e[i] = __builtin_amdgcn_exp2f(x[i] - mu);
            l += e[i];
        }
        const v8bf pb = __builtin_bit_cast(v8bf, u32x4{bf16_pack2(e[0], e[1]), bf16_pack2(e[2], e[3]),
                                                       bf16_pack2(e[4], e[5]), bf16_pack2(e[6], e[7])});
        const float sc[8] = {scale_of<0>(vs.x), scale_of<1>(vs.x), scale_of<2>(vs.x), scale_of<3>(vs.x),
                             scale_of<0>(vs.y), scale_of<1>(vs.y), scale_of<2>(vs.y), scale_of<3>(vs.y)};
        v8bf c0, c1;
#define PV(B)                                                                                 \
    unpack_cols<B>(vw, sc, c0, c1);                                                           \
    acc[2 * B] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(c0, pb, acc[2 * B], 0, 0, 0);        \
    acc[2 * B + 1] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(c1, pb, acc[2 * B + 1], 0, 0, 0);
        PV(0)
        PV(1)
        if constexpr (D == 128) {
            PV(2)
            PV(3)
        }
#undef PV
    }

    // the waves join: maxima, then sums and outputs over the common maximum, in wave order
    __shared__ float sm[NW][16], sl_[NW][16];
    __shared__ __attribute__((aligned(16))) float so[NW][16][D + 4];
    l += __shfl_xor(l, 16, 64);
    l += __shfl_xor(l, 32, 64);
    if (h == 0) {
        sm[wave][n] = m;
        sl_[wave][n] = l;
    }
    // element (j, r): column (4 h + r) J + j of row n
#pragma unroll
    for (int r = 0; r < 4; ++r)
#pragma unroll
        for (int j = 0; j < J; j += 4)
            *reinterpret_cast<float4 *>(&so[wave][n][(4 * h + r) * J + j]) =
                make_float4(acc[j][r], acc[j + 1][r], acc[j + 2][r], acc[j + 3][r]);
    __syncthreads();
    for (int i = threadIdx.x; i < 16 * (D / 4); i += 64 * NW) {
        const int r = i / (D / 4), col = i % (D / 4) * 4;
        if (row0 + r >= sp.rows) continue;
        float M = sm[0][r], L = 0.0f;
#pragma unroll
        for (int w = 1; w < NW; ++w) M = fmaxf(M, sm[w][r]);
        const float mu = M == -INFINITY ? 0.0f : M;
        float o[4] = {0, 0, 0, 0};
#pragma unroll
        for (int w = 0; w < NW; ++w) {
            const float f = __builtin_amdgcn_exp2f(sm[w][r] - mu);
            L += sl_[w][r] * f;
            const float4 v = *reinterpret_cast<const float4 *>(&so[w][r][col]);
            o[0] += v.x * f;
            o[1] += v.y * f;
            o[2] += v.z * f;
            o[3] += v.w * f;
        }
        if (p.splits == 1) {
            const int64_t out = (int64_t)(sp.qbeg + (row0 + r) / p.g) * a.hq + head * p.g + (row0 + r) % p.g;
            const float inv = L == 0.0f ? 0.0f : 1.0f / L;
            *reinterpret_cast<uint2 *>(a.o + out * D + col) =
                make_uint2(bf16_pack2(o[0] * inv, o[1] * inv), bf16_pack2(o[2] * inv, o[3] * inv));
            if (a.lse && col == 0) a.lse[out] = L == 0.0f ? -INFINITY : (M + __builtin_amdgcn_logf(L)) * LN2;
        } else {
            // partial row: D sums, then the maximum and the sum of the split
            float *w = reinterpret_cast<float *>(a.ws) +
                       ((((int64_t)seq * p.rt + rt) * a.geo.hkv + head) * p.splits + split) * 16 * (D + 4) + r * (D + 4);
            *reinterpret_cast<float4 *>(w + col) = make_float4(o[0], o[1], o[2], o[3]);
            if (col == 0) {
                w[D] = M;
                w[D + 1] = L;
            }
        }
    }
}

// Joins the splits of a (sequence, head): one wave a row, splits in ascending order.
template <int D>
__global__ __launch_bounds__(256) void k_kv4_join(DecArgs p) {
    const Kv4Attn &a = p.a;
    const int lane = threadIdx.x & 63;
    int64_t id = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
    const int r = (int)(id % 16); id /= 16;
    const int head = (int)(id % a.geo.hkv); id /= a.geo.hkv;
    const int rt = (int)(id % p.rt);
    const int seq = (int)(id / p.rt);
    if (seq >= a.b) return;
    const Span sp = span_of(a, p.g, seq, rt * 16, 16);
    const int row = rt * 16 + r;
    if (row >= sp.rows) return;
    const int ns = sp.hi > sp.lo ? (sp.hi - sp.lo + p.chunk - 1) / p.chunk : 0;
    const float *w = reinterpret_cast<const float *>(a.ws) +
                     (((int64_t)seq * p.rt + rt) * a.geo.hkv + head) * p.splits * 16 * (D + 4) + r * (D + 4);
    constexpr int SS = 16 * (D + 4);
    float M = -INFINITY;
    for (int s = lane; s < ns; s += 64) M = fmaxf(M, w[(int64_t)s * SS + D]);
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) M = fmaxf(M, __shfl_xor(M, off, 64));
    const float mu = M == -INFINITY ? 0.0f : M;
    constexpr int E = D / 64;
    float o[E] = {}, L = 0.0f;
    for (int s = 0; s < ns; ++s) {
        const float *x = w + (int64_t)s * SS;
        const float f = __builtin_amdgcn_exp2f(x[D] - mu);
        L += x[D + 1] * f;
#pragma unroll
        for (int i = 0; i < E; ++i) o[i] += x[lane * E + i] * f;
    }
    const float inv = L == 0.0f ? 0.0f : 1.0f / L;
    const int64_t out = (int64_t)(sp.qbeg + row / p.g) * a.hq + head * p.g + row % p.g;
    if constexpr (E == 2)
        *reinterpret_cast<uint32_t *>(a.o + out * D + lane * 2) = bf16_pack2(o[0] * inv, o[1] * inv);
    else
        a.o[out * D + lane] = (uint16_t)bf16_pack2(o[0] * inv, 0.0f);
    if (a.lse && lane == 0) a.lse[out] = L == 0.0f ? -INFINITY : (M + __builtin_amdgcn_logf(L)) * LN2;
}

namespace {
constexpr int64_t WANT = 1024;  // workgroups of a call, where its tokens allow: four a CU
// The split of a call along the tokens: WANT workgroups in all, each with at least one round of its
// waves' tiles.
void plan(int b, int max_q, int hq, const Kv4Geom &g, int width, int window, DecArgs &p) {
    p.g = hq / g.hkv;
    p.rt = (int)(((int64_t)max_q * p.g + 15) / 16);
    const int64_t groups = (int64_t)b * g.hkv * p.rt, unit = NW * TT;
    int64_t span = (int64_t)width << g.page_log2;
    if (window) span = std::min<int64_t>(span, (int64_t)window + 16 / p.g + 1 + TT);  // + the start's rounding down
    int64_t splits = (WANT + groups - 1) / groups;
    splits = std::max<int64_t>(1, std::min(splits, (span + unit - 1) / unit));
    const int64_t chunk = ((span + splits - 1) / splits + unit - 1) / unit * unit;
    p.chunk = (int)chunk;
    p.splits = (int)((span + chunk - 1) / chunk);
}
}  // namespace

// Enough for every window: a window only shortens the span, so the bound on the splits falls.
size_t kv4_attn_ws_bytes(int b, int max_q, int hq, const Kv4Geom &g, int width) {
    const int64_t rt = ((int64_t)max_q * (hq / g.hkv) + 15) / 16, groups = (int64_t)b * g.hkv * rt, unit = NW * TT;
    const int64_t splits = std::min((WANT + groups - 1) / groups, (((int64_t)width << g.page_log2) + unit - 1) / unit);
    return splits <= 1 ? 0 : (size_t)(groups * splits) * 16 * (g.d + 4) * 4;
}

hipError_t launch_kv4_attn(const Kv4Attn &a, hipStream_t s) {
    DecArgs p;
    p.a = a;
    p.c = a.scale * LOG2E;
    plan(a.b, a.max_q, a.hq, a.geo, a.width, a.window, p);
    const int64_t tiles = (int64_t)a.b * p.rt * a.geo.hkv;
    const dim3 grid((unsigned)(tiles * p.splits));
    if (a.geo.d == 128) hipLaunchKernelGGL(k_kv4_decode<128>, grid, dim3(64 * NW), 0, s, p);
    else hipLaunchKernelGGL(k_kv4_decode<64>, grid, dim3(64 * NW), 0, s, p);
    hipError_t e = hipGetLastError();
    if (e == hipSuccess && p.splits > 1) {
        const dim3 jg((unsigned)(tiles * 4));
        if (a.geo.d == 128) hipLaunchKernelGGL(k_kv4_join<128>, jg, dim3(256), 0, s, p);
        else hipLaunchKernelGGL(k_kv4_join<64>, jg, dim3(256), 0, s, p);
        e = hipGetLastError();
    }
    return e;
}

}  // namespace fp4
