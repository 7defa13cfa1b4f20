// Norm of queries and keys for each head with the rotation of their positions, its gradients, and the same with keys
// and values written into the 4-bit cache (layout: kv4.h).
//
//      r = 1 / sqrt(mean(x^2) + eps),  y = x r w,  then over the first rot columns
//      (a, b) -> (a cos - b sin, b cos + a sin) for pairs (i, i + rot / 2), or (2 i, 2 i + 1) if interleaved
//
// Gradients: g = the rotation by the opposite angle of dy, dw = sum over tokens and heads of g x r, and with h = g w
// dx = r (h - x r mean(h x r)).
//
// Each value is read once and written once (backward: x and dy once, dx once): bound by memory.  A lane holds 8 columns,
// d / 8 lanes a row (rounded up to a power of two, L); a lane group stays with one token and goes through a
// run of its heads, so that angles and weights are fetched once a run and not once a row.
// Keys are made in 64 bits and rounded to fp32 and then to the type, so that their values do not depend on the order of
// a sum: the fused write puts into the cache what the norm and kv4_write put there one after the other, bit for bit, and a
// code of the cache next to a border is the right one.  Queries and gradients are made in fp32 (36.3 instead of
// 39.8 us for the layer's forward below), but for rows whose mean square leaves 2^-80 .. 2^120.
// A layer's forward (8192 tokens of 32 + 8 heads of 128, bf16: 168 MB) takes 36.6 us, 4.6 TB/s where a large copy reaches
// 4.8; its gradients (252 MB) 48 and the weights' sums 5; 16384 tokens into the cache (353 MB) 81 to 83.
#include <algorithm>

#include "block8.h"
#include "serve.h"

namespace fp4 {

namespace {

// Heads of a run of a large call, in bf16 and in fp32.  The angles and weights of a run cost about as much as two rows:
// a layer's forward (8192 tokens of 40 heads of 128, bf16) takes 45 us with runs of 2, 38 of 4, 36 of 8, 39.5 of 16; the write into the
// cache (16384 tokens, 32 and 8 heads) 95 of 2, 82 of 4, 86 of 8, whose registers leave two waves.
constexpr int FWD16 = 8, FWD32 = 4, FILL16 = 4, FILL32 = 2, BWD16 = 4, BWD32 = 2;
constexpr int BWD_BLOCKS = 1024;  // workgroups of a backward at most: rows of partial weight gradients

// A launch has fewer than 2^32 threads along x, and the largest calls more: workgroups lie in rows of 2^23 at most, numbered on.
// The last row's surplus finds no token of its own.
__device__ __forceinline__ uint32_t workgroup() { return blockIdx.y * gridDim.x + blockIdx.x; }
dim3 grid_of(int64_t workgroups) {
    const int64_t rows = (workgroups + (1 << 23) - 1) >> 23;
    return dim3((unsigned)((workgroups + rows - 1) / rows), (unsigned)rows);
}

// x of another lane of the 16 that a DPP row is.
template <int CTRL>
__device__ __forceinline__ float lane_of(float x) {
    return __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(x), CTRL, 0xF, 0xF, true));
}
template <int CTRL>
__device__ __forceinline__ double lane_of(double x) {
    const uint64_t b = __builtin_bit_cast(uint64_t, x);
    const uint32_t lo = (uint32_t)__builtin_amdgcn_mov_dpp((int)b, CTRL, 0xF, 0xF, true);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_mov_dpp((int)(b >> 32), CTRL, 0xF, 0xF, true);
    return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
// Sum over the L lanes of a group, in each of them: neighbours, neighbouring pairs, then mirrored halves of 8 and of 16,
// whose lanes hold the same by then.
template <int L, typename T>
__device__ __forceinline__ T group_sum(T x) {
    x += lane_of<0xB1>(x);   // quad_perm 1 0 3 2
    x += lane_of<0x4E>(x);   // quad_perm 2 3 0 1
    if constexpr (L >= 8) x += lane_of<0x141>(x);   // row_half_mirror
    if constexpr (L >= 16) x += lane_of<0x140>(x);  // row_mirror
    if constexpr (L >= 32) x += __shfl_xor(x, 16, 64);
    return x;
}

// 1 / sqrt(v) from the instruction's 2^-23 by one step of the series (1 - e)^(-1/2) = 1 + e / 2 + 3 e^2 / 8 + ...
__device__ __forceinline__ double rsqrt64(double v) {
    const double r = __builtin_amdgcn_rsq(v);
    const double e = __builtin_fma(-v * r, r, 1.0);
    return __builtin_fma(r * e, __builtin_fma(0.375, e, 0.5), r);
}

template <int DT>
struct Raw {
    u32x4 w[DT == DT_BF16 ? 1 : 2];
};

template <int DT>
__device__ __forceinline__ Raw<DT> load_raw(const void *x, int64_t elem, bool live) {
    Raw<DT> r;
#pragma unroll
    for (auto &q : r.w) q = u32x4{0, 0, 0, 0};
    if (!live) return r;
    if constexpr (DT == DT_BF16) {
        r.w[0] = *reinterpret_cast<const ua_u32x4 *>(static_cast<const uint16_t *>(x) + elem);
    } else {
        const float *p = static_cast<const float *>(x) + elem;
        r.w[0] = *reinterpret_cast<const ua_u32x4 *>(p);
        r.w[1] = *reinterpret_cast<const ua_u32x4 *>(p + 4);
    }
    return r;
}

template <int DT>
__device__ __forceinline__ void values(const Raw<DT> &r, float (&v)[8]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (DT == DT_BF16) {
            v[2 * i] = __uint_as_float(r.w[0][i] << 16);
            v[2 * i + 1] = __uint_as_float(r.w[0][i] & 0xFFFF0000u);
        } else {
            v[i] = __uint_as_float(r.w[0][i]);
            v[4 + i] = __uint_as_float(r.w[1][i]);
        }
    }
}

// The values that the lane's are paired with: of another lane, or its own neighbours; zeros where the lane's columns are not
// rotated (`mask` 0 instead of ~0).  They stand there beside a sine of 0, and an infinity would make that NaN.
template <int DT, bool IL>
__device__ __forceinline__ void partners(const Raw<DT> &r, int from, uint32_t mask, float (&v)[8]) {
    Raw<DT> p;
#pragma unroll
    for (int q = 0; q < (DT == DT_BF16 ? 1 : 2); ++q)
#pragma unroll
        for (int i = 0; i < 4; ++i) p.w[q][i] = (IL ? r.w[q][i] : (uint32_t)__shfl((int)r.w[q][i], from, 64)) & mask;
    if constexpr (IL) {
        float u[8];
        values<DT>(p, u);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = u[i ^ 1];
    } else {
        values<DT>(p, v);
    }
}

// PAST: past the caches, which leaves them to the inputs.
template <int DT, bool PAST>
__device__ __forceinline__ void store_row(void *y, int64_t elem, const float (&v)[8]) {
    auto put = [](ua_u32x4 w, void *p) {
        if constexpr (PAST) __builtin_nontemporal_store(w, static_cast<ua_u32x4 *>(p));
        else *static_cast<ua_u32x4 *>(p) = w;
    };
    if constexpr (DT == DT_BF16) {
        put(ua_u32x4{bf16_pack2(v[0], v[1]), bf16_pack2(v[2], v[3]), bf16_pack2(v[4], v[5]), bf16_pack2(v[6], v[7])},
            static_cast<uint16_t *>(y) + elem);
    } else {
        float *p = static_cast<float *>(y) + elem;
        put(__builtin_bit_cast(ua_u32x4, v4f{v[0], v[1], v[2], v[3]}), p);
        put(__builtin_bit_cast(ua_u32x4, v4f{v[4], v[5], v[6], v[7]}), p + 4);
    }
}

// Eight weights from a column on.
__device__ __forceinline__ void weights_at(const NormRope &a, const void *w, int col, float (&v)[8]) {
    if (!w) {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = 1.0f;
    } else if (a.w_dt == DT_BF16) {
        values<DT_BF16>(load_raw<DT_BF16>(w, col, true), v);
    } else {
        values<DT_F32>(load_raw<DT_F32>(w, col, true), v);
    }
}

// A lane's part of a token: its columns, their partners' place, the angles.  A position past the table gives NaN angles.
template <bool IL>
struct Turn {
    int col;         // first of the lane's 8 columns
    bool live, zero; // its columns are the row's; the token's rows are zeros (a negative position)
    uint32_t mask;   // ~0 if its columns are rotated (all eight are, or none), else 0
    int from;        // lane of the partners
    float c[8], s[8];

    __device__ __forceinline__ Turn(const NormRope &a, int64_t t, int lane, int lanes) {
        col = lane * 8;
        live = col < a.d;
        zero = false;
        mask = col < a.rot ? ~0u : 0u;
        const int me = threadIdx.x & 63, half = a.rot / 16;
        from = IL || lane >= 2 * half ? me : lane < half ? me + half : me - half;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            c[i] = 1.0f;
            s[i] = 0.0f;
        }
        if (!a.rot) return;
        const int pos = a.positions[t];
        zero = pos < 0;
        if (col >= a.rot) return;
        const bool in = (uint64_t)pos < (uint64_t)a.max_pos;
        const float *row = a.table + (in ? (int64_t)pos : 0) * a.rot;
        if constexpr (IL) {
            const float4 x = *reinterpret_cast<const float4 *>(row + col / 2);
            const float4 y = *reinterpret_cast<const float4 *>(row + a.rot / 2 + col / 2);
            const float cs[4] = {x.x, x.y, x.z, x.w}, sn[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                c[i] = cs[i >> 1];
                s[i] = i & 1 ? sn[i >> 1] : -sn[i >> 1];
            }
        } else {
            const bool second = lane >= half;
            const float4 *p = reinterpret_cast<const float4 *>(row + (second ? col - a.rot / 2 : col));
            const float4 x = p[0], y = p[1], z = p[a.rot / 8], w = p[a.rot / 8 + 1];
            const float cs[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w}, sn[8] = {z.x, z.y, z.z, z.w, w.x, w.y, w.z, w.w};
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                c[i] = cs[i];
                s[i] = second ? sn[i] : -sn[i];
            }
        }
        if (!in && !zero) {
#pragma unroll
            for (int i = 0; i < 8; ++i) c[i] = s[i] = __uint_as_float(0x7FC00000u);
        }
    }
};

// A token's weights times its angles: y = r (x u + partner v).  Where the lane's columns are not rotated, partners are 0, u is
// the weight and v -0, so that y is r x u, a zero's sign with it.
template <bool IL, typename T>
__device__ __forceinline__ void factors(const NormRope &a, const void *w, const Turn<IL> &t, T (&u)[8], T (&v)[8]) {
    float own[8], other[8];
    const int half = a.rot / 2;
    weights_at(a, w, t.live ? t.col : 0, own);
    if constexpr (IL) {
#pragma unroll
        for (int i = 0; i < 8; ++i) other[i] = own[i ^ 1];
    } else {
        weights_at(a, w, t.col >= a.rot ? 0 : t.col < half ? t.col + half : t.col - half, other);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {  // (columns past the rotated ones: c = 1; past the row's: x = 0)
        u[i] = (T)own[i] * (T)t.c[i];
        v[i] = t.mask ? (T)other[i] * (T)t.s[i] : (T)-0.0f;
    }
}

// 1 / sqrt(mean(x^2) + eps) of the lane group's row.
template <int L>
__device__ __forceinline__ double row_scale64(const NormRope &a, const float (&x)[8]) {
    double ss = 0.0;
#pragma unroll
    for (int i = 0; i < 8; ++i) ss = __builtin_fma((double)x[i], (double)x[i], ss);
    return rsqrt64(__builtin_fma(group_sum<L>(ss), a.inv_d, (double)a.eps));
}
// The same in fp32; false where the row's squares may have left fp32's range.
template <int L>
__device__ __forceinline__ bool row_scale32(const NormRope &a, const float (&x)[8], float &r) {
    float ss = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) ss = __builtin_fmaf(x[i], x[i], ss);
    const float v = __builtin_fmaf(group_sum<L>(ss), (float)a.inv_d, a.eps);
    r = __builtin_amdgcn_rsqf(v);
    return v >= 0x1p-80f && v <= 0x1p120f;
}

template <int DT, int L, bool IL>
__device__ __forceinline__ void turn_row(const NormRope &a, const Raw<DT> &raw, const Turn<IL> &t, const double (&u)[8],
                                         const double (&v)[8], float (&y)[8]) {
    float x[8], p[8];
    values<DT>(raw, x);
    partners<DT, IL>(raw, t.from, t.mask, p);
    const double r = a.norm ? row_scale64<L>(a, x) : 1.0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float f = (float)(r * __builtin_fma((double)p[i], v[i], (double)x[i] * u[i]));
        y[i] = t.zero ? 0.0f : f;
    }
}
template <int DT, int L, bool IL>
__device__ __forceinline__ void turn_row(const NormRope &a, const Raw<DT> &raw, const Turn<IL> &t, const float (&u)[8],
                                         const float (&v)[8], float (&y)[8]) {
    float x[8], p[8];
    values<DT>(raw, x);
    partners<DT, IL>(raw, t.from, t.mask, p);
    float r = 1.0f;
    const bool fits = !a.norm || row_scale32<L>(a, x, r);
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = r * __builtin_fmaf(p[i], v[i], x[i] * u[i]);
    if (__builtin_amdgcn_ballot_w64(!fits) != 0) {  // the other rows of the wave keep what they have
        const double rd = row_scale64<L>(a, x);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float f = (float)(rd * __builtin_fma((double)p[i], (double)v[i], (double)x[i] * (double)u[i]));
            y[i] = fits ? y[i] : f;
        }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = t.zero ? 0.0f : y[i];
}

struct FwdArgs {
    NormRope a;
    void *qo, *ko;
    int qc, kc;           // runs of query heads and of key heads
};

}  // namespace

// HP: heads of a run, all of whose loads are on their way before the first is used.
template <int DT, int L, bool IL, int HP>
__global__ __launch_bounds__(256) void k_norm_rope(FwdArgs f) {
    const NormRope &a = f.a;
    const int lane = threadIdx.x % L;
    const uint32_t id = workgroup(), runs = f.qc + f.kc;
    int run = (int)(id % runs);
    const int64_t t = (int64_t)(id / runs) * (256 / L) + threadIdx.x / L;
    const int64_t tc = min(t, a.n - 1);  // lanes past the last token stay for the exchanges, with its data
    const bool isq = run < f.qc;
    const HeadRows in = isq ? a.q : a.k;
    void *out = isq ? f.qo : f.ko;
    run = isq ? run : run - f.qc;
    const int h0 = run * HP, h1 = min(h0 + HP, in.heads);
    const int64_t row = tc * in.ts + lane * 8;
    Raw<DT> raw[HP];
#pragma unroll
    for (int j = 0; j < HP; ++j) raw[j] = load_raw<DT>(in.x, row + min(h0 + j, h1 - 1) * in.hs, lane * 8 < a.d);
    const Turn<IL> turn(a, tc, lane, L);
    auto rows = [&](auto zero) {
        decltype(zero) u[8], v[8];
        factors<IL>(a, in.w, turn, u, v);
#pragma unroll
        for (int j = 0; j < HP; ++j) {
            if (h0 + j >= h1) break;
            float y[8];
            turn_row<DT, L, IL>(a, raw[j], turn, u, v, y);
            if (turn.live && t < a.n) store_row<DT, (HP > 1)>(out, (t * in.heads + h0 + j) * a.d + turn.col, y);
        }
    };
    if (isq) rows(0.0f);
    else rows(0.0);
}

namespace {

struct FillArgs {
    NormRope a;
    HeadRows v;
    void *qo;
    uint8_t *cache;
    Kv4Geom g;
    const void *slots;
    bool slots64;
    int qc, kc;
};

}  // namespace

// Queries as above; a key/value head's rows of a token go into the cache as k_kv4_write puts them there.
template <int DT, int D, bool IL, int HP>
__global__ __launch_bounds__(256) void k_norm_rope_kv4(FillArgs f) {
    constexpr int L = D / 8;
    const NormRope &a = f.a;
    const int lane = threadIdx.x % L;
    const uint32_t id = workgroup(), runs = f.qc + f.kc;
    int run = (int)(id % runs);
    const int64_t t = (int64_t)(id / runs) * (256 / L) + threadIdx.x / L;
    const int64_t tc = min(t, a.n - 1);
    const bool isq = run < f.qc;
    const HeadRows in = isq ? a.q : a.k;
    run = isq ? run : run - f.qc;
    const int h0 = run * HP, h1 = min(h0 + HP, in.heads);
    const int64_t row = tc * in.ts + lane * 8, vrow = tc * f.v.ts + lane * 8;
    Raw<DT> raw[HP], vraw[HP];
#pragma unroll
    for (int j = 0; j < HP; ++j) raw[j] = load_raw<DT>(in.x, row + min(h0 + j, h1 - 1) * in.hs, true);
    if (!isq) {
#pragma unroll
        for (int j = 0; j < HP; ++j) vraw[j] = load_raw<DT>(f.v.x, vrow + min(h0 + j, h1 - 1) * f.v.hs, true);
    }
    const Turn<IL> turn(a, tc, lane, L);
    if (isq) {
        float u[8], v[8];
        factors<IL>(a, in.w, turn, u, v);
#pragma unroll
        for (int j = 0; j < HP; ++j) {
            if (h0 + j >= h1) break;
            float y[8];
            turn_row<DT, L, IL>(a, raw[j], turn, u, v, y);
            if (t < a.n) store_row<DT, (HP > 1)>(f.qo, (t * in.heads + h0 + j) * D + turn.col, y);
        }
        return;
    }
    const int64_t slot = f.slots64 ? static_cast<const int64_t *>(f.slots)[tc] : static_cast<const int32_t *>(f.slots)[tc];
    const bool ok = t < a.n && slot >= 0 && slot < f.g.pages << f.g.page_log2;
    const int P = 1 << f.g.page_log2, tok = ok ? (int)(slot & (P - 1)) : 0;
    double u[8], v[8];
    factors<IL>(a, in.w, turn, u, v);
#pragma unroll
    for (int j = 0; j < HP; ++j) {
        const int h = h0 + j;
        if (h >= h1) break;
        float y[8], z[8];
        turn_row<DT, L, IL>(a, raw[j], turn, u, v, y);
        values<DT>(vraw[j], z);
        if constexpr (DT == DT_BF16) {  // the key as the norm's own output holds it
#pragma unroll
            for (int i = 0; i < 8; i += 2) {
                const uint32_t b = bf16_pack2(y[i], y[i + 1]);
                y[i] = __uint_as_float(b << 16);
                y[i + 1] = __uint_as_float(b & 0xFFFF0000u);
            }
        }
        uint32_t mk = amax8(y), mv = amax8(z);
#pragma unroll
        for (int off = 2; off > 0; off >>= 1) {
            mk = max(mk, (uint32_t)__shfl_xor((int)mk, off, 64));
            mv = max(mv, (uint32_t)__shfl_xor((int)mv, off, 64));
        }
        const uint64_t bad_all = __builtin_amdgcn_ballot_w64(max(mk, mv) >= 0x7F800000u);
        const bool bad = ((bad_all >> ((threadIdx.x & 63) / L * L)) & ((1ull << L) - 1)) != 0;
        const uint32_t ek = min(e8m0_of(mk, 2), 252u), ev = min(e8m0_of(mv, 2), 252u);
        const float fk = e8m0_inv(ek), fv = e8m0_inv(ev);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            y[i] *= fk;
            z[i] *= fv;
        }
        if (!ok) continue;
        uint8_t *base = f.cache + ((slot >> f.g.page_log2) * f.g.hkv + h) * f.g.region();
        *reinterpret_cast<uint32_t *>(base + tok * (D / 2) + lane * 4) = bad ? 0u : e2m1_pack8(y);
        *reinterpret_cast<uint32_t *>(base + f.g.v_off() + ((tok >> 3) * L + lane) * 32 + (tok & 7) * 4) = bad ? 0u : e2m1_pack8(z);
        if ((lane & 3) == 0) {
            base[f.g.ks_off() + (lane >> 2) * P + tok] = (uint8_t)(bad ? 255u : ek);
            base[f.g.vs_off() + (lane >> 2) * P + tok] = (uint8_t)(bad ? 0u : ev);
        }
    }
}

namespace {

struct BwdArgs {
    NormRope a;
    RopeGrads g;
    int qc, kc;        // as above
    int qb, kb;        // workgroups of queries and of keys
    float *part;       // a row of d sums each, or NULL
};

}  // namespace

template <int DT, int L, bool IL, int HP>
__global__ __launch_bounds__(256) void k_norm_rope_bwd(BwdArgs f) {
    const NormRope &a = f.a;
    const int lane = threadIdx.x % L;
    const bool isq = (int)blockIdx.x < f.qb;
    const HeadRows in = isq ? a.q : a.k, dy = isq ? f.g.dq : f.g.dk;
    void *dx = isq ? f.g.dxq : f.g.dxk;
    const int64_t dx_ts = isq ? f.g.dxq_ts : f.g.dxk_ts, dx_hs = isq ? f.g.dxq_hs : f.g.dxk_hs;
    const int runs = isq ? f.qc : f.kc, blocks = isq ? f.qb : f.kb, me = isq ? blockIdx.x : blockIdx.x - f.qb;
    const int64_t items = (a.n + 256 / L - 1) / (256 / L) * runs;
    float dw[8] = {0, 0, 0, 0, 0, 0, 0, 0}, w[8];
    weights_at(a, in.w, lane * 8 < a.d ? lane * 8 : 0, w);
    for (int64_t item = me; item < items; item += blocks) {
        const int64_t t = item / runs * (256 / L) + threadIdx.x / L, tc = min(t, a.n - 1);
        const int h0 = (int)(item % runs) * HP, h1 = min(h0 + HP, in.heads);
        const int64_t xr = tc * in.ts + lane * 8, yr = tc * dy.ts + lane * 8;
        Raw<DT> xw[HP], yw[HP];
#pragma unroll
        for (int j = 0; j < HP; ++j) {
            const int h = min(h0 + j, h1 - 1);
            xw[j] = load_raw<DT>(in.x, xr + h * in.hs, lane * 8 < a.d);
            yw[j] = load_raw<DT>(dy.x, yr + h * dy.hs, lane * 8 < a.d);
        }
        const Turn<IL> turn(a, tc, lane, L);
        const bool off = turn.zero || t >= a.n;
#pragma unroll
        for (int j = 0; j < HP; ++j) {
            if (h0 + j >= h1) break;
            float x[8], y[8], p[8], g[8];
            values<DT>(xw[j], x);
            values<DT>(yw[j], y);
            partners<DT, IL>(yw[j], turn.from, turn.mask, p);
#pragma unroll
            for (int i = 0; i < 8; ++i) g[i] = __builtin_fmaf(-turn.s[i], p[i], y[i] * turn.c[i]);
            if (a.norm) {
                float r, dot = 0.0f;
                const bool fits = row_scale32<L>(a, x, r);
                if (__builtin_amdgcn_ballot_w64(!fits) != 0) {
                    const double rd = row_scale64<L>(a, x);
#pragma unroll
                    for (int i = 0; i < 8; ++i) x[i] = fits ? x[i] * r : (float)(x[i] * rd);
                    r = fits ? r : (float)rd;
                } else {
#pragma unroll
                    for (int i = 0; i < 8; ++i) x[i] *= r;
                }
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float e = off ? 0.0f : g[i] * x[i];
                    dw[i] += e;
                    g[i] *= w[i];
                    dot = __builtin_fmaf(g[i], x[i], dot);
                }
                dot = group_sum<L>(dot) * (float)a.inv_d;
#pragma unroll
                for (int i = 0; i < 8; ++i) g[i] = r * __builtin_fmaf(-x[i], dot, g[i]);
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) g[i] = off ? 0.0f : g[i];
            if (turn.live && t < a.n) store_row<DT, (HP > 1)>(dx, t * dx_ts + (h0 + j) * dx_hs + turn.col, g);
        }
    }
    if (!f.part) return;
    // the lane groups' sums in order: those of a wave by exchanges, then the waves'
    __shared__ float sums[4][L * 8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int off = L; off < 64; off <<= 1) dw[i] += __shfl_xor(dw[i], off, 64);
    if ((threadIdx.x & 63) < L) {
#pragma unroll
        for (int i = 0; i < 8; ++i) sums[threadIdx.x >> 6][lane * 8 + i] = dw[i];
    }
    __syncthreads();
    if ((int)threadIdx.x < a.d)
        f.part[(int64_t)blockIdx.x * a.d + threadIdx.x] =
            (sums[0][threadIdx.x] + sums[1][threadIdx.x]) + (sums[2][threadIdx.x] + sums[3][threadIdx.x]);
}

// Partial weight gradients (rows of d) to their sums: 64 rows at once for 16 columns, then the 64 in order.
__global__ __launch_bounds__(1024) void k_rope_dw(const float *__restrict__ part, int qb, int kb, int d, float *dwq, float *dwk) {
    const bool isq = blockIdx.y == 0;
    float *out = isq ? dwq : dwk;
    if (!out) return;
    const int first = isq ? 0 : qb, rows = isq ? qb : kb;
    const int col = blockIdx.x * 16 + threadIdx.x % 16, r = threadIdx.x / 16;
    float s = 0.0f;
    if (col < d) {
#pragma unroll 8
        for (int i = r; i < rows; i += 64) s += part[(int64_t)(first + i) * d + col];
    }
    __shared__ float sums[64][17];
    sums[r][threadIdx.x % 16] = s;
    __syncthreads();
    if (r == 0 && col < d) {
        s = 0.0f;
#pragma unroll
        for (int i = 0; i < 64; ++i) s += sums[i][threadIdx.x];
        out[col] = s;
    }
}

// cos and sin of (pos / factor) * base^(-2 i / rot), in 64 bits, rounded once.
__global__ __launch_bounds__(256) void k_rope_table(float *__restrict__ table, int64_t max_pos, int rot, double base, double factor) {
    const int64_t id = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const int half = rot / 2;
    if (id >= max_pos * half) return;
    const int64_t pos = id / half;
    const int i = (int)(id % half);
    double s, c;
    sincos((double)pos / factor * pow(base, -2.0 * i / rot), &s, &c);
    table[pos * rot + i] = (float)c;
    table[pos * rot + half + i] = (float)s;
}

hipError_t launch_rope_table(float *table, int64_t max_pos, int rot, double base, double factor, hipStream_t s) {
    hipLaunchKernelGGL(k_rope_table, dim3((unsigned)((max_pos * (rot / 2) + 255) / 256)), dim3(256), 0, s, table, max_pos, rot,
                       base, factor);
    return hipGetLastError();
}

namespace {

int lanes_of(int d) { return d <= 32 ? 4 : d <= 64 ? 8 : d <= 128 ? 16 : 32; }

// One head a run where `most` would leave fewer than 1024 workgroups.
int heads_a_run(int64_t n, int d, int heads, int most) {
    const int64_t blocks = (n + 256 / lanes_of(d) - 1) / (256 / lanes_of(d));
    return blocks * heads >= 1024 * most ? most : 1;
}

}  // namespace

#define ROPE_L(KERNEL, DT, IL, HP, ...)                                                                  \
    switch (lanes_of(a.d)) {                                                                             \
        case 4: hipLaunchKernelGGL((KERNEL<DT, 4, IL, HP>), grid, dim3(256), 0, s, __VA_ARGS__); break;  \
        case 8: hipLaunchKernelGGL((KERNEL<DT, 8, IL, HP>), grid, dim3(256), 0, s, __VA_ARGS__); break;  \
        case 16: hipLaunchKernelGGL((KERNEL<DT, 16, IL, HP>), grid, dim3(256), 0, s, __VA_ARGS__); break; \
        default: hipLaunchKernelGGL((KERNEL<DT, 32, IL, HP>), grid, dim3(256), 0, s, __VA_ARGS__);       \
    }
#define ROPE_HP(KERNEL, DT, IL, HP, ...)                            \
    do {                                                            \
        if (hp == 1) { ROPE_L(KERNEL, DT, IL, 1, __VA_ARGS__) }     \
        else { ROPE_L(KERNEL, DT, IL, HP, __VA_ARGS__) }            \
    } while (0)
#define ROPE_DISPATCH(KERNEL, H16, H32, ...)                                                 \
    do {                                                                                     \
        if (a.dt == DT_BF16 && a.interleaved) ROPE_HP(KERNEL, DT_BF16, true, H16, __VA_ARGS__); \
        else if (a.dt == DT_BF16) ROPE_HP(KERNEL, DT_BF16, false, H16, __VA_ARGS__);         \
        else if (a.interleaved) ROPE_HP(KERNEL, DT_F32, true, H32, __VA_ARGS__);             \
        else ROPE_HP(KERNEL, DT_F32, false, H32, __VA_ARGS__);                               \
    } while (0)

hipError_t launch_norm_rope(const NormRope &a, void *qo, void *ko, hipStream_t s) {
    FwdArgs f;
    f.a = a;
    f.qo = qo;
    f.ko = ko;
    const int hp = heads_a_run(a.n, a.d, a.q.heads + a.k.heads, a.dt == DT_BF16 ? FWD16 : FWD32);
    f.qc = (a.q.heads + hp - 1) / hp;
    f.kc = (a.k.heads + hp - 1) / hp;
    const int per = 256 / lanes_of(a.d);
    const dim3 grid = grid_of((a.n + per - 1) / per * (f.qc + f.kc));
    ROPE_DISPATCH(k_norm_rope, FWD16, FWD32, f);
    return hipGetLastError();
}

hipError_t launch_norm_rope_kv4(const NormRope &a, const HeadRows &v, void *qo, uint8_t *cache, const Kv4Geom &g,
                                const void *slots, bool slots64, hipStream_t s) {
    FillArgs f;
    f.a = a;
    f.v = v;
    f.qo = qo;
    f.cache = cache;
    f.g = g;
    f.slots = slots;
    f.slots64 = slots64;
    const int hp = heads_a_run(a.n, a.d, a.q.heads + 2 * a.k.heads, a.dt == DT_BF16 ? FILL16 : FILL32);
    f.qc = (a.q.heads + hp - 1) / hp;
    f.kc = (a.k.heads + hp - 1) / hp;
    const int per = 256 / lanes_of(a.d);
    const dim3 grid = grid_of((a.n + per - 1) / per * (f.qc + f.kc));
#define FILL_HP(DT, D, HP)                                                                                \
    do {                                                                                                  \
        if (a.interleaved) hipLaunchKernelGGL((k_norm_rope_kv4<DT, D, true, HP>), grid, dim3(256), 0, s, f); \
        else hipLaunchKernelGGL((k_norm_rope_kv4<DT, D, false, HP>), grid, dim3(256), 0, s, f);           \
    } while (0)
#define FILL(DT, D, HP)                       \
    do {                                      \
        if (hp == 1) FILL_HP(DT, D, 1);       \
        else FILL_HP(DT, D, HP);              \
    } while (0)
    if (a.dt == DT_BF16 && a.d == 128) FILL(DT_BF16, 128, FILL16);
    else if (a.dt == DT_BF16) FILL(DT_BF16, 64, FILL16);
    else if (a.d == 128) FILL(DT_F32, 128, FILL32);
    else FILL(DT_F32, 64, FILL32);
#undef FILL_HP
#undef FILL
    return hipGetLastError();
}

static void bwd_blocks(const NormRope &a, BwdArgs &f, int hp) {
    f.qc = (a.q.heads + hp - 1) / hp;
    f.kc = (a.k.heads + hp - 1) / hp;
    const int per = 256 / lanes_of(a.d);
    const int64_t tb = (a.n + per - 1) / per, qi = tb * f.qc, ki = tb * f.kc;
    const int64_t all = qi + ki, most = std::min<int64_t>(all, BWD_BLOCKS);
    // shared in proportion to the work, one at least for each tensor
    f.kb = ki ? (int)std::max<int64_t>(1, std::min(ki, most * ki / all)) : 0;
    f.qb = (int)std::min(qi, std::max<int64_t>(1, most - f.kb));
}

size_t norm_rope_bwd_ws_bytes(int d) { return (size_t)(BWD_BLOCKS + 1) * d * 4; }

hipError_t launch_norm_rope_bwd(const NormRope &a, const RopeGrads &g, float *ws, hipStream_t s) {
    BwdArgs f;
    f.a = a;
    f.g = g;
    f.part = a.norm && (g.dwq || g.dwk) ? ws : nullptr;
    const int hp = heads_a_run(a.n, a.d, a.q.heads + a.k.heads, a.dt == DT_BF16 ? BWD16 : BWD32);
    bwd_blocks(a, f, hp);
    const dim3 grid((unsigned)(f.qb + f.kb));
    ROPE_DISPATCH(k_norm_rope_bwd, BWD16, BWD32, f);
    hipError_t e = hipGetLastError();
    if (f.part && e == hipSuccess) {
        hipLaunchKernelGGL(k_rope_dw, dim3((unsigned)((a.d + 15) / 16), 2), dim3(1024), 0, s, ws, f.qb, f.kb, a.d, g.dwq, g.dwk);
        e = hipGetLastError();
    }
    return e;
}

}  // namespace fp4
