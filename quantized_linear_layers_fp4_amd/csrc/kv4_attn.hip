// Attention of packed queries over the 4-bit paged cache (layout: kv4.h).
//
//      s = scale * q . k   over the visible tokens: j <= p, and if there is a window j > p - window or j < sinks
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
// bf16; P is rounded to bf16 (2^-8 of each term, as the output itself is), the sum of P is taken
// before that rounding.
#include <algorithm>
#include <type_traits>

#include "block8.h"
#include "kv4.h"

namespace fp4 {

typedef float v16f __attribute__((ext_vector_type(16)));
typedef __bf16 v2bf __attribute__((ext_vector_type(2)));

namespace {

constexpr int TT = 32;       // tokens a wave takes at once
constexpr int CT = 64;       // tokens a workgroup of the many-rows kernel takes at once
constexpr int FEW = 32;      // rows a (sequence, head) up to which the decode kernel takes them
constexpr float LN2 = 0.69314718055994530942f;
constexpr float LOG2E = 1.44269504088896340736f;

// What a kernel's tokens are.
//   PLAIN   a sequence's, or those of its window
//   SINKS   those of its window and the first a.sinks ones: tokens are counted along an axis that leaves out those
//           between (Span::turn, gap), so the tiles, splits and joins are those of PLAIN
//   PREFIX  the first a.shared pages of row 0 of the table, for the queries of all sequences at once: rows are those of one
//           long sequence, and more rows a tile read the bytes once
//   OWN     a sequence's after those
//   WHOLE   PLAIN's, their first a.shared pages looked up in row 0: where sharing their bytes would cost more than it saves
// PREFIX leaves partial results; OWN takes them in itself, or, where its own tokens are split too or PREFIX's splits are many,
// leaves partial results as well, and the join brings both together.
enum : int { PLAIN, SINKS, PREFIX, OWN, WHOLE };

struct DecArgs {
    Kv4Attn a;
    int g, rt;        // heads a group; row tiles a (sequence, head)
    int tr;           // rows of a tile: 16, or 128 or 256 (the many-rows kernel, 32 a wave)
    int pr;           // rows a partial result holds: min(tr, max_q * g)
    int nw;           // waves of a workgroup
    int splits;       // workgroups along the tokens
    int chunk;        // tokens each takes (a multiple of the unit, nw * TT or CT)
    int work, blanks; // workgroups that attend; those after them, for the queries of no row tile
    float c;          // scale * log2(e)
    float *part;      // partial results
    // of OWN: PREFIX's tile rows, rows a partial holds, splits and partial results
    int ptr_, ppr, psplits;
    const float *ppart;
    bool takes;       // it takes PREFIX's results in itself: it has one split, and they are few for a wave
};

// Entry i of a table that no kernel here writes: a scalar load where i is uniform, though other code of the kernel
// stores first (as vector loads: 77 instead of 69 us for 64 sequences to 8192 tokens).
__device__ __forceinline__ int fixed(const int32_t *p, int64_t i) {
    return ((const __attribute__((address_space(4))) int32_t *)p)[i];
}

// What one workgroup's rows see: rows of sequence `seq`, tile rt.
struct Span {
    int len, qlen, qbeg;
    int rows;         // qlen * g
    int lo, hi;       // tokens any of the tile's rows sees: [lo, hi), lo a multiple of TT
    int full_lo, full_hi;  // tokens that all of its rows see
    // SINKS: token t of the axis stands for t, or from `turn` on (a multiple of CT) for t + gap; the window's tokens
    int turn, gap, wlo, whi;
};

// The first token that a query at position p sees (0 for p below 0, which sees none); no difference here leaves the
// integers, whatever the window.
__device__ __forceinline__ int first_seen(int window, int p) { return window && p >= window ? p - window + 1 : 0; }

// The query at offset entry i, inside the queries whatever the entry says.
__device__ __forceinline__ int query_at(const Kv4Attn &a, int i) { return min(max(fixed(a.q_start, i), 0), a.nq); }

// The tokens that all rows share.
__device__ __forceinline__ int prefix_of(const Kv4Attn &a) { return a.shared << a.geo.page_log2; }

template <int MODE>
__device__ __forceinline__ Span span_of(const Kv4Attn &a, int g, int seq, int row0, int nrows) {
    Span s;
    if constexpr (MODE == PREFIX) {
        s.len = s.hi = s.full_hi = prefix_of(a);
        s.qbeg = s.lo = s.full_lo = 0;
        s.qlen = a.nq;
        s.rows = a.nq * g;
        return s;
    }
    s.len = max(fixed(a.lens, seq), 0);
    s.qbeg = a.q_start ? query_at(a, seq) : seq;
    s.qlen = a.q_start ? query_at(a, seq + 1) - s.qbeg : 1;
    s.rows = min(max(s.qlen, 0), a.max_q) * g;
    const int cap = min(s.len, a.width << a.geo.page_log2);
    s.lo = s.hi = s.full_lo = s.full_hi = 0;
    if constexpr (MODE == SINKS) s.turn = s.gap = s.wlo = s.whi = 0;
    if (row0 >= s.rows) return s;
    const int j0 = row0 / g, j1 = min(row0 + nrows - 1, s.rows - 1) / g;
    const int p0 = s.len - s.qlen + j0, p1 = s.len - s.qlen + j1;
    const int lo = (MODE == OWN ? prefix_of(a) : first_seen(a.window, p0)) & ~(TT - 1), hi = max(min(p1 + 1, cap), 0);
    if constexpr (MODE == SINKS) {
        s.wlo = lo;
        s.whi = hi;
        if (hi <= 0) return s;
        const int turn = (int)(((int64_t)min(a.sinks, hi) + CT - 1) & ~(int64_t)(CT - 1));
        if (lo >= hi) {  // the table's row ends before the window: the first tokens alone
            s.hi = min(turn, hi);
        } else if (turn < lo) {
            s.turn = turn;
            s.gap = lo - turn;
            s.hi = turn + hi - lo;
        } else {
            s.hi = hi;
        }
    } else {
        if (lo >= hi) return s;
        s.lo = lo;
        s.hi = hi;
    }
    s.full_lo = MODE == OWN ? prefix_of(a) : first_seen(a.window, p1);
    s.full_hi = min(p0 + 1, cap);
    return s;
}

// A place of the axis as a token.
template <int MODE>
__device__ __forceinline__ int token_at(const Span &s, int t) {
    if constexpr (MODE == SINKS) return t >= s.turn ? t + s.gap : t;
    return t;
}

// The sequence that owns a query, -1 if none does or if it is past the sequence's first max_q.
__device__ __forceinline__ int owner_of(const Kv4Attn &a, int query) {
    if (!a.q_start) return query;
    int lo = 0, hi = a.b + 1;  // the number of offsets up to `query`
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (a.q_start[mid] <= query) lo = mid + 1;
        else hi = mid;
    }
    if (lo == 0 || lo > a.b || query - query_at(a, lo - 1) >= a.max_q) return -1;
    return lo - 1;
}

// PREFIX's partial result of a row of the call's, for OWN and the join: column c of split s is sums[s * split + (c / 8) *
// eight + c % 8], and the maximum and sum ml[s * split].  The decode kernel leaves a row's d columns side by side (eight = 8); the
// many-rows kernel eight columns of 32 rows, which is 1 KB of a wave's store instruction (row by row it wrote pieces of 32
// bytes: 53 against 49 us for 256 rows a head over 32768 tokens).
struct PrefixRow {
    const float *sums, *ml;
    int64_t split;
    int eight;
};
__device__ __forceinline__ PrefixRow prefix_row(const DecArgs &p, int head, int64_t row) {
    const int d = p.a.geo.d, r = (int)(row % p.ptr_);
    const float *block = p.ppart + (row / p.ptr_ * p.a.geo.hkv + head) * p.psplits * p.ppr * (d + 4);
    PrefixRow x;
    x.split = (int64_t)p.ppr * (d + 4);
    x.eight = p.ptr_ > 16 ? 256 : 8;
    if (p.ptr_ > 16) {
        block += (r >> 5) * 32 * (d + 4);
        x.sums = block + (r & 31) * 8;
        x.ml = block + 32 * d + (r & 31) * 2;
    } else {
        x.sums = block + r * (d + 4);
        x.ml = x.sums + d;
    }
    return x;
}

// PREFIX: whether some sequence has queries that do not see all shared tokens (all threads of the workgroup call it).
__device__ __forceinline__ bool some_short(const Kv4Attn &a, int threads) {
    bool s = false;
    for (int i = threadIdx.x; i < a.b; i += threads) {
        const int ql = a.q_start ? query_at(a, i + 1) - query_at(a, i) : 1;
        s = s || (ql > 0 && (int64_t)max(a.lens[i], 0) - ql + 1 < prefix_of(a));
    }
    return __syncthreads_or(s) != 0;
}

// PREFIX: the number of shared tokens that a row sees, `row` one of the call's.
__device__ __forceinline__ int prefix_seen(const Kv4Attn &a, int g, int row) {
    const int query = row / g, seq = owner_of(a, query);
    if (seq < 0) return prefix_of(a);  // of a row that nothing is made of
    const int beg = a.q_start ? query_at(a, seq) : query, ql = a.q_start ? query_at(a, seq + 1) - beg : 1;
    return (int)min(max((int64_t)max(a.lens[seq], 0) - ql + (query - beg) + 1, (int64_t)0), (int64_t)prefix_of(a));
}

// Queries that no sequence's row tiles cover get zeros and lse = -inf: those past a sequence's first max_q, before
// q_start[0] and from q_start[b] on (a padded batch).  Workgroups of their own at the grid's end do it, `id` the
// sequence's and every p.blanks-th of the others.
__device__ __forceinline__ void blank_rows(const DecArgs &p, int id, int threads) {
    const Kv4Attn &a = p.a;
    auto blank = [&](int from, int to, int step) {
        for (int64_t i = from; i < to; i += step) {
            u32x4 *o = reinterpret_cast<u32x4 *>(a.o + i * a.hq * a.geo.d);
            for (int j = threadIdx.x; j < a.hq * a.geo.d / 8; j += threads) o[j] = u32x4{0, 0, 0, 0};
            if (a.lse)
                for (int j = threadIdx.x; j < a.hq; j += threads) a.lse[i * a.hq + j] = -INFINITY;
        }
    };
    const int first = query_at(a, 0), end = query_at(a, a.b);
    if (id < first) blank(id, first, p.blanks);
    if (id < a.nq - end) blank(end + id, a.nq, p.blanks);
    if (id < a.b && query_at(a, id + 1) - query_at(a, id) > a.max_q) blank(query_at(a, id) + a.max_q, query_at(a, id + 1), 1);
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

// The largest of three, NaN if one is: one instruction, where fmaxf would first quiet each operand.  A NaN
// score that a row sees makes the row NaN in any case.
__device__ __forceinline__ float max3(float a, float b, float c) {
    return __builtin_elementwise_maximum(__builtin_elementwise_maximum(a, b), c);
}
// Largest over the four lanes n, n + 16, n + 32, n + 48, in each of them.
__device__ __forceinline__ float half_max(float x) {
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ __forceinline__ float quarter_max(float x) {
    const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return half_max(fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1])));
}

}  // namespace

// Few rows (single tokens, drafts): 16 rows of one (sequence, key/value head) a workgroup, its NW
// waves taking tiles of 32 tokens in turn and joining in LDS; `splits` workgroups share the tokens.
// Bound by the cache's bytes.
// ONE: a tile lies in one page (of 32 tokens or more), so its addresses are a scalar base and constants of the
// lane: about 45 of 270 vector instructions a tile.
template <int D, int NW, bool ONE, int MODE>
__global__ __launch_bounds__(64 * NW, NW == 4 ? 3 : 1) void k_kv4_decode(DecArgs p) {
    constexpr int J = D / 16;   // columns a lane owns in the O^T tiles: J n + j
    constexpr int KS = D / 32;  // contraction steps of the scores
    const Kv4Attn &a = p.a;
    const int lane = threadIdx.x & 63, n = lane & 15, h = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    // heads first, splits last: consecutive workgroups go to different XCDs, and with splits first each of
    // eight XCDs would have one split of every sequence, the far ones mostly empty (85 against 62 us for 64
    // sequences of unlike lengths); so the empty ones also come at the end
    int id = blockIdx.x;
    if (id >= p.work) return blank_rows(p, id - p.work, 64 * NW);
    const int head = id % a.geo.hkv; id /= a.geo.hkv;
    const int rt = id % p.rt; id /= p.rt;
    const int seq = MODE == PREFIX ? 0 : id % a.b, split = MODE == PREFIX ? id : id / a.b;
    const int row0 = rt * 16;
    Span sp = span_of<MODE>(a, p.g, seq, row0, 16);
    if (row0 >= sp.rows) return;
    const int beg = sp.lo + split * p.chunk, end = min(sp.hi, beg + p.chunk);
    if ((MODE == OWN ? !p.takes : p.splits > 1 || MODE == PREFIX) && beg >= end) return;  // the join counts the splits the same way

    // this lane's row
    const int row = row0 + n;
    const bool live = row < sp.rows;
    const int qi = live ? row / p.g : 0, qh = live ? head * p.g + row % p.g : 0;
    const int pos = sp.len - sp.qlen + qi;
    int vhi = live ? (MODE == PREFIX ? sp.len : pos + 1) : 0;
    const int vlo = MODE == OWN ? prefix_of(a) : first_seen(a.window, pos);
    if constexpr (MODE == PREFIX) {
        if (some_short(a, 64 * NW)) {
            vhi = live ? prefix_seen(a, p.g, row) : 0;
            sp.full_hi = 0;
        }
    }
    // the first token that nobody sees: of the window where the axis has two parts
    const int stop = MODE == SINKS ? sp.whi : end;
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

    const int lg = a.geo.page_log2, P = 1 << lg;
    const int64_t region = a.geo.region();
    const int32_t *table = a.pages + (int64_t)seq * a.page_rs;
    v4f acc[J];
#pragma unroll
    for (int j = 0; j < J; ++j) acc[j] = v4f{0, 0, 0, 0};
    float m = -INFINITY, l = 0.0f;

    // A lane's part of a tile of 32 tokens.  Tokens of the scores' row n in half s: 8 (n / 4) + 4 s +
    // n % 4; of V's step: 8 h + 0..7.  Nothing is masked here: the page index is clamped into the
    // table's row and into the cache, whose bytes are finite numbers wherever a score is masked away.
    struct Tile {
        uint32_t kw[2][KS], vw[8];
        uint32_t ks[2];
        uint2 vs;
        bool okk;  // the page is one of the cache's (K's lane; V's tokens are the same pages)
    };
    auto page_at = [&](int t) {
        const int c = min(t, stop - 1) >> lg;
        return fixed(MODE == WHOLE && c < a.shared ? a.pages : table, c);
    };
    auto fetch = [&](int at, int pk, int pv, Tile &x) {
        const int t0 = token_at<MODE>(sp, at);
        x.okk = (uint32_t)pk < (uint64_t)a.geo.pages;
        const bool okv = (uint32_t)pv < (uint64_t)a.geo.pages;
        // codes' and scales' bases of K and of V; then a lane's token in them
        const int64_t pk0 = x.okk ? pk : 0, pv0 = okv ? pv : 0;
        const int in = ONE ? t0 & (P - 1) : 0;
        const uint8_t *kc = a.cache + (pk0 * a.geo.hkv + head) * region + in * (D / 2), *ks = kc + a.geo.ks_off() + in - in * (D / 2);
        const uint8_t *vc = a.cache + (pv0 * a.geo.hkv + head) * region + a.geo.v_off() + in * (D / 2);
        const uint8_t *vs = vc + P * (D / 2) + in - in * (D / 2);
        const int tk = (ONE ? 8 * (n >> 2) : (t0 + 8 * (n >> 2)) & (P - 1)) + (n & 3), tv = ONE ? 8 * h : (t0 + 8 * h) & (P - 1);
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            const int tok = tk + 4 * s;
            if constexpr (D == 128) {
                const u32x4 w = *reinterpret_cast<const u32x4 *>(kc + (uint32_t)(tok * (D / 2) + h * (D / 8)));
#pragma unroll
                for (int i = 0; i < 4; ++i) x.kw[s][i] = w[i];
            } else {
                const uint2 w = *reinterpret_cast<const uint2 *>(kc + (uint32_t)(tok * (D / 2) + h * (D / 8)));
                x.kw[s][0] = w.x;
                x.kw[s][1] = w.y;
            }
            x.ks[s] = ks[(uint32_t)((h * D / 128) * P + tok)];
        }
        const int dw = D == 128 ? n : n >> 1;
        const u32x4 *src = reinterpret_cast<const u32x4 *>(vc + (uint32_t)(((tv >> 3) * (D / 8) + dw) * 32));
        const u32x4 y0 = src[0], y1 = src[1];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x.vw[i] = y0[i];
            x.vw[4 + i] = y1[i];
        }
        x.vs = *reinterpret_cast<const uint2 *>(vs + (uint32_t)((n * J / 32) * P + tv));
    };

    // two tiles of loads in flight: the next tile's bytes and the page indices of the one after it
    const int first = beg + wave * TT;
    Tile even, odd;
    int pk = 0, pv = 0;
    auto pages_of = [&](int at) {
        const int t0 = token_at<MODE>(sp, at);
        pk = page_at(ONE ? t0 : t0 + 8 * (n >> 2));
        pv = ONE ? pk : page_at(t0 + 8 * h);
    };
    auto tile = [&](Tile &cur, Tile &nxt, int at) {
        fetch(at + NW * TT, pk, pv, nxt);
        pages_of(at + 2 * NW * TT);
        const int t0 = token_at<MODE>(sp, at);
        if constexpr (D == 64) {
#pragma unroll
            for (int i = 0; i < 8; ++i) cur.vw[i] >>= 16 * (n & 1);
        }
        // scores: element r of half s is token t0 + 8 h + 4 s + r, row n
        float x[8];
        const uint64_t okm = __builtin_amdgcn_ballot_w64(cur.okk);
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            v4f d = v4f{0, 0, 0, 0};
            v8bf kf[KS];
            unpack_row<KS>(cur.kw[s], cur.ks[s], kf);
#pragma unroll
            for (int i = 0; i < KS; ++i) d = __builtin_amdgcn_mfma_f32_16x16x32_bf16(kf[i], qf[i], d, 0, 0, 0);
#pragma unroll
            for (int r = 0; r < 4; ++r) x[4 * s + r] = d[r] * p.c;
        }
        if (okm != ~0ull || (t0 < sp.full_lo && !(MODE == SINKS && t0 + TT <= a.sinks)) ||
            t0 + TT > min(sp.full_hi, stop)) {  // some token is masked
            const bool okp = ((okm >> (4 * h)) & 1) != 0;  // of the lane's score tokens' page
            const int hi = okp ? min(vhi, stop) : 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int tok = t0 + 8 * h + i;
                x[i] = tok < hi && (tok >= vlo || (MODE == SINKS && tok < a.sinks)) ? x[i] : -INFINITY;
            }
        }
        const float mx = fmaxf(m, quarter_max(max3(max3(x[0], x[1], x[2]), max3(x[3], x[4], x[5]), fmaxf(x[6], x[7]))));
        // Rarely, after a row's first tiles.  (Letting factors grow to 2^8 before the maximum moves saved 1 to 3 %
        // and cost a dominant token its exact factor of 1: 0.0021 instead of 0.0017 off in the mean.)
        if (__builtin_amdgcn_ballot_w64(mx != m) != 0) {
            const float alpha = m == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f(m - mx);
            m = mx;
            l *= alpha;
#pragma unroll
            for (int j = 0; j < J; ++j) acc[j] *= alpha;
        }
        const float mu = m == -INFINITY ? 0.0f : m;
        float e[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) e[i] = __builtin_amdgcn_exp2f(x[i] - mu);
        l += ((e[0] + e[1]) + (e[2] + e[3])) + ((e[4] + e[5]) + (e[6] + e[7]));
        const v8bf pb = __builtin_bit_cast(v8bf, u32x4{bf16_pack2(e[0], e[1]), bf16_pack2(e[2], e[3]),
                                                       bf16_pack2(e[4], e[5]), bf16_pack2(e[6], e[7])});
        const uint2 vs = cur.vs;
        const float sc[8] = {scale_of<0>(vs.x), scale_of<1>(vs.x), scale_of<2>(vs.x), scale_of<3>(vs.x),
                             scale_of<0>(vs.y), scale_of<1>(vs.y), scale_of<2>(vs.y), scale_of<3>(vs.y)};
        v8bf c0, c1;
#define PV(B)                                                                                 \
    unpack_cols<B>(cur.vw, sc, c0, c1);                                                       \
    acc[2 * B] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(c0, pb, acc[2 * B], 0, 0, 0);        \
    acc[2 * B + 1] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(c1, pb, acc[2 * B + 1], 0, 0, 0);
        PV(0)
        PV(1)
        if constexpr (D == 128) {
            PV(2)
            PV(3)
        }
#undef PV
    };
    if (first < end) {
        pages_of(first);
        fetch(first, pk, pv, even);
        pages_of(first + NW * TT);
    }
    // OWN: the shared tokens' partial results, by turns of the waves: columns (4 h + r) J .. + J - 1 of the row, as
    // acc holds them
    auto take_prefix = [&] {
        const PrefixRow w = prefix_row(p, head, (int64_t)sp.qbeg * p.g + row);
        if (p.takes && live) {
#pragma unroll 2
            for (int s = wave; s < p.psplits; s += NW) {
                const float *ws = w.sums + s * w.split + (h * J / 2) * w.eight;
                const float2 ml = *reinterpret_cast<const float2 *>(w.ml + s * w.split);
                float4 v[J];
#pragma unroll
                for (int i = 0; i < J; ++i) v[i] = *reinterpret_cast<const float4 *>(ws + (i >> 1) * w.eight + 4 * (i & 1));
                const float nm = fmaxf(m, ml.x), mu = nm == -INFINITY ? 0.0f : nm;
                const float f0 = __builtin_amdgcn_exp2f(m - mu), f1 = __builtin_amdgcn_exp2f(ml.x - mu);
                m = nm;
                l = l * f0 + (h == 0 ? ml.y * f1 : 0.0f);
                // column c of the lane's 4 J: element c / J of tile c % J
#pragma unroll
                for (int i = 0; i < J; ++i) {
                    const float x[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
                    for (int u = 0; u < 4; ++u) {
                        const int c = 4 * i + u;
                        acc[c % J][c / J] = acc[c % J][c / J] * f0 + x[u] * f1;
                    }
                }
            }
        }
    };
    // while the first tile is on its way; the 128 registers of 16 waves have no room for both
    if constexpr (MODE == OWN && NW == 4) take_prefix();
    if constexpr (ONE || NW == 4 || D == 64) {
        for (int t0 = first; t0 < end; t0 += 2 * NW * TT) {
            tile(even, odd, t0);
            if (t0 + NW * TT < end) tile(odd, even, t0 + NW * TT);
        }
    } else {  // the 128 registers of 16 waves do not hold both tiles' addresses (9.2 | 14.8 us at 777 tokens)
        for (int t0 = first; t0 < end; t0 += NW * TT) {
            tile(even, odd, t0);
            even = odd;
        }
    }

    if constexpr (MODE == OWN && NW != 4) take_prefix();

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
        if (MODE == OWN ? p.takes : p.splits == 1 && MODE != PREFIX) {
            const int64_t out = (int64_t)(sp.qbeg + (row0 + r) / p.g) * a.hq + head * p.g + (row0 + r) % p.g;
            const float inv = L == 0.0f ? 0.0f : 1.0f / L;
            *reinterpret_cast<uint2 *>(a.o + out * D + col) =
                make_uint2(bf16_pack2(o[0] * inv, o[1] * inv), bf16_pack2(o[2] * inv, o[3] * inv));
            if (a.lse && col == 0) a.lse[out] = L == 0.0f ? -INFINITY : (M + __builtin_amdgcn_logf(L)) * LN2;
        } else {
            // partial row: D sums, then the maximum and the sum of the split
            float *w = p.part +
                       (((((int64_t)seq * p.rt + rt) * a.geo.hkv + head) * p.splits + split) * p.pr + r) * (D + 4);
            *reinterpret_cast<float4 *>(w + col) = make_float4(o[0], o[1], o[2], o[3]);
            if (col == 0) {
                w[D] = M;
                w[D + 1] = L;
            }
        }
    }
}

// Many rows (chunks of prompts): rows of one (sequence, key/value head), 32 a wave, NT / 2 a workgroup.
// Every tile of 64 tokens is unpacked to bf16 once by the whole workgroup into one of two LDS
// buffers, while the waves multiply the other: with 16 rows a wave, as above, unpacking in registers
// would take more time than the products.  Tokens are rows of K's operand with bits 2 and 3 of their
// index exchanged, so that a lane's eight scores of one V step are eight consecutive tokens.
// Eight waves a CU in either size.  2 x 1024 queries of 32 heads over 8192 tokens (d 128, 8 key/value heads), us:
// 16 rows a wave 700; this with four waves 362, page indices looked up a tile earlier 341, the maximum
// in one instruction for two scores 322; with eight waves, which halves a thread's unpacking, and bytes two
// tiles ahead 305 (short runs; 276 once the clock is up), with scalar pages and addresses 268 (0.96 PFLOP/s).  Of a busy CU's cycles matrix instructions
// take 44 %, vector instructions (the exponentials first) 61 % and LDS 34 %: a deeper interleaving within a wave
// (64 rows, 512 registers) was slower.
template <int D, int NT, int MODE>
__global__ __launch_bounds__(NT, 2) void k_kv4_chunk(DecArgs p) {
    constexpr int CR = NT / 2;        // rows of the workgroup
    constexpr int KC = D / 8;     // 16-byte pieces of a token's K row
    constexpr int KS = D / 16;    // contraction steps of the scores
    constexpr int DT = D / 32;    // tiles of 32 columns
    constexpr int KD = 8 * D / NT;  // dwords of K, and tokens of V, that a thread unpacks
    constexpr int TPT = NT / 64;  // threads a token of K
    static_assert(KD == 2 || KD == 4, "what fetch and unpack know");
    __shared__ __attribute__((aligned(16))) uint8_t sk0[CT * D * 2], sv0[D * CT * 2], sk1[CT * D * 2], sv1[D * CT * 2];
    const Kv4Attn &a = p.a;
    const int tid = threadIdx.x, lane = tid & 63, n = lane & 31, h = lane >> 5;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    int id = blockIdx.x;
    if (id >= p.work) return blank_rows(p, id - p.work, NT);
    const int head = id % a.geo.hkv; id /= a.geo.hkv;
    const int rt = p.rt - 1 - id % p.rt; id /= p.rt;  // the longest first
    const int seq = MODE == PREFIX ? 0 : id % a.b, split = MODE == PREFIX ? id : id / a.b;
    const int row0 = rt * CR;
    const Span sp = span_of<MODE>(a, p.g, seq, row0, CR);
    if (row0 >= sp.rows) return;
    const int beg = sp.lo + split * p.chunk, end = min(sp.hi, beg + p.chunk);
    if ((MODE == OWN ? !p.takes : p.splits > 1 || MODE == PREFIX) && beg >= end) return;  // the join counts the splits the same way
    const int stop = MODE == SINKS ? sp.whi : end;  // the first token that nobody sees

    // this lane's row, and what the wave's rows see
    const int row = row0 + wave * 32 + n;
    const bool live = row < sp.rows;
    const int qi = live ? row / p.g : 0, qh = live ? head * p.g + row % p.g : 0;
    const int pos = sp.len - sp.qlen + qi;
    int vhi = live ? min(MODE == PREFIX ? sp.len : pos + 1, stop) : 0;
    const int vlo = MODE == OWN ? prefix_of(a) : first_seen(a.window, pos);
    Span sw = span_of<MODE>(a, p.g, seq, row0 + wave * 32, 32);
    if constexpr (MODE == PREFIX) {
        if (row0 + wave * 32 >= sp.rows) sw.hi = 0;
        if (some_short(a, NT)) {
            vhi = live ? min(prefix_seen(a, p.g, row), stop) : 0;
            sw.full_hi = 0;
        }
    }
    const bool neg = p.c < 0.0f;  // the maximum is taken before the scale: a negative one goes to q
    // A scale of 0 becomes the smallest float: a masked score, -inf here, stays -inf under it (-inf * 0 would be
    // NaN), and a finite one stays below 2^-21, as good as 0.
    const float c = p.c == 0.0f ? 0x1p-149f : neg ? -p.c : p.c;
    v8bf qf[KS];
#pragma unroll
    for (int i = 0; i < KS; ++i) {
        u32x4 x = {0, 0, 0, 0};
        if (live)
            x = *reinterpret_cast<const ua_u32x4 *>(a.q + (int64_t)(sp.qbeg + qi) * a.q_ts + (int64_t)qh * a.q_hs +
                                                    16 * i + 8 * h);
        if (neg) x ^= 0x80008000u;
        qf[i] = __builtin_bit_cast(v8bf, x);
    }

    // SINKS: tokens vlo .. vlo + vcount - 1 and those below vsinks (three comparisons instead cost 30 registers, a wave)
    const uint32_t vcount = max(vhi - vlo, 0);
    const int vsinks = min(a.sinks, vhi);
    // What a thread unpacks: KD dwords of one token's K (of one group of 32), and eight columns of KD
    // consecutive tokens' V.
    const int lg = a.geo.page_log2, P = 1 << lg;
    const int64_t region = a.geo.region();
    const int32_t *table = a.pages + (int64_t)seq * a.page_rs;
    const int kt = tid / TPT, kq = tid % TPT;
    constexpr int VP = 8 / KD;
    const int vp = tid % VP, vn = tid / VP % (D / 8), vt = tid / VP / (D / 8);
    // A wave's tokens, of K as of V, are WT consecutive ones, so they lie in one page, and page and address are scalars.
    constexpr int WT = 64 * 64 / NT;
    const int wt = wave * WT, ktok = kt - wt, vtok = vt * 8 + vp * KD - wt;
    // the bytes of two tiles on their way: an even tile's in set 0, an odd one's in set 1
    uint32_t kw[2][KD], vw[2][KD], ks[2], vs[2];
    const uint8_t *const headp = a.cache + (int64_t)head * region;
    const int64_t pstride = (int64_t)a.geo.hkv * region;
    auto page_at = [&](int t) {
        const int c = min(t, stop - 1) >> lg;
        return fixed(MODE == WHOLE && c < a.shared ? a.pages : table, c);
    };
    const uint32_t ko = ktok * (D / 2) + kq * (KD * 4), vo = ((vtok >> 3) * (D / 8) + vn) * 32 + (vtok & 7) * 4;
    const uint32_t kso = (kq * KD / 4) * P + ktok, vso = (vn >> 2) * P + vtok;
    // pages outside the cache: their tokens' bytes are any page's, and their scores are masked
    bool okk[2];
    auto fetch = [&](auto set, int at, int pg) {
        constexpr int z = decltype(set)::value;
        okk[z] = (uint32_t)pg < (uint64_t)a.geo.pages;
        const int in = (token_at<MODE>(sp, at) + wt) & (P - 1);  // a multiple of 8
        const uint8_t *base = headp + (okk[z] ? pg : 0) * pstride;
        const uint8_t *ka = base + in * (D / 2), *va = base + a.geo.v_off() + in * (D / 2);
        const uint8_t *ksa = base + a.geo.ks_off() + in, *vsa = base + a.geo.vs_off() + in;
        if constexpr (KD == 4) {
            const u32x4 x = *reinterpret_cast<const u32x4 *>(ka + ko), y = *reinterpret_cast<const u32x4 *>(va + vo);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                kw[z][i] = x[i];
                vw[z][i] = y[i];
            }
            vs[z] = *reinterpret_cast<const uint32_t *>(vsa + vso);
        } else {
            const uint2 x = *reinterpret_cast<const uint2 *>(ka + ko), y = *reinterpret_cast<const uint2 *>(va + vo);
            kw[z][0] = x.x;
            kw[z][1] = x.y;
            vw[z][0] = y.x;
            vw[z][1] = y.y;
            vs[z] = *reinterpret_cast<const uint16_t *>(vsa + vso);
        }
        ks[z] = ksa[kso];
    };
    // K rows: KC pieces, turned so that 16 rows of one piece lie on 16 places; V rows (columns): 8
    // pieces of eight tokens, turned for the reads (32 consecutive columns) and the writes (every eighth)
    auto kpiece = [](int r, int ch) { return D == 128 ? r * 16 + (ch ^ (r & 15)) : r * 8 + (ch ^ ((r >> 1) & 7)); };
    auto vpiece = [](int col, int ch) { return col * 8 + (ch ^ (((col >> 1) ^ (col >> 4)) & 7)); };
    // the reads' places: row n (+ 32 u: a constant further on) at piece 2 i + h, and column n + 32 j at
    // piece 2 k + h, where j turns the piece by 2 j
    int ka[KS], va[4];
#pragma unroll
    for (int i = 0; i < KS; ++i) ka[i] = kpiece(n, 2 * i + h) * 16;
#pragma unroll
    for (int i = 0; i < 4; ++i) va[i] = vpiece(n, 2 * i + h) * 16;
    const int krow = (kt & ~12) | ((kt & 4) << 1) | ((kt & 8) >> 1);
    int kst[KD], vst[8];
#pragma unroll
    for (int i = 0; i < KD; ++i) kst[i] = kpiece(krow, kq * KD + i) * 16;
#pragma unroll
    for (int j = 0; j < 8; ++j) vst[j] = vpiece(vn * 8 + j, vt) * 16 + vp * KD * 2;
    auto unpack = [&](auto set, uint8_t *dk, uint8_t *dv) {
        constexpr int z = decltype(set)::value;
        v8bf kf[KD];
        unpack_row<KD>(kw[z], okk[z] ? ks[z] : 0u, kf);
#pragma unroll
        for (int i = 0; i < KD; ++i) *reinterpret_cast<v8bf *>(dk + kst[i]) = kf[i];
        const float sc[4] = {scale_of<0>(vs[z]), scale_of<1>(vs[z]), scale_of<2>(vs[z]), scale_of<3>(vs[z])};
        uint32_t x[KD][4];
#pragma unroll
        for (int t = 0; t < KD; ++t) {
            x[t][0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(vw[z][t], sc[t], 0));
            x[t][1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(vw[z][t], sc[t], 1));
            x[t][2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(vw[z][t], sc[t], 2));
            x[t][3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(vw[z][t], sc[t], 3));
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const uint32_t sel = j & 1 ? 0x07060302u : 0x05040100u;
            uint8_t *d = dv + vst[j];
            if constexpr (KD == 4)
                *reinterpret_cast<uint2 *>(d) = make_uint2(__builtin_amdgcn_perm(x[1][j >> 1], x[0][j >> 1], sel),
                                                           __builtin_amdgcn_perm(x[3][j >> 1], x[2][j >> 1], sel));
            else
                *reinterpret_cast<uint32_t *>(d) = __builtin_amdgcn_perm(x[1][j >> 1], x[0][j >> 1], sel);
        }
    };

    v16f acc[DT];
#pragma unroll
    for (int j = 0; j < DT; ++j)
#pragma unroll
        for (int r = 0; r < 16; ++r) acc[j][r] = 0.0f;
    float m = -INFINITY, l = 0.0f;  // m: of the unscaled scores

    // whether some page of a tile lies outside the cache, from the waves that unpacked it
    __shared__ uint32_t bad[2][TPT];
    // tile t0 is multiplied while t0 + CT is unpacked, the bytes of the next two are on their way and the page
    // indices of t0 + 4 CT
    using I0 = std::integral_constant<int, 0>;
    using I1 = std::integral_constant<int, 1>;
    int pg = 0;
    auto pages_of = [&](int at) { pg = page_at(token_at<MODE>(sp, at) + wt); };
    if (beg < end) {
        pages_of(beg);
        fetch(I0{}, beg, pg);
        pages_of(beg + CT);
        fetch(I1{}, beg + CT, pg);
        pages_of(beg + 2 * CT);
        if (lane == 0) bad[0][wave] = !okk[0];
        unpack(I0{}, sk0, sv0);
        fetch(I0{}, beg + 2 * CT, pg);
        pages_of(beg + 3 * CT);
    }
    auto tile = [&](auto buf, int at, const uint8_t *ck, const uint8_t *cv, uint8_t *nk, uint8_t *nv) {
        constexpr int b = decltype(buf)::value;
        __syncthreads();  // tile t0 is in buffer b, and nobody reads the other any more
        // the next tile is unpacked whether there is one or not (the fetched bytes are always some page's), so
        // that it lies beside the products, which are matrix instructions
        auto next = [&] {
            using Set = std::integral_constant<int, b ^ 1>;
            if (lane == 0) bad[b ^ 1][wave] = !okk[b ^ 1];
            unpack(Set{}, nk, nv);
            fetch(Set{}, at + 3 * CT, pg);
            pages_of(at + 4 * CT);
        };
        const int t0 = token_at<MODE>(sp, at);
        // (named truth values here cost 20 registers and spills)
        if (t0 >= (MODE == SINKS ? sw.whi : sw.hi) ||
            (t0 + CT <= (MODE == SINKS ? sw.wlo : sw.lo) && (MODE != SINKS || t0 >= a.sinks))) {  // the wave's rows see nothing of it
            next();
            return;
        }
        v16f s[2];
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int r = 0; r < 16; ++r) s[u][r] = 0.0f;
        __builtin_amdgcn_sched_barrier(0);
        next();
#pragma unroll
        for (int i = 0; i < KS; ++i)
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const v8bf kf = *reinterpret_cast<const v8bf *>(ck + ka[i] + u * (64 * D));
                s[u] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(kf, qf[i], s[u], 0, 0, 0);
            }
        __builtin_amdgcn_sched_barrier(0);
        // element r of block u: token t0 + 32 u + 16 (r / 8) + 8 h + r % 8 of row n
        uint32_t any = 0;
#pragma unroll
        for (int w = 0; w < TPT; ++w) any |= bad[b][w];
        const bool anybad = __builtin_amdgcn_readfirstlane((int)any) != 0;
        const bool before = t0 < sw.full_lo && !(MODE == SINKS && t0 + CT <= a.sinks);
        if (anybad || before || t0 + CT > min(sw.full_hi, stop)) {
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int r = 0; r < 16; ++r) {
                    const int q = 32 * u + 16 * (r >> 3) + 8 * h + (r & 7), tok = t0 + q;
                    const bool ok = bad[b][q / WT] == 0;
                    const bool see = MODE == SINKS ? (uint32_t)(tok - vlo) < vcount || tok < vsinks : tok < vhi && tok >= vlo;
                    s[u][r] = ok && see ? s[u][r] : -INFINITY;
                }
        }
        float mx = m;
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int r = 0; r < 16; r += 2) mx = max3(mx, s[u][r], s[u][r + 1]);
        mx = half_max(mx);
        if (__builtin_amdgcn_ballot_w64(mx != m) != 0) {
            const float alpha = m == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f((m - mx) * c);
            m = mx;
            l *= alpha;
#pragma unroll
            for (int j = 0; j < DT; ++j) acc[j] *= alpha;
        }
        const float mu = m == -INFINITY ? 0.0f : m * c;
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            float e[8];
#pragma unroll
            for (int r = 0; r < 8; ++r) e[r] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[k >> 1][8 * (k & 1) + r], c, -mu));
            l += ((e[0] + e[1]) + (e[2] + e[3])) + ((e[4] + e[5]) + (e[6] + e[7]));
            const v8bf pb = __builtin_bit_cast(v8bf, u32x4{bf16_pack2(e[0], e[1]), bf16_pack2(e[2], e[3]),
                                                           bf16_pack2(e[4], e[5]), bf16_pack2(e[6], e[7])});
#pragma unroll
            for (int j = 0; j < DT; ++j) {
                const v8bf vf = *reinterpret_cast<const v8bf *>(cv + va[k ^ j] + j * 4096);
                acc[j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(vf, pb, acc[j], 0, 0, 0);
            }
        }
    };
    for (int t0 = beg; t0 < end; t0 += 2 * CT) {
        tile(I0{}, t0, sk0, sv0, sk1, sv1);
        if (t0 + CT < end) tile(I1{}, t0 + CT, sk1, sv1, sk0, sv0);
    }
    l += __shfl_xor(l, 32, 64);
    if (!live) return;
    float ms = m == -INFINITY ? m : m * c;  // of the scaled scores
    if constexpr (MODE == OWN) {
        const PrefixRow w = prefix_row(p, head, (int64_t)sp.qbeg * p.g + row);
        if (p.takes) {
            for (int s = 0; s < p.psplits; ++s) {
                const float *ws = w.sums + s * w.split + 4 * h;
                const float2 ml = *reinterpret_cast<const float2 *>(w.ml + s * w.split);
                const float nm = fmaxf(ms, ml.x), mu = nm == -INFINITY ? 0.0f : nm;
                const float f0 = __builtin_amdgcn_exp2f(ms - mu), f1 = __builtin_amdgcn_exp2f(ml.x - mu);
                ms = nm;
                l = l * f0 + ml.y * f1;
#pragma unroll
                for (int j = 0; j < DT; ++j)
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const float4 v = *reinterpret_cast<const float4 *>(ws + (4 * j + q) * w.eight);
                        const float x[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                        for (int u = 0; u < 4; ++u) acc[j][4 * q + u] = acc[j][4 * q + u] * f0 + x[u] * f1;
                    }
            }
        }
    }
    // element r of tile j: column 32 j + 8 (r / 4) + 4 h + r % 4 of row n
    if (MODE == OWN ? p.takes : p.splits == 1 && MODE != PREFIX) {
        const int64_t out = (int64_t)(sp.qbeg + qi) * a.hq + qh;
        const float inv = l == 0.0f ? 0.0f : 1.0f / l;
#pragma unroll
        for (int j = 0; j < DT; ++j)
#pragma unroll
            for (int q = 0; q < 4; ++q)
                *reinterpret_cast<uint2 *>(a.o + out * D + 32 * j + 8 * q + 4 * h) =
                    make_uint2(bf16_pack2(acc[j][4 * q] * inv, acc[j][4 * q + 1] * inv),
                               bf16_pack2(acc[j][4 * q + 2] * inv, acc[j][4 * q + 3] * inv));
        if (a.lse && h == 0) a.lse[out] = l == 0.0f ? -INFINITY : (ms + __builtin_amdgcn_logf(l)) * LN2;
    } else {
        float *w = p.part +
                   (((((int64_t)seq * p.rt + rt) * a.geo.hkv + head) * p.splits + split) * p.pr + wave * 32) * (D + 4);
        float *ml = w + (MODE == PREFIX ? 32 * D + n * 2 : n * (D + 4) + D);  // (PREFIX: as PrefixRow says)
        w += MODE == PREFIX ? n * 8 : n * (D + 4);
#pragma unroll
        for (int j = 0; j < DT; ++j)
#pragma unroll
            for (int q = 0; q < 4; ++q)
                *reinterpret_cast<float4 *>(w + (4 * j + q) * (MODE == PREFIX ? 256 : 8) + 4 * h) =
                    make_float4(acc[j][4 * q], acc[j][4 * q + 1], acc[j][4 * q + 2], acc[j][4 * q + 3]);
        if (h == 0) {
            ml[0] = ms;
            ml[1] = l;
        }
    }
}

// Joins the splits of a row: D / 4 lanes to a split's columns, so a workgroup has 8 (D = 128) or 16 lane
// groups; G of them read a row's splits at once (all, or one where there are few splits and many rows).
// Each group sums its splits in ascending order, then the groups are summed in order.
template <int D, int G, int MODE>
__global__ __launch_bounds__(256) void k_kv4_join(DecArgs p) {
    constexpr int L = D / 4, RW = 256 / L / G;  // RW rows a workgroup
    const Kv4Attn &a = p.a;
    const int lane = threadIdx.x % L, grp = threadIdx.x / L % G;
    int64_t id = (int64_t)blockIdx.x * RW + threadIdx.x / L / G;
    const int r = (int)(id % p.pr); id /= p.pr;
    const int head = (int)(id % a.geo.hkv); id /= a.geo.hkv;
    const int rt = (int)(id % p.rt);
    const int seq = (int)(id / p.rt);
    if (seq >= a.b) return;  // (of a workgroup that joins one row, all or none)
    const Span sp = span_of<MODE>(a, p.g, seq, rt * p.tr, p.tr);
    const int row = rt * p.tr + r;
    if (row >= sp.rows) return;
    const int ns = sp.hi > sp.lo ? (sp.hi - sp.lo + p.chunk - 1) / p.chunk : 0;
    const int64_t SS = (int64_t)p.pr * (D + 4);
    const float *w = p.part + ((((int64_t)seq * p.rt + rt) * a.geo.hkv + head) * p.splits * p.pr + r) * (D + 4);
    PrefixRow pw{};  // the shared tokens' partial results of the row
    if constexpr (MODE == OWN) pw = prefix_row(p, head, (int64_t)sp.qbeg * p.g + row);
    float M = -INFINITY, Lsum = 0.0f, o[4] = {0, 0, 0, 0};
    const int parts = MODE == OWN ? ns + p.psplits : ns;
#pragma unroll 4
    for (int s = grp; s < parts; s += G) {
        const bool pre = MODE == OWN && s >= ns;
        const float *ws = pre ? pw.sums + (s - ns) * pw.split + (lane >> 1) * pw.eight + (lane & 1) * 4 : w + s * SS + lane * 4;
        const float4 v = *reinterpret_cast<const float4 *>(ws);
        const float2 ml = *reinterpret_cast<const float2 *>(pre ? pw.ml + (s - ns) * pw.split : w + s * SS + D);
        const float nm = fmaxf(M, ml.x), mu = nm == -INFINITY ? 0.0f : nm;
        const float f0 = __builtin_amdgcn_exp2f(M - mu), f1 = __builtin_amdgcn_exp2f(ml.x - mu);
        M = nm;
        Lsum = Lsum * f0 + ml.y * f1;
        o[0] = o[0] * f0 + v.x * f1;
        o[1] = o[1] * f0 + v.y * f1;
        o[2] = o[2] * f0 + v.z * f1;
        o[3] = o[3] * f0 + v.w * f1;
    }
    if constexpr (G > 1) {
        __shared__ __attribute__((aligned(16))) float so[G][D + 4];
        *reinterpret_cast<float4 *>(&so[grp][lane * 4]) = make_float4(o[0], o[1], o[2], o[3]);
        if (lane == 0) {
            so[grp][D] = M;
            so[grp][D + 1] = Lsum;
        }
        __syncthreads();
        if (grp != 0) return;
#pragma unroll
        for (int i = 1; i < G; ++i) M = fmaxf(M, so[i][D]);
        const float mu = M == -INFINITY ? 0.0f : M;
        Lsum = 0.0f;
        o[0] = o[1] = o[2] = o[3] = 0.0f;
#pragma unroll
        for (int i = 0; i < G; ++i) {
            const float f = __builtin_amdgcn_exp2f(so[i][D] - mu);
            const float4 v = *reinterpret_cast<const float4 *>(&so[i][lane * 4]);
            Lsum += so[i][D + 1] * f;
            o[0] += v.x * f;
            o[1] += v.y * f;
            o[2] += v.z * f;
            o[3] += v.w * f;
        }
    }
    const float inv = Lsum == 0.0f ? 0.0f : 1.0f / Lsum;
    const int64_t out = (int64_t)(sp.qbeg + row / p.g) * a.hq + head * p.g + row % p.g;
    *reinterpret_cast<uint2 *>(a.o + out * D + lane * 4) =
        make_uint2(bf16_pack2(o[0] * inv, o[1] * inv), bf16_pack2(o[2] * inv, o[3] * inv));
    if (a.lse && lane == 0) a.lse[out] = Lsum == 0.0f ? -INFINITY : (M + __builtin_amdgcn_logf(Lsum)) * LN2;
}

namespace {

constexpr int64_t WANT = 1024;  // workgroups of a call, where its tokens allow: four a CU
constexpr int64_t FAR = 1024;   // tokens after which a workgroup's share is split all the same ...
constexpr int64_t FAR_SPLITS = 64;  // ... into at most this many: sequences of unlike lengths balance

// A call of few (sequence, head, tile)s over few tokens goes to workgroups of WIDE waves instead of several
// of four: they join in LDS, which saves the second launch (about 4 us of the host's time).  On the
// device, split | wide, us, d 128: 8 groups 7.1 | 7.0 at 512 tokens, 7.2 | 8.8 at 1024, 7.6 | 12.4 at 2048;
// 64 groups 9.0 | 9.1 at 1024, 12.1 | 13.1 at 2048; 256 groups 12.5 | 8.5 at 512, 15.1 | 12.0 at 1024,
// 30.5 | 28.9 at 4096, 53.1 | 51.4 at 8192 (where unlike lengths would leave CUs idle).
constexpr int WIDE = 16;
bool wide(int64_t groups, int64_t span) { return groups <= 256 && span <= (groups >= 128 ? 4096 : groups >= 64 ? 2048 : 1024); }

// Rows and tiles of a call: up to FEW rows a (sequence, head) go to the decode kernel.  Eight waves unpack a
// tile for 256 rows; heads of 64 have too little to unpack for that.
void tiles_of(int max_q, int g, int d, DecArgs &p) {
    const int64_t rows = (int64_t)max_q * g;
    p.g = g;
    p.tr = rows <= FEW ? 16 : d == 128 && rows >= 256 ? 256 : 128;
    p.pr = (int)std::min<int64_t>(rows, p.tr);
    p.rt = (int)((rows + p.tr - 1) / p.tr);
}
// The split of a call along `span` tokens, at most (it does not fall as the span grows).
int64_t splits_of(const DecArgs &p, int64_t groups, int64_t span) {
    const int64_t unit = p.tr > 16 ? CT : 4 * TT, want = p.tr == 256 ? WANT / 4 : p.tr == 128 ? WANT / 2 : WANT;
    int64_t splits = (want + groups - 1) / groups;
    // (a launch has at most 2^22 workgroups, far below the 2^32 threads that it may have)
    if (p.tr == 16)
        splits = std::max(splits, std::min({(span + FAR - 1) / FAR, FAR_SPLITS, ((int64_t)1 << 22) / std::max<int64_t>(groups, 1)}));
    return std::max<int64_t>(1, std::min(splits, (span + unit - 1) / unit));
}
// The split of a many-rows call of SINKS, PREFIX or OWN, at most `most`, by the time that it would take.  A tile takes
// 2.3 us of a workgroup of eight waves; one of four has company on its CU: 1.1, 1.6 and 2.0 us with one to three of them
// at heads of 64, 1.6 and 2.4 with two at 128.  A turn of workgroups costs 5 us besides; partial results are written and
// read at 4.8 TB/s; `always`: one split leaves them too, and otherwise more than one costs the join's launch.
// Against the rule above, splits and us: 17 x 75 queries of 20 heads of 64 behind 4000 shared tokens 4 -> 5 and 101 -> 53 with
// its join gone.  (2 x 1000 of them through a window of 1500 keep their two splits.)
int64_t turns_of(const DecArgs &p, int64_t groups, int64_t span, int64_t most, bool always, float &us) {
    const int64_t tiles = (span + CT - 1) / CT;
    const bool wide_tile = p.tr == 256, small_head = p.a.geo.d == 64;
    const int64_t company = wide_tile ? 1 : small_head ? 3 : 2;
    const float one = wide_tile ? 2.3f : small_head ? 1.13f : 1.6f, more = small_head ? 0.43f : 0.8f;
    const float parts = (float)groups * p.pr * (p.a.geo.d + 4) * (8.0f / 4.8e6f);
    int64_t best = 1;
    for (int64_t n = 1; n <= std::min({most, tiles, (int64_t)64}); ++n) {
        const int64_t on_cu = (groups * n + 255) / 256, full = on_cu / company, rest = on_cu % company;
        const float tile = full * (one + (company - 1) * more) + (rest ? one + (rest - 1) * more : 0.0f);
        const float t = tile * ((tiles + n - 1) / n) + 5.0f * (full + (rest != 0)) + (always || n > 1 ? parts * n : 0.0f) +
                        (!always && n > 1 ? 4.0f : 0.0f);
        if (n == 1 || t < us) {
            us = t;
            best = n;
        }
    }
    return best;
}

// A decode call of 256 groups or more through a window with sinks, in a table at least twice as wide as that: most of its sequences
// are past the window and alike long, so one split of four waves a group needs no join; past a span that grows with
// the groups, four splits cost alike lengths 5 % at most and balance unlike ones, whose number a call does not know.
// One split | four | as many as splits_of says | wide workgroups, us, sequences past the window; in brackets lengths of 32 to 131072
// tokens, even in their logarithm; heads of 128:
//    256 groups    2048: 17 | 22 | 22 | 20 (16 | 18 | 18 | 18)     8192: 61 | 62 | 63 | 67 (51 | 38 | 40 | 53)
//    320           1024: 15 | 19 | 19 | 24 (14 | 17 | 17 | 19)     4096: 45 | 44 | 45 | 64 (38 | 29 | 30 | 36)
//    512           8192: 108 | 113 | 117 | 127 (72 | 72 | 75 | 105)  16384: 201 | 210 | 224 | 233 (133 | 114 | 120 | 173)
//   1024           8192: 205 | 220 | 232 | 246 (120 | 120 | 126 | 164)  32768: 787 | 798 | 887 | 865 (368 | 276 | 308 | 424)
// heads of 64:
//    256           1024: 10 | 13 | 13 | 9 (10 | 13 | 13 | 9)       4096: 24 | 21 | 22 | 18 (23 | 21 | 20 | 17)
//    512           2048: 20 | 25 | 24 | 22 (18 | 23 | 23 | 21)     8192: 71 | 67 | 72 | 62 (59 | 49 | 50 | 55)
// A batch of sequences shorter than the window is quickest with one split: 10 | 14 | 14 | 13 of 256 groups.
int64_t sinks_splits(int64_t groups, int64_t span, int d, int64_t splits) {
    const int64_t one = (groups > 256 && groups < 512 ? FAR * 5 / 2 : FAR * groups / 64) * d / 128;
    return span <= one ? 1 : std::min<int64_t>(splits, 4);
}

// The rest of a call's plan: `groups` of rows, each over `span` tokens at most, of the `full` that the table's rows hold.
// Returns about how many us it takes, launch and all (not of PLAIN's many-rows kernels): the decode kernel 6 and what
// the bytes take, of the last-level cache where they are shared, 7.9 TB/s at heads of 128 and 5.8 at 64.
float split(DecArgs &p, int64_t groups, int64_t span, int64_t full, int mode) {
    int64_t splits = splits_of(p, groups, span);
    const int d = p.a.geo.d;
    float us = 0.0f;
    if (p.tr > 16) {
        if (mode == SINKS) splits = turns_of(p, groups, span, splits, false, us);  // (PLAIN's workspace)
        else if (mode != PLAIN) splits = turns_of(p, groups, span, 64, mode == PREFIX, us);
        us += 4.0f;
    } else {
        // (256 groups of heads of 64 are quicker in the wide workgroups)
        const bool many = groups >= 256 && !(d == 64 && wide(groups, span));
        if (mode == SINKS && many && 2 * span <= full) splits = sinks_splits(groups, span, d, splits);
        // then no join.  One | many | wide, us: 64 sequences of 8 heads of 128 over 16384 shared tokens and up to 450 of their own
        // 41 | 60 | 48, to 1900 52 | 71 | 65; 32 of them 31 | 45 | 32 and 38 | 51 | 38, at heads of 64 36 | 36 | 23 and 40 | 40 | 27
        if (mode == OWN && many && span <= 2 * FAR) splits = 1;
    }
    p.nw = p.tr == 16 && splits > 1 && wide(groups, span) ? WIDE : 4;
    if (p.nw == WIDE) splits = 1;
    if (p.tr == 16)
        us = 6.0f + (float)groups * span * p.a.geo.d * (17.0f / 16.0f) / (p.a.geo.d == 128 ? 7.9e6f : 5.8e6f) +
             (mode == WHOLE && splits > 1 ? 4.0f : 0.0f);
    const int64_t unit = p.tr > 16 ? CT : p.nw * TT;
    const int64_t chunk = ((span + splits - 1) / splits + unit - 1) / unit * unit;
    p.chunk = (int)chunk;
    p.splits = (int)((span + chunk - 1) / chunk);
    p.work = (int)(groups * p.splits);  // below 2^23
    p.blanks = 0;
    return us;
}

DecArgs args_of(const Kv4Attn &a) {
    DecArgs p{};
    p.a = a;
    p.c = a.scale * LOG2E;
    p.part = reinterpret_cast<float *>(a.ws);
    return p;
}

// A call with shared pages: in two parts, or (`whole`) as one; and the bytes of its partial results, OWN's or WHOLE's,
// if they leave any, then PREFIX's.
struct SharedPlan {
    DecArgs pre, own;
    bool whole;
    size_t bytes;
};
SharedPlan plan_shared(const Kv4Attn &a) {
    SharedPlan s;
    const int g = a.hq / a.geo.hkv, row = (a.geo.d + 4) * 4;
    s.pre = s.own = args_of(a);
    tiles_of(a.nq, g, a.geo.d, s.pre);
    if (s.pre.tr > 16) s.pre.pr = (s.pre.pr + 31) & ~31;  // whole waves' rows
    tiles_of(a.max_q, g, a.geo.d, s.own);
    const int64_t pg = (int64_t)a.geo.hkv * s.pre.rt, og = (int64_t)a.b * a.geo.hkv * s.own.rt;
    const int64_t shared = (int64_t)a.shared << a.geo.page_log2, all = (int64_t)a.width << a.geo.page_log2, rest = all - shared + TT;
    // OWN takes PREFIX's results in, one split after the other in a wave, about 1 us each; or a join does, 6 us and their bytes
    float two = split(s.pre, pg, shared, shared, PREFIX);
    DecArgs joined = s.own, one = s.own;
    const float taken = split(s.own, og, rest, rest, OWN) +
                        (s.own.tr == 16 ? 1.2f * ((s.pre.splits + s.own.nw - 1) / s.own.nw) : 1.0f * s.pre.splits);
    const float left = split(joined, og, rest, rest, PREFIX) + 6.0f +
                       (float)a.nq * a.hq * (s.pre.splits + joined.splits) * row / 4.8e6f;
    s.own.takes = s.own.splits == 1 && taken <= left;
    if (!s.own.takes) s.own = joined;
    two += s.own.takes ? taken : left;
    // Two parts | one, us, heads of 128 in groups of four over 8, 16384 shared tokens: 28 | 15 for one single token, 27 | 29
    // for 8, 30 | 47 for 16, 47 | 146 for 64; 2048: 14 | 13 for 8, 27 | 33 for 64; 8 x 40 tokens 44 | 40 behind 2048, 107 | 153
    // behind 16384.
    s.whole = split(one, og, all, all, WHOLE) <= two;
    if (s.whole) {
        s.own = one;
        s.bytes = one.splits > 1 ? (size_t)(og * one.splits) * one.pr * row : 0;
        return s;
    }
    const size_t first = !s.own.takes ? ((size_t)(og * s.own.splits) * s.own.pr * row + 255) & ~(size_t)255 : 0;
    s.pre.part = reinterpret_cast<float *>(a.ws + first);
    s.own.ptr_ = s.pre.tr;
    s.own.ppr = s.pre.pr;
    s.own.psplits = s.pre.splits;
    s.own.ppart = s.pre.part;
    s.bytes = first + (size_t)(pg * s.pre.splits) * s.pre.pr * row;
    return s;
}

template <int MODE>
hipError_t launch_attend(const DecArgs &p, hipStream_t s) {
    const Kv4Attn &a = p.a;
    const dim3 grid((unsigned)(p.work + p.blanks));
    if (p.tr > 16) {
        if (p.tr == 256) hipLaunchKernelGGL((k_kv4_chunk<128, 512, MODE>), grid, dim3(512), 0, s, p);
        else if (a.geo.d == 128) hipLaunchKernelGGL((k_kv4_chunk<128, 256, MODE>), grid, dim3(256), 0, s, p);
        else hipLaunchKernelGGL((k_kv4_chunk<64, 256, MODE>), grid, dim3(256), 0, s, p);
    } else {
#define DECODE(D, NW)                                                                                              \
    do {                                                                                                           \
        if (a.geo.page_log2 >= 5) hipLaunchKernelGGL((k_kv4_decode<D, NW, true, MODE>), grid, dim3(64 * NW), 0, s, p); \
        else hipLaunchKernelGGL((k_kv4_decode<D, NW, false, MODE>), grid, dim3(64 * NW), 0, s, p);                   \
    } while (0)
        if (a.geo.d == 128 && p.nw == WIDE) DECODE(128, WIDE);
        else if (a.geo.d == 128) DECODE(128, 4);
        else if (p.nw == WIDE) DECODE(64, WIDE);
        else DECODE(64, 4);
#undef DECODE
    }
    return hipGetLastError();
}

template <int MODE>
hipError_t launch_join(const DecArgs &p, hipStream_t s) {
    const Kv4Attn &a = p.a;
    const int64_t tiles = (int64_t)a.b * p.rt * a.geo.hkv;
    // one group a row where a row has no more splits than four groups' turns and the rows fill the device
    const int parts = p.splits + p.psplits;
    const int groups = 1024 / a.geo.d, per = (parts <= 4 && tiles * p.pr >= 8192) || tiles * p.pr >= 1 << 22 ? groups : 1;
    const dim3 jg((unsigned)((tiles * p.pr + per - 1) / per));
    if (a.geo.d == 128 && per > 1) hipLaunchKernelGGL((k_kv4_join<128, 1, MODE>), jg, dim3(256), 0, s, p);
    else if (a.geo.d == 128) hipLaunchKernelGGL((k_kv4_join<128, 8, MODE>), jg, dim3(256), 0, s, p);
    else if (per > 1) hipLaunchKernelGGL((k_kv4_join<64, 1, MODE>), jg, dim3(256), 0, s, p);
    else hipLaunchKernelGGL((k_kv4_join<64, 16, MODE>), jg, dim3(256), 0, s, p);
    return hipGetLastError();
}

template <int MODE>
hipError_t attend_and_join(const DecArgs &p, hipStream_t s) {
    const hipError_t e = launch_attend<MODE>(p, s);
    return e == hipSuccess && p.splits > 1 ? launch_join<MODE>(p, s) : e;
}

int blanks_of(const Kv4Attn &a) { return a.q_start ? std::max(a.b, std::min(a.nq, 64)) : 0; }

}  // namespace

// Enough for every window: a window only shortens the span, so the bound on the splits falls (and a call
// that goes to the wide workgroups needs none of it).
size_t kv4_attn_ws_bytes(int b, int max_q, int hq, const Kv4Geom &g, int width) {
    DecArgs p;
    tiles_of(max_q, hq / g.hkv, g.d, p);
    const int64_t groups = (int64_t)b * g.hkv * p.rt, splits = splits_of(p, groups, (int64_t)width << g.page_log2);
    return splits <= 1 ? 0 : (size_t)(groups * splits) * p.pr * (g.d + 4) * 4;
}

hipError_t launch_kv4_attn(const Kv4Attn &a, hipStream_t s) {
    DecArgs p = args_of(a);
    tiles_of(a.max_q, a.hq / a.geo.hkv, a.geo.d, p);
    const int64_t full = (int64_t)a.width << a.geo.page_log2;
    int64_t span = full;
    // a window's span: that of the tile's first to its last query, and the start's rounding down; and the sinks'
    const bool sinks = a.window && a.sinks;
    if (a.window) span = std::min<int64_t>(span, (int64_t)a.window + p.tr / p.g + 1 + CT + (sinks ? (int64_t)a.sinks + CT : 0));
    split(p, (int64_t)a.b * a.geo.hkv * p.rt, span, full, sinks ? SINKS : PLAIN);
    p.blanks = blanks_of(a);
    return sinks ? attend_and_join<SINKS>(p, s) : attend_and_join<PLAIN>(p, s);
}

static SharedPlan plan_shared(int64_t nq, int b, int max_q, int hq, const Kv4Geom &g, int width, int shared) {
    Kv4Attn a{};
    a.geo = g;
    a.nq = (int)nq;
    a.b = b;
    a.max_q = max_q;
    a.hq = hq;
    a.width = width;
    a.shared = shared;
    return plan_shared(a);
}
int kv4_attn_shared_parts(int64_t nq, int b, int max_q, int hq, const Kv4Geom &g, int width, int shared) {
    return plan_shared(nq, b, max_q, hq, g, width, shared).whole ? 1 : 2;
}
size_t kv4_attn_shared_ws_bytes(int64_t nq, int b, int max_q, int hq, const Kv4Geom &g, int width, int shared) {
    return plan_shared(nq, b, max_q, hq, g, width, shared).bytes;
}

hipError_t launch_kv4_attn_shared(const Kv4Attn &a, hipStream_t s) {
    SharedPlan p = plan_shared(a);
    p.own.blanks = blanks_of(a);
    if (p.whole) {
        const hipError_t e = launch_attend<WHOLE>(p.own, s);
        return e == hipSuccess && p.own.splits > 1 ? launch_join<PLAIN>(p.own, s) : e;
    }
    hipError_t e = launch_attend<PREFIX>(p.pre, s);
    if (e == hipSuccess) e = launch_attend<OWN>(p.own, s);
    return e == hipSuccess && !p.own.takes ? launch_join<OWN>(p.own, s) : e;
}

}  // namespace fp4
