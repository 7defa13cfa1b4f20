// C ABI of the block-scaled FP8 layer and of the 4-bit key/value cache (declared in
// include/fp4lin.h): host-side argument checks, workspace carving and launches.  Every check runs
// before the first HIP call.
#include <hip/hip_runtime.h>

#include "block8.h"
#include "fp4_host.h"
#include "fp4lin.h"
#include "kv4.h"

using namespace fp4;

namespace {

constexpr int64_t SIDE_MAX = ((int64_t)1 << 23) - 128;  // a product tile's 256 rows stay below 2^31 bytes
constexpr int64_t ELEMS_MAX = (int64_t)1 << 34;       // threads of a quantizer's launch at most 2^31

size_t up256(size_t x) { return (x + 255) & ~(size_t)255; }
bool al16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool al_elem(const void *p, int32_t dt) { return (reinterpret_cast<uintptr_t>(p) & (dt == FP4_BF16 ? 1u : 3u)) == 0; }
bool dt_ok(int32_t d) { return d == FP4_F32 || d == FP4_BF16; }
int dt_in(int32_t d) { return d == FP4_BF16 ? DT_BF16 : DT_F32; }
bool mode_ok(int32_t m) { return m == FP4_BLOCK_VECTOR || m == FP4_BLOCK_SQUARE; }
int64_t up128(int64_t x) { return (x + 127) / 128 * 128; }
bool mat_ok(int64_t r, int64_t c) {
    return r >= 1 && c >= 1 && r <= SIDE_MAX && c <= SIDE_MAX && up128(r) * up128(c) <= ELEMS_MAX;
}

Op8 op8(const uint8_t *codes, const uint8_t *scales, int64_t rows, int64_t L, int32_t mode) {
    Op8 o;
    o.codes = codes;
    o.scales = reinterpret_cast<const uint32_t *>(scales);
    o.ld = up128(L);
    o.srows = (int)(mode == FP4_BLOCK_SQUARE ? (rows + 127) / 128 : rows);
    o.sshift = mode == FP4_BLOCK_SQUARE ? 7 : 0;
    return o;
}

hipStream_t hs(void *s) { return reinterpret_cast<hipStream_t>(s); }

}  // namespace

extern "C" {

size_t fp4_block8_codes_bytes(int64_t rows, int64_t L) {
    return mat_ok(rows, L) ? (size_t)rows * (size_t)up128(L) : 0;
}

size_t fp4_block8_scales_bytes(int64_t rows, int64_t L, int32_t mode) {
    if (!mat_ok(rows, L) || !mode_ok(mode)) return 0;
    const int64_t srows = mode == FP4_BLOCK_SQUARE ? (rows + 127) / 128 : rows;
    return (size_t)((L + 511) / 512) * (size_t)srows * 4;
}

fp4_status fp4_block8_quantize(const void *X, int32_t x_dtype, int64_t R, int64_t C, int64_t ld, int32_t mode,
                               uint8_t *row_codes, uint8_t *row_scales, uint8_t *col_codes, uint8_t *col_scales,
                               void *stream) {
    if (!X || (!row_codes && !col_codes) || !row_codes != !row_scales || !col_codes != !col_scales) return FP4_ERR_NULL;
    if (!dt_ok(x_dtype) || !mode_ok(mode)) return FP4_ERR_DTYPE;
    if (!mat_ok(R, C) || ld < C) return FP4_ERR_SHAPE;
    if (!al_elem(X, x_dtype) || !al16(row_codes) || !al16(row_scales) || !al16(col_codes) || !al16(col_scales))
        return FP4_ERR_ALIGN;
    int cus;
    const fp4_status st = device_check(&cus);
    if (st != FP4_OK) return st;
    return hip_status(launch_block8_quant(X, dt_in(x_dtype), R, C, ld, mode == FP4_BLOCK_SQUARE, row_codes, row_scales,
                                          col_codes, col_scales, hs(stream)));
}

fp4_status fp4_block8_dequantize(const uint8_t *codes, const uint8_t *scales, int64_t rows, int64_t L, int32_t mode,
                                 void *Y, int32_t y_dtype, void *stream) {
    if (!codes || !scales || !Y) return FP4_ERR_NULL;
    if (!dt_ok(y_dtype) || !mode_ok(mode)) return FP4_ERR_DTYPE;
    if (!mat_ok(rows, L)) return FP4_ERR_SHAPE;
    if (!al16(codes) || !al16(scales) || !al_elem(Y, y_dtype)) return FP4_ERR_ALIGN;
    int cus;
    const fp4_status st = device_check(&cus);
    if (st != FP4_OK) return st;
    return hip_status(launch_block8_dequant(codes, scales, rows, L, mode == FP4_BLOCK_SQUARE, Y, dt_in(y_dtype),
                                            hs(stream)));
}

fp4_status fp4_block8_gemm(const uint8_t *a_codes, const uint8_t *a_scales, int32_t a_mode, const uint8_t *b_codes,
                           const uint8_t *b_scales, int32_t b_mode, int64_t M, int64_t N, int64_t K, void *Y,
                           int32_t y_dtype, void *stream) {
    if (!a_codes || !a_scales || !b_codes || !b_scales || !Y) return FP4_ERR_NULL;
    if (!dt_ok(y_dtype) || !mode_ok(a_mode) || !mode_ok(b_mode)) return FP4_ERR_DTYPE;
    if (!mat_ok(M, K) || !mat_ok(N, K) || !mat_ok(M, N)) return FP4_ERR_SHAPE;
    if (!al16(a_codes) || !al16(a_scales) || !al16(b_codes) || !al16(b_scales) || !al_elem(Y, y_dtype))
        return FP4_ERR_ALIGN;
    int cus;
    const fp4_status st = device_check(&cus);
    if (st != FP4_OK) return st;
    return hip_status(launch_block8_gemm(op8(a_codes, a_scales, M, K, a_mode), op8(b_codes, b_scales, N, K, b_mode), M,
                                         N, K, Y, dt_in(y_dtype), cus, hs(stream)));
}

size_t fp4_block8_linear_workspace_bytes(int64_t M, int64_t K, int64_t N) {
    if (!mat_ok(M, K) || !mat_ok(N, K) || !mat_ok(M, N)) return 0;
    return up256(fp4_block8_codes_bytes(M, K)) + up256(fp4_block8_scales_bytes(M, K, FP4_BLOCK_VECTOR));
}

fp4_status fp4_block8_linear(const void *X, int32_t x_dtype, int64_t M, int64_t K, int64_t ldx, const uint8_t *w_codes,
                             const uint8_t *w_scales, int32_t w_mode, int64_t N, void *Y, int32_t y_dtype,
                             uint8_t *xt_codes, uint8_t *xt_scales, void *workspace, size_t ws_bytes, void *stream) {
    if (!X || !w_codes || !w_scales || !Y || !workspace || !xt_codes != !xt_scales) return FP4_ERR_NULL;
    if (!dt_ok(x_dtype) || !dt_ok(y_dtype) || !mode_ok(w_mode)) return FP4_ERR_DTYPE;
    if (!mat_ok(M, K) || !mat_ok(N, K) || !mat_ok(M, N) || ldx < K) return FP4_ERR_SHAPE;
    if (ws_bytes < fp4_block8_linear_workspace_bytes(M, K, N)) return FP4_ERR_WORKSPACE;
    if (!al_elem(X, x_dtype) || !al16(w_codes) || !al16(w_scales) || !al_elem(Y, y_dtype) || !al16(xt_codes) ||
        !al16(xt_scales) || !al16(workspace))
        return FP4_ERR_ALIGN;
    int cus;
    const fp4_status st = device_check(&cus);
    if (st != FP4_OK) return st;
    if (!xt_codes && block8_few_direct(M, N, K))
        return hip_status(launch_block8_few_direct(X, dt_in(x_dtype), ldx, op8(w_codes, w_scales, N, K, w_mode), M, N, K, Y,
                                                   dt_in(y_dtype), hs(stream)));
    uint8_t *xc = static_cast<uint8_t *>(workspace), *xs = xc + up256(fp4_block8_codes_bytes(M, K));
    hipError_t e = launch_block8_quant(X, dt_in(x_dtype), M, K, ldx, false, xc, xs, xt_codes, xt_scales, hs(stream));
    if (e == hipSuccess)
        e = launch_block8_gemm(op8(xc, xs, M, K, FP4_BLOCK_VECTOR), op8(w_codes, w_scales, N, K, w_mode), M, N, K, Y,
                               dt_in(y_dtype), cus, hs(stream));
    return hip_status(e);
}

size_t fp4_block8_backward_workspace_bytes(int64_t M, int64_t N) {
    if (!mat_ok(M, N)) return 0;
    return up256(fp4_block8_codes_bytes(M, N)) + up256(fp4_block8_scales_bytes(M, N, FP4_BLOCK_VECTOR)) +
           up256(fp4_block8_codes_bytes(N, M)) + up256(fp4_block8_scales_bytes(N, M, FP4_BLOCK_VECTOR));
}

fp4_status fp4_block8_backward(const void *dY, int32_t dy_dtype, int64_t M, int64_t K, int64_t N, int64_t lddy,
                               const uint8_t *w_codes, const uint8_t *w_scales, int32_t w_mode,
                               const uint8_t *xt_codes, const uint8_t *xt_scales, void *dX, int32_t dx_dtype, void *dW,
                               int32_t dw_dtype, void *workspace, size_t ws_bytes, void *stream) {
    if (!dY || !workspace || (!dX && !dW)) return FP4_ERR_NULL;
    if ((dX && (!w_codes || !w_scales)) || (dW && (!xt_codes || !xt_scales))) return FP4_ERR_NULL;
    if (!dt_ok(dy_dtype) || (dX && (!dt_ok(dx_dtype) || !mode_ok(w_mode))) || (dW && !dt_ok(dw_dtype)))
        return FP4_ERR_DTYPE;
    if (!mat_ok(M, N) || !mat_ok(M, K) || !mat_ok(K, N) || lddy < N) return FP4_ERR_SHAPE;
    if (ws_bytes < fp4_block8_backward_workspace_bytes(M, N)) return FP4_ERR_WORKSPACE;
    if (!al_elem(dY, dy_dtype) || !al16(workspace) || (dX && (!al16(w_codes) || !al16(w_scales) || !al_elem(dX, dx_dtype))) ||
        (dW && (!al16(xt_codes) || !al16(xt_scales) || !al_elem(dW, dw_dtype))))
        return FP4_ERR_ALIGN;
    int cus;
    const fp4_status st = device_check(&cus);
    if (st != FP4_OK) return st;
    uint8_t *rc = static_cast<uint8_t *>(workspace), *rs = rc + up256(fp4_block8_codes_bytes(M, N));
    uint8_t *cc = rs + up256(fp4_block8_scales_bytes(M, N, FP4_BLOCK_VECTOR));
    uint8_t *cs = cc + up256(fp4_block8_codes_bytes(N, M));
    hipError_t e = launch_block8_quant(dY, dt_in(dy_dtype), M, N, lddy, false, dX ? rc : nullptr, dX ? rs : nullptr,
                                       dW ? cc : nullptr, dW ? cs : nullptr, hs(stream));
    if (dX && e == hipSuccess)
        e = launch_block8_gemm(op8(rc, rs, M, N, FP4_BLOCK_VECTOR), op8(w_codes, w_scales, K, N, w_mode), M, K, N, dX,
                               dt_in(dx_dtype), cus, hs(stream));
    if (dW && e == hipSuccess)
        e = launch_block8_gemm(op8(xt_codes, xt_scales, K, M, FP4_BLOCK_VECTOR), op8(cc, cs, N, M, FP4_BLOCK_VECTOR), K,
                               N, M, dW, dt_in(dw_dtype), cus, hs(stream));
    return hip_status(e);
}

// ----------------------------------------------------------------------------- key/value cache
static bool geom(int64_t pages, int32_t page, int32_t hkv, int32_t d, Kv4Geom &g) {
    if (pages < 1 || page < 16 || page > 1024 || (page & (page - 1)) || hkv < 1 || hkv > 65536 || (d != 64 && d != 128))
        return false;
    g.pages = pages;
    g.page_log2 = __builtin_ctz((unsigned)page);
    g.hkv = hkv;
    g.d = d;
    return pages <= ((int64_t)1 << 46) / ((int64_t)hkv * g.region()) && pages <= 0x7FFFFFFF;
}

size_t fp4_kv4_cache_bytes(int64_t pages, int32_t page, int32_t hkv, int32_t d) {
    Kv4Geom g;
    return geom(pages, page, hkv, d, g) ? (size_t)(pages * hkv * g.region()) : 0;
}

fp4_status fp4_kv4_write(uint8_t *cache, int64_t pages, int32_t page, int32_t hkv, int32_t d, const void *K,
                         const void *V, int32_t dtype, int64_t n, int64_t k_token_stride, int64_t k_head_stride,
                         int64_t v_token_stride, int64_t v_head_stride, const void *slots, int32_t slot_bytes,
                         void *stream) {
    if (!cache || !K || !V || !slots) return FP4_ERR_NULL;
    if (!dt_ok(dtype) || (slot_bytes != 4 && slot_bytes != 8)) return FP4_ERR_DTYPE;
    Kv4Geom g;
    if (!geom(pages, page, hkv, d, g) || n < 1 || n > ((int64_t)1 << 27) / hkv) return FP4_ERR_SHAPE;
    if (!al16(cache) || !al_elem(K, dtype) || !al_elem(V, dtype) ||
        (reinterpret_cast<uintptr_t>(slots) & (uintptr_t)(slot_bytes - 1)))
        return FP4_ERR_ALIGN;
    int cus;
    const fp4_status st = device_check(&cus);
    if (st != FP4_OK) return st;
    return hip_status(launch_kv4_write(cache, g, K, V, dt_in(dtype), n, k_token_stride, k_head_stride, v_token_stride,
                                       v_head_stride, slots, slot_bytes == 8, hs(stream)));
}

fp4_status fp4_kv4_read(const uint8_t *cache, int64_t pages, int32_t page, int32_t hkv, int32_t d, const void *slots,
                        int32_t slot_bytes, int64_t n, void *K, void *V, int32_t dtype, void *stream) {
    if (!cache || !K || !V || !slots) return FP4_ERR_NULL;
    if (!dt_ok(dtype) || (slot_bytes != 4 && slot_bytes != 8)) return FP4_ERR_DTYPE;
    Kv4Geom g;
    if (!geom(pages, page, hkv, d, g) || n < 1 || n > ((int64_t)1 << 27) / hkv) return FP4_ERR_SHAPE;
    if (!al16(cache) || !al16(K) || !al16(V) || (reinterpret_cast<uintptr_t>(slots) & (uintptr_t)(slot_bytes - 1)))
        return FP4_ERR_ALIGN;
    int cus;
    const fp4_status st = device_check(&cus);
    if (st != FP4_OK) return st;
    return hip_status(launch_kv4_read(cache, g, slots, slot_bytes == 8, n, K, V, dt_in(dtype), hs(stream)));
}

static bool attn_shape(int32_t b, int32_t max_q, int32_t hq, int32_t hkv, int32_t width, int32_t page, int32_t window) {
    if (b < 1 || max_q < 1 || hq < 1 || hq % hkv || width < 1 || window < 0) return false;
    if ((int64_t)max_q * (hq / hkv) >= (1 << 24) || (int64_t)width * page > (1 << 30)) return false;
    // workgroups of a launch: at most 1024 splits of (sequence, head, row tile)
    return (int64_t)b * hkv * (((int64_t)max_q * (hq / hkv) + 15) / 16) < (1 << 22);
}

size_t fp4_kv4_attention_workspace_bytes(int32_t b, int32_t max_q, int32_t hq, int32_t hkv, int32_t d, int32_t page,
                                         int32_t width) {
    Kv4Geom g;
    if (!geom(1, page, hkv, d, g) || !attn_shape(b, max_q, hq, hkv, width, page, 0)) return 0;
    return kv4_attn_ws_bytes(b, max_q, hq, g, width);
}

// What the attention calls check and hand over alike; need: the workspace's bytes.
static fp4_status attention_check(const void *q, int64_t nq, int32_t hq, const int32_t *q_start, const int32_t *lens, int32_t b,
                                  int32_t max_q, const int32_t *table, int64_t table_stride, int32_t width,
                                  const uint8_t *cache, void *o, float *lse, void *workspace, size_t ws_bytes, size_t need) {
    if (nq < 1 || nq > 0x7FFFFFFF / hq || table_stride < width || (!q_start && (nq != b || max_q != 1)))
        return FP4_ERR_SHAPE;
    if (need && !workspace) return FP4_ERR_NULL;
    if (ws_bytes < need) return FP4_ERR_WORKSPACE;
    if (!al_elem(q, FP4_BF16) || !al16(cache) || !al16(o) || !al_elem(lse, FP4_F32) || !al16(workspace) ||
        !al_elem(lens, FP4_F32) || !al_elem(table, FP4_F32) || !al_elem(q_start, FP4_F32))
        return FP4_ERR_ALIGN;
    int cus;
    return device_check(&cus);
}

static Kv4Attn attention_args(const void *q, int64_t q_token_stride, int64_t q_head_stride, int64_t nq, int32_t hq,
                              const int32_t *q_start, const int32_t *lens, int32_t b, int32_t max_q, const int32_t *table,
                              int64_t table_stride, int32_t width, const uint8_t *cache, const Kv4Geom &g, float scale,
                              void *o, float *lse, void *workspace) {
    Kv4Attn a{};
    a.q = static_cast<const uint16_t *>(q);
    a.q_ts = q_token_stride;
    a.q_hs = q_head_stride;
    a.q_start = q_start;
    a.lens = lens;
    a.pages = table;
    a.page_rs = table_stride;
    a.width = width;
    a.cache = cache;
    a.geo = g;
    a.b = b;
    a.nq = (int)nq;
    a.hq = hq;
    a.max_q = max_q;
    a.scale = scale;
    a.o = static_cast<uint16_t *>(o);
    a.lse = lse;
    a.ws = static_cast<uint8_t *>(workspace);
    return a;
}

fp4_status fp4_kv4_attention_sinks(const void *q, int64_t q_token_stride, int64_t q_head_stride, int64_t nq, int32_t hq,
                                   const int32_t *q_start, const int32_t *lens, int32_t b, int32_t max_q,
                                   const int32_t *table, int64_t table_stride, int32_t width, const uint8_t *cache,
                                   int64_t pages, int32_t page, int32_t hkv, int32_t d, int32_t window, int32_t sinks,
                                   float scale, void *o, float *lse, void *workspace, size_t ws_bytes, void *stream) {
    if (!q || !lens || !table || !cache || !o) return FP4_ERR_NULL;
    Kv4Geom g;
    if (!geom(pages, page, hkv, d, g) || !attn_shape(b, max_q, hq, hkv, width, page, window) || sinks < 0) return FP4_ERR_SHAPE;
    const fp4_status st = attention_check(q, nq, hq, q_start, lens, b, max_q, table, table_stride, width, cache, o, lse,
                                          workspace, ws_bytes, kv4_attn_ws_bytes(b, max_q, hq, g, width));
    if (st != FP4_OK) return st;
    Kv4Attn a = attention_args(q, q_token_stride, q_head_stride, nq, hq, q_start, lens, b, max_q, table, table_stride, width,
                               cache, g, scale, o, lse, workspace);
    a.window = window;
    a.sinks = sinks;
    return hip_status(launch_kv4_attn(a, hs(stream)));
}

fp4_status fp4_kv4_attention(const void *q, int64_t q_token_stride, int64_t q_head_stride, int64_t nq, int32_t hq,
                             const int32_t *q_start, const int32_t *lens, int32_t b, int32_t max_q,
                             const int32_t *table, int64_t table_stride, int32_t width, const uint8_t *cache,
                             int64_t pages, int32_t page, int32_t hkv, int32_t d, int32_t window, float scale, void *o,
                             float *lse, void *workspace, size_t ws_bytes, void *stream) {
    return fp4_kv4_attention_sinks(q, q_token_stride, q_head_stride, nq, hq, q_start, lens, b, max_q, table, table_stride,
                                   width, cache, pages, page, hkv, d, window, 0, scale, o, lse, workspace, ws_bytes, stream);
}

// The shared pages' rows are all queries': the limits of attn_shape, as of one sequence with nq queries.
static bool shared_shape(int64_t nq, int32_t b, int32_t max_q, int32_t hq, int32_t hkv, int32_t width, int32_t page, int32_t shared) {
    return attn_shape(b, max_q, hq, hkv, width, page, 0) && shared >= 1 && shared <= width && nq >= 1 && nq <= (1 << 24) &&
           attn_shape(1, (int32_t)nq, hq, hkv, width, page, 0);
}

int32_t fp4_kv4_attention_shared_parts(int64_t nq, int32_t b, int32_t max_q, int32_t hq, int32_t hkv, int32_t d, int32_t page,
                                       int32_t width, int32_t shared) {
    Kv4Geom g;
    if (!geom(1, page, hkv, d, g) || !shared_shape(nq, b, max_q, hq, hkv, width, page, shared)) return 0;
    return kv4_attn_shared_parts(nq, b, max_q, hq, g, width, shared);
}

size_t fp4_kv4_attention_shared_workspace_bytes(int64_t nq, int32_t b, int32_t max_q, int32_t hq, int32_t hkv, int32_t d,
                                                int32_t page, int32_t width, int32_t shared) {
    Kv4Geom g;
    if (!geom(1, page, hkv, d, g) || !shared_shape(nq, b, max_q, hq, hkv, width, page, shared)) return 0;
    return kv4_attn_shared_ws_bytes(nq, b, max_q, hq, g, width, shared);
}

fp4_status fp4_kv4_attention_shared(const void *q, int64_t q_token_stride, int64_t q_head_stride, int64_t nq, int32_t hq,
                                    const int32_t *q_start, const int32_t *lens, int32_t b, int32_t max_q,
                                    const int32_t *table, int64_t table_stride, int32_t width, const uint8_t *cache,
                                    int64_t pages, int32_t page, int32_t hkv, int32_t d, int32_t shared, float scale, void *o,
                                    float *lse, void *workspace, size_t ws_bytes, void *stream) {
    if (!q || !lens || !table || !cache || !o) return FP4_ERR_NULL;
    Kv4Geom g;
    if (!geom(pages, page, hkv, d, g) || !shared_shape(nq, b, max_q, hq, hkv, width, page, shared)) return FP4_ERR_SHAPE;
    const fp4_status st = attention_check(q, nq, hq, q_start, lens, b, max_q, table, table_stride, width, cache, o, lse,
                                          workspace, ws_bytes, kv4_attn_shared_ws_bytes(nq, b, max_q, hq, g, width, shared));
    if (st != FP4_OK) return st;
    Kv4Attn a = attention_args(q, q_token_stride, q_head_stride, nq, hq, q_start, lens, b, max_q, table, table_stride, width,
                               cache, g, scale, o, lse, workspace);
    a.shared = shared;
    return hip_status(launch_kv4_attn_shared(a, hs(stream)));
}

}  // extern "C"
