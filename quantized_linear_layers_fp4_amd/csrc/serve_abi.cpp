// C ABI of the page tables and of the query/key norm with rotation (declared in include/fp4lin.h): host-side argument
// checks and launches.  Every check runs before the first HIP call.
#include <hip/hip_runtime.h>

#include "block8.h"
#include "fp4_host.h"
#include "fp4lin.h"
#include "serve.h"

using namespace fp4;

namespace {

bool al(const void *p, unsigned n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
bool dt_ok(int32_t d) { return d == FP4_F32 || d == FP4_BF16; }
int dt_in(int32_t d) { return d == FP4_BF16 ? DT_BF16 : DT_F32; }
unsigned size_of(int32_t d) { return d == FP4_BF16 ? 2 : 4; }
hipStream_t hs(void *s) { return reinterpret_cast<hipStream_t>(s); }

bool tables_ok(int32_t b, int32_t width, int64_t stride, int32_t page, int64_t pages) {
    return b >= 1 && b <= (1 << 20) && width >= 1 && stride >= width && page >= 16 && page <= 1024 && !(page & (page - 1)) &&
           pages >= 1 && pages <= 0x7FFFFFFF && (int64_t)width * page <= (1 << 30) && (int64_t)b * width < ((int64_t)1 << 31);
}

PageTables tables_of(int32_t *table, int64_t stride, int32_t b, int32_t width, int32_t *lens, int32_t *free, int32_t *count,
                     int64_t pages, int32_t page) {
    PageTables t;
    t.table = table;
    t.table_rs = stride;
    t.width = width;
    t.lens = lens;
    t.b = b;
    t.free = free;
    t.count = count;
    t.pages = (int32_t)pages;
    t.page_log2 = __builtin_ctz((unsigned)page);
    return t;
}

// The arguments that the three calls over rows of heads share.
fp4_status rows_check(int64_t n, int32_t hq, int32_t hkv, int32_t d, int32_t dtype, int32_t w_dtype, const void *qw,
                      const void *kw, float eps, const int32_t *positions, const float *table, int64_t max_pos, int32_t rot) {
    if (rot && (!positions || !table)) return FP4_ERR_NULL;
    if (!dt_ok(dtype) || ((qw || kw) && !dt_ok(w_dtype))) return FP4_ERR_DTYPE;
    if (n < 1 || n > (1 << 24) || hq < 1 || hkv < 0 || n * ((int64_t)hq + hkv) > ((int64_t)1 << 29)) return FP4_ERR_SHAPE;
    if (d < 32 || d > 256 || d % 8 || rot < 0 || rot % 16 || rot > d || (rot && max_pos < 1)) return FP4_ERR_SHAPE;
    if (!(eps >= 0.0f || eps == -1.0f) || (eps < 0.0f && (qw || kw))) return FP4_ERR_SHAPE;
    if ((rot && (!al(positions, 4) || !al(table, 16))) || ((qw || kw) && (!al(qw, size_of(w_dtype)) || !al(kw, size_of(w_dtype)))))
        return FP4_ERR_ALIGN;
    return FP4_OK;
}

NormRope rows_of(const void *q, int64_t q_ts, int64_t q_hs, int32_t hq, const void *k, int64_t k_ts, int64_t k_hs, int32_t hkv,
                 int64_t n, int32_t d, int32_t dtype, const void *qw, const void *kw, int32_t w_dtype, float eps,
                 const int32_t *positions, const float *table, int64_t max_pos, int32_t rot, int32_t interleaved) {
    NormRope a;
    a.q = HeadRows{q, q_ts, q_hs, hq, qw};
    a.k = HeadRows{k, k_ts, k_hs, hkv, kw};
    a.dt = dt_in(dtype);
    a.w_dt = dt_in(w_dtype);
    a.d = d;
    a.n = n;
    a.positions = positions;
    a.table = table;
    a.max_pos = max_pos;
    a.rot = rot;
    a.interleaved = interleaved != 0;
    a.norm = eps >= 0.0f;
    a.eps = eps;
    a.inv_d = 1.0 / d;
    return a;
}

}  // namespace

extern "C" {

size_t fp4_kv4_extend_workspace_bytes(int32_t b, int64_t n) {
    return b < 1 || b > (1 << 20) || n < 0 || n >= 0x7FFFFFFF ? 0 : pages_extend_ws_bytes(b, n);
}

fp4_status fp4_kv4_extend(int32_t *table, int64_t table_stride, int32_t b, int32_t width, int32_t *lens, int32_t *free_pages,
                          int32_t *free_count, int64_t pages, int32_t page, const int32_t *new_tokens, int64_t n, int64_t *slots,
                          int32_t *positions, int32_t *q_start, void *workspace, size_t ws_bytes, void *stream) {
    if (!table || !lens || !free_pages || !free_count || (n > 0 && (!slots || !positions))) return FP4_ERR_NULL;
    if (!tables_ok(b, width, table_stride, page, pages) || n < 0 || n >= 0x7FFFFFFF || (!q_start && n != b)) return FP4_ERR_SHAPE;
    const size_t need = q_start ? pages_extend_ws_bytes(b, n) : 0;
    if (need && !workspace) return FP4_ERR_NULL;
    if (ws_bytes < need) return FP4_ERR_WORKSPACE;
    if (!al(table, 4) || !al(lens, 4) || !al(free_pages, 4) || !al(free_count, 4) || !al(new_tokens, 4) || !al(slots, 8) ||
        !al(positions, 4) || !al(q_start, 4) || !al(workspace, 4))
        return FP4_ERR_ALIGN;
    int cus;
    const fp4_status st = device_check(&cus);
    if (st != FP4_OK) return st;
    return hip_status(launch_pages_extend(tables_of(table, table_stride, b, width, lens, free_pages, free_count, pages, page),
                                          new_tokens, n, slots, positions, q_start, static_cast<int32_t *>(workspace), hs(stream)));
}

size_t fp4_kv4_release_workspace_bytes(int32_t b, int32_t width) {
    return b < 1 || b > (1 << 20) || width < 1 ? 0 : pages_release_ws_bytes(b, width);
}

fp4_status fp4_kv4_release(int32_t *table, int64_t table_stride, int32_t b, int32_t width, int32_t *lens, int32_t *free_pages,
                           int32_t *free_count, int64_t pages, int32_t page, const int32_t *keep, int32_t window,
                           int32_t sinks, int32_t shared, void *workspace, size_t ws_bytes, void *stream) {
    if (!table || !lens || !free_pages || !free_count) return FP4_ERR_NULL;
    if (!tables_ok(b, width, table_stride, page, pages) || window < 0 || sinks < 0 || shared < 0) return FP4_ERR_SHAPE;
    const size_t need = pages_release_ws_bytes(b, width);
    if (need && !workspace) return FP4_ERR_NULL;
    if (ws_bytes < need) return FP4_ERR_WORKSPACE;
    if (!al(table, 4) || !al(lens, 4) || !al(free_pages, 4) || !al(free_count, 4) || !al(keep, 4) || !al(workspace, 4))
        return FP4_ERR_ALIGN;
    int cus;
    const fp4_status st = device_check(&cus);
    if (st != FP4_OK) return st;
    return hip_status(launch_pages_release(tables_of(table, table_stride, b, width, lens, free_pages, free_count, pages, page),
                                           keep, window, sinks, shared, static_cast<int32_t *>(workspace), hs(stream)));
}

fp4_status fp4_rope_table(float *table, int64_t max_pos, int32_t rot, double base, double factor, void *stream) {
    if (!table) return FP4_ERR_NULL;
    if (max_pos < 1 || rot < 16 || rot > 256 || rot % 16 || max_pos > ((int64_t)1 << 32) / rot || !(base > 0.0) || !(factor > 0.0))
        return FP4_ERR_SHAPE;
    if (!al(table, 16)) return FP4_ERR_ALIGN;
    int cus;
    const fp4_status st = device_check(&cus);
    if (st != FP4_OK) return st;
    return hip_status(launch_rope_table(table, max_pos, rot, base, factor, hs(stream)));
}

fp4_status fp4_qk_norm_rope(const void *q, int64_t q_token_stride, int64_t q_head_stride, int32_t hq, const void *k,
                            int64_t k_token_stride, int64_t k_head_stride, int32_t hkv, int64_t n, int32_t d, int32_t dtype,
                            const void *q_weight, const void *k_weight, int32_t w_dtype, float eps, const int32_t *positions,
                            const float *table, int64_t max_pos, int32_t rot, int32_t interleaved, void *q_out, void *k_out,
                            void *stream) {
    if (!q || !q_out || (hkv > 0 && (!k || !k_out))) return FP4_ERR_NULL;
    fp4_status st = rows_check(n, hq, hkv, d, dtype, w_dtype, q_weight, k_weight, eps, positions, table, max_pos, rot);
    if (st != FP4_OK) return st;
    const unsigned es = size_of(dtype);
    if (!al(q, es) || !al(k, es) || !al(q_out, es) || !al(k_out, es)) return FP4_ERR_ALIGN;
    int cus;
    st = device_check(&cus);
    if (st != FP4_OK) return st;
    return hip_status(launch_norm_rope(rows_of(q, q_token_stride, q_head_stride, hq, k, k_token_stride, k_head_stride, hkv, n, d,
                                               dtype, q_weight, k_weight, w_dtype, eps, positions, table, max_pos, rot,
                                               interleaved), q_out, k_out, hs(stream)));
}

fp4_status fp4_kv4_norm_rope(uint8_t *cache, int64_t pages, int32_t page, const void *q, int64_t q_token_stride,
                             int64_t q_head_stride, int32_t hq, const void *k, int64_t k_token_stride, int64_t k_head_stride,
                             const void *v, int64_t v_token_stride, int64_t v_head_stride, int32_t hkv, int64_t n, int32_t d,
                             int32_t dtype, const void *slots, int32_t slot_bytes, const void *q_weight, const void *k_weight,
                             int32_t w_dtype, float eps, const int32_t *positions, const float *table, int64_t max_pos,
                             int32_t rot, int32_t interleaved, void *q_out, void *stream) {
    if (!cache || !q || !k || !v || !slots || !q_out) return FP4_ERR_NULL;
    if (slot_bytes != 4 && slot_bytes != 8) return FP4_ERR_DTYPE;
    if (!fp4_kv4_cache_bytes(pages, page, hkv, d)) return FP4_ERR_SHAPE;
    fp4_status st = rows_check(n, hq, hkv, d, dtype, w_dtype, q_weight, k_weight, eps, positions, table, max_pos, rot);
    if (st != FP4_OK) return st;
    const unsigned es = size_of(dtype);
    if (!al(cache, 16) || !al(q, es) || !al(k, es) || !al(v, es) || !al(q_out, es) || !al(slots, (unsigned)slot_bytes))
        return FP4_ERR_ALIGN;
    int cus;
    st = device_check(&cus);
    if (st != FP4_OK) return st;
    Kv4Geom g;
    g.pages = pages;
    g.page_log2 = __builtin_ctz((unsigned)page);
    g.hkv = hkv;
    g.d = d;
    return hip_status(launch_norm_rope_kv4(
        rows_of(q, q_token_stride, q_head_stride, hq, k, k_token_stride, k_head_stride, hkv, n, d, dtype, q_weight, k_weight,
                w_dtype, eps, positions, table, max_pos, rot, interleaved),
        HeadRows{v, v_token_stride, v_head_stride, hkv, nullptr}, q_out, cache, g, slots, slot_bytes == 8, hs(stream)));
}

size_t fp4_qk_norm_rope_backward_workspace_bytes(int32_t d) {
    return d < 32 || d > 256 || d % 8 ? 0 : norm_rope_bwd_ws_bytes(d);
}

fp4_status fp4_qk_norm_rope_backward(const void *dq, int64_t dq_token_stride, int64_t dq_head_stride, const void *dk,
                                     int64_t dk_token_stride, int64_t dk_head_stride, const void *q, int64_t q_token_stride,
                                     int64_t q_head_stride, int32_t hq, const void *k, int64_t k_token_stride,
                                     int64_t k_head_stride, int32_t hkv, int64_t n, int32_t d, int32_t dtype,
                                     const void *q_weight, const void *k_weight, int32_t w_dtype, float eps,
                                     const int32_t *positions, const float *table, int64_t max_pos, int32_t rot,
                                     int32_t interleaved, void *q_grad, int64_t qg_token_stride, int64_t qg_head_stride,
                                     void *k_grad, int64_t kg_token_stride, int64_t kg_head_stride, float *q_weight_grad,
                                     float *k_weight_grad, void *workspace, size_t ws_bytes, void *stream) {
    if (!dq || !q || !q_grad || (hkv > 0 && (!dk || !k || !k_grad))) return FP4_ERR_NULL;
    fp4_status st = rows_check(n, hq, hkv, d, dtype, w_dtype, q_weight, k_weight, eps, positions, table, max_pos, rot);
    if (st != FP4_OK) return st;
    if ((q_weight_grad || k_weight_grad) && eps < 0.0f) return FP4_ERR_SHAPE;
    if (k_weight_grad && hkv == 0) return FP4_ERR_SHAPE;
    const size_t need = q_weight_grad || k_weight_grad ? norm_rope_bwd_ws_bytes(d) : 0;
    if (need && !workspace) return FP4_ERR_NULL;
    if (ws_bytes < need) return FP4_ERR_WORKSPACE;
    const unsigned es = size_of(dtype);
    if (!al(dq, es) || !al(dk, es) || !al(q, es) || !al(k, es) || !al(q_grad, es) || !al(k_grad, es) || !al(q_weight_grad, 4) ||
        !al(k_weight_grad, 4) || !al(workspace, 4))
        return FP4_ERR_ALIGN;
    int cus;
    st = device_check(&cus);
    if (st != FP4_OK) return st;
    RopeGrads g;
    g.dq = HeadRows{dq, dq_token_stride, dq_head_stride, hq, nullptr};
    g.dk = HeadRows{dk, dk_token_stride, dk_head_stride, hkv, nullptr};
    g.dxq = q_grad;
    g.dxk = k_grad;
    g.dxq_ts = qg_token_stride;
    g.dxq_hs = qg_head_stride;
    g.dxk_ts = kg_token_stride;
    g.dxk_hs = kg_head_stride;
    g.dwq = q_weight_grad;
    g.dwk = k_weight_grad;
    return hip_status(launch_norm_rope_bwd(rows_of(q, q_token_stride, q_head_stride, hq, k, k_token_stride, k_head_stride, hkv, n,
                                                   d, dtype, q_weight, k_weight, w_dtype, eps, positions, table, max_pos, rot,
                                                   interleaved), g, static_cast<float *>(workspace), hs(stream)));
}

}  // extern "C"
