// What a step over the 4-bit cache needs beside its projections and attention: page tables and slots, and the norm of
// queries and keys with the rotation of positions (internal; the C ABI is include/fp4lin.h).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "kv4.h"

namespace fp4 {

// Page tables of b sequences: rows table_rs apart of `width` entries, tokens of each, and a stack of free pages.
struct PageTables {
    int32_t *table;
    int64_t table_rs;
    int32_t width;
    int32_t *lens;
    int32_t b;
    int32_t *free, *count;   // `pages` entries, of which the first *count are free; the last of these is taken first
    int32_t pages;
    int page_log2;
};

size_t pages_extend_ws_bytes(int b, int64_t n);
hipError_t launch_pages_extend(const PageTables &t, const int32_t *add, int64_t n, int64_t *slots, int32_t *positions,
                               int32_t *q_start, int32_t *ws, hipStream_t s);
size_t pages_release_ws_bytes(int b, int width);
hipError_t launch_pages_release(const PageTables &t, const int32_t *keep, int window, int sinks, int shared, int32_t *ws,
                                hipStream_t s);

// Heads of one tensor: rows of d values, strides in elements.
struct HeadRows {
    const void *x;
    int64_t ts, hs;
    int heads;
    const void *w;           // d weights, or NULL: ones
};

struct NormRope {
    HeadRows q, k;
    int dt, w_dt, d;
    int64_t n;
    const int32_t *positions;
    const float *table;      // max_pos rows of rot / 2 cosines and rot / 2 sines
    int64_t max_pos;
    int rot;
    bool interleaved, norm;
    float eps;
    double inv_d;            // 1 / d
};

hipError_t launch_rope_table(float *table, int64_t max_pos, int rot, double base, double factor, hipStream_t s);
hipError_t launch_norm_rope(const NormRope &a, void *qo, void *ko, hipStream_t s);
// K and V into the cache instead (v's d and dtype are k's; its rows are not changed)
hipError_t launch_norm_rope_kv4(const NormRope &a, const HeadRows &v, void *qo, uint8_t *cache, const Kv4Geom &g,
                                const void *slots, bool slots64, hipStream_t s);
size_t norm_rope_bwd_ws_bytes(int d);
// a.q and a.k are the forward's inputs; dq, dk its outputs' gradients; dxq, dxk (strides as given) the inputs'
struct RopeGrads {
    HeadRows dq, dk;
    void *dxq, *dxk;
    int64_t dxq_ts, dxq_hs, dxk_ts, dxk_hs;
    float *dwq, *dwk;        // or NULL
};
hipError_t launch_norm_rope_bwd(const NormRope &a, const RopeGrads &g, float *ws, hipStream_t s);

}  // namespace fp4
