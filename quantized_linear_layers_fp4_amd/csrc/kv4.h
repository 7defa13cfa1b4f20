// The 4-bit paged key/value cache: its layout and launchers (internal; the C ABI is
// include/fp4lin.h).
//
// One contiguous region per (page, key/value head), so that a tile of tokens of one head is one
// run of memory.  With P tokens a page and head size D:
//   K codes   P x D/2 bytes, token-major: the matrix instruction's own FP4 operand (a lane takes a
//             token's 16 bytes of one group of 32)
//   K scales  D/32 x P E8M0 bytes, group-major
//   V codes   eight tokens interleaved by dwords (8 columns of one token): dword n of token t at
//             ((t / 8) * (D / 8) + n) * 32 + (t % 8) * 4, so a lane that owns 8 columns reads the
//             eight tokens of one contraction step as 32 contiguous bytes
//   V scales  D/32 x P E8M0 bytes, group-major: eight tokens' bytes of a group are 8 bytes
// A token whose key or value holds a NaN or an infinity (in that head) has K scale bytes 255 and
// all codes and V scales 0: its scores are NaN where it is visible, and it adds nothing elsewhere.
// Other scale bytes are 0 .. 252, under which every code is finite.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace fp4 {

struct Kv4Geom {
    int64_t pages;   // pages in the cache
    int page_log2;   // tokens a page
    int hkv, d;
    __host__ __device__ int64_t region() const { return ((int64_t)1 << page_log2) * (d + d / 16); }
    __host__ __device__ int64_t ks_off() const { return ((int64_t)1 << page_log2) * (d / 2); }
    __host__ __device__ int64_t v_off() const { return ((int64_t)1 << page_log2) * (d / 2 + d / 32); }
    __host__ __device__ int64_t vs_off() const { return ((int64_t)1 << page_log2) * (d + d / 32); }
};

struct Kv4Attn {
    const uint16_t *q;          // bf16, last dimension contiguous
    int64_t q_ts, q_hs;         // its token and head strides (elements)
    const int32_t *q_start;     // b + 1 offsets, or NULL: one query a sequence
    const int32_t *lens;        // b
    const int32_t *pages;       // b rows, page_rs apart, `width` entries each
    int64_t page_rs;
    int width;
    const uint8_t *cache;
    Kv4Geom geo;
    int b, nq, hq, max_q, window;
    int sinks;                  // with a window: first tokens that stay visible
    int shared;                 // first pages that all rows have in common (launch_kv4_attn_shared)
    float scale;                // of the scores
    uint16_t *o;                // nq x hq x d bf16
    float *lse;                 // nq x hq, or NULL
    uint8_t *ws;
};

hipError_t launch_kv4_write(uint8_t *cache, const Kv4Geom &g, const void *K, const void *V, int dt, int64_t n,
                            int64_t k_ts, int64_t k_hs, int64_t v_ts, int64_t v_hs, const void *slots, bool slots64,
                            hipStream_t s);
hipError_t launch_kv4_read(const uint8_t *cache, const Kv4Geom &g, const void *slots, bool slots64, int64_t n, void *K,
                           void *V, int dt, hipStream_t s);
size_t kv4_attn_ws_bytes(int b, int max_q, int hq, const Kv4Geom &g, int width);
hipError_t launch_kv4_attn(const Kv4Attn &a, hipStream_t s);
int kv4_attn_shared_parts(int64_t nq, int b, int max_q, int hq, const Kv4Geom &g, int width, int shared);
size_t kv4_attn_shared_ws_bytes(int64_t nq, int b, int max_q, int hq, const Kv4Geom &g, int width, int shared);
hipError_t launch_kv4_attn_shared(const Kv4Attn &a, hipStream_t s);

}  // namespace fp4
