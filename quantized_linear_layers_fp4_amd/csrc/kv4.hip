// Writing keys and values into the 4-bit paged cache, and reading them back (layout: kv4.h).
//
// Groups of 32 values along the head take one E8M0 scale: e is the smallest exponent >= -127 with
// max|x| <= 7 * 2^e, and codes are the nearest E2M1 values of x * 2^-e, ties to even, saturating at
// 6: a group's maximum in (6, 7] * 2^e loses at most a seventh, which is no more than the half step
// of 1 that rounding costs there anyway, and the group's other values keep the finer scale.  Both
// kernels move each byte once and are bound by memory; 8 values a lane, D/8 lanes a (token, head).
#include "block8.h"
#include "kv4.h"

namespace fp4 {

template <bool S64>
__device__ __forceinline__ int64_t slot_at(const void *slots, int64_t i) {
    if constexpr (S64) return static_cast<const int64_t *>(slots)[i];
    else return static_cast<const int32_t *>(slots)[i];
}

// A workgroup takes 16 (D = 128) or 32 (D = 64) consecutive tokens of one head.
template <int DT, int D, bool S64>
__global__ __launch_bounds__(256) void k_kv4_write(uint8_t *__restrict__ cache, Kv4Geom g, const void *__restrict__ K,
                                                   const void *__restrict__ V, int64_t n, int64_t k_ts, int64_t k_hs,
                                                   int64_t v_ts, int64_t v_hs, const void *__restrict__ slots) {
    constexpr int L = D / 8;  // lanes a token
    const int head = blockIdx.x % g.hkv, lane = threadIdx.x % L;
    const int64_t t = (int64_t)(blockIdx.x / g.hkv) * (256 / L) + threadIdx.x / L;
    // lanes past the last token stay for the shuffles, with its data, and store nothing
    const int64_t tc = min(t, n - 1);
    const int64_t slot = slot_at<S64>(slots, tc);
    float k[8], v[8];
    load8_any<DT>(K, tc * k_ts + head * k_hs + lane * 8, 8, k);
    load8_any<DT>(V, tc * v_ts + head * v_hs + lane * 8, 8, v);
    uint32_t mk = amax8(k), mv = amax8(v);
#pragma unroll
    for (int off = 2; off > 0; off >>= 1) {
        mk = max(mk, (uint32_t)__shfl_xor((int)mk, off, 64));
        mv = max(mv, (uint32_t)__shfl_xor((int)mv, off, 64));
    }
    const uint64_t bad_all = __builtin_amdgcn_ballot_w64(max(mk, mv) >= 0x7F800000u);
    const bool bad = ((bad_all >> ((threadIdx.x & 63) / L * L)) & ((1ull << L) - 1)) != 0;
    if (t >= n || slot < 0 || slot >= (g.pages << g.page_log2)) return;
    uint32_t ek = e8m0_of(mk, 2), ev = e8m0_of(mv, 2), ck = 0, cv = 0;
    if (!bad) {
        const float fk = e8m0_inv(ek), fv = e8m0_inv(ev);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            k[i] *= fk;
            v[i] *= fv;
        }
        // 4 * 2^126 is no fp32 number: there 3 is the largest code, so that whatever is held stays
        // finite where its token is masked (0 * inf would be NaN)
        if (ek == 253u) {
#pragma unroll
            for (int i = 0; i < 8; ++i) k[i] = fminf(fmaxf(k[i], -3.0f), 3.0f);
        }
        if (ev == 253u) {
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = fminf(fmaxf(v[i], -3.0f), 3.0f);
        }
        ck = e2m1_pack8(k);
        cv = e2m1_pack8(v);
    } else {
        ek = 255u;
        ev = 0u;
    }
    const int P = 1 << g.page_log2, tok = (int)(slot & (P - 1));
    uint8_t *base = cache + ((slot >> g.page_log2) * g.hkv + head) * g.region();
    *reinterpret_cast<uint32_t *>(base + tok * (D / 2) + lane * 4) = ck;
    *reinterpret_cast<uint32_t *>(base + g.v_off() + ((tok >> 3) * L + lane) * 32 + (tok & 7) * 4) = cv;
    if ((lane & 3) == 0) {
        base[g.ks_off() + (lane >> 2) * P + tok] = (uint8_t)ek;
        base[g.vs_off() + (lane >> 2) * P + tok] = (uint8_t)ev;
    }
}

// Eight E2M1 codes -> fp32 values times s (a power of two; NaN poisons all).
__device__ __forceinline__ void e2m1_unpack8(uint32_t w, float s, float v[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        // magnitude bits e e m: 0, 0.5, then (1 + m / 2) * 2^(e - 1); as a float: e m << 22 plus a
        // rebias of 126 exponents, 0.5 being the one subnormal
        const uint32_t c = (w >> (4 * i)) & 15u, em = c & 7u;
        const float mag = em < 2 ? 0.5f * (float)em : __uint_as_float((em << 22) + (126u << 23));
        v[i] = ((c & 8u) ? -mag : mag) * s;
    }
}

template <int DT>
__device__ __forceinline__ void store8(void *Y, int64_t elem, const float v[8]) {
    if constexpr (DT == DT_BF16) {
        *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(Y) + elem) = make_uint4(
            bf16_pack2(v[0], v[1]), bf16_pack2(v[2], v[3]), bf16_pack2(v[4], v[5]), bf16_pack2(v[6], v[7]));
    } else {
        float4 *y = reinterpret_cast<float4 *>(static_cast<float *>(Y) + elem);
        y[0] = make_float4(v[0], v[1], v[2], v[3]);
        y[1] = make_float4(v[4], v[5], v[6], v[7]);
    }
}

template <int DT, int D, bool S64>
__global__ __launch_bounds__(256) void k_kv4_read(const uint8_t *__restrict__ cache, Kv4Geom g,
                                                  const void *__restrict__ slots, int64_t n, void *__restrict__ K,
                                                  void *__restrict__ V) {
    constexpr int L = D / 8;
    const int head = blockIdx.x % g.hkv, lane = threadIdx.x % L;
    const int64_t t = (int64_t)(blockIdx.x / g.hkv) * (256 / L) + threadIdx.x / L;
    if (t >= n) return;
    const int64_t slot = slot_at<S64>(slots, t);
    uint32_t ck = 0, cv = 0, ek = 0, ev = 0;
    if (slot >= 0 && slot < (g.pages << g.page_log2)) {
        const int P = 1 << g.page_log2, tok = (int)(slot & (P - 1));
        const uint8_t *base = cache + ((slot >> g.page_log2) * g.hkv + head) * g.region();
        ck = *reinterpret_cast<const uint32_t *>(base + tok * (D / 2) + lane * 4);
        cv = *reinterpret_cast<const uint32_t *>(base + g.v_off() + ((tok >> 3) * L + lane) * 32 + (tok & 7) * 4);
        ek = base[g.ks_off() + (lane >> 2) * P + tok];
        ev = ek == 255u ? 255u : base[g.vs_off() + (lane >> 2) * P + tok];
    }
    float k[8], v[8];
    e2m1_unpack8(ck, e8m0_value(ek), k);
    e2m1_unpack8(cv, e8m0_value(ev), v);
    const int64_t out = (t * g.hkv + head) * D + lane * 8;
    store8<DT>(K, out, k);
    store8<DT>(V, out, v);
}

#define KV4_DISPATCH(KERNEL, DT, ...)                                                                        \
    do {                                                                                                     \
        const int per = 256 / (g.d / 8);                                                                     \
        const dim3 grid((unsigned)((n + per - 1) / per * g.hkv)), blk(256);                                  \
        if (g.d == 128) {                                                                                    \
            if (slots64) hipLaunchKernelGGL((KERNEL<DT, 128, true>), grid, blk, 0, s, __VA_ARGS__);          \
            else hipLaunchKernelGGL((KERNEL<DT, 128, false>), grid, blk, 0, s, __VA_ARGS__);                 \
        } else {                                                                                             \
            if (slots64) hipLaunchKernelGGL((KERNEL<DT, 64, true>), grid, blk, 0, s, __VA_ARGS__);           \
            else hipLaunchKernelGGL((KERNEL<DT, 64, false>), grid, blk, 0, s, __VA_ARGS__);                  \
        }                                                                                                    \
        return hipGetLastError();                                                                            \
    } while (0)

hipError_t launch_kv4_write(uint8_t *cache, const Kv4Geom &g, const void *K, const void *V, int dt, int64_t n,
                            int64_t k_ts, int64_t k_hs, int64_t v_ts, int64_t v_hs, const void *slots, bool slots64,
                            hipStream_t s) {
    if (dt == DT_BF16) KV4_DISPATCH(k_kv4_write, DT_BF16, cache, g, K, V, n, k_ts, k_hs, v_ts, v_hs, slots);
    KV4_DISPATCH(k_kv4_write, DT_F32, cache, g, K, V, n, k_ts, k_hs, v_ts, v_hs, slots);
}

hipError_t launch_kv4_read(const uint8_t *cache, const Kv4Geom &g, const void *slots, bool slots64, int64_t n, void *K,
                           void *V, int dt, hipStream_t s) {
    if (dt == DT_BF16) KV4_DISPATCH(k_kv4_read, DT_BF16, cache, g, slots, n, K, V);
    KV4_DISPATCH(k_kv4_read, DT_F32, cache, g, slots, n, K, V);
}

}  // namespace fp4
