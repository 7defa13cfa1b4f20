// Writing keys and values into the 4-bit paged cache, and reading them back (layout: kv4.h).
//
// Groups of 32 values along the head take one E8M0 scale: e is the smallest exponent of -127 .. 125 with
// max|x| <= 7 * 2^e (125 if there is none), and codes are the nearest E2M1 values of x * 2^-e, ties to even, saturating at
// 6: a group's maximum in (6, 7] * 2^e loses at most a seventh, which is no more than the half step
// of 1 that rounding costs there anyway, and the group's other values keep the finer scale.  Both
// kernels move each byte once and are bound by memory; 8 values a lane and token, D/8 lanes a (token, head).
#include "block8.h"
#include "kv4.h"

namespace fp4 {

template <bool S64>
__device__ __forceinline__ int64_t slot_at(const void *slots, int64_t i) {
    if constexpr (S64) return static_cast<const int64_t *>(slots)[i];
    else return static_cast<const int32_t *>(slots)[i];
}

// A lane takes 8 columns of U consecutive tokens of one head: U = 4 in long calls, so that the values of
// four tokens are on their way at once, and tokens that lie side by side in the cache (a prompt's) have
// their four V dwords stored and read as one 16-byte piece; U = 1 in short ones.
template <int U, bool S64>
__device__ __forceinline__ bool slots_at(const void *slots, int64_t t, int64_t n, int64_t total, int64_t (&slot)[U],
                                         bool (&ok)[U]) {
    bool run = true;
#pragma unroll
    for (int u = 0; u < U; ++u) {
        slot[u] = slot_at<S64>(slots, min(t + u, n - 1));
        ok[u] = t + u < n && slot[u] >= 0 && slot[u] < total;
        run = run && ok[u] && slot[u] == slot[0] + u;
    }
    return U == 4 && run && (slot[0] & 3) == 0;  // four tokens of one group of eight
}

template <int DT, int D, bool S64, int U>
__global__ __launch_bounds__(256) void k_kv4_write(uint8_t *__restrict__ cache, Kv4Geom g, const void *__restrict__ K,
                                                   const void *__restrict__ V, int64_t n, int64_t k_ts, int64_t k_hs,
                                                   int64_t v_ts, int64_t v_hs, const void *__restrict__ slots) {
    constexpr int L = D / 8;  // lanes a token
    const int lane = threadIdx.x % L;
    // U = 4: two lane groups take eight tokens of a head (whole lines of V), the next two the next head's, so a
    // wave reads longer pieces of a token
    const int64_t item = (int64_t)blockIdx.x * (256 / L) + threadIdx.x / L;
    const int head = U == 1 ? blockIdx.x % g.hkv : (int)((item >> 1) % g.hkv);
    const int64_t t = (U == 1 ? (int64_t)(blockIdx.x / g.hkv) * (256 / L) + threadIdx.x / L : (item >> 1) / g.hkv * 2 + (item & 1)) * U;
    // tokens past the last stay for the shuffles, with its data, and are not stored
    float k[U][8], v[U][8];
    int64_t slot[U];
    bool ok[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int64_t tc = min(t + u, n - 1);
        load8_any<DT>(K, tc * k_ts + head * k_hs + lane * 8, 8, k[u]);
        load8_any<DT>(V, tc * v_ts + head * v_hs + lane * 8, 8, v[u]);
    }
    const bool run = slots_at<U, S64>(slots, t, n, g.pages << g.page_log2, slot, ok);
    uint32_t ck[U], cv[U], ek[U], ev[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        uint32_t mk = amax8(k[u]), mv = amax8(v[u]);
#pragma unroll
        for (int off = 2; off > 0; off >>= 1) {
            mk = max(mk, (uint32_t)__shfl_xor((int)mk, off, 64));
            mv = max(mv, (uint32_t)__shfl_xor((int)mv, off, 64));
        }
        const uint64_t bad_all = __builtin_amdgcn_ballot_w64(max(mk, mv) >= 0x7F800000u);
        const bool bad = ((bad_all >> ((threadIdx.x & 63) / L * L)) & ((1ull << L) - 1)) != 0;
        // at most 125: 6 * 2^125 is the largest code under any scale byte, so whatever a token's bytes are, of two
        // tokens written at once even, they stay finite where the token is masked (0 * inf would be NaN)
        ek[u] = min(e8m0_of(mk, 2), 252u);
        ev[u] = min(e8m0_of(mv, 2), 252u);
        const float fk = e8m0_inv(ek[u]), fv = e8m0_inv(ev[u]);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            k[u][i] *= fk;
            v[u][i] *= fv;
        }
        ck[u] = bad ? 0u : e2m1_pack8(k[u]);
        cv[u] = bad ? 0u : e2m1_pack8(v[u]);
        ek[u] = bad ? 255u : ek[u];
        ev[u] = bad ? 0u : ev[u];
    }
    const int P = 1 << g.page_log2;
    if (run) {
        const int tok = (int)(slot[0] & (P - 1));
        uint8_t *base = cache + ((slot[0] >> g.page_log2) * g.hkv + head) * g.region();
#pragma unroll
        for (int u = 0; u < U; ++u)
            __builtin_nontemporal_store(ck[u], reinterpret_cast<uint32_t *>(base + (tok + u) * (D / 2) + lane * 4));
        __builtin_nontemporal_store(u32x4{cv[0], cv[U > 1 ? 1 : 0], cv[U > 2 ? 2 : 0], cv[U > 3 ? 3 : 0]},
                                    reinterpret_cast<u32x4 *>(base + g.v_off() + ((tok >> 3) * L + lane) * 32 + (tok & 4) * 4));
        if ((lane & 3) == 0) {
            uint32_t wk = 0, wv = 0;
#pragma unroll
            for (int u = 0; u < U; ++u) {
                wk |= ek[u] << (8 * u);
                wv |= ev[u] << (8 * u);
            }
            *reinterpret_cast<uint32_t *>(base + g.ks_off() + (lane >> 2) * P + tok) = wk;
            *reinterpret_cast<uint32_t *>(base + g.vs_off() + (lane >> 2) * P + tok) = wv;
        }
        return;
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        if (!ok[u]) continue;
        const int tok = (int)(slot[u] & (P - 1));
        uint8_t *base = cache + ((slot[u] >> g.page_log2) * g.hkv + head) * g.region();
        *reinterpret_cast<uint32_t *>(base + tok * (D / 2) + lane * 4) = ck[u];
        *reinterpret_cast<uint32_t *>(base + g.v_off() + ((tok >> 3) * L + lane) * 32 + (tok & 7) * 4) = cv[u];
        if ((lane & 3) == 0) {
            base[g.ks_off() + (lane >> 2) * P + tok] = (uint8_t)ek[u];
            base[g.vs_off() + (lane >> 2) * P + tok] = (uint8_t)ev[u];
        }
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
        __builtin_nontemporal_store(
            u32x4{bf16_pack2(v[0], v[1]), bf16_pack2(v[2], v[3]), bf16_pack2(v[4], v[5]), bf16_pack2(v[6], v[7])},
            reinterpret_cast<u32x4 *>(static_cast<uint16_t *>(Y) + elem));
    } else {
        v4f *y = reinterpret_cast<v4f *>(static_cast<float *>(Y) + elem);
        __builtin_nontemporal_store(v4f{v[0], v[1], v[2], v[3]}, y);
        __builtin_nontemporal_store(v4f{v[4], v[5], v[6], v[7]}, y + 1);
    }
}

template <int DT, int D, bool S64, int U>
__global__ __launch_bounds__(256) void k_kv4_read(const uint8_t *__restrict__ cache, Kv4Geom g,
                                                  const void *__restrict__ slots, int64_t n, void *__restrict__ K,
                                                  void *__restrict__ V) {
    constexpr int L = D / 8;
    const int head = blockIdx.x % g.hkv, lane = threadIdx.x % L;
    const int64_t t = ((int64_t)(blockIdx.x / g.hkv) * (256 / L) + threadIdx.x / L) * U;
    if (t >= n) return;
    int64_t slot[U];
    bool ok[U];
    const bool run = slots_at<U, S64>(slots, t, n, g.pages << g.page_log2, slot, ok);
    const int P = 1 << g.page_log2;
    uint32_t ck[U], cv[U], ek[U], ev[U];
    if (run) {
        const int tok = (int)(slot[0] & (P - 1));
        const uint8_t *base = cache + ((slot[0] >> g.page_log2) * g.hkv + head) * g.region();
#pragma unroll
        for (int u = 0; u < U; ++u) ck[u] = *reinterpret_cast<const uint32_t *>(base + (tok + u) * (D / 2) + lane * 4);
        const uint4 w = *reinterpret_cast<const uint4 *>(base + g.v_off() + ((tok >> 3) * L + lane) * 32 + (tok & 4) * 4);
        const uint32_t wk = *reinterpret_cast<const uint32_t *>(base + g.ks_off() + (lane >> 2) * P + tok);
        const uint32_t wv = *reinterpret_cast<const uint32_t *>(base + g.vs_off() + (lane >> 2) * P + tok);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            cv[u] = u == 0 ? w.x : u == 1 ? w.y : u == 2 ? w.z : w.w;
            ek[u] = (wk >> (8 * u)) & 255u;
            ev[u] = ek[u] == 255u ? 255u : (wv >> (8 * u)) & 255u;
        }
    } else {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            ck[u] = cv[u] = ek[u] = ev[u] = 0;
            if (!ok[u]) continue;
            const int tok = (int)(slot[u] & (P - 1));
            const uint8_t *base = cache + ((slot[u] >> g.page_log2) * g.hkv + head) * g.region();
            ck[u] = *reinterpret_cast<const uint32_t *>(base + tok * (D / 2) + lane * 4);
            cv[u] = *reinterpret_cast<const uint32_t *>(base + g.v_off() + ((tok >> 3) * L + lane) * 32 + (tok & 7) * 4);
            ek[u] = base[g.ks_off() + (lane >> 2) * P + tok];
            ev[u] = ek[u] == 255u ? 255u : base[g.vs_off() + (lane >> 2) * P + tok];
        }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        if (t + u >= n) break;
        float k[8], v[8];
        e2m1_unpack8(ck[u], e8m0_value(ek[u]), k);
        e2m1_unpack8(cv[u], e8m0_value(ev[u]), v);
        const int64_t out = ((t + u) * g.hkv + head) * D + lane * 8;
        store8<DT>(K, out, k);
        store8<DT>(V, out, v);
    }
}

// U = 4 from two workgroups a CU on (of 256): measured on 16384 tokens of 32 heads, U = 1 | 4: write 82 | 78 us,
// read 89 | 67 us; with U = 4's stores past the caches, which leaves them to the inputs, write 51 us
#define KV4_LAUNCH(KERNEL, DT, D, S, U, ...)                                                              \
    do {                                                                                                  \
        const int per = 256 / (D / 8) * U;                                                                \
        hipLaunchKernelGGL((KERNEL<DT, D, S, U>), dim3((unsigned)((n + per - 1) / per * g.hkv)), dim3(256), 0, s, \
                           __VA_ARGS__);                                                                  \
    } while (0)
#define KV4_DISPATCH(KERNEL, DT, ...)                                                                     \
    do {                                                                                                  \
        const bool many = n * g.hkv >= 512 * 4 * (2048 / g.d);                                            \
        if (g.d == 128) {                                                                                 \
            if (many && slots64) KV4_LAUNCH(KERNEL, DT, 128, true, 4, __VA_ARGS__);                       \
            else if (many) KV4_LAUNCH(KERNEL, DT, 128, false, 4, __VA_ARGS__);                            \
            else if (slots64) KV4_LAUNCH(KERNEL, DT, 128, true, 1, __VA_ARGS__);                          \
            else KV4_LAUNCH(KERNEL, DT, 128, false, 1, __VA_ARGS__);                                      \
        } else {                                                                                          \
            if (many && slots64) KV4_LAUNCH(KERNEL, DT, 64, true, 4, __VA_ARGS__);                        \
            else if (many) KV4_LAUNCH(KERNEL, DT, 64, false, 4, __VA_ARGS__);                             \
            else if (slots64) KV4_LAUNCH(KERNEL, DT, 64, true, 1, __VA_ARGS__);                           \
            else KV4_LAUNCH(KERNEL, DT, 64, false, 1, __VA_ARGS__);                                       \
        }                                                                                                 \
        return hipGetLastError();                                                                         \
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
