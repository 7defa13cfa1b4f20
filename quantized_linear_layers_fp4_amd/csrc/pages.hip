// Page tables of a paged cache kept on the GPU: appending tokens and giving pages back (declared in serve.h).
//
// extend: sequence i asks for add_i tokens: with have_i = ceil(len_i / P) and need_i = ceil((len_i + add_i) / P) the
// pages have_i .. need_i - 1 of its row come off the stack, in the order of (i, page).  A sequence that does not fit (its
// row's width, the stack, the n tokens of the call) gets nothing.  What fits is decided by prefix sums over all
// sequences, so the refused are the last ones that ask for a page (or a token), whatever order threads run in.
// release: the pages past a sequence's kept tokens, and those that no later query sees, go back to the stack, so
// that the first of them, in the order of (i, page), is the next to be taken: cutting and appending the same number of
// tokens gives the same table again.
//
// Nothing here is arithmetic or bandwidth: a call is a chain of a few dependent loads, scans and stores, and its time
// that of launches.  So one workgroup does a whole small call; large calls do the scan (extend) or the count (release) in
// one launch and write tokens or entries in a second one from many workgroups.
#include "serve.h"

namespace fp4 {

namespace {

constexpr int NT = 1024;             // threads of a workgroup, and sequences that it holds at once
constexpr int64_t ONE_TOKENS = 8192; // tokens and
constexpr int64_t ONE_ENTRIES = 16384;  // table entries up to which one workgroup does a call
constexpr int RELEASE_WGS = 1024;

// Inclusive sum over the workgroup's threads, and their total; all of them call it.
template <typename T>
__device__ __forceinline__ T block_scan(T x, T *sums, T &total) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
        const T y = __shfl_up(x, off, 64);
        if (lane >= off) x += y;
    }
    __syncthreads();  // the last scan's sums have been read
    if (lane == 63) sums[wave] = x;
    __syncthreads();
    T before = 0;
    total = 0;
#pragma unroll
    for (int w = 0; w < NT / 64; ++w) {
        const T s = sums[w];
        before += w < wave ? s : T(0);
        total += s;
    }
    return x + before;
}

// Two of them at once.
__device__ __forceinline__ void block_scan2(int64_t &x, int64_t &y, int64_t *sums, int64_t &tx, int64_t &ty) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
        const int64_t u = __shfl_up(x, off, 64), v = __shfl_up(y, off, 64);
        if (lane >= off) {
            x += u;
            y += v;
        }
    }
    __syncthreads();
    if (lane == 63) {
        sums[wave] = x;
        sums[NT / 64 + wave] = y;
    }
    __syncthreads();
    tx = ty = 0;
    int64_t bx = 0, by = 0;
#pragma unroll
    for (int w = 0; w < NT / 64; ++w) {
        const int64_t u = sums[w], v = sums[NT / 64 + w];
        bx += w < wave ? u : 0;
        by += w < wave ? v : 0;
        tx += u;
        ty += v;
    }
    x += bx;
    y += by;
}

// The number of entries of the ascending p[0 .. n) that are at most x.
template <typename T>
__device__ __forceinline__ int at_most(const T *p, int n, T x) {
    int lo = 0, hi = n;
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (p[mid] <= x) lo = mid + 1;
        else hi = mid;
    }
    return lo;
}

__device__ __forceinline__ int pages_of(int tokens, int lg) { return (int)(((int64_t)tokens + (1 << lg) - 1) >> lg); }

// Slot of a token at pos of sequence i, whose pages from `have` on are the stack's entries top - excl - (page - have);
// writes the table's entry if the token is a new page's first.
__device__ __forceinline__ int64_t place(const PageTables &t, int i, int pos, int have, int excl, int count) {
    const int k = pos >> t.page_log2, in = pos & ((1 << t.page_log2) - 1);
    int32_t *entry = t.table + i * t.table_rs + k;
    int page;
    if (k < have) page = *entry;
    else {
        page = t.free[count - 1 - (excl + k - have)];
        if (in == 0) *entry = page;
    }
    return (uint32_t)page < (uint32_t)t.pages ? ((int64_t)page << t.page_log2) + in : -1;
}

}  // namespace

// One workgroup: who gets what, the new lengths, the offsets, the stack's new height; and, where `small`, the tokens.
// PACKED: tokens lie one sequence after the other; otherwise token i is sequence i's only one.
template <bool PACKED>
__global__ __launch_bounds__(NT) void k_pages_extend(PageTables t, const int32_t *__restrict__ add, int64_t n,
                                                     int64_t *__restrict__ slots, int32_t *__restrict__ positions,
                                                     int32_t *__restrict__ q_start, int32_t *__restrict__ ws, bool small) {
    __shared__ int64_t sums[2 * NT / 64];
    __shared__ int32_t s_start[NT + 1], s_old[NT], s_excl[NT];
    const int count = min(max(*t.count, 0), t.pages);
    int64_t pages = 0, asked = 0, given = 0, taken = 0;  // sums over the sequences before this turn's
    for (int base = 0; base < t.b; base += NT) {
        const int i = base + threadIdx.x;
        const bool in = i < t.b;
        const int old = in ? max(t.lens[i], 0) : 0;
        int64_t a = in ? (add ? max(add[i], 0) : 1) : 0;
        if constexpr (!PACKED) a = min(a, (int64_t)1);
        bool ok = old + a <= ((int64_t)t.width << t.page_log2);
        const int have = pages_of(old, t.page_log2);
        const int64_t need = ok ? pages_of((int)(old + a), t.page_log2) - have : 0;
        int64_t pi = need, ti = ok ? a : 0, total, tokens;
        block_scan2(pi, ti, sums, total, tokens);
        pi += pages;
        ti += asked;
        bool short_ = in && a > 0 && (!ok || (need > 0 && pi > count) || (PACKED && ti > n));
        if (__syncthreads_or(short_) || asked != given) {  // somebody gets nothing: who, and the sums of what the others get
            ok = ok && (need == 0 || pi <= count);
            a = ok ? a : 0;
            if constexpr (PACKED) {
                ti = asked + block_scan(a, sums, tokens);
                ok = ok && (a == 0 || ti <= n);
                asked += tokens;
                a = ok ? a : 0;
                ti = given + block_scan(a, sums, tokens);
                given += tokens;
            }
            pages += total;
            block_scan(ok ? need : 0, sums, total);
            taken += total;
        } else {
            asked += tokens;
            given += tokens;
            pages += total;
            taken += total;
        }
        const int64_t want = ok ? need : 0;
        const int excl = (int)(pi - want);
        if (in) {
            t.lens[i] = old + (int)a;
            if constexpr (PACKED) {
                if (i == 0) q_start[0] = 0;
                q_start[i + 1] = (int32_t)ti;
                if (!small) {
                    ws[2 + 2 * i] = old;
                    ws[3 + 2 * i] = excl;
                }
            } else {
                slots[i] = a ? place(t, i, old, have, excl, count) : -1;
                positions[i] = a ? old : -1;
            }
        }
        if constexpr (PACKED) {
            if (small) {
                s_start[threadIdx.x + 1] = (int32_t)ti;
                s_old[threadIdx.x] = old;
                s_excl[threadIdx.x] = excl;
            }
        }
    }
    __syncthreads();  // every thread has read the height
    if (threadIdx.x == 0) {
        *t.count = count - (int)taken;
        if (PACKED && !small) ws[0] = count;
    }
    if constexpr (PACKED) {
        if (!small) return;
        if (threadIdx.x == 0) s_start[0] = 0;
        __syncthreads();
        const int end = s_start[t.b];
        for (int64_t j = threadIdx.x; j < n; j += NT) {
            int64_t slot = -1;
            int pos = -1;
            if (j < end) {
                const int i = at_most(s_start + 1, t.b - 1, (int32_t)j);
                pos = s_old[i] + (int)j - s_start[i];
                slot = place(t, i, pos, pages_of(s_old[i], t.page_log2), s_excl[i], count);
            }
            slots[j] = slot;
            positions[j] = pos;
        }
    }
}

// The tokens of a large call, from what k_pages_extend left: ws[0] the stack's old height, then each sequence's old
// length and the pages taken before its own.
__global__ __launch_bounds__(256) void k_pages_tokens(PageTables t, int64_t n, int64_t *__restrict__ slots,
                                                      int32_t *__restrict__ positions, const int32_t *__restrict__ q_start,
                                                      const int32_t *__restrict__ ws) {
    const int64_t j = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (j >= n) return;
    int64_t slot = -1;
    int pos = -1;
    if (j < q_start[t.b]) {
        const int i = at_most(q_start + 1, t.b - 1, (int32_t)j);
        const int old = ws[2 + 2 * i];
        pos = old + (int)j - q_start[i];
        slot = place(t, i, pos, pages_of(old, t.page_log2), ws[3 + 2 * i], ws[0]);
    }
    slots[j] = slot;
    positions[j] = pos;
}

// PHASE 0: one workgroup, all of it.  1: workgroup w counts what its sequences (`per` of them) give back into ws[w], ws[G]
// the stack's height.  2: it pushes them, knowing everybody's counts.
template <int PHASE>
__global__ __launch_bounds__(NT) void k_pages_release(PageTables t, const int32_t *__restrict__ keep, int window, int sinks,
                                                      int shared, int per, int32_t *__restrict__ ws) {
    __shared__ int32_t sums[NT / 64];
    __shared__ int32_t s_end[NT], s_tail[NT], s_mid[NT], s_cut[NT];
    const int first = blockIdx.x * per, mine = min(per, t.b - first);
    // candidates of a sequence: columns [mid, mid + m) that its window has left, then [tail, ...) past its kept tokens
    int old = 0, kept = 0, m = 0, tail = 0, mid = 0, rest = 0;
    if ((int)threadIdx.x < mine) {
        const int i = first + threadIdx.x;
        old = max(t.lens[i], 0);
        kept = keep ? min(max(keep[i], 0), old) : old;
        const int end = min(pages_of(old, t.page_log2), t.width), from = min(pages_of(kept, t.page_log2), t.width);
        tail = max(from, shared);
        rest = max(end - tail, 0);
        if (window) {
            mid = max((int)(((int64_t)sinks + (1 << t.page_log2) - 1) >> t.page_log2), shared);
            const int64_t gone = (int64_t)kept - window + 1;  // tokens before this one are seen by no query from `kept` on
            m = max(min((int)(gone > 0 ? gone >> t.page_log2 : 0), from) - mid, 0);
        }
    }
    int total;
    s_end[threadIdx.x] = block_scan(m + rest, sums, total);
    s_tail[threadIdx.x] = tail;
    s_mid[threadIdx.x] = mid;
    s_cut[threadIdx.x] = m;
    __syncthreads();
    auto entry_of = [&](int c) -> int32_t * {
        const int i = at_most(s_end, mine - 1, c);
        const int at = c - (i ? s_end[i - 1] : 0);
        return t.table + (int64_t)(first + i) * t.table_rs + (at < s_cut[i] ? s_mid[i] + at : s_tail[i] + at - s_cut[i]);
    };
    int height = 0, before = 0, all = 0;  // the stack's; pages that earlier workgroups give; pages that all give
    if constexpr (PHASE != 1) {
        if constexpr (PHASE == 2) {
            const int G = gridDim.x, w = threadIdx.x;
            static_assert(RELEASE_WGS <= NT, "a count a thread");
            const int x = w < G ? ws[w] : 0;
            block_scan(w < (int)blockIdx.x ? x : 0, sums, before);
            block_scan(x, sums, all);
            height = ws[G];
        } else {
            height = min(max(*t.count, 0), t.pages);
        }
    }
    if constexpr (PHASE == 0) {
        if (total <= NT) {  // the usual call: each entry is read once, and one scan says where it goes
            int32_t *e = (int)threadIdx.x < total ? entry_of(threadIdx.x) : nullptr;
            const int page = e ? *e : -1;
            const bool good = (uint32_t)page < (uint32_t)t.pages;
            const int rank = block_scan((int)good, sums, all) - 1;
            const int64_t at = (int64_t)height + all - 1 - rank;
            if (good && at < t.pages) t.free[at] = page;
            if (e) *e = -1;
            if ((int)threadIdx.x < mine) t.lens[first + threadIdx.x] = kept;
            if (threadIdx.x == 0) *t.count = (int)min((int64_t)height + all, (int64_t)t.pages);
            return;
        }
    }
    if constexpr (PHASE != 2) {
        int mycount = 0;
        for (int c = threadIdx.x; c < total; c += NT) mycount += (uint32_t)*entry_of(c) < (uint32_t)t.pages;
        int got;
        block_scan(mycount, sums, got);
        if constexpr (PHASE == 1) {
            if (threadIdx.x == 0) {
                ws[blockIdx.x] = got;
                if (blockIdx.x == 0) ws[gridDim.x] = min(max(*t.count, 0), t.pages);
            }
            return;
        }
        all = got;
    }
    int done = before;
    for (int c0 = 0; c0 < total; c0 += NT) {
        const int c = c0 + threadIdx.x;
        int32_t *e = c < total ? entry_of(c) : nullptr;
        const int page = e ? *e : -1;
        const bool good = (uint32_t)page < (uint32_t)t.pages;
        int got;
        const int rank = done + block_scan((int)good, sums, got) - 1;
        done += got;
        if (good) {
            const int64_t at = (int64_t)height + all - 1 - rank;  // below the stack's end unless a page was in it twice
            if (at < t.pages) t.free[at] = page;
        }
        if (e) *e = -1;
    }
    if ((int)threadIdx.x < mine) t.lens[first + threadIdx.x] = kept;
    if (threadIdx.x == 0 && blockIdx.x == 0) *t.count = (int)min((int64_t)height + all, (int64_t)t.pages);
}

// One launch up to ONE_TOKENS tokens and NT sequences.
static bool extend_small(int b, int64_t n) { return b <= NT && n <= ONE_TOKENS; }
size_t pages_extend_ws_bytes(int b, int64_t n) { return extend_small(b, n) ? 0 : (2 + 2 * (size_t)b) * 4; }

hipError_t launch_pages_extend(const PageTables &t, const int32_t *add, int64_t n, int64_t *slots, int32_t *positions,
                               int32_t *q_start, int32_t *ws, hipStream_t s) {
    const bool small = extend_small(t.b, n);
    if (!q_start) {
        hipLaunchKernelGGL((k_pages_extend<false>), dim3(1), dim3(NT), 0, s, t, add, n, slots, positions, q_start, ws, small);
        return hipGetLastError();
    }
    hipLaunchKernelGGL((k_pages_extend<true>), dim3(1), dim3(NT), 0, s, t, add, n, slots, positions, q_start, ws, small);
    hipError_t e = hipGetLastError();
    if (e == hipSuccess && !small && n > 0) {
        hipLaunchKernelGGL(k_pages_tokens, dim3((unsigned)((n + 255) / 256)), dim3(256), 0, s, t, n, slots, positions,
                           q_start, ws);
        e = hipGetLastError();
    }
    return e;
}

static bool release_small(int b, int width) { return b <= NT && (int64_t)b * width <= ONE_ENTRIES; }
size_t pages_release_ws_bytes(int b, int width) { return release_small(b, width) ? 0 : (RELEASE_WGS + 1) * 4; }

hipError_t launch_pages_release(const PageTables &t, const int32_t *keep, int window, int sinks, int shared, int32_t *ws,
                                hipStream_t s) {
    if (release_small(t.b, t.width)) {
        hipLaunchKernelGGL((k_pages_release<0>), dim3(1), dim3(NT), 0, s, t, keep, window, sinks, shared, t.b, ws);
        return hipGetLastError();
    }
    const int per = (t.b + RELEASE_WGS - 1) / RELEASE_WGS, G = (t.b + per - 1) / per;
    hipLaunchKernelGGL((k_pages_release<1>), dim3(G), dim3(NT), 0, s, t, keep, window, sinks, shared, per, ws);
    hipError_t e = hipGetLastError();
    if (e == hipSuccess) {
        hipLaunchKernelGGL((k_pages_release<2>), dim3(G), dim3(NT), 0, s, t, keep, window, sinks, shared, per, ws);
        e = hipGetLastError();
    }
    return e;
}

}  // namespace fp4
