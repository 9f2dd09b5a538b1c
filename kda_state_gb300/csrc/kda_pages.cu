// Pages of a cache: handing out, forking, freeing, copying, compacting.
//
// refs[page] counts the rows of the page table that hold a page; a page with 0
// is free.  Free pages are handed out lowest number first, found by a scan of
// refs: no free list has to be kept, the result does not depend on the order of
// atomics, and a pool stays dense at its lower end.  Row b holds
// ceil(lens[b] / P) pages; only full pages are ever shared.
//
// The scans are one CTA's work (16 K pages are 64 KB of refs, a few us); the
// page data moves in a launch of its own, HBM-bound, over all layers' pools.
#include "kda_common.cuh"
#include "kda_internal.h"

namespace kda {
namespace {

enum { DEVERR_PAGE_RANGE = 32, DEVERR_PAGES = 64 };

constexpr int SCAN = 1024;             // threads of a scanning CTA
constexpr int PER = 16;                // refs a thread looks at in one step

// Exclusive prefix sum over the CTA; total to every thread.
template <typename T>
__device__ __forceinline__ T cta_scan(T x, T &total) {
    __shared__ T warp_sum[33];
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    T in = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const T y = __shfl_up_sync(~0u, in, o);
        if (lane >= o) in += y;
    }
    __syncthreads();                   // the last call's readers are done
    if (lane == 31) warp_sum[w] = in;
    __syncthreads();
    if (w == 0) {
        const T s = lane < (int)(blockDim.x >> 5) ? warp_sum[lane] : 0;
        T t = s;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const T y = __shfl_up_sync(~0u, t, o);
            if (lane >= o) t += y;
        }
        warp_sum[lane] = t - s;
        if (lane == 31) warp_sum[32] = t;
    }
    __syncthreads();
    total = warp_sum[32];
    return warp_sum[w] + in - x;
}

// refs of pages p0 .. p0 + PER - 1 (p0 a multiple of PER); `past` beyond the last page.
__device__ __forceinline__ void load_refs(const int32_t *refs, int num_pages, int p0, int past, int (&r)[PER]) {
    if (p0 + PER <= num_pages && (reinterpret_cast<uintptr_t>(refs) & 15) == 0) {
#pragma unroll
        for (int i = 0; i < PER; i += 4) {
            const int4 x = *reinterpret_cast<const int4 *>(refs + p0 + i);
            r[i] = x.x, r[i + 1] = x.y, r[i + 2] = x.z, r[i + 3] = x.w;
        }
    } else {
#pragma unroll
        for (int i = 0; i < PER; ++i) r[i] = p0 + i < num_pages ? refs[p0 + i] : past;
    }
}

// Hands out `want` free pages from page `cursor` on, lowest first: take(k, page)
// is called for the k-th, by any thread.  Returns how many there were, and leaves
// the cursor at the step that may have more (the caller has counted those it took
// by then).  Every thread of the CTA calls it.
template <typename Take>
__device__ int hand_out(const int32_t *refs, int num_pages, int &cursor, int want, Take take) {
    int got = 0;
    while (got < want && cursor < num_pages) {
        const int p0 = cursor + (int)threadIdx.x * PER;
        int r[PER];
        int free_here = 0;
        load_refs(refs, num_pages, p0, 1, r);
#pragma unroll
        for (int i = 0; i < PER; ++i) free_here += r[i] == 0;
        int total;
        int k = cta_scan(free_here, total) + got;
#pragma unroll
        for (int i = 0; i < PER; ++i)
            if (r[i] == 0) {
                if (k < want) take(k, p0 + i);
                ++k;
            }
        got += total;
        if (got <= want) cursor += SCAN * PER;
    }
    return min(got, want);
}

// The first i in [0, n) with upto[i] > k.
template <typename T>
__device__ __forceinline__ int which(const T *upto, int n, int k) {
    int lo = 0, hi = n;
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (upto[mid] > k) hi = mid; else lo = mid + 1;
    }
    return lo;
}

__device__ __forceinline__ int pages_of(int tokens, int shift) {
    return (int)(((long long)tokens + (1 << shift) - 1) >> shift);
}

// One holder less of the page that a table's entry names; the entry becomes -1.
__device__ __forceinline__ void let_go(const PageArgs &a, int32_t *entry) {
    const int page = *entry;
    if (page < 0 || page >= a.num_pages) report(a.err, DEVERR_PAGE_RANGE);
    else if (atomicSub(&a.refs[page], 1) <= 0) {           // it was free already
        atomicAdd(&a.refs[page], 1);
        report(a.err, DEVERR_PAGES);
    }
    *entry = -1;
}

__global__ void __launch_bounds__(SCAN) alloc_kernel(const PageArgs a, const int32_t *__restrict__ grow) {
    __shared__ long long upto[SCAN];   // (what 1024 rows ask for may pass 32 bits)
    __shared__ int have_s[SCAN], need_s[SCAN];
    int cursor = 0;
    // Rows that shrink come first: all of them are looked at before any lets go of a page, so that what a row may do
    // does not depend on when another's count went down.  (65536 rows in one go: a bit each of a thread's 64.)
    bool any = false;
    for (int b = threadIdx.x; b < a.B; b += SCAN) any |= grow[b] < 0;
    if (__syncthreads_or(any)) {
        for (int g0 = 0; g0 < a.B; g0 += 64 * SCAN) {
            unsigned long long shrinks = 0;
            for (int i = 0; i < 64; ++i) {
                const int b = g0 + i * SCAN + (int)threadIdx.x;
                if (b >= a.B || grow[b] >= 0) continue;
                const int len = a.lens[b];
                const long long to = (long long)len + grow[b];
                if (to < 0 || (long long)len > ((long long)a.max_pages << a.page_shift)) {
                    report(a.err, DEVERR_SEQLENS);
                    continue;
                }
                if (to & ((1 << a.page_shift) - 1)) {      // its new last page is one it will write to: not a shared one
                    const int page = a.page_table[(size_t)b * a.max_pages + (to >> a.page_shift)];
                    if (page < 0 || page >= a.num_pages) {
                        report(a.err, DEVERR_PAGE_RANGE);
                        continue;
                    }
                    if (a.refs[page] > 1) {
                        report(a.err, DEVERR_PAGES);
                        continue;
                    }
                }
                shrinks |= 1ull << i;
            }
            __syncthreads();
            for (int i = 0; i < 64; ++i) {
                if (!(shrinks >> i & 1)) continue;
                const int b = g0 + i * SCAN + (int)threadIdx.x, len = a.lens[b], to = len + grow[b];
                for (int j = pages_of(to, a.page_shift); j < pages_of(len, a.page_shift); ++j) let_go(a, a.page_table + (size_t)b * a.max_pages + j);
                a.lens[b] = to;
            }
            __syncthreads();
        }
    }
    bool out = false;                  // the pool has run out: later rows that need pages get none
    for (int b0 = 0; b0 < a.B; b0 += SCAN) {
        const int b = b0 + threadIdx.x, n = min(SCAN, a.B - b0);
        int need = 0, have = 0, g = 0;
        bool bad = false;
        if (b < a.B) {
            const int len = a.lens[b];
            g = grow[b];
            const long long to = (long long)len + g;
            bad = g < 0 || len < 0 || to > ((long long)a.max_pages << a.page_shift);
            if (bad) {
                if (g >= 0) report(a.err, DEVERR_SEQLENS);
            } else {
                have = pages_of(len, a.page_shift);
                need = pages_of((int)to, a.page_shift) - have;
            }
        }
        long long total;
        const long long before = cta_scan((long long)need, total);
        upto[threadIdx.x] = before + need;
        have_s[threadIdx.x] = have;
        need_s[threadIdx.x] = need;
        __syncthreads();
        int got = 0;
        if (!out)
            got = hand_out(a.refs, a.num_pages, cursor, (int)min(total, 0x7fffffffLL), [&](int k, int page) {
                const int i = which(upto, n, k);
                a.page_table[(size_t)(b0 + i) * a.max_pages + have_s[i] + k - (int)(upto[i] - need_s[i])] = page;
            });
        if (got < total) out = true;
        __syncthreads();
        if (b < a.B && !bad) {
            int32_t *row = a.page_table + (size_t)b * a.max_pages;
            if (need == 0 || before + need <= got) {
                for (int j = have; j < have + need; ++j) a.refs[row[j]] = 1;
                a.lens[b] += g;
            } else {                   // a row is served whole or not at all
                for (int j = 0; j < need && before + j < got; ++j) row[have + j] = -1;
                report(a.err, DEVERR_PAGES);
            }
        }
        __syncthreads();
    }
}

// Forks: tables and counts here; the partial last pages to copy go to moves[2 i]
// (from) and moves[2 i + 1] (to), -1 where there is none.  While a step's forks are
// made the length of a row forked to holds a negative mark of the first fork to it.
__global__ void __launch_bounds__(SCAN) fork_kernel(const PageArgs a, const int32_t *__restrict__ src,
                                                    const int32_t *__restrict__ dst, int n_forks, int32_t *moves) {
    __shared__ int upto[SCAN], fresh_s[SCAN];
    __shared__ int4 share_s[SCAN];     // of each fork that is made: from row, to row, full pages, pages
    int cursor = 0;
    bool out = false;
    for (int f0 = 0; f0 < n_forks; f0 += SCAN) {
        const int f = f0 + threadIdx.x, n = min(SCAN, n_forks - f0);
        int need = 0, s = -1, d = -1, len = 0, full = 0;
        if (f < n_forks) {
            s = src[f], d = dst[f];
            if (s < 0 || s >= a.B || d < 0 || d >= a.B || s == d) {
                report(a.err, DEVERR_SLOT_RANGE);
                s = -1;
            } else {
                len = a.lens[s];
                if (len < 0 || (long long)len > ((long long)a.max_pages << a.page_shift) || a.lens[d] != 0) {
                    report(a.err, DEVERR_SEQLENS);   // the row forked to has to be empty
                    s = -1;
                }
            }
        }
        __syncthreads();
        if (s >= 0) atomicMin(&a.lens[d], (int)threadIdx.x - SCAN);
        __syncthreads();
        if (s >= 0 && __ldcg(&a.lens[d]) != (int)threadIdx.x - SCAN) {
            report(a.err, DEVERR_SEQLENS);           // another fork to this row comes first
            s = -1;
        }
        const bool mine = s >= 0;
        if (mine) {
            full = len >> a.page_shift;
            need = (len & ((1 << a.page_shift) - 1)) != 0;
        }
        int total;
        const int before = cta_scan(need, total);
        upto[threadIdx.x] = before + need;
        __syncthreads();
        int got = 0;
        if (!out)
            got = hand_out(a.refs, a.num_pages, cursor, total,
                           [&](int k, int page) { fresh_s[which(upto, n, k)] = page; });
        if (got < total) out = true;
        __syncthreads();
        int from = -1, to = -1;
        bool served = mine;
        if (served && need) {
            served = before + need <= got;
            if (!served) report(a.err, DEVERR_PAGES);
            else {
                from = a.page_table[(size_t)s * a.max_pages + full];
                to = fresh_s[threadIdx.x];
                a.refs[to] = 1;
                a.page_table[(size_t)d * a.max_pages + full] = to;
                if (from < 0 || from >= a.num_pages) {
                    report(a.err, DEVERR_PAGE_RANGE);
                    from = to = -1;
                }
            }
        }
        if (f < n_forks) {
            moves[2 * f] = from;
            moves[2 * f + 1] = to;
        }
        share_s[threadIdx.x] = served ? make_int4(s, d, full, full + need) : make_int4(-1, 0, 0, 0);
        __syncthreads();
        // the full pages are shared: a warp copies one row's entries at a time
        for (int i = threadIdx.x >> 5; i < n; i += SCAN / 32) {
            const int4 x = share_s[i];
            if (x.x < 0) continue;
            for (int j = threadIdx.x & 31; j < a.max_pages; j += 32) {
                if (j < x.z) {
                    const int page = a.page_table[(size_t)x.x * a.max_pages + j];
                    a.page_table[(size_t)x.y * a.max_pages + j] = page;
                    if (page < 0 || page >= a.num_pages) report(a.err, DEVERR_PAGE_RANGE);
                    else atomicAdd(&a.refs[page], 1);
                } else if (j >= x.w) {
                    a.page_table[(size_t)x.y * a.max_pages + j] = -1;
                }
            }
        }
        if (mine) a.lens[d] = served ? len : 0;
        __syncthreads();
    }
}

__global__ void __launch_bounds__(128) free_kernel(const PageArgs a, const int32_t *__restrict__ rows) {
    const int b = rows[blockIdx.x];
    if (b < 0 || b >= a.B) {
        if (threadIdx.x == 0) report(a.err, DEVERR_SLOT_RANGE);
        return;
    }
    const int len = a.lens[b];
    if (len < 0 || (long long)len > ((long long)a.max_pages << a.page_shift)) {
        if (threadIdx.x == 0) report(a.err, DEVERR_SEQLENS);
        return;
    }
    const int held = pages_of(len, a.page_shift);
    for (int j = threadIdx.x; j < a.max_pages; j += blockDim.x) {
        int32_t *entry = a.page_table + (size_t)b * a.max_pages + j;
        if (j < held) let_go(a, entry);
        else *entry = -1;
    }
    __syncthreads();
    if (threadIdx.x == 0) a.lens[b] = 0;
}

// Compaction: ws[0] moves, moves list at ws + 16 (pairs), map at ws + 16 + 2 N.
__global__ void __launch_bounds__(SCAN) compact_plan_kernel(const PageArgs a, int32_t *ws, int32_t *live_out) {
    const int N = a.num_pages;
    int32_t *moves = ws + 16, *map = ws + 16 + 2 * (size_t)N;
    int live = 0;
    {
        int mine = 0;
        for (int p0 = (int)threadIdx.x * PER; p0 < N; p0 += SCAN * PER) {
            int r[PER];
            load_refs(a.refs, N, p0, 0, r);
#pragma unroll
            for (int i = 0; i < PER; ++i) mine += r[i] != 0;
        }
        cta_scan(mine, live);
    }
    int holes = 0, movers = 0;         // found so far; one scan counts both, 16384 at most of each in a step
    for (int p0 = 0; p0 < N; p0 += SCAN * PER) {
        const int p1 = p0 + (int)threadIdx.x * PER;
        int r[PER], h = 0, m = 0;
        load_refs(a.refs, N, p1, 0, r);
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int p = p1 + i;
            h += r[i] == 0 && p < live;
            m += r[i] != 0 && p >= live;
        }
        int both;
        const int before = cta_scan(h | m << 16, both);
        int kh = holes + (before & 0xffff), km = movers + (before >> 16);
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int p = p1 + i;
            if (p >= N) continue;
            if (r[i] == 0 && p < live) moves[2 * kh++ + 1] = p;
            if (p >= live) {
                if (r[i] != 0) moves[2 * km++] = p;
                else map[p] = p;               // free: an entry that names it all the same stays
            }
        }
        holes += both & 0xffff;
        movers += both >> 16;
    }
    __syncthreads();
    for (int k = threadIdx.x; k < movers; k += SCAN) {
        const int from = moves[2 * k], to = moves[2 * k + 1];
        map[from] = to;
        a.refs[to] = a.refs[from];
        a.refs[from] = 0;
    }
    if (threadIdx.x == 0) {
        ws[0] = movers;
        ws[1] = live;
        *live_out = live;
    }
}

constexpr int COPY_THREADS = 256;
constexpr int COPY_VEC = 8;
constexpr size_t COPY_CHUNK = (size_t)COPY_THREADS * COPY_VEC * 16;     // bytes per CTA and step

// dst page <- src page in every pool: pair i at src[i * step], dst[i * step]; n from the device where n_dev is given.
// A compaction's page table follows in the same launch: entries past the live pages go through the plan's map.
__global__ void __launch_bounds__(COPY_THREADS) page_copy_kernel(const __grid_constant__ PageCopyParams p) {
    for (long long i = (long long)blockIdx.x * COPY_THREADS + threadIdx.x; i < p.cells; i += (long long)gridDim.x * COPY_THREADS) {
        const int page = p.table[i];
        if (page >= p.num_pages) report(p.err, DEVERR_PAGE_RANGE);
        else if (page >= p.n_dev[1]) p.table[i] = p.map[page];
    }
    const long long n = p.n_dev ? *p.n_dev : p.n;
    const long long units = n * p.P * p.chunks;
    for (long long u = blockIdx.x; u < units; u += gridDim.x) {
        const int chunk = (int)(u % p.chunks);
        const long long pair = u / p.chunks;
        const int pool = (int)(pair % p.P);
        const long long i = pair / p.P;
        const int s = p.src[i * p.step], d = p.dst[i * p.step];
        if (s == -1 && d == -1 && p.step == 2) continue;      // a fork that copies nothing
        if (s < 0 || s >= p.num_pages || d < 0 || d >= p.num_pages) {
            if (threadIdx.x == 0 && chunk == 0 && pool == 0) report(p.err, DEVERR_PAGE_RANGE);
            continue;
        }
        const uint4 *from = reinterpret_cast<const uint4 *>(p.pool[pool] + (size_t)s * p.page_bytes);
        uint4 *to = reinterpret_cast<uint4 *>(p.pool[pool] + (size_t)d * p.page_bytes);
        // the chunks of a page are of one size
        const size_t all = p.page_bytes / 16, part = (all + p.chunks - 1) / p.chunks;
        const size_t nvec = min(all, (chunk + 1) * part), v0 = chunk * part + threadIdx.x;
        uint4 buf[COPY_VEC];
#pragma unroll
        for (int j = 0; j < COPY_VEC; ++j) {
            const size_t v = v0 + (size_t)j * COPY_THREADS;
            if (v < nvec) buf[j] = __ldcs(from + v);
        }
#pragma unroll
        for (int j = 0; j < COPY_VEC; ++j) {
            const size_t v = v0 + (size_t)j * COPY_THREADS;
            if (v < nvec) __stcs(to + v, buf[j]);
        }
    }
}

}  // namespace

cudaError_t launch_page_alloc(const PageArgs &a, const int32_t *grow, cudaStream_t s) {
    alloc_kernel<<<1, SCAN, 0, s>>>(a, grow);
    return cudaGetLastError();
}

cudaError_t launch_page_copy(const PageCopyParams &p_in, cudaStream_t s) {
    PageCopyParams p = p_in;
    p.chunks = (int)((p.page_bytes + COPY_CHUNK - 1) / COPY_CHUNK);
    const long long most = p.n_dev ? 152 * 8 : (long long)p.n * p.P * p.chunks;
    if (most == 0) return cudaSuccess;
    const unsigned grid = (unsigned)(most > 0x7fffffffLL ? 0x7fffffffLL : most);
    page_copy_kernel<<<grid, COPY_THREADS, 0, s>>>(p);
    return cudaGetLastError();
}

cudaError_t launch_page_fork(const PageArgs &a, const int32_t *src, const int32_t *dst, int n, PageCopyParams p,
                             int32_t *ws, cudaStream_t s) {
    fork_kernel<<<1, SCAN, 0, s>>>(a, src, dst, n, ws);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    p.n = n;
    p.n_dev = nullptr;
    p.src = ws;
    p.dst = ws + 1;
    p.step = 2;
    return launch_page_copy(p, s);
}

cudaError_t launch_page_free(const PageArgs &a, const int32_t *rows, int n, cudaStream_t s) {
    free_kernel<<<(unsigned)n, 128, 0, s>>>(a, rows);
    return cudaGetLastError();
}

cudaError_t launch_page_compact(const PageArgs &a, PageCopyParams p, int32_t *ws, int32_t *live, cudaStream_t s) {
    compact_plan_kernel<<<1, SCAN, 0, s>>>(a, ws, live);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    p.cells = (long long)a.B * a.max_pages;
    p.table = a.page_table;
    p.map = ws + 16 + 2 * (size_t)a.num_pages;
    p.n_dev = ws;
    p.src = ws + 16;
    p.dst = ws + 17;
    p.step = 2;
    return launch_page_copy(p, s);
}

}  // namespace kda
