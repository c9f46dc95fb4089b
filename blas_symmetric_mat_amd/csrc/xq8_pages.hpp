// xq8_pages.hpp -- kernels on the pages of a cache of 8-bit rows: sequences
// grown, forked and freed, the used pages moved together, pages copied.
//
// A page is free where refs[page] is 0.  What has to be decided in order (which
// fork or sequence gets which free page) is decided by one workgroup of 1024
// threads: the lists are short, and a second workgroup would have to wait for the
// first one's counts, which between the chip's dies costs what a launch does.  A
// fork or grow of a few sequences takes 9 us and 4, the lists of 4096 pages 8.
// All numbers that come from device arrays are checked where they are used.
#pragma once

#include "xq8_cache.hpp"

namespace xsymv {

constexpr int PG_THREADS = 1024;
constexpr int PG_MOST = 8192;  // sequences of one call of fork or grow (LDS)
constexpr int PG_CHUNK = 16;   // refs a thread looks at in one go

// Exclusive sums over the workgroup's threads; `total` is theirs together.
// `waves`: a number of LDS for each wave, free again after the next barrier.
template <class V>
__device__ __forceinline__ V pg_scan(V v, V* waves, V& total)
{
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    V sum = v;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const V o = __shfl_up(sum, d, 64);
        if (lane >= d) sum += o;
    }
    __syncthreads();
    if (lane == 63) waves[wave] = sum;
    __syncthreads();
    V before = 0;
    total = 0;
#pragma unroll
    for (int w = 0; w < PG_THREADS / 64; ++w) {
        const V s = waves[w];
        before += w < wave ? s : 0;
        total += s;
    }
    return before + sum - v;
}

// Calls take(page, rank) for the first `want` free pages in ascending order and
// returns how many there are (at most want, as far as looked).
template <class F>
__device__ int pg_free(const PgCache& c, int want, int* waves, F&& take)
{
    int found = 0;
    // (unsigned: the last stretch reaches past the largest int)
    for (unsigned base = 0; base < (unsigned)c.pages && found < want; base += PG_THREADS * PG_CHUNK) {
        const unsigned first = base + threadIdx.x * PG_CHUNK;
        unsigned mask = 0;
#pragma unroll
        for (int e = 0; e < PG_CHUNK; ++e)
            if (first + e < (unsigned)c.pages && c.refs[first + e] == 0) mask |= 1u << e;
        int total = 0;
        int rank = found + pg_scan((int)__popc(mask), waves, total);
        while (mask != 0 && rank < want) {
            take((int)first + __ffs((int)mask) - 1, rank++);
            mask &= mask - 1;
        }
        found += total;
    }
    return found < want ? found : want;
}

// Lets the first of the list's entries that name a sequence keep it: `mine(i)`
// is the sequence of entry i (< 0: none), and keep(i, yes) is called for those
// that have one.  Uses len as the place to meet; the caller has read what it
// needs of it, and writes it again for those that keep theirs.
template <class M, class K>
__device__ void pg_claim(const PgCache& c, int n, M&& mine, K&& keep)
{
    auto all = [&](auto&& f) {
        for (int i = threadIdx.x; i < n; i += PG_THREADS)
            if (mine(i) >= 0) f(i, &c.len[mine(i)]);
        __threadfence_block();
        __syncthreads();
    };
    __syncthreads();
    all([](int, int* p) {
        __hip_atomic_store(p, (int)0x80000000, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    });
    all([](int i, int* p) { atomicMax(p, -1 - i); });
    all([&](int i, int* p) {
        keep(i, __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == -1 - i);
    });
}

// ------------------------------------------------------------------ growing
struct PgGrowArgs {
    PgCache c;
    const int *seq, *add;
    int* got;
    int n;
};

__global__ __launch_bounds__(PG_THREADS) void q8_pages_grow(PgGrowArgs a)
{
    // tokens before, of those that grow (-1: left as it is); pages of those before it;
    // what the lengths are, in range or not
    __shared__ int before[PG_MOST], start[PG_MOST + 1], was[PG_MOST], waves[PG_THREADS / 64];
    __shared__ long long wide[PG_THREADS / 64];
    const PgCache& c = a.c;
    for (int i = threadIdx.x; i < a.n; i += PG_THREADS) {
        const int s = a.seq[i];
        before[i] = c.is_seq(s) ? c.length(s, was[i]) : -1;
    }
    pg_claim(c, a.n, [&](int i) { return before[i] < 0 ? -1 : a.seq[i]; },
             [&](int i, bool yes) { start[i] = yes; });
    // the claims are off: every sequence has its length again
    for (int i = threadIdx.x; i < a.n; i += PG_THREADS)
        if (before[i] >= 0) c.len[a.seq[i]] = was[i];
    __syncthreads();
    auto held = [&](long long tokens) { return (tokens + c.ps - 1) / c.ps; };
    long long sum = 0;
    for (int base = 0; base < a.n; base += PG_THREADS) {
        const int i = base + (int)threadIdx.x;
        long long need = 0;
        if (i < a.n) {
            const int old = before[i];
            const long long more = old >= 0 ? a.add[i] : 0;
            if (old >= 0 && start[i] != 0 && more > 0 && old + more <= (long long)c.ldt * c.ps &&
                old + more <= 0x7fffffff)
                need = held(old + more) - held(old);
            else
                before[i] = -1;
        }
        long long total = 0;
        const long long at = sum + pg_scan(need, wide, total);
        // (the largest int stands for more pages than there can be)
        if (i < a.n) start[i] = (int)min(at, 0x7fffffffll);
        sum += total;
        __syncthreads();
    }
    if (threadIdx.x == 0) start[a.n] = (int)min(sum, 0x7fffffffll);
    __syncthreads();
    const int found = pg_free(c, start[a.n], waves, [&](int page, int rank) {
        int lo = 0, hi = a.n - 1;  // the last entry that starts at or before the rank
        while (lo < hi) {
            const int mid = (lo + hi + 1) / 2;
            if (start[mid] <= rank)
                lo = mid;
            else
                hi = mid - 1;
        }
        c.row(a.seq[lo])[held(before[lo]) + rank - start[lo]] = page;
        c.refs[page] = 1;
    });
    __threadfence_block();
    __syncthreads();
    for (int i = threadIdx.x; i < a.n; i += PG_THREADS) {
        int got = 0;
        if (before[i] >= 0) {
            const int old = before[i], more = a.add[i];
            if (start[i + 1] <= found || held((long long)old + more) == held(old)) {
                got = more;
                c.len[a.seq[i]] = old + more;
            } else {  // what it was given of too few goes back
                for (int r = start[i]; r < found; ++r) {
                    int* e = &c.row(a.seq[i])[held(old) + r - start[i]];
                    c.refs[*e] = 0;
                    *e = -1;
                }
            }
        }
        a.got[i] = got;
    }
}

// -------------------------------------------------------------------- slots
struct PgSlotArgs {
    PgCache c;
    const int* start;
    int* slot;
    int rows, kvheads;
};

__global__ __launch_bounds__(256) void q8_pages_slots(PgSlotArgs a)
{
    const PgCache& c = a.c;
    const long long all = (long long)a.rows * a.kvheads;
    for (long long i = blockIdx.x * 256ll + threadIdx.x; i < all; i += gridDim.x * 256ll) {
        const int r = (int)(i / a.kvheads), h = (int)(i % a.kvheads);
        const int s = pg_sequence(a.start, c.seqs, r);
        if (s < 0) continue;
        const int behind = a.start ? a.start[s + 1] - 1 - r : 0;
        const long long t = (long long)c.length(s) - 1 - behind;
        int slot = -1;
        if (t >= 0) {
            const int page = c.row(s)[t / c.ps];
            if (c.is_page(page)) slot = (page * a.kvheads + h) * c.ps + (int)(t % c.ps);
        }
        a.slot[i] = slot;
    }
}

// ------------------------------------------------------------------ forking
struct PgForkArgs {
    PgCache c;
    const int *parent, *child;
    int *src, *dst;
    int n, whole;  // whole: the tables are written by the same launch
};

// Entries of a forked sequence's row of the table, and their counts; `t` of
// `threads` share it.  dst: its own last page, where it has one.
__device__ __forceinline__ void pg_inherit(const PgCache& c, int parent, int child, int length, int dst,
                                           int t, int threads)
{
    const int full = length / c.ps;
    const int* from = c.row(parent);
    int* to = c.row(child);
    for (int j = t; j < full; j += threads) {
        const int page = from[j];
        to[j] = page;
        if (c.is_page(page)) atomicAdd(&c.refs[page], 1);
    }
    if (t == 0 && dst >= 0) to[full] = dst;
}

__global__ __launch_bounds__(PG_THREADS) void q8_pages_fork(PgForkArgs a)
{
    __shared__ int tokens[PG_MOST], page_of[PG_MOST], was[PG_MOST], waves[PG_THREADS / 64];
    const PgCache& c = a.c;
    for (int i = threadIdx.x; i < a.n; i += PG_THREADS) {
        const int p = a.parent[i], s = a.child[i];
        int n = -1;
        if (c.is_seq(p) && c.is_seq(s) && c.length(s, was[i]) == 0) n = c.length(p);
        tokens[i] = n;
    }
    pg_claim(c, a.n, [&](int i) { return tokens[i] < 0 ? -1 : a.child[i]; },
             [&](int i, bool yes) { page_of[i] = yes; });
    for (int i = threadIdx.x; i < a.n; i += PG_THREADS) {
        if (tokens[i] < 0) continue;
        c.len[a.child[i]] = was[i];
        if (page_of[i] == 0) tokens[i] = -1;
    }
    __syncthreads();
    int sum = 0;  // page_of: the rank of the page that a fork needs, -1: none
    for (int base = 0; base < a.n; base += PG_THREADS) {
        const int i = base + (int)threadIdx.x;
        const bool cut = i < a.n && tokens[i] > 0 && tokens[i] % c.ps != 0;
        int total = 0;
        const int at = pg_scan((int)cut, waves, total);
        if (i < a.n) page_of[i] = cut ? sum + at : -1;
        sum += total;
        __syncthreads();
    }
    // src takes the pages by rank before it takes what the caller wants
    const int found = pg_free(c, sum, waves, [&](int page, int rank) { a.src[rank] = page; });
    __threadfence_block();
    __syncthreads();
    // ranks to pages, before src and dst take their own
    for (int i = threadIdx.x; i < a.n; i += PG_THREADS) {
        if (page_of[i] >= found)
            tokens[i] = -1;
        else if (page_of[i] >= 0)
            page_of[i] = a.src[page_of[i]];
    }
    __syncthreads();
    for (int i = threadIdx.x; i < a.n; i += PG_THREADS) {
        const int n = tokens[i], page = page_of[i];
        int from = n < 0 ? -2 : -1, to = from;
        if (n >= 0) {
            c.len[a.child[i]] = n;
            if (page >= 0) {
                from = c.row(a.parent[i])[n / c.ps];
                to = page;
                c.refs[page] = 1;
            }
        }
        a.src[i] = from;
        a.dst[i] = to;
    }
    if (!a.whole) return;
    __syncthreads();
    for (int i = 0; i < a.n; ++i)
        if (tokens[i] > 0)
            pg_inherit(c, a.parent[i], a.child[i], tokens[i], page_of[i], threadIdx.x, PG_THREADS);
}

// The tables of many forks or of long ones: a workgroup a fork.
__global__ __launch_bounds__(256) void q8_pages_inherit(PgForkArgs a)
{
    for (int i = blockIdx.x; i < a.n; i += gridDim.x) {
        const int to = a.dst[i];
        if (to == -2) continue;
        // (the parent's own row may name no page where a copy is due: src is -1 then,
        // and the child still has its page)
        pg_inherit(a.c, a.parent[i], a.child[i], a.c.length(a.child[i]), to, threadIdx.x, 256);
    }
}

// ------------------------------------------------------------------ freeing
struct PgFreeArgs {
    PgCache c;
    const int* seq;
    int n;
};

__global__ __launch_bounds__(256) void q8_pages_free(PgFreeArgs a)
{
    __shared__ int shared;
    const PgCache& c = a.c;
    for (int i = blockIdx.x; i < a.n; i += gridDim.x) {
        const int s = a.seq[i];
        if (!c.is_seq(s)) continue;
        __syncthreads();
        // whoever takes the length frees the sequence: one of those that list it
        if (threadIdx.x == 0) shared = atomicExch(&c.len[s], 0);
        __syncthreads();
        const long long n = shared, room = (long long)c.ldt * c.ps;
        const int held = n <= 0 ? 0 : (int)(((n < room ? n : room) + c.ps - 1) / c.ps);
        int* row = c.row(s);
        for (int j = threadIdx.x; j < held; j += 256) {
            const int page = row[j];
            row[j] = -1;
            if (c.is_page(page)) atomicSub(&c.refs[page], 1);
        }
    }
}

// --------------------------------------------------------------- compacting
struct PgCompactArgs {
    const int *table, *refs;
    int *out, *rout, *src, *dst, *live;
    int seqs, ldt, ldo, pages;
};

// The lists of what moves where, by one workgroup: it counts the live pages,
// then ranks the holes before and the live ones behind that place.
__global__ __launch_bounds__(PG_THREADS) void q8_pages_plan(PgCompactArgs a)
{
    __shared__ int waves[PG_THREADS / 64];
    const int half = a.pages / 2;
    constexpr int STEP = PG_THREADS * PG_CHUNK;
    auto used = [&](unsigned base) {
        const unsigned first = base + threadIdx.x * PG_CHUNK;
        unsigned mask = 0;
#pragma unroll
        for (int e = 0; e < PG_CHUNK; ++e)
            if (first + e < (unsigned)a.pages && a.refs[first + e] != 0) mask |= 1u << e;
        return mask;
    };
    int live = 0;
    for (unsigned base = 0; base < (unsigned)a.pages; base += STEP) live += __popc(used(base));
    int total = 0;
    (void)pg_scan(live, waves, total);
    live = total;
    int holes = 0, movers = 0;
    for (unsigned base = 0; base < (unsigned)a.pages; base += STEP) {
        const unsigned first = base + threadIdx.x * PG_CHUNK;
        const int have = first < (unsigned)a.pages ? min(a.pages - (int)first, PG_CHUNK) : 0;
        const int low = first < (unsigned)live ? min(live - (int)first, have) : 0;  // before place `live`
        const unsigned mask = used(base), below = (1u << low) - 1, valid = (1u << have) - 1;
        unsigned hole = ~mask & below, mover = mask & valid & ~below;
        int more = 0;
        int rank = holes + pg_scan((int)__popc(hole), waves, more);
        holes += more;
        for (; hole != 0; hole &= hole - 1) a.dst[rank++] = (int)first + __ffs((int)hole) - 1;
        rank = movers + pg_scan((int)__popc(mover), waves, more);
        movers += more;
        for (; mover != 0; mover &= mover - 1) a.src[rank++] = (int)first + __ffs((int)mover) - 1;
    }
    for (int i = movers + (int)threadIdx.x; i < half; i += PG_THREADS) a.src[i] = a.dst[i] = -1;
    if (threadIdx.x == 0) a.live[0] = live;
}

// Number of entries of an ascending list below `v`; entries of -1 lie behind the
// list's end and count as above everything.
__device__ __forceinline__ int pg_below(const int* list, int n, int v)
{
    int lo = 0, hi = n;
    while (lo < hi) {
        const int mid = (lo + hi) / 2;
        if ((unsigned)list[mid] < (unsigned)v)
            lo = mid + 1;
        else
            hi = mid;
    }
    return lo;
}

__global__ __launch_bounds__(256) void q8_pages_rename(PgCompactArgs a)
{
    const int live = a.live[0], half = a.pages / 2;
    const long long entries = (long long)a.seqs * a.ldt, all = entries + a.pages;
    for (long long i = blockIdx.x * 256ll + threadIdx.x; i < all; i += gridDim.x * 256ll) {
        if (i < entries) {
            const long long s = i / a.ldt, j = i % a.ldt;
            const int page = a.table[i];
            int to = -1;
            if ((unsigned)page < (unsigned)a.pages) {
                if (page >= live) {
                    const int k = pg_below(a.src, half, page);
                    if (k < half && a.src[k] == page) to = a.dst[k];
                } else {
                    const int k = pg_below(a.dst, half, page);
                    if (k >= half || a.dst[k] != page) to = page;  // not a hole
                }
            }
            a.out[s * a.ldo + j] = to;
        } else {
            // a moved page's count is read and written by one thread, so that rout
            // may be refs
            const int page = (int)(i - entries);
            if (page < live) {
                const int k = pg_below(a.dst, half, page);
                if (k >= half || a.dst[k] != page) a.rout[page] = a.refs[page];
            } else {
                const int k = pg_below(a.src, half, page);
                if (k < half && a.src[k] == page) a.rout[a.dst[k]] = a.refs[page];
                a.rout[page] = 0;
            }
        }
    }
}

// ------------------------------------------------------------------ copying
struct PgCopyArgs {
    const int *src, *dst;
    signed char *k, *v;
    float *ks, *vs;
    int n, pages, rows, hd, ldk, ldv, layers, stride;
    int pieces;  // of a page's codes of one matrix and layer
};

// Bytes of a piece, where a page's codes lie in one run, and rows of one, where
// they do not: 256 threads with a few 16-byte loads each in flight.
constexpr int PG_PIECE = 256 * 16 * 4, PG_ROWS = 64;

// n bytes by `threads` threads of which this is `t`, 16 at a time, U of these in
// flight; the last 16 overlap those before them.
template <int U>
__device__ __forceinline__ void pg_bytes(signed char* to, const signed char* from, int n, int t, int threads)
{
    typedef int vec __attribute__((ext_vector_type(4), aligned(1)));
    if (n < 16) {
        for (int i = t; i < n; i += threads) to[i] = from[i];
        return;
    }
    const int chunks = (n + 15) / 16;
    for (int c = t; c < chunks; c += threads * U) {
        vec x[U];
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (c + u * threads < chunks) x[u] = *(const vec*)(from + min((c + u * threads) * 16, n - 16));
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (c + u * threads < chunks) *(vec*)(to + min((c + u * threads) * 16, n - 16)) = x[u];
    }
}

// Bound by HBM: 1638 pages of 64 tokens, 8 heads of 128 codes (134 MB and back), in
// 43 us, 6.3 TB/s.
__global__ __launch_bounds__(256) void q8_pages_copy(PgCopyArgs a)
{
    const bool run = a.ldk == a.hd && (a.v == nullptr || a.ldv == a.hd);
    const int both = a.v != nullptr ? 2 : 1;
    const long long each = (long long)both * a.layers * a.pieces, all = a.n * each;
    for (long long i = blockIdx.x; i < all; i += gridDim.x) {
        const int pair = (int)(i / each), from = a.src[pair], to = a.dst[pair];
        if ((unsigned)from >= (unsigned)a.pages || (unsigned)to >= (unsigned)a.pages || from == to) continue;
        const long long rest = i % each;
        const int piece = (int)(rest % a.pieces), of = (int)(rest / a.pieces);
        const int layer = of / both;
        const bool values = of % both != 0;
        const long long base = (long long)layer * a.stride;
        const long long rf = base + (long long)from * a.rows, rt = base + (long long)to * a.rows;
        const int ld = values ? a.ldv : a.ldk;
        signed char* m = values ? a.v : a.k;
        float* s = values ? a.vs : a.ks;
        if (run) {
            const long long bytes = (long long)a.rows * a.hd, at = (long long)piece * PG_PIECE;
            const int have = (int)min(bytes - at, (long long)PG_PIECE);
            pg_bytes<4>(m + rt * ld + at, m + rf * ld + at, have, threadIdx.x, 256);
        } else {
            // eight threads a row
            const int first = piece * PG_ROWS, last = min(first + PG_ROWS, a.rows);
            for (int r = first + (int)threadIdx.x / 8; r < last; r += 32)
                pg_bytes<4>(m + (rt + r) * ld, m + (rf + r) * ld, a.hd, threadIdx.x & 7, 8);
        }
        if (piece == 0)
            for (int r = threadIdx.x; r < a.rows; r += 256) s[rt + r] = s[rf + r];
    }
}

}  // namespace xsymv
