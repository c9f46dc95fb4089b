// xq8_attn_plan.hpp -- how the attention's work is cut into jobs and pieces.
//
// An entry is a stretch of rows of q with the tokens that they read: first the
// groups (rows of their sequences, the shared tokens), then the sequences (their
// rows, the tokens that are not read for a group).  Each head of keys and each
// block of an entry's rows is a job.  A row of an entry is a row of q and one of
// the `share` heads of q that read the same keys; blocks are of 16 rows where an
// entry has no more (narrow), else of 128 (wide).
//
// Jobs lie one after the other in a line of costs (entries, heads, blocks), of
// which every workgroup takes AtPlan's quota.  A job's tiles of 128 tokens lie in
// its costs from the start; a tile is taken by the workgroup in whose piece it
// begins.  Costs need not be exact, only the same wherever they are computed: the
// kernel's workgroups and the join each do that from the arrays on the device, so
// that a captured call follows them.
#pragma once

#include <hip/hip_runtime.h>

#include "xq8_cache.hpp"

namespace xsymv {

constexpr int AT_LOW = 16, AT_HD = 256;  // least and widest head
constexpr int AT_NARROW = 16;  // rows of a narrow job, and of a slab
constexpr int AT_WIDE = 128;   // rows of a wide job
constexpr int AT_TILE = 128;   // tokens of a tile
// Costs in tokens of a narrow job: those of a wide one, and of a job besides.
constexpr int AT_WEIGHT = 2, AT_OVER = 64;
// A workgroup's piece is a wide tile at least, so that each has one of every job
// that it is in the middle of.
constexpr int AT_LEAST = AT_TILE * AT_WEIGHT;

// Floats of a slab, the results of 16 rows in a part of a job: m and l of each,
// then their out, not yet divided by l.
__host__ __device__ __forceinline__ size_t at_slab(int hd) { return (size_t)AT_NARROW * (2 + hd); }

struct AtPlan {
    const int *start, *len, *table, *first, *shared;
    int rows, heads, kvheads, share, hd, seqs, ldt, groups, pages, ps;
    int grid;    // workgroups
    int whole;   // no job is cut, nothing is shared: no workspace
    int blocks;  // slabs of a part of a cut job: 8, or 1 where no job is wide
    long long slabs;  // of the workspace; what starts that do not ascend would have beyond is left out
    // workspace: the quota, and where each entry's costs and whole parts begin
    long long* quota;
    long long *cost_at, *slab_at;

    __device__ __forceinline__ int entries() const { return groups + seqs; }
    __device__ __forceinline__ int length(int s) const
    {
        const long long room = min((long long)ldt * ps, 0x7fffff00ll);
        return (int)min((long long)max(len[s], 0), room);
    }
    __device__ __forceinline__ int row_of(int s) const { return start != nullptr ? min(max(start[s], 0), rows) : s; }
};

struct AtEntry {
    int row0, rows;  // the first row of q; rows of the entry
    int t0, t1;      // tokens
    int before;      // tokens before the first row's own (a sequence's)
    int table;       // the row of the table that is read
    int blocks;
    bool wide, group, joined;
    long long cost;  // of one head

    __device__ __forceinline__ int block_slabs() const { return wide ? AT_WIDE / AT_NARROW : 1; }
    __device__ __forceinline__ long long slabs() const { return joined ? (long long)blocks * block_slabs() : 0; }
    // costs of the blocks before block b
    __device__ __forceinline__ long long before_block(const AtPlan& p, long long b) const
    {
        if (p.whole) return b;
        if (!wide || group) return b * (AT_OVER + (long long)(t1 - t0) * (wide ? AT_WEIGHT : 1));
        const int step = (AT_WIDE + p.share - 1) / p.share;  // rows of q a block
        return b * (AT_OVER + (long long)AT_WEIGHT * max(before - t0, 0)) + AT_WEIGHT * step * (b * (b + 1) / 2);
    }
    __device__ __forceinline__ int block_rows() const { return wide ? AT_WIDE : AT_NARROW; }
    // end of the tokens that block b sees
    __device__ __forceinline__ int end(const AtPlan& p, int b) const
    {
        if (group) return t1;
        const long long last = min((long long)(b + 1) * block_rows(), (long long)rows) - 1;
        return (int)min(max(before + last / p.share + 1, (long long)t0), (long long)t1);
    }
    __device__ __forceinline__ int tiles(const AtPlan& p, int b) const { return max(1, (end(p, b) - t0 + AT_TILE - 1) / AT_TILE); }
    __device__ __forceinline__ int tile_cost() const { return AT_TILE * (wide ? AT_WEIGHT : 1); }
    __device__ __forceinline__ void shape(const AtPlan& p)
    {
        wide = rows > AT_NARROW;
        blocks = (rows + block_rows() - 1) / block_rows();
        cost = blocks == 0 ? 0 : before_block(p, blocks);
    }
};

// Group g: its sequences, its shared tokens; whether reading these once is less
// work than for each sequence.
struct AtGroup {
    int s0, s1, row0, rows, tokens;
    bool pays;
    __device__ __forceinline__ AtGroup(const AtPlan& p, int g)
    {
        s0 = min(max(p.first[g], 0), p.seqs);
        s1 = min(max(p.first[g + 1], s0), p.seqs);
        const long long room = min((long long)p.ldt * p.ps, 0x7fffff00ll);
        tokens = (int)min((long long)max(p.shared[g], 0), room);
        row0 = p.row_of(s0);
        rows = max(p.row_of(s1) - row0, 0);
        const int count = s1 - s0;
        pays = false;
        if (tokens > 0 && count > 1 && rows > 0) {
            const long long one = ((long long)rows + count - 1) / count * p.share, all = (long long)rows * p.share;
            pays = work(all) < count * work(one);
        }
    }
    static __device__ __forceinline__ long long work(long long rows)
    {
        return rows <= AT_NARROW ? 1 : (rows + AT_WIDE - 1) / AT_WIDE * AT_WEIGHT;
    }
};

// The group that sequence s reads its first tokens with, -1: none.
__device__ __forceinline__ int at_group(const AtPlan& p, int s, int& tokens)
{
    tokens = 0;
    if (p.whole || p.groups == 0) return -1;
    int lo = 0, hi = p.groups;  // the last group that begins at or before s
    while (lo < hi) {
        const int mid = lo + (hi - lo) / 2;
        if (p.first[mid + 1] <= s)
            lo = mid + 1;
        else
            hi = mid;
    }
    if (lo >= p.groups) return -1;
    const AtGroup g(p, lo);
    if (!g.pays || s < g.s0 || s >= g.s1) return -1;
    tokens = g.tokens;
    return lo;
}

__device__ __forceinline__ AtEntry at_entry(const AtPlan& p, int e)
{
    AtEntry x{};
    if (e < p.groups) {
        x.group = x.joined = true;
        if (!p.whole) {
            const AtGroup g(p, e);
            if (g.pays) {
                x.row0 = g.row0;
                x.rows = g.rows * p.share;
                x.t1 = g.tokens;
                x.table = g.s0;
            }
        }
    } else {
        const int s = e - p.groups, from = p.row_of(s), count = max(p.row_of(s + 1) - from, 0);
        const int len = p.length(s);
        x.row0 = from;
        x.rows = count * p.share;
        x.joined = at_group(p, s, x.t0) >= 0;
        x.t1 = max(len, x.t0);
        x.before = len - count;
        x.table = s;
    }
    x.shape(p);
    return x;
}

// A piece of work: rows of an entry, a head of keys.
struct AtJob {
    int head, rows, rho0, row0, end, before, table;
    bool wide, group;
    // row n's row and head of q
    __device__ __forceinline__ int place(const AtPlan& p, int n, size_t& row) const
    {
        const int rho = rho0 + n;
        row = (size_t)row0 + rho / p.share;
        return head * p.share + rho % p.share;
    }
    // tokens that row n sees
    __device__ __forceinline__ int limit(const AtPlan& p, int n) const
    {
        const int at = (rho0 + n) / p.share;
        if (!group) return before + at + 1;
        const int row = row0 + at, s = pg_sequence(p.start, p.seqs, row);
        if (s < 0) return 0;
        return p.length(s) - (p.row_of(s + 1) - 1 - row);
    }
};

struct AtScan {
    long long cost[257], slab[257], wave_cost[4], wave_slab[4];
};

// Least and largest of a number that lanes n, n + 16, ... have alike.
__device__ __forceinline__ int at_least(int v)
{
#pragma unroll
    for (int d = 8; d > 0; d >>= 1) v = min(v, __shfl_xor(v, d, 64));
    return __builtin_amdgcn_readfirstlane(v);
}
__device__ __forceinline__ int at_most(int v)
{
#pragma unroll
    for (int d = 8; d > 0; d >>= 1) v = max(v, __shfl_xor(v, d, 64));
    return __builtin_amdgcn_readfirstlane(v);
}
// What a wave wrote to LDS is there for all its lanes.
__device__ __forceinline__ void at_wave_sync()
{
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}
template <int I>
struct AtIndex {
    static constexpr int value = I;
};
template <int N, int I = 0, class F>
__device__ __forceinline__ void at_each(F&& f)
{
    if constexpr (I < N) {
        f(AtIndex<I>{});
        at_each<N, I + 1>(f);
    }
}
__device__ __forceinline__ long long at_uniform(long long v)
{
    const int lo = __builtin_amdgcn_readfirstlane((int)v), hi = __builtin_amdgcn_readfirstlane((int)(v >> 32));
    return (long long)hi << 32 | (unsigned)lo;
}

// An entry that all lanes have alike.
__device__ __forceinline__ AtEntry at_uniform(const AtEntry& x)
{
    AtEntry u;
    u.row0 = __builtin_amdgcn_readfirstlane(x.row0);
    u.rows = __builtin_amdgcn_readfirstlane(x.rows);
    u.t0 = __builtin_amdgcn_readfirstlane(x.t0);
    u.t1 = __builtin_amdgcn_readfirstlane(x.t1);
    u.before = __builtin_amdgcn_readfirstlane(x.before);
    u.table = __builtin_amdgcn_readfirstlane(x.table);
    u.blocks = __builtin_amdgcn_readfirstlane(x.blocks);
    u.wide = __builtin_amdgcn_readfirstlane(x.wide);
    u.group = __builtin_amdgcn_readfirstlane(x.group);
    u.joined = __builtin_amdgcn_readfirstlane(x.joined);
    u.cost = at_uniform(x.cost);
    return u;
}

// A workgroup's way through its piece of the line.
struct AtCursor {
    long long pos, end, quota;
    long long base, slab;  // where the entry's costs, and its whole parts, begin
    int worker, entry;
    AtEntry of;

    __device__ __forceinline__ AtCursor(const AtPlan& p, AtScan& scan)
    {
        // workgroups of one die, which takes every eighth, have pieces side by side
        const int per = p.grid / 8;
        worker = p.grid % 8 == 0 ? (int)(blockIdx.x % 8) * per + (int)blockIdx.x / 8 : (int)blockIdx.x;
        const int t = threadIdx.x, lane = t & 63, wave = t >> 6;
        const int entries = p.entries(), chunk = (entries + 255) / 256;
        long long cost = 0;
        long long slabs = 0;
        for (int e = t * chunk; e < min((t + 1) * chunk, entries); ++e) {
            const AtEntry x = at_entry(p, e);
            cost += x.cost * p.kvheads;
            slabs += x.slabs() * p.kvheads;
        }
        long long c = cost;
        long long s = slabs;
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            const long long oc = __shfl_up(c, d, 64);
            const long long os = __shfl_up(s, d, 64);
            if (lane >= d) {
                c += oc;
                s += os;
            }
        }
        if (lane == 63) {
            scan.wave_cost[wave] = c;
            scan.wave_slab[wave] = s;
        }
        __syncthreads();
        for (int w = 0; w < wave; ++w) {
            c += scan.wave_cost[w];
            s += scan.wave_slab[w];
        }
        scan.cost[t + 1] = c;
        scan.slab[t + 1] = s;
        if (t == 0) {
            scan.cost[0] = 0;
            scan.slab[0] = 0;
        }
        __syncthreads();
        const long long total = at_uniform(scan.cost[256]);
        quota = (total + p.grid - 1) / p.grid;
        if (!p.whole) {
            quota = max(quota, (long long)AT_LEAST);
            if (blockIdx.x == 0) {  // for the join
                if (t == 0) p.quota[0] = quota;
                long long at = c - cost;
                long long sl = s - slabs;
                for (int e = t * chunk; e < min((t + 1) * chunk, entries); ++e) {
                    const AtEntry x = at_entry(p, e);
                    p.cost_at[e] = at;
                    p.slab_at[e] = sl;
                    at += x.cost * p.kvheads;
                    sl += x.slabs() * p.kvheads;
                }
            }
        }
        pos = worker * quota;
        end = min(pos + quota, total);
        if (pos >= end) return;
        int lo = 0, hi = 255;  // the last chunk that begins at or before pos
        while (lo < hi) {
            const int mid = (lo + hi + 1) / 2;
            if (scan.cost[mid] <= pos)
                lo = mid;
            else
                hi = mid - 1;
        }
        lo = __builtin_amdgcn_readfirstlane(lo);
        base = at_uniform(scan.cost[lo]);
        slab = at_uniform(scan.slab[lo]);
        entry = lo * chunk;
        of = at_uniform(at_entry(p, entry));
        settle(p);
    }
    // to the entry that holds pos
    __device__ __forceinline__ void settle(const AtPlan& p)
    {
        while (entry + 1 < p.entries() && pos >= base + of.cost * p.kvheads) {
            base += of.cost * p.kvheads;
            slab += of.slabs() * p.kvheads;
            of = at_uniform(at_entry(p, ++entry));
        }
    }
    // The next job with tiles in the piece: its tokens from `from` to `to`, and the
    // slab for its results (-1: they are whole, and go to out).
    __device__ __forceinline__ bool next(const AtPlan& p, AtJob& job, int& from, int& to, long long& part)
    {
        while (pos < end) {
            settle(p);
            if (of.cost <= 0) return false;
            const long long in = pos - base, head = in / of.cost, rest = in - head * of.cost;
            if (head >= p.kvheads) return false;
            int lo = 0, hi = of.blocks - 1;  // the last block that begins at or before it
            while (lo < hi) {
                const int mid = (lo + hi + 1) / 2;
                if (of.before_block(p, mid) <= rest)
                    lo = mid;
                else
                    hi = mid - 1;
            }
            const int b = lo, tiles = of.tiles(p, b), weight = of.tile_cost();
            const long long c0 = of.before_block(p, b), c1 = of.before_block(p, b + 1);
            const long long x = rest - c0, y = min(x + end - pos, c1 - c0);
            pos += y - x;
            int t0 = 0, t1 = tiles;
            if (!p.whole) {
                t0 = (int)min((x + weight - 1) / weight, (long long)tiles);
                t1 = (int)min((y + weight - 1) / weight, (long long)tiles);
            }
            if (t0 >= t1) continue;
            job.head = (int)head;
            job.rho0 = b * of.block_rows();
            job.rows = min(of.rows - job.rho0, of.block_rows());
            job.row0 = of.row0;
            job.end = of.end(p, b);
            job.before = of.before;
            job.table = of.table;
            job.wide = of.wide;
            job.group = of.group;
            from = of.t0 + t0 * AT_TILE;
            to = min(of.t0 + t1 * AT_TILE, job.end);
            part = -1;
            if (!p.whole) {
                if (t0 > 0 || t1 < tiles)
                    part = (2ll * worker + (t0 == 0)) * p.blocks;
                else if (of.joined)
                    part = 2ll * p.grid * p.blocks + slab + head * of.slabs() + (long long)b * of.block_slabs();
                if (part + of.block_slabs() > p.slabs) continue;
            }
            return true;
        }
        return false;
    }
};

// Where the results of a row of q lie, for one head of keys and one of its entries.
struct AtParts {
    const AtPlan* plan;
    AtEntry of;
    long long base, quota;
    long long slab0;
    int kv, rho;  // rho: the entry's row of the first head
    bool some;

    __device__ __forceinline__ void set(const AtPlan& p, int e, int row, int head)
    {
        plan = &p;
        of = at_entry(p, e);
        base = p.cost_at[e];
        slab0 = p.slab_at[e];
        quota = p.quota[0];
        kv = head;
        rho = (row - of.row0) * p.share;
        some = row >= of.row0 && rho < of.rows;
    }
    __device__ __forceinline__ int block(int h) const { return (rho + h) / of.block_rows(); }
    __device__ __forceinline__ int row(int h) const { return (rho + h) % of.block_rows(); }
    // the workgroups that the job's first and last tiles are taken by
    __device__ __forceinline__ void workers(int h, int& w0, int& w1) const
    {
        const int b = block(h);
        const long long at = base + kv * of.cost + of.before_block(*plan, b);
        w0 = (int)(at / quota);
        w1 = (int)((at + (long long)(of.tiles(*plan, b) - 1) * of.tile_cost()) / quota);
    }
    __device__ __forceinline__ int count(int h) const
    {
        if (!some) return 0;
        int w0, w1;
        workers(h, w0, w1);
        return w1 - w0 + 1;
    }
    // slab of part i of head h's job, -1: there is none
    __device__ __forceinline__ long long slab(int h, int i) const
    {
        int w0, w1;
        workers(h, w0, w1);
        const long long at = w0 == w1 ? 2ll * plan->grid * plan->blocks + slab0 + kv * of.slabs() +
                                            (long long)block(h) * of.block_slabs()
                                      : (2ll * (w0 + i) + (i == 0)) * plan->blocks;
        return at + of.block_slabs() > plan->slabs ? -1 : at + row(h) / AT_NARROW;
    }
};

// A row's parts: of its group's tokens, and of its own; false where the row has
// none that are to be added.
__device__ __forceinline__ bool at_parts(const AtPlan& p, int row, int kv, AtParts (&parts)[2])
{
    const int s = pg_sequence(p.start, p.seqs, row);
    if (s < 0) return false;
    parts[1].set(p, p.groups + s, row, kv);
    parts[0].some = false;
    int tokens;
    const int g = at_group(p, s, tokens);
    if (g >= 0) {
        parts[0].set(p, g, row, kv);
        return true;
    }
    for (int h = 0; h < p.share; h += parts[1].of.block_rows())
        if (parts[1].count(h) > 1) return true;
    return parts[1].count(p.share - 1) > 1;
}

}  // namespace xsymv
