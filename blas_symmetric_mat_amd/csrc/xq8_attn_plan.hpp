// xq8_attn_plan.hpp -- how the attention's work is cut into jobs and pieces.
//
// An entry is a stretch of rows of q with the tokens that they read: first the
// groups (rows of their sequences, the shared tokens), then the sequences (their
// rows, the tokens that are not read for a group).  Each head of keys and each
// block of an entry's rows is a job.  A row of an entry is a row of q and one of
// the `share` heads of q that read the same keys; blocks are of 16 rows where an
// entry has no more (narrow), else of 128 (wide).
//
// There are two lines of jobs, one after the other by entry, head and block, each
// with a cost in tokens: wide jobs, of which every workgroup takes an equal piece,
// and narrow ones, of which every wave does.  A job's tiles (32 tokens of a narrow
// job, 64 of a wide one) lie in its costs from the start; a tile is taken by the
// worker in whose piece it begins.  Costs need not be exact, only the same for all
// workers, which compute them from the arrays on the device, so that a captured call
// follows what these hold.
//
// Who takes a job's first tile writes down, for each of its rows, where the parts of
// its results are; the join reads that.
#pragma once

#include <hip/hip_runtime.h>

#include "xq8_cache.hpp"

namespace xsymv {

constexpr int AT_LOW = 16, AT_HD = 256;  // least and widest head
constexpr int AT_NARROW = 16;            // rows of a narrow job, and of a slab
constexpr int AT_WIDE = 128;             // rows of a wide job
constexpr int AT_SLABS = AT_WIDE / AT_NARROW;
constexpr int AT_TILE[2] = {32, 64};  // tokens of a narrow and of a wide tile
constexpr int AT_OVER = 48;           // cost of a job besides its tokens
// A piece is two tiles at least: so that each worker has one of every job that it is
// in the middle of, and for the join's sake.
constexpr int AT_LEAST[2] = {64, 128};

// Floats of a slab, the results of 16 rows in a part of a job: m and l of each,
// then their out, not yet divided by l.
__host__ __device__ inline size_t at_slab(int hd) { return (size_t)AT_NARROW * (2 + hd); }

// Quotients of numbers below 2^31 by one that the host knows.
struct AtDivisor {
    unsigned d, mul, shift;
    AtDivisor(int by = 1)
    {
        d = (unsigned)by;
        shift = 0;
        while (((unsigned long long)1 << shift) < d) ++shift;
        mul = (unsigned)((((unsigned long long)1 << 32) * (((unsigned long long)1 << shift) - d)) / d + 1);
    }
    __device__ __forceinline__ int of(int n) const
    {
        return (int)((__umulhi((unsigned)n, mul) + (unsigned)n) >> shift);
    }
};

struct AtPlan {
    const int *start, *len, *table, *first, *shared;
    int rows, heads, kvheads, share, hd, seqs, ldt, groups, pages, ps;
    AtDivisor by_share, by_page;
    int grid;   // workgroups
    int whole;  // no job is cut, nothing is shared: no workspace
    // Workspace: slabs (of cut wide jobs' parts, two of 128 rows a workgroup; of cut
    // narrow ones', two a wave; of whole parts) and, for each row and head, where its
    // own parts and its group's are.
    long long slabs, narrow_at, whole_at;
    int2 *own, *shared_parts;

    __device__ __forceinline__ int entries() const { return groups + seqs; }
    __device__ __forceinline__ int room() const { return (int)min((long long)ldt * ps, 0x7fffff00ll); }
    __device__ __forceinline__ int length(int s) const { return min(max(len[s], 0), room()); }
    __device__ __forceinline__ int row_of(int s) const
    {
        return start != nullptr ? min(max(start[s], 0), rows) : s;
    }
};

// Floor of a / b for 0 <= a < 2^62, b > 0 and a quotient that an int holds: a
// division in 32-bit floating point, put right.
__device__ __forceinline__ int at_quotient(long long a, long long b)
{
    int q = (int)fminf((float)a / (float)b, 2.1e9f);
    while ((long long)q * b > a) --q;
    while ((long long)(q + 1) * b <= a) ++q;
    return q;
}

struct AtEntry {
    int row0, rows;  // the first row of q; rows of the entry
    int t0, t1;      // tokens
    int before;      // tokens before the first row's own (a sequence's)
    int table;       // the row of the table that is read
    int blocks;
    int wide, group, joined;
    long long cost;  // of one head

    __device__ __forceinline__ int block_rows() const { return wide ? AT_WIDE : AT_NARROW; }
    __device__ __forceinline__ int block_slabs() const { return wide ? AT_SLABS : 1; }
    __device__ __forceinline__ long long slabs() const { return joined ? (long long)blocks * block_slabs() : 0; }
    // costs of the blocks before block b
    __device__ __forceinline__ long long before_block(const AtPlan& p, int b) const
    {
        if (p.whole) return b;
        if (!wide || group) return (long long)b * (AT_OVER + t1 - t0);
        const int step = p.by_share.of(AT_WIDE + p.share - 1);  // rows of q a block
        return (long long)b * (AT_OVER + max(before - t0, 0)) + step * ((long long)b * (b + 1) / 2);
    }
    // end of the tokens that block b sees
    __device__ __forceinline__ int end(const AtPlan& p, int b) const
    {
        if (group) return t1;
        const int last = (int)min((long long)(b + 1) * block_rows(), (long long)rows) - 1;
        return min(max(before + p.by_share.of(last) + 1, t0), t1);
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
        tokens = min(max(p.shared[g], 0), p.room());
        row0 = p.row_of(s0);
        rows = max(p.row_of(s1) - row0, 0);
        const int count = s1 - s0;
        pays = false;
        if (tokens > 0 && count > 1 && rows > 0) {
            const long long one = (long long)((rows + count - 1) / count) * p.share;
            pays = work((long long)rows * p.share) < count * work(one);
        }
    }
    // a wide tile of tokens takes about as long as two narrow ones
    static __device__ __forceinline__ long long work(long long rows)
    {
        return rows <= AT_NARROW ? 1 : (rows + AT_WIDE - 1) / AT_WIDE * 2;
    }
};

// The tokens that sequence s reads with its group, 0: none.
__device__ __forceinline__ int at_shared(const AtPlan& p, int s)
{
    if (p.whole || p.groups == 0) return 0;
    int lo = 0, hi = p.groups;  // the last group that begins at or before s
    while (lo < hi) {
        const int mid = lo + (hi - lo) / 2;
        if (p.first[mid + 1] <= s)
            lo = mid + 1;
        else
            hi = mid;
    }
    if (lo >= p.groups) return 0;
    const AtGroup g(p, lo);
    return g.pays && s >= g.s0 && s < g.s1 ? g.tokens : 0;
}

// MIXED: the call has groups, several rows a sequence or many heads that share keys.
template <bool MIXED>
__device__ __forceinline__ AtEntry at_entry(const AtPlan& p, int e)
{
    AtEntry x{};
    if (MIXED && e < p.groups) {
        x.group = x.joined = 1;
        if (!p.whole) {
            const AtGroup g(p, e);
            if (g.pays) {
                x.row0 = g.row0;
                x.rows = g.rows * p.share;
                x.t1 = g.tokens;
                x.table = g.s0;
            }
        }
    } else if (MIXED) {
        const int s = e - p.groups, from = p.row_of(s), count = max(p.row_of(s + 1) - from, 0);
        const int len = p.length(s);
        x.row0 = from;
        x.rows = count * p.share;
        x.t0 = at_shared(p, s);
        x.joined = x.t0 > 0;
        x.t1 = max(len, x.t0);
        x.before = len - count;
        x.table = s;
    } else {
        x.row0 = x.table = e;
        x.rows = p.share;
        x.t1 = p.length(e);
        x.before = x.t1 - 1;
    }
    x.wide = MIXED && x.rows > AT_NARROW;
    x.blocks = x.wide ? (x.rows + AT_WIDE - 1) / AT_WIDE : x.rows > 0;
    x.cost = x.blocks == 0 ? 0 : x.before_block(p, x.blocks);
    return x;
}

// A piece of work: rows of an entry, a head of keys.
struct AtJob {
    int head, rows, rho0, row0, end, before, table, group;
    // row n's row and head of q
    __device__ __forceinline__ int place(const AtPlan& p, int n, size_t& row) const
    {
        const int rho = rho0 + n, at = p.by_share.of(rho);
        row = (size_t)row0 + at;
        return head * p.share + rho - at * p.share;
    }
    // tokens that row n sees
    __device__ __forceinline__ int limit(const AtPlan& p, int n) const
    {
        const int at = p.by_share.of(rho0 + n);
        if (!group) return before + at + 1;
        const int row = row0 + at, s = pg_sequence(p.start, p.seqs, row);
        if (s < 0) return 0;
        return p.length(s) - (p.row_of(s + 1) - 1 - row);
    }
};

struct AtScan {
    long long cost[2][257], slab[257], wave[3][4];
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
// Lane `from`'s number, the same for all.
__device__ __forceinline__ int at_lane(int v, int from) { return __builtin_amdgcn_readlane(v, from); }
__device__ __forceinline__ long long at_lane(long long v, int from)
{
    const int lo = __builtin_amdgcn_readlane((int)v, from), hi = __builtin_amdgcn_readlane((int)(v >> 32), from);
    return (long long)hi << 32 | (unsigned)lo;
}
// Sums of the lanes up to and with this one.
__device__ __forceinline__ long long at_sums(long long v, int lane)
{
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const long long o = __shfl_up(v, d, 64);
        v += lane >= d ? o : 0;
    }
    return v;
}

// The lines' costs, by the whole workgroup: 256 stretches of entries.
template <bool MIXED>
__device__ __forceinline__ void at_scan(const AtPlan& p, AtScan& scan)
{
    const int t = threadIdx.x, lane = t & 63, wave = t >> 6;
    const int entries = p.entries(), chunk = (entries + 255) / 256;
    long long v[3] = {0, 0, 0};  // narrow, wide, slabs
    for (int e = t * chunk; e < min((t + 1) * chunk, entries); ++e) {
        const AtEntry x = at_entry<MIXED>(p, e);
        const long long cost = x.cost * p.kvheads;
        v[0] += x.wide ? 0 : cost;
        if (MIXED) {
            v[1] += x.wide ? cost : 0;
            v[2] += x.slabs() * p.kvheads;
        }
    }
    constexpr int N = MIXED ? 3 : 1;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        v[i] = at_sums(v[i], lane);
        if (lane == 63) scan.wave[i][wave] = v[i];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i)
        for (int w = 0; w < wave; ++w) v[i] += scan.wave[i][w];
    scan.cost[0][t + 1] = v[0];
    if (MIXED) {
        scan.cost[1][t + 1] = v[1];
        scan.slab[t + 1] = v[2];
    }
    if (t == 0) scan.cost[0][0] = scan.cost[1][0] = scan.slab[0] = 0;
    __syncthreads();
}

// A worker's way through its piece of a line: a wave's (narrow jobs) or a
// workgroup's (wide ones).
template <bool MIXED, bool WIDE>
struct AtCursor {
    static constexpr int TILE = AT_TILE[WIDE];
    long long pos, end, quota;
    long long base, slab;  // where the entry's costs, and its whole parts, begin
    int worker, entry;
    AtEntry of;

    __device__ __forceinline__ AtCursor(const AtPlan& p, const AtScan& scan, int worker_, int workers)
    {
        worker = worker_;
        const int lane = threadIdx.x & 63;
        const long long total = at_lane(scan.cost[WIDE][256], 0);
        // a little more than total / workers, which need not be exact
        quota = (long long)((float)total / (float)workers * 1.000001f) + 1;
        if (!p.whole) quota = max(quota, (long long)AT_LEAST[WIDE]);
        pos = worker * quota;
        end = min(pos + quota, total);
        of.cost = 0;
        base = slab = 0;
        entry = 0;
        if (pos >= end) return;
        // the last stretch that begins at or before pos: of 256, four to a lane
        int last = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const unsigned long long at = __ballot(scan.cost[WIDE][64 * i + lane] <= pos);
            if (at != 0) last = 64 * i + 63 - __builtin_clzll(at);
        }
        const int chunk = (p.entries() + 255) / 256;
        base = at_lane(scan.cost[WIDE][last], 0);
        if (MIXED) slab = at_lane(scan.slab[last], 0);
        entry = last * chunk;
    }
    // To the entry that holds pos; each lane looks at one.
    __device__ __forceinline__ bool settle(const AtPlan& p)
    {
        const int lane = threadIdx.x & 63, entries = p.entries();
        for (; entry < entries; entry += 64) {
            AtEntry x{};
            if (entry + lane < entries) x = at_entry<MIXED>(p, entry + lane);
            const long long cost = x.wide == (int)WIDE ? x.cost * p.kvheads : 0;
            const long long sums = at_sums(cost, lane);
            long long slabs = 0, part = 0;
            if (MIXED) {
                part = x.slabs() * p.kvheads;
                slabs = at_sums(part, lane);
            }
            const unsigned long long found = __ballot(base + sums > pos);
            if (found == 0) {
                base += at_lane(sums, 63);
                slab += at_lane(slabs, 63);
                continue;
            }
            const int at = __builtin_ctzll(found);
            base += at_lane(sums - cost, at);
            slab += at_lane(slabs - part, at);
            entry += at;
            of.row0 = at_lane(x.row0, at);
            of.rows = at_lane(x.rows, at);
            of.t0 = at_lane(x.t0, at);
            of.t1 = at_lane(x.t1, at);
            of.before = at_lane(x.before, at);
            of.table = at_lane(x.table, at);
            of.blocks = at_lane(x.blocks, at);
            of.wide = WIDE;
            of.group = at_lane(x.group, at);
            of.joined = at_lane(x.joined, at);
            of.cost = at_lane(x.cost, at);
            return true;
        }
        return false;
    }
    // The next job with tiles in the piece: its tokens from `from` to `to`, and the
    // slab for its results (-1: they are whole, and go to out).
    __device__ __forceinline__ bool next(const AtPlan& p, AtJob& job, int& from, int& to, long long& part)
    {
        while (pos < end) {
            if (of.cost == 0) {
                if (!settle(p)) return false;
            } else if (pos >= base + of.cost * p.kvheads) {
                of.cost = 0;
                continue;
            }
            const int head = at_quotient(pos - base, of.cost);
            const long long rest = pos - base - head * of.cost;
            int b = 0;  // the last block that begins at or before it
            if (WIDE)
                for (int hi = of.blocks - 1; b < hi;) {
                    const int mid = (b + hi + 1) / 2;
                    if (of.before_block(p, mid) <= rest)
                        b = mid;
                    else
                        hi = mid - 1;
                }
            const long long c0 = of.before_block(p, b), c1 = of.before_block(p, b + 1);
            const long long x = rest - c0, y = min(x + end - pos, c1 - c0);
            job.end = of.end(p, b);
            const int tiles = max(1, (job.end - of.t0 + TILE - 1) / TILE);
            int t0 = 0, t1 = tiles;
            if (!p.whole) {
                t0 = (int)min((x + TILE - 1) / TILE, (long long)tiles);
                t1 = (int)min((y + TILE - 1) / TILE, (long long)tiles);
            }
            pos += y - x;
            if (t0 >= t1) continue;
            job.head = head;
            job.rho0 = b * of.block_rows();
            job.rows = min(of.rows - job.rho0, of.block_rows());
            job.row0 = of.row0;
            job.before = of.before;
            job.table = of.table;
            job.group = of.group;
            from = of.t0 + t0 * TILE;
            to = min(of.t0 + t1 * TILE, job.end);
            part = -1;
            if (p.whole) return true;
            if (t0 > 0 || t1 < tiles)
                part = WIDE ? (2ll * worker + (t0 == 0)) * AT_SLABS : p.narrow_at + 2ll * worker + (t0 == 0);
            else if (of.joined)
                part = p.whole_at + slab + head * of.slabs() + (long long)b * of.block_slabs();
            if (part + of.block_slabs() > p.slabs) continue;  // (starts that do not ascend)
            if (t0 == 0) note(p, job, part, t1 < tiles ? c0 + (long long)(tiles - 1) * TILE - rest - (y - x) : -1);
            return true;
        }
        return false;
    }
    // For the join: where the parts of the job's rows are.  behind: how far behind the
    // piece the last tile begins, -1 where the job is whole.
    __device__ __forceinline__ void note(const AtPlan& p, const AtJob& job, long long part, long long behind)
    {
        const int count = behind >= 0 ? 2 + at_quotient(behind, quota) : of.joined;
        const int n = WIDE ? threadIdx.x : threadIdx.x & 63;
        if (n < job.rows) {
            size_t row;
            const int head = job.place(p, n, row);
            // the number of parts, the row in its slab, whether shared parts are to be added
            const int what = count == 0 ? 0 : count | (n % AT_NARROW) << 16 | of.joined << 24 | (int)WIDE << 25;
            (job.group ? p.shared_parts : p.own)[row * p.heads + head] =
                make_int2(part < 0 ? 0 : (int)(part + n / AT_NARROW), what);
        }
    }
};

// Slab of part i of a row: the first one's, then one of each of the next workers.
__device__ __forceinline__ long long at_part(int2 where, int i)
{
    const int step = where.y >> 25 & 1 ? AT_SLABS : 1;
    return where.x + (i == 0 ? 0ll : (2ll * i - 1) * step);
}

}  // namespace xsymv
