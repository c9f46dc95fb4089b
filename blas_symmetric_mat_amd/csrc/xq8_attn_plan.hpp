// xq8_attn_plan.hpp -- how the attention's work is cut into jobs and pieces.
//
// An entry is a stretch of rows of q with the tokens that they read: first the
// groups (rows of their sequences, the shared tokens), then the sequences (their
// rows, the tokens that are not read for a group).  Each head of keys and each
// block of an entry's rows is a job.  A row of an entry is a row of q and one of
// the `share` heads of q that read the same keys; blocks are of 16 rows where an
// entry has no more (narrow), else of 256 (wide; 128 where registers hold no more).
//
// There are two lines of jobs, one after the other by entry, head and block: wide
// jobs, of which every workgroup of q8_attn_wide takes an equal piece, and narrow
// ones, of which every wave of q8_attn_narrow does.  Lines are counted in tiles (32
// tokens): a job's tiles come first in its stretch of the line, then some that stand
// for what a job takes besides.  Stretches may be longer than need be, but have to be
// the same for all workers, which compute them from the arrays on the device, so that
// a captured call follows what these hold.  A single sequence's step waits for
// this: it is some hundred instructions, with sums over lanes (64 entries at a time).
//
// Who takes a job's first tile writes down, for each of its rows, where the parts of
// its results are; the join reads that.
#pragma once

#include <hip/hip_runtime.h>

#include "xq8_cache.hpp"

namespace xsymv {

constexpr int AT_LOW = 16, AT_HD = 256;  // least and widest head
constexpr int AT_NARROW = 16;            // rows of a narrow job, and of a slab
constexpr int AT_TILE = 32;              // tokens of a tile
// Tiles that a job takes besides its own: a narrow one, a wide one (20 us for its rows
// of q and its results, when a step of 128 tokens takes 7).  In us, one state of 32 heads
// on 8 at a time (64 tokens behind 16384 shared ones and 600 each, 200 over 500 each; two
// times 100 rows behind 4096): narrow 0, 3, 8: 85, 81, 84 and 45, 42, 46; wide 4, 12, 30:
// 86, 81, 81 and 61, 58, 63.
constexpr int AT_OVER = 3, AT_OVER_WIDE = 12;
// A piece is so many tiles at least, for the join's sake (narrow, wide: a step).  Narrow
// 1, 2, 6: one token over 1000 14.5, 15.2, 18.9, the 64 tokens 81, 81, 87; wide 4, 12: nine
// sequences of 5 rows behind 1500 tokens 38, 48.
constexpr int AT_LEAST = 2, AT_LEAST_WIDE = 4;
// Entries of a call at most: windows of 64, of which LDS holds the sums.
constexpr int AT_WINDOWS = 1024, AT_ENTRIES = 64 * AT_WINDOWS;

// Floats of a slab, the results of 16 rows in a part of a job: m and l of each, then
// their out, not yet divided by l, in the order in which a wave stores it (at_part_of).
__host__ __device__ inline size_t at_slab(int hd)
{
    return (size_t)AT_NARROW * (2 + (hd <= 64 ? 64 : hd <= 128 ? 128 : 256));
}

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
    int wide_log;  // of a wide job's rows
    __host__ __device__ __forceinline__ int wide_rows() const { return 1 << wide_log; }
    __host__ __device__ __forceinline__ int wide_slabs() const { return 1 << wide_log >> 4; }
    // Workspace: slabs (of cut wide jobs' parts, two a workgroup; of cut
    // narrow ones', two a wave; of whole parts) and, for each row and head, where its
    // own parts and its group's are.
    int slabs, narrow_at, whole_at;
    int2 *own, *shared_parts;

    int wide_entries;  // of the first, those that can be wide
    __device__ __forceinline__ int room() const { return (int)min((long long)ldt * ps, 0x7fffff00ll); }
    __device__ __forceinline__ int length(int s) const { return min(max(len[s], 0), room()); }
    __device__ __forceinline__ int row_of(int s) const
    {
        return start != nullptr ? min(max(start[s], 0), rows) : s;
    }
};

// Floor of a / b for a >= 0, b > 0: a division in floating point, put right.
__device__ __forceinline__ int at_quotient(int a, int b)
{
    int q = (int)((float)a * __builtin_amdgcn_rcpf((float)b));
    q = min(q, a);
    while ((long long)q * b > a) --q;
    while ((long long)(q + 1) * b <= a) ++q;
    return q;
}

struct AtEntry {
    int row0, rows;  // the first row of q; rows of the entry
    int t0, t1;      // tokens
    int before;      // tokens before the first row's own (a sequence's)
    int table;       // the row of the table that is read
    int wide, group, joined;
    int mine;  // whether its jobs are of the kernel's kind
    int cost;  // tiles of one head

    __device__ __forceinline__ int block_slabs(const AtPlan& p) const { return wide ? p.wide_slabs() : 1; }
    __device__ __forceinline__ int blocks(const AtPlan& p) const
    {
        return wide ? (rows + p.wide_rows() - 1) >> p.wide_log : rows > 0;
    }
    __device__ __forceinline__ int slabs(const AtPlan& p) const { return joined ? blocks(p) * block_slabs(p) : 0; }
    static __device__ __forceinline__ int tiles(int tokens) { return (tokens + AT_TILE - 1) / AT_TILE; }
    // length of the blocks before block b, of an entry of the kernel's kind
    template <bool WIDE>
    __device__ __forceinline__ int before_block(const AtPlan& p, int b) const
    {
        if (p.whole) return b;
        if constexpr (!WIDE) return b * (AT_OVER + tiles(t1 - t0));
        // (more rows than tokens, or heads of a row than a block: any block as one that sees all.
        // The sums below are of steps of whole tokens, of which such blocks have none or less
        // than one each, and no int would hold them: from 370000 blocks on.)
        if (group || before < 0 || p.share >= p.wide_rows()) return b * (AT_OVER_WIDE + tiles(t1 - t0));
        // block b sees up to step * (b + 1) tokens more than what lies before the
        // rows; the sums of these are rounded down, for which one tile makes up
        const int step = p.by_share.of(p.wide_rows() + p.share - 1);
        return b * (AT_OVER_WIDE + 1 + tiles(max(before - t0, 0))) +
               (int)((long long)b * (b + 1) / 2 * step / AT_TILE);
    }
    // end of the tokens that block b sees
    __device__ __forceinline__ int end(const AtPlan& p, int b) const
    {
        if (group) return t1;
        const int last = wide ? (int)min((long long)(b + 1) << p.wide_log, (long long)rows) - 1 : rows - 1;
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
            // A quarter less, as rows that have two entries are added by the join.  Counted is
            // work alone, so short stretches are shared though starts and ends then cost more
            // than is saved: in us, never and always shared, 64 tokens behind 16384 276, 81;
            // two and three behind 65536 56, 42 and 75, 42; but eight behind 4096 30, 37, nine
            // sequences of 5 rows behind 1500 28, 37; prompts of 1024 rows, which the rule
            // leaves alone, 690, 738.
            pays = work(p, (long long)rows * p.share) * 4 <= count * work(p, one) * 3;
        }
    }
    // The sequence whose row of the table is read: the first one that has all the shared
    // tokens, else the longest (others may have ended, and their pages be free).
    __device__ __forceinline__ int table(const AtPlan& p) const
    {
        int best = s0, most = -1;
        for (int s = s0; s < s1 && most < tokens; s += 8) {
            int len[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) len[i] = s + i < s1 ? p.length(s + i) : -1;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                if (most < tokens && len[i] > most) {
                    most = len[i];
                    best = s + i;
                }
            }
        }
        return best;
    }
    // A wide job counts as two narrow ones with as many tokens, which the times above bear out
    // for long stretches.  (In a compute unit's time a tile of a full wide job is a quarter of 7
    // us, one of a narrow job 0.3 us where memory is the bound.)
    static __device__ __forceinline__ long long work(const AtPlan& p, long long rows)
    {
        return rows <= AT_NARROW ? 1 : (rows + p.wide_rows() - 1) >> p.wide_log << 1;
    }
};

// The tokens that sequence s reads with its group, 0: none.
__device__ __forceinline__ int at_shared(const AtPlan& p, int s)
{
    if (p.whole || p.groups == 0) return 0;
    int lo = 0, hi = p.groups > 1 ? p.groups : 0;  // the last group that begins at or before s
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

// Which jobs a kernel makes: wide ones, narrow ones, or all of a call that has neither
// groups nor several rows a sequence nor many heads that share keys.
enum AtKind { AT_WIDE_JOBS, AT_NARROW_JOBS, AT_SINGLE_JOBS };

template <AtKind KIND>
__device__ __forceinline__ AtEntry at_entry(const AtPlan& p, int e)
{
    constexpr bool MIXED = KIND != AT_SINGLE_JOBS;
    AtEntry x{};
    if (MIXED && e < p.groups) {
        x.group = x.joined = 1;
        if (!p.whole) {
            const AtGroup g(p, e);
            if (g.pays) {
                x.row0 = g.row0;
                x.rows = g.rows * p.share;
                x.t1 = g.tokens;
                x.table = g.table(p);
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
    x.mine = MIXED ? x.wide == (KIND == AT_WIDE_JOBS) : 1;
    x.cost = x.before_block<KIND == AT_WIDE_JOBS>(p, x.blocks(p));
    return x;
}

// A piece of work: rows of an entry, a head of keys.
struct AtJob {
    int head, rows, rho0, row0, before, table, group;
    int end;  // of the piece's tokens
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

// Sums of 64 entries each: tiles, slabs.
template <AtKind KIND>
struct AtScan {
    int sums[KIND == AT_SINGLE_JOBS ? 1 : 2][AT_WINDOWS];
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
// Sums of the lanes up to and with this one.
__device__ __forceinline__ int at_sums(int v)
{
    // within rows of 16 lanes, then the last lanes of the rows before
    v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xf, 0xf, true);  // from 1, 2, 4, 8 lanes before
    v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xf, 0xf, true);
    v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xf, 0xf, true);
    v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xf, 0xf, true);
    v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xa, 0xf, true);  // lane 15 to row 1, 47 to row 3
    v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xc, 0xf, true);  // lane 31 to rows 2 and 3
    return v;
}

// 64 entries, one a lane, and their sums up to and with the lane's.
template <AtKind KIND>
struct AtWindow {
    static constexpr int N = KIND == AT_SINGLE_JOBS ? 1 : 2;
    AtEntry x;
    int own[N], sums[N];  // tiles, slabs
    static __device__ __forceinline__ int entries(const AtPlan& p)
    {
        return KIND == AT_WIDE_JOBS ? p.wide_entries : p.groups + p.seqs;
    }
    __device__ __forceinline__ void load(const AtPlan& p, int window)
    {
        const int e = window * 64 + (threadIdx.x & 63);
        x = AtEntry{};
        if (e < entries(p)) x = at_entry<KIND>(p, e);
        own[0] = x.mine ? x.cost * p.kvheads : 0;
        if constexpr (N > 1) own[1] = x.slabs(p) * p.kvheads;
#pragma unroll
        for (int i = 0; i < N; ++i) sums[i] = at_sums(own[i]);
    }
    __device__ __forceinline__ int all(int i) const { return at_lane(sums[i], 63); }
};

// The whole line: its length, and with more than 64 entries the windows' sums.
template <AtKind KIND>
struct AtLines {
    AtWindow<KIND> w;
    int total, windows;
    __device__ __forceinline__ AtLines(const AtPlan& p, AtScan<KIND>& scan)
    {
        const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
        windows = (AtWindow<KIND>::entries(p) + 63) / 64;
        if (windows <= 1) {
            w.load(p, 0);
            total = w.all(0);
            return;
        }
        for (int i = wave; i < windows; i += (int)blockDim.x >> 6) {
            w.load(p, i);
            if (lane == 63)
#pragma unroll
                for (int j = 0; j < AtWindow<KIND>::N; ++j) scan.sums[j][i] = w.sums[j];
        }
        __syncthreads();
        total = 0;
        for (int i = 0; i < windows; i += 64)
            total += at_lane(at_sums(i + lane < windows ? scan.sums[0][i + lane] : 0), 63);
    }
};

// A worker's way through its piece of a line: a wave's (narrow jobs) or a
// workgroup's (wide ones).
template <AtKind KIND>
struct AtCursor {
    static constexpr bool WIDE = KIND == AT_WIDE_JOBS, MIXED = KIND != AT_SINGLE_JOBS;
    int pos, end, quota;
    int base, slab;  // where the window's tiles, and its whole parts, begin
    int worker, window, windows;
    int first, parts;  // the same of the entry
    AtEntry of;

    __device__ __forceinline__ AtCursor(const AtPlan& p, const AtScan<KIND>& scan, const AtLines<KIND>& lines,
                                        int worker_, int workers)
    {
        AtWindow<KIND> w = lines.w;
        worker = worker_;
        const int lane = threadIdx.x & 63, total = lines.total;
        // a little more than total / workers, which need not be exact
        quota = (int)((float)total * __builtin_amdgcn_rcpf((float)workers) * 1.00001f) + 1;
        if (!p.whole) quota = max(quota, WIDE ? AT_LEAST_WIDE : AT_LEAST);
        const long long at = (long long)worker * quota;
        pos = (int)min(at, (long long)total);
        end = (int)min(at + quota, (long long)total);
        base = slab = window = 0;
        windows = lines.windows;
        if (pos >= end) return;
        if (windows > 1) {
            for (int i = 0; i < windows; i += 64) {
                const bool some = i + lane < windows;
                const int v = some ? scan.sums[0][i + lane] : 0, sums = at_sums(v);
                int part = 0, slabs = 0;
                if constexpr (MIXED) {
                    part = some ? scan.sums[1][i + lane] : 0;
                    slabs = at_sums(part);
                }
                const unsigned long long found = __ballot(base + sums > pos);
                if (found != 0) {
                    const int in = __builtin_ctzll(found);
                    window = i + in;
                    base += at_lane(sums - v, in);
                    slab += at_lane(slabs - part, in);
                    break;
                }
                base += at_lane(sums, 63);
                slab += at_lane(slabs, 63);
            }
            w.load(p, window);
        }
        if (!find(w)) end = pos;
    }
    // The window's entry that holds pos.
    __device__ __forceinline__ bool find(const AtWindow<KIND>& w)
    {
        const unsigned long long found = __ballot(base + w.sums[0] > pos);
        if (found == 0) return false;
        const int at = __builtin_ctzll(found);
        first = base + at_lane(w.sums[0] - w.own[0], at);
        parts = 0;
        if constexpr (MIXED) parts = slab + at_lane(w.sums[1] - w.own[1], at);
        of.row0 = at_lane(w.x.row0, at);
        of.rows = at_lane(w.x.rows, at);
        of.t0 = at_lane(w.x.t0, at);
        of.t1 = at_lane(w.x.t1, at);
        of.before = at_lane(w.x.before, at);
        of.table = at_lane(w.x.table, at);
        of.wide = WIDE;
        of.group = MIXED ? at_lane(w.x.group, at) : 0;
        of.joined = MIXED ? at_lane(w.x.joined, at) : 0;
        of.cost = at_lane(w.x.cost, at);
        return of.cost > 0;
    }
    // To the entry that holds pos, in this window or one behind it.  (Read again rather
    // than kept in registers while jobs run.)
    __device__ __forceinline__ bool settle(const AtPlan& p)
    {
        for (; window < windows; ++window) {
            AtWindow<KIND> w;
            w.load(p, window);
            if (find(w)) return true;
            base += w.all(0);
            if constexpr (MIXED) slab += w.all(1);
        }
        return false;
    }
    // The next job with tiles in the piece: its tokens from `from` to `to`, and the
    // slab for its results (-1: they are whole, and go to out).
    __device__ __forceinline__ bool next(const AtPlan& p, AtJob& job, int& from, int& to, int& part)
    {
        while (pos < end) {
            if (pos - first >= of.cost * p.kvheads && !settle(p)) return false;
            const int head = at_quotient(pos - first, of.cost), rest = pos - first - head * of.cost;
            int b = 0;  // the last block that begins at or before it
            if (WIDE)
                for (int hi = of.blocks(p) - 1; b < hi;) {
                    const int mid = (b + hi + 1) / 2;
                    if (of.template before_block<WIDE>(p, mid) <= rest)
                        b = mid;
                    else
                        hi = mid - 1;
                }
            const int c0 = WIDE ? of.template before_block<WIDE>(p, b) : 0;
            const int c1 = WIDE ? of.template before_block<WIDE>(p, b + 1) : of.cost;
            const int x = rest - c0, y = min(x + end - pos, c1 - c0);
            // (starts that do not ascend: sums that no int holds)
            if ((unsigned)head >= (unsigned)p.kvheads || y <= x) return false;
            job.end = of.end(p, b);
            const int tiles = max(1, of.tiles(job.end - of.t0));
            const int t0 = p.whole ? 0 : min(x, tiles), t1 = p.whole ? tiles : min(y, tiles);
            pos += y - x;
            if (t0 >= t1) continue;
            job.head = head;
            job.rho0 = WIDE ? b << p.wide_log : 0;
            job.rows = min(of.rows - job.rho0, WIDE ? p.wide_rows() : AT_NARROW);
            job.row0 = of.row0;
            job.before = of.before;
            job.table = of.table;
            job.group = of.group;
            from = of.t0 + t0 * AT_TILE;
            to = min(of.t0 + t1 * AT_TILE, job.end);
            job.end = to;
            part = -1;
            if (p.whole) return true;
            if (t0 > 0 || t1 < tiles)
                part = WIDE ? (2 * worker + (t0 == 0)) * p.wide_slabs() : p.narrow_at + 2 * worker + (t0 == 0);
            else if (of.joined)
                part = p.whole_at + parts + head * of.slabs(p) + b * of.block_slabs(p);
            if (part < -1 || part > p.slabs - of.block_slabs(p)) continue;  // (the same)
            if (t0 == 0) note(p, job, part, t1 < tiles ? tiles - 1 - y : -1);
            return true;
        }
        return false;
    }
    // For the join: where the parts of the job's rows are.  behind: how far behind the
    // piece the last tile begins, -1 where the job is whole.
    __device__ __forceinline__ void note(const AtPlan& p, const AtJob& job, int part, int behind)
    {
        const int count = behind >= 0 ? 2 + at_quotient(behind, quota) : of.joined;
        const int n = WIDE ? threadIdx.x : threadIdx.x & 63;
        if (n < job.rows) {
            size_t row;
            const int head = job.place(p, n, row);
            // the number of parts, the row in its slab, whether shared parts are to be added
            const int what = count == 0 ? 0 : count | (n % AT_NARROW) << 16 | of.joined << 24 | (int)WIDE << 25;
            (job.group ? p.shared_parts : p.own)[row * p.heads + head] =
                make_int2(part < 0 ? 0 : part + n / AT_NARROW, what);
        }
    }
};

// Slab of part i of a row: the first one's, then one of each of the next workers.
__device__ __forceinline__ long long at_part(const AtPlan& p, int2 where, int i)
{
    const int step = where.y >> 25 & 1 ? p.wide_slabs() : 1;
    return where.x + (i == 0 ? 0ll : (2ll * i - 1) * step);
}

}  // namespace xsymv
