// xq8_attn_run.hpp -- a call of the attention over a cache of 8-bit rows: checks
// and launch (kernels: xq8_attn.hpp).  The units xq8_attn_[shb].hip compile it.
#pragma once

#include "xq8_attn.hpp"
#include "xq8_host.hpp"

#include <cmath>

namespace xsymv {

// Workgroups at most: what two a compute unit are.
constexpr int AT_GRID = 512;

// A call of single tokens with nothing in common and few heads that share keys has
// narrow jobs alone.
inline bool attn_mixed(int heads, int kvheads, int groups, bool single)
{
    return !single || groups > 0 || heads / kvheads > AT_NARROW;
}

// Rows of a wide job: 256, or 128 (AtWide::ROWS).
constexpr int AT_WIDE = 256, AT_LESS = 128;

// Workspace: where the rows' parts are, and their slabs: of cut jobs (two a worker),
// and where groups share tokens of whole ones.
struct AttnSpace {
    size_t shared, parts, narrow, whole, slabs, bytes;
    AttnSpace(int rows, int heads, int kvheads, int hd, int seqs, int groups, bool single)
    {
        const size_t share = heads / kvheads, table = align_up((size_t)rows * heads * sizeof(int2));
        shared = table;
        parts = groups > 0 ? 2 * table : table;
        // (256 workgroups of 256 rows)
        narrow = attn_mixed(heads, kvheads, groups, single) ? 2 * (size_t)AT_GRID * AT_LESS / AT_NARROW : 0;
        whole = narrow + 2 * 4 * (size_t)AT_GRID;
        slabs = whole;
        if (groups > 0) {
            const size_t most = AT_WIDE / AT_NARROW, all = (size_t)rows * share / AT_NARROW;
            const size_t own = single && share <= AT_NARROW ? seqs : all + seqs * most;
            slabs += kvheads * (own + all + groups * most);
        }
        bytes = parts + slabs * at_slab(hd) * sizeof(float);
    }
};

// Workgroups of a kernel: as many for every die, and no more than can have work.
template <class K>
int attn_grid(K* kernel, int threads, long long most, int& grid)
{
    int resident = 0;
    const int rc = resident_blocks(reinterpret_cast<const void*>(kernel), threads, &resident);
    const long long room = std::min((long long)resident, (long long)AT_GRID * 256 / threads);
    grid = (int)std::max(8ll, std::min(room / 8, std::max(1ll, (most + 7) / 8)) * 8);
    return rc;
}

template <class T, int LANES>
int attn_join(const AttnArgs<T>& a, hipStream_t stream, hipEvent_t stop)
{
    // More waves for rows and heads where there are few, which may have many parts: two
    // rows of 32 heads over 131072 tokens, 128 parts each, take 14 us by four waves and 9
    // by sixteen; one over 1000, 16 parts each, 2 us more by sixteen than by four.
    const long long all = (long long)a.p.rows * a.p.heads;
    const int waves = all <= 256 && (long long)a.p.ldt * a.p.ps > 4096 ? 16 : all <= 4096 ? 4 : 1;
    const long long each = 64 / LANES * (waves > 1 ? 1 : 4);
    XSYMV_HIP(launch_k(waves == 16  ? &q8_attn_join<T, LANES, 16>
                       : waves == 4 ? &q8_attn_join<T, LANES, 4>
                                    : &q8_attn_join<T, LANES, 1>,
                       dim3((unsigned)((all + each - 1) / each)), dim3(waves > 4 ? 64 * waves : 256), stream, a,
                       nullptr, stop));
    return 0;
}

template <class T, int HD>
int attn_launch(AttnArgs<T> a, hipStream_t stream)
{
    AtPlan& p = a.p;
    const bool single = p.start == nullptr, mixed = attn_mixed(p.heads, p.kvheads, p.groups, single);
    // Tiles that a line has at most.  (Where an int might not count them, no job is cut;
    // the call takes minutes.)
    const double blocks = (double)p.rows * p.share / AT_LESS + p.seqs + p.groups;
    const double line = blocks * p.kvheads * (((double)p.ldt * p.ps) / AT_TILE + AT_OVER_WIDE + 2);
    // Sequences of a piece at most are whole as they are: one launch.
    const bool cut = line < 2e9 && (p.groups > 0 || (long long)p.ldt * p.ps > AT_LEAST * AT_TILE);
    const AttnSpace space(p.rows, p.heads, p.kvheads, p.hd, p.seqs, p.groups, single);
    return q8_with_workspace(cut ? space.bytes : 0, true, stream, [&](void* ws, const TimedCall& tc) -> int {
        constexpr int threads = 64 * AtWide<T, HD>::WAVES;
        p.whole = ws == nullptr;
        p.wide_log = AtWide<T, HD>::ROWS == AT_WIDE ? 8 : 7;
        if (!p.whole) {
            char* at = static_cast<char*>(ws);
            p.own = reinterpret_cast<int2*>(at);
            p.shared_parts = reinterpret_cast<int2*>(at + space.shared);
            p.slabs = (int)space.slabs;
            p.narrow_at = (int)space.narrow;
            p.whole_at = (int)space.whole;
            a.slabs = reinterpret_cast<float*>(at + space.parts);
        }
        hipEvent_t start = tc.e0;
        if (mixed) {
            // Single tokens of few heads are narrow jobs: only groups' may be wide.
            p.wide_entries = p.groups + (single && p.share <= AT_NARROW ? 0 : p.seqs);
            if (p.whole && single && p.share <= AT_NARROW) p.wide_entries = 0;
            // (a launch without jobs: one token over 1000 21 us with it, 15 without)
            if ((long long)p.rows * p.share <= AT_NARROW) p.wide_entries = 0;
            const long long most = p.whole ? (long long)std::min(blocks * p.kvheads, 1e9) : 1ll << 30;
            const int rc = p.wide_entries > 0 ? attn_grid(&q8_attn_wide<T, HD>, threads, most, p.grid) : 0;
            if (rc) return rc;
            if (p.wide_entries > 0) {
                XSYMV_HIP(launch_k(&q8_attn_wide<T, HD>, dim3(p.grid), dim3(threads), stream, a, start, nullptr));
                start = nullptr;
            }
        }
        // A line of narrow jobs has no more tiles than this.
        const double tiles = p.whole ? 1.0 : ((double)p.ldt * p.ps / AT_TILE + 1 + AT_OVER) / AT_LEAST;
        const long long most = (long long)std::min(((double)p.seqs + p.groups) * p.kvheads * tiles / 4 + 1, 1e9);
        auto* narrow = mixed ? &q8_attn_narrow<T, HD, AT_NARROW_JOBS> : &q8_attn_narrow<T, HD, AT_SINGLE_JOBS>;
        const int rc = attn_grid(narrow, 256, most, p.grid);
        if (rc) return rc;
        XSYMV_HIP(launch_k(narrow, dim3(p.grid), dim3(256), stream, a, start, tc.e1));
        if (p.whole) return 0;
        return HD == 64 ? attn_join<T, 16>(a, stream, tc.e2)
                        : HD == 128 ? attn_join<T, 32>(a, stream, tc.e2) : attn_join<T, 64>(a, stream, tc.e2);
    });
}

template <class T>
int attn_run(int rows, int heads, int kvheads, int hd, const T* q, int ldq, int seqs, const int* start,
             const int* len, const int* table, int ldt, int groups, const int* first, const int* shared,
             const signed char* k, int ldk, const float* ks, const signed char* v, int ldv, const float* vs,
             int pages, int ps, float scale, T* out, int ldo, float* lse, hipStream_t stream)
{
    if (rows < 0) return -1;
    if (heads < 1 || (kvheads >= 1 && heads % kvheads != 0)) return -2;
    if (kvheads < 1) return -3;
    if ((long long)rows * heads > 0x7fffffffll) return -1;
    if (hd < AT_LOW || hd > AT_HD) return -4;
    const long long wide = (long long)heads * hd;
    if (wide > 0x7fffffffll) return -2;
    const bool some = rows > 0 && (seqs > 0 || start == nullptr);
    if (some && q == nullptr) return -5;
    if (ldq < wide) return -6;
    if (seqs < 0 || (start == nullptr && seqs != rows) || seqs > AT_ENTRIES) return -7;
    const bool tokens = some && ldt > 0 && pages > 0;
    if (some && len == nullptr) return -9;
    if (tokens && table == nullptr) return -10;
    if (ldt < 0) return -11;
    if (groups < 0 || groups > AT_ENTRIES - seqs) return -12;
    if (tokens && groups > 0 && first == nullptr) return -13;
    if (tokens && groups > 0 && shared == nullptr) return -14;
    if (tokens && k == nullptr) return -15;
    if (ldk < hd) return -16;
    if (tokens && ks == nullptr) return -17;
    if (tokens && v == nullptr) return -18;
    if (ldv < hd) return -19;
    if (tokens && vs == nullptr) return -20;
    if (pages < 0) return -21;
    if (ps >= 1 && ((long long)pages * ps > 0x7fffffffll || (long long)pages * ps * kvheads > 0x7fffffffll))
        return -21;
    if (ps < 1) return -22;
    if (!std::isfinite(scale)) return -23;
    if (some && out == nullptr) return -24;
    if (ldo < wide) return -25;
    if (!some) return 0;
    AttnArgs<T> a{};
    AtPlan& p = a.p;
    p.start = start;
    p.len = len;
    p.table = table;
    p.first = first;
    p.shared = shared;
    p.rows = rows;
    p.heads = heads;
    p.kvheads = kvheads;
    p.share = heads / kvheads;
    p.hd = hd;
    p.seqs = seqs;
    p.ldt = tokens ? ldt : 0;
    p.groups = tokens ? groups : 0;
    p.pages = pages;
    p.ps = ps;
    p.by_share = AtDivisor(p.share);
    p.by_page = AtDivisor(ps);
    a.q = q;
    a.out = out;
    a.lse = lse;
    a.k = k;
    a.v = v;
    a.ks = ks;
    a.vs = vs;
    a.scale = scale * 1.4426950408889634f;
    a.ldq = ldq;
    a.ldk = ldk;
    a.ldv = ldv;
    a.ldo = ldo;
    if (hd <= 64) return attn_launch<T, 64>(a, stream);
    if (hd <= 128) return attn_launch<T, 128>(a, stream);
    return attn_launch<T, 256>(a, stream);
}

}  // namespace xsymv

#define XSYMV_Q8_ATTN(L, CT, T)                                                                               \
    extern "C" int xsymv_q8attn_##L(int rows, int heads, int kvheads, int hd, const CT* q, int ldq,           \
                                    int seqs, const int* start, const int* len, const int* table,             \
                                    int ldt, int groups, const int* first, const int* shared,                 \
                                    const signed char* k, int ldk, const float* ks, const signed char* v,     \
                                    int ldv, const float* vs, int pages, int ps, float scale, CT* out,        \
                                    int ldo, float* lse, void* stream)                                        \
    {                                                                                                         \
        return xsymv::q8_guard([&] {                                                                          \
            return xsymv::attn_run<T>(rows, heads, kvheads, hd, reinterpret_cast<const T*>(q), ldq, seqs,     \
                                      start, len, table, ldt, groups, first, shared, k, ldk, ks, v, ldv, vs,  \
                                      pages, ps, scale, reinterpret_cast<T*>(out), ldo, lse,                  \
                                      (hipStream_t)stream);                                                   \
        });                                                                                                   \
    }
