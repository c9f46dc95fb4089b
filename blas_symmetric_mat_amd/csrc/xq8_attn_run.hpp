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

// Workspace: where the rows' parts are, and their slabs: of cut jobs (two a worker),
// and where groups share tokens of whole ones.
struct AttnSpace {
    size_t shared, parts, narrow, whole, slabs, bytes;
    AttnSpace(int rows, int heads, int kvheads, int hd, int seqs, int groups, bool single)
    {
        const size_t share = heads / kvheads, table = align_up((size_t)rows * heads * sizeof(int2));
        shared = table;
        parts = groups > 0 ? 2 * table : table;
        narrow = attn_mixed(heads, kvheads, groups, single) ? 2 * (size_t)AT_GRID * AT_SLABS : 0;
        whole = narrow + 2 * 4 * (size_t)AT_GRID;
        slabs = whole;
        if (groups > 0) {
            const size_t blocks = (size_t)rows * share / AT_WIDE;
            const size_t own = single ? seqs * (share <= AT_NARROW ? 1 : (share + AT_WIDE - 1) / AT_WIDE * AT_SLABS)
                                      : (blocks + seqs) * AT_SLABS;
            slabs += kvheads * (own + (blocks + groups) * AT_SLABS);
        }
        bytes = parts + slabs * at_slab(hd) * sizeof(float);
    }
};

template <class T, int HD, bool MIXED>
int attn_launch(AttnArgs<T> a, hipStream_t stream)
{
    AtPlan& p = a.p;
    // Tiles that a line has at most.  (Where an int might not count them, no job is cut;
    // the call takes minutes.)
    const double blocks = (double)p.rows * p.share / AT_WIDE + p.seqs + p.groups;
    const double line = blocks * p.kvheads * (((double)p.ldt * p.ps) / AT_TILE[0] + AT_OVER + 2);
    // Sequences of a piece at most are whole as they are: one launch.
    const bool cut = line < 2e9 && (p.groups > 0 || (long long)p.ldt * p.ps > AT_LEAST * AT_TILE[0]);
    const AttnSpace space(p.rows, p.heads, p.kvheads, p.hd, p.seqs, p.groups, p.start == nullptr);
    int resident = 0;
    const int rc = resident_blocks(reinterpret_cast<const void*>(&q8_attn<T, HD, MIXED>), 256, &resident);
    if (rc) return rc;
    return q8_with_workspace(cut ? space.bytes : 0, true, stream, [&](void* ws, const TimedCall& tc) -> int {
        p.whole = ws == nullptr;
        // no more than there can be pieces
        const long long jobs = ((long long)p.rows * p.share / AT_WIDE + p.seqs) * p.kvheads;
        const long long tiles = p.whole ? 1 : (long long)p.ldt * p.ps / AT_TILE[0] + 1 + AT_OVER;
        // (as many for every die, and for the four engines of each)
        const long long most = MIXED ? jobs * tiles + p.groups : (jobs * tiles + 3) / 4;
        const long long step = MIXED ? 32 : 8;
        p.grid = (int)std::min(std::min((long long)resident, (long long)AT_GRID) / step * step,
                               std::max(1ll, (most + step - 1) / step) * step);
        if (!p.whole) {
            char* at = static_cast<char*>(ws);
            p.own = reinterpret_cast<int2*>(at);
            p.shared_parts = reinterpret_cast<int2*>(at + space.shared);
            p.slabs = (int)space.slabs;
            p.narrow_at = (int)space.narrow;
            p.whole_at = (int)space.whole;
            a.slabs = reinterpret_cast<float*>(at + space.parts);
        }
        XSYMV_HIP(launch_k(&q8_attn<T, HD, MIXED>, dim3(MIXED ? 2 * p.grid : p.grid), dim3(256), stream, a, tc.e0, tc.e1));
        if (p.whole) return 0;
        // Four waves for a row and head where there are few, else one for several.
        const long long all = (long long)p.rows * p.heads;
        const bool few = all <= 4096;
        a.per = few ? 1 : (int)std::min(std::max(all / 8192, 1ll), 64ll);
        const long long each = few ? 1 : 4 * a.per;
        XSYMV_HIP(launch_k(few ? &q8_attn_join<T, 4> : &q8_attn_join<T, 1>, dim3((unsigned)((all + each - 1) / each)),
                           dim3(256), stream, a, nullptr, tc.e2));
        return 0;
    });
}

template <class T, int HD>
int attn_width(const AttnArgs<T>& a, hipStream_t stream)
{
    const AtPlan& p = a.p;
    return attn_mixed(p.heads, p.kvheads, p.groups, p.start == nullptr) ? attn_launch<T, HD, true>(a, stream)
                                                                        : attn_launch<T, HD, false>(a, stream);
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
    if ((long long)rows * heads > 0x7fffffffll) return -1;
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
    if (hd <= 64) return attn_width<T, 64>(a, stream);
    if (hd <= 128) return attn_width<T, 128>(a, stream);
    return attn_width<T, 256>(a, stream);
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
