// xq8_attn_run.hpp -- a call of the attention over a cache of 8-bit rows: checks
// and launch (kernels: xq8_attn.hpp).  The units xq8_attn_[shb].hip compile it.
#pragma once

#include "xq8_attn.hpp"
#include "xq8_host.hpp"

#include <cmath>

namespace xsymv {

// Workgroups at most: what two a compute unit are.
constexpr int AT_GRID = 512;

// Slabs of a part of a cut job: no job is wide where rows are single tokens' and
// few heads share keys.
inline int attn_blocks(int heads, int kvheads, int groups, bool single)
{
    return single && groups == 0 && heads / kvheads <= AT_NARROW ? 1 : AT_WIDE / AT_NARROW;
}

// Workspace: the quota, the entries' places in the line, parts of cut jobs (two a
// workgroup), and where groups share tokens the whole parts.
struct AttnSpace {
    size_t costs, slabs, parts, count, bytes;
    AttnSpace(int rows, int heads, int kvheads, int hd, int seqs, int groups, bool single)
    {
        const size_t entries = (size_t)groups + seqs, share = heads / kvheads;
        costs = align_up(sizeof(long long));
        slabs = costs + align_up(entries * sizeof(long long));
        parts = slabs + align_up(entries * sizeof(long long));
        constexpr size_t wide = AT_WIDE / AT_NARROW;
        count = 2 * (size_t)AT_GRID * attn_blocks(heads, kvheads, groups, single);
        if (groups > 0) {
            const size_t blocks = (size_t)rows * share / AT_WIDE;
            const size_t own = single ? seqs * (share <= AT_NARROW ? 1 : (share + AT_WIDE - 1) / AT_WIDE * wide)
                                      : (blocks + seqs) * wide;
            count += kvheads * (own + (blocks + groups) * wide);
        }
        bytes = parts + count * at_slab(hd) * sizeof(float);
    }
};

template <class T, int HD>
int attn_launch(AttnArgs<T> a, hipStream_t stream)
{
    AtPlan& p = a.p;
    const bool single = p.start == nullptr;
    // Sequences of a tile at most are whole as they are: one launch.
    const bool cut = p.groups > 0 || (long long)p.ldt * p.ps > AT_TILE;
    const AttnSpace space(p.rows, p.heads, p.kvheads, p.hd, p.seqs, p.groups, single);
    int resident = 0;
    const int rc = resident_blocks(reinterpret_cast<const void*>(&q8_attn<T, HD>), 256, &resident);
    if (rc) return rc;
    return q8_with_workspace(cut ? space.bytes : 0, true, stream, [&](void* ws, const TimedCall& tc) -> int {
        p.whole = ws == nullptr;
        p.blocks = attn_blocks(p.heads, p.kvheads, p.groups, single);
        // no more than there can be tiles
        const long long blocks = (long long)p.rows * p.share / AT_WIDE + 1ll * p.seqs;
        const long long tiles = p.whole ? 1 : ((long long)p.ldt * p.ps + AT_TILE - 1) / AT_TILE;
        p.grid = (int)std::min((long long)std::min(resident, AT_GRID), std::max(1ll, blocks * p.kvheads * tiles));
        if (!p.whole) {
            char* at = static_cast<char*>(ws);
            p.quota = reinterpret_cast<long long*>(at);
            p.cost_at = reinterpret_cast<long long*>(at + space.costs);
            p.slab_at = reinterpret_cast<long long*>(at + space.slabs);
            p.slabs = (long long)space.count;
            a.slabs = reinterpret_cast<float*>(at + space.parts);
        }
        XSYMV_HIP(launch_k(&q8_attn<T, HD>, dim3(p.grid), dim3(256), stream, a, tc.e0, tc.e1));
        if (p.whole) return 0;
        const long long all = (long long)p.rows * p.kvheads;
        AttnJoinArgs<T> j{a, (int)std::min(std::max(all / 2048, 1ll), 64ll)};
        XSYMV_HIP(launch_k(&q8_attn_join<T>, dim3((unsigned)((all + j.per - 1) / j.per)), dim3(256), stream, j,
                           nullptr, tc.e2));
        return 0;
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
    if (hd < AT_LOW || hd > AT_HD) return -4;
    const long long wide = (long long)heads * hd;
    if (wide > 0x7fffffffll) return -2;
    const bool some = rows > 0 && (seqs > 0 || start == nullptr);
    if (some && q == nullptr) return -5;
    if (ldq < wide) return -6;
    if (seqs < 0 || (start == nullptr && seqs != rows)) return -7;
    const bool tokens = some && ldt > 0 && pages > 0;
    if (some && len == nullptr) return -9;
    if (tokens && table == nullptr) return -10;
    if (ldt < 0) return -11;
    if (groups < 0) return -12;
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
    const AtPlan p{start, len,  table, tokens ? first : nullptr, shared, rows, heads, kvheads, heads / kvheads,
                   hd,    seqs, pages > 0 ? ldt : 0, tokens ? groups : 0, pages, ps};
    const AttnArgs<T> a{p, q, out, lse, k, v, ks, vs, scale * 1.4426950408889634f, ldq, ldk, ldv, ldo, nullptr};
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
