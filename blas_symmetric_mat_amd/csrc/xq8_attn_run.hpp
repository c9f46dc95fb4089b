// xq8_attn_run.hpp -- a call of the attention over a cache of 8-bit rows: checks
// and launch (kernels: xq8_attn.hpp).  The units xq8_attn_[shb].hip compile it.
#pragma once

#include "xq8_attn.hpp"
#include "xq8_host.hpp"

#include <cmath>

namespace xsymv {

template <class T>
int attn_run(int rows, int heads, int kvheads, int hd, const T* q, int ldq, int seqs, const int* start,
             const int* len, const int* table, int ldt, int groups, const int* first, const int* shared,
             const signed char* k, int ldk, const float* ks, const signed char* v, int ldv, const float* vs,
             int pages, int ps, float scale, T* out, int ldo, float* lse, hipStream_t stream)
{
    if (rows < 0) return -1;
    if (heads < 1 || (kvheads >= 1 && heads % kvheads != 0)) return -2;
    if (kvheads < 1) return -3;
    if (hd < 1 || hd > AT_HD) return -4;
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
    const AttnArgs<T> a{q, out, lse, start, len, table, first, shared, k, v, ks, vs, scale, rows, heads, kvheads,
                        hd, ldq, seqs, pages > 0 ? ldt : 0, groups, ldk, ldv, pages, ps, ldo};
    const unsigned grid = (unsigned)std::min((long long)rows * heads, 1ll << 20);
    return q8_launch(&q8_attn_simple<T>, grid, 256, stream, a);
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
