// xq8_attn.hpp -- attention over a cache of 8-bit rows in pages.
//
//   s_t = scale * ks_t * sum_d q_d kc_td,  m = max_t s_t,  l = sum_t e^(s_t - m)
//   out = sum_t e^(s_t - m) vs_t vc_t / l,  lse = m + log l
#pragma once

#include <hip/hip_runtime.h>

#include "xq8_cache.hpp"
#include "xq8_rows.hpp"

namespace xsymv {

constexpr int AT_HD = 256;  // widest head

template <class T>
struct AttnArgs {
    const T* q;
    T* out;
    float* lse;
    const int *start, *len, *table, *first, *shared;
    const signed char *k, *v;
    const float *ks, *vs;
    float scale;
    int rows, heads, kvheads, hd, ldq, seqs, ldt, groups, ldk, ldv, pages, ps, ldo;
};

// One workgroup a row and head.
template <class T>
__global__ __launch_bounds__(256) void q8_attn_simple(AttnArgs<T> a)
{
    __shared__ float q[AT_HD], p[256], of_wave[4];
    __shared__ int at[256];
    const int t = threadIdx.x;
    for (long long item = blockIdx.x; item < (long long)a.rows * a.heads; item += gridDim.x) {
        const int r = (int)(item / a.heads), h = (int)(item % a.heads), g = h / (a.heads / a.kvheads);
        const int s = pg_sequence(a.start, a.seqs, r);
        if (s < 0) continue;
        const long long room = (long long)a.ldt * a.ps;
        const int behind = a.start ? a.start[s + 1] - 1 - r : 0;
        const long long seen = min((long long)a.len[s], room) - behind;
        const int* row = a.table + (size_t)s * a.ldt;
        __syncthreads();
        if (t < a.hd) q[t] = (float)a.q[(size_t)r * a.ldq + (size_t)h * a.hd + t];
        float m = -INFINITY, l = 0.0f, o = 0.0f;
        for (long long base = 0; base < seen; base += 256) {
            __syncthreads();
            const long long tok = base + t;
            float x = -INFINITY, vs = 0.0f;
            at[t] = -1;
            if (tok < seen) {
                const int page = row[tok / a.ps];
                if ((unsigned)page < (unsigned)a.pages) {
                    const int c = (page * a.kvheads + g) * a.ps + (int)(tok % a.ps);
                    at[t] = c;
                    const signed char* k = a.k + (size_t)c * a.ldk;
                    float dot = 0.0f;
                    for (int d = 0; d < a.hd; ++d) dot = __builtin_fmaf(q[d], (float)k[d], dot);
                    x = dot * a.ks[c] * a.scale;
                    vs = a.vs[c];
                }
            }
            float most = x;
            for (int d = 32; d > 0; d >>= 1) most = fmaxf(most, __shfl_xor(most, d, 64));
            if ((t & 63) == 0) of_wave[t / 64] = most;
            __syncthreads();
            most = fmaxf(fmaxf(of_wave[0], of_wave[1]), fmaxf(of_wave[2], of_wave[3]));
            most = fmaxf(m, most);
            const float keep = most == -INFINITY ? 1.0f : expf(m - most);
            const float e = at[t] < 0 ? 0.0f : expf(x - (most == -INFINITY ? 0.0f : most));
            m = most;
            float sum = e;
            for (int d = 32; d > 0; d >>= 1) sum += __shfl_xor(sum, d, 64);
            __syncthreads();
            if ((t & 63) == 0) of_wave[t / 64] = sum;
            p[t] = e * vs;
            __syncthreads();
            l = l * keep + of_wave[0] + of_wave[1] + of_wave[2] + of_wave[3];
            o *= keep;
            if (t < a.hd)
                for (int j = 0; j < 256; ++j)
                    if (at[j] >= 0) o = __builtin_fmaf(p[j], (float)a.v[(size_t)at[j] * a.ldv + t], o);
        }
        if (t < a.hd) a.out[(size_t)r * a.ldo + (size_t)h * a.hd + t] = (T)(l == 0.0f ? 0.0f : o / l);
        if (t == 0 && a.lse) a.lse[item] = l == 0.0f ? -INFINITY : m + logf(l);
    }
}

}  // namespace xsymv
