// xlogp.hpp -- log probabilities of a row of logits: of a given token, the
// entropy, and the most likely tokens.
//
//   lse = log sum_j e^(x_j),  logp = x[token] - lse,
//   entropy = -sum_j p_j log p_j = log l - s / l,  l = sum_j e^(x_j - c),  s = sum_j e^(x_j - c) (x_j - c)
//
// for any c; one pass keeps c at a thread's largest logit so far.  A row's largest
// `top` logits are found in the same pass: each thread remembers the largest of
// its own and where, the top-th largest of these bounds the row's top-th logit
// from below, and only the few threads that hold one above it read theirs again.
//
// Bound by the reads where rows are many and long: 2048 rows of 131072 bfloat16
// logits in 100 us, 5.5 TB/s, the sums' some nine instructions a logit behind
// them (at eleven, with room for five waves a SIMD instead of eight, 129 us).  A
// single row of 32000 is dealt over 16 workgroups; the rest of its 11 us is the
// two launches and what each does one after the other.
#pragma once

#include <hip/hip_runtime.h>

#include "xq8_rows.hpp"

namespace xsymv {

constexpr int LP_THREADS = 256;
constexpr int LP_MOST = 0x7fffffff - 4095;  // logits of a row at most: a round of loads further is an int
constexpr int LP_TOP = 128;     // alternatives of one row at most
constexpr int LP_FEW = 32;      // alternatives that 64 bounds find
constexpr int LP_CAP = 1024;    // candidates ranked at once
constexpr int LP_PARTS = 64;    // workgroups that share a row at most
constexpr int LP_LISTS = 2048;  // alternatives of all parts of a row at most

typedef unsigned long long lp_key;

// What a row is reduced to: c, l and s above, s in units of log 2.
struct LpSums {
    float c, l, s;
};

template <class T>
struct LpArgs {
    const T* x;
    const int* token;
    float *logp, *entropy, *lse;
    int* index;
    float* value;
    int m, n, ldx, top, ldt;
    int parts, each;  // workgroups that share a row, logits of one (a multiple of 8)
    LpSums* sums;     // where there are several: of row i's part p at i * parts + p
    lp_key* keys;     // top keys of each, the largest first, 0 behind the last
};

// Order of the logits as whole numbers: the larger value first, the lower index
// of equal ones (and -0 equals 0).  0 stands below every logit.
__device__ __forceinline__ lp_key lp_order(float v, unsigned index)
{
    const unsigned b = __float_as_uint(v + 0.0f);
    // (a NaN above all: every stretch of a row has its share of the order)
    const unsigned u = v != v ? 0xffffffffu : b ^ ((unsigned)((int)b >> 31) | 0x80000000u);
    return (lp_key)u << 32 | (0xffffffffu - index);
}
__device__ __forceinline__ float lp_value(lp_key k)
{
    const unsigned u = (unsigned)(k >> 32);
    return __uint_as_float(u & 0x80000000u ? u ^ 0x80000000u : ~u);
}
__device__ __forceinline__ int lp_index(lp_key k) { return (int)(0xffffffffu - (unsigned)k); }

// Of a wave's keys, those above one.
__device__ __forceinline__ int lp_rank(lp_key k)
{
    int rank = 0;
#pragma unroll
    for (int o = 0; o < 64; ++o) {
        const unsigned lo = __builtin_amdgcn_readlane((unsigned)k, o);
        const unsigned hi = __builtin_amdgcn_readlane((unsigned)(k >> 32), o);
        rank += ((lp_key)hi << 32 | lo) > k;
    }
    return rank;
}

constexpr float LP_LOG2E = 1.4426950408889634f, LP_LN2 = 0.6931471805599453f;
constexpr float LP_LOWEST = -3.4028234663852886e38f;

// Sums for another reference c.  The difference is bounded, so that nothing (l =
// s = 0) stays nothing.
__device__ __forceinline__ void lp_move(LpSums& a, float c)
{
    const float d = fmaxf((a.c - c) * LP_LOG2E, -1e5f), f = __builtin_amdgcn_exp2f(d);
    a.s = f * (a.s + a.l * d);
    a.l *= f;
    a.c = c;
}
__device__ __forceinline__ void lp_add(LpSums& a, LpSums b)
{
    const float c = fmaxf(a.c, b.c);
    lp_move(a, c);
    lp_move(b, c);
    a.l += b.l;
    a.s += b.s;
}

// Eight logits, -infinity behind a row's last.
template <class T>
__device__ __forceinline__ void lp_load(const T* x, int have, float (&v)[8])
{
    q8_load(x, have, v);
    if (have < 8) {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (e >= have) v[e] = -INFINITY;
    }
}

// Adds eight logits.  c follows each larger one: results are differences of log l and
// a logit's distance from c, which are near 0 for a row that is sure of its token, and
// keep their bits if c is its logit (with c up to 20 below they were off by 2e-6;
// following late is no faster, 2048 rows of 131072 in 101 us, and 100 so).  The eight are summed by
// themselves first: a sum of n in this order is off by some n / 8 + 8 roundings.
__device__ __forceinline__ float lp_take(LpSums& a, const float (&v)[8])
{
    float most = v[0];  // (a NaN passes: fmaxf would quiet each first)
#pragma unroll
    for (int e = 1; e < 8; ++e) most = __builtin_elementwise_maximum(most, v[e]);
    if (most > a.c) lp_move(a, most);
    float l = 0.0f, s = 0.0f;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        // the difference first: c itself has power 1, and masks of the type's lowest
        // value, times log2(e), would be no numbers
        const float z = (v[e] - a.c) * LP_LOG2E, p = __builtin_amdgcn_exp2f(z);
        l += p;
        s = __builtin_fmaf(p, fmaxf(z, -1e30f), s);  // -infinity has no part; p is a NaN where z is one
    }
    a.l += l;
    a.s += s;
    return most;
}

// What a row's sums give: log probabilities are (x - c) - log_l, so that they
// keep their bits where c is large.
struct LpRow {
    float c, log_l;
    bool none;  // nothing but -infinity
    __device__ float of(float x) const { return none ? -INFINITY : (x - c) - log_l; }
};

template <class T>
__device__ __forceinline__ LpRow lp_finish(const LpArgs<T>& a, int row, LpSums t, bool write)
{
    const float log_l = logf(t.l);
    const LpRow r{t.c, log_l, t.l == 0.0f};
    if (write) {
        if (a.token != nullptr) {
            const int k = a.token[row];
            a.logp[row] = (unsigned)k < (unsigned)a.n ? r.of((float)a.x[(size_t)row * a.ldx + k]) : 0.0f;
        }
        if (a.entropy != nullptr) a.entropy[row] = r.none ? 0.0f : log_l - t.s / t.l * LP_LN2;
        if (a.lse != nullptr) a.lse[row] = r.none ? -INFINITY : t.c + log_l;
    }
    return r;
}

template <class T>
__device__ __forceinline__ void lp_alternative(const LpArgs<T>& a, int row, int rank, lp_key k, const LpRow& r)
{
    const size_t at = (size_t)row * a.ldt + rank;
    a.index[at] = lp_index(k);
    if (a.value != nullptr) a.value[at] = r.of(lp_value(k));
}

template <class T, bool TOP>
__global__ __launch_bounds__(LP_THREADS, 8) void logp_rows(LpArgs<T> a)
{
    __shared__ LpSums of_wave[LP_THREADS / 64];
    __shared__ lp_key bound[TOP ? LP_THREADS : 1], found[TOP ? LP_CAP : 1], least;
    __shared__ int chosen[TOP ? LP_THREADS : 1], chosen_n, found_n;
    const int t = threadIdx.x;
    const long long all = (long long)a.m * a.parts;
    for (long long item = blockIdx.x; item < all; item += gridDim.x) {
        const int row = (int)(item / a.parts), part = (int)(item % a.parts);
        const int from = part * a.each, have = min(a.n - from, a.each), vecs = (have + 7) / 8;
        const T* x = a.x + (size_t)row * a.ldx + from;
        LpSums sum{LP_LOWEST, 0.0f, 0.0f};
        float best = -INFINITY;
        int best_at = t;
        auto take = [&](const float (&e)[8], int v) {
            const float most = lp_take(sum, e);
            if (TOP && most > best) {
                best = most;
                best_at = v;
            }
        };
        // Four loads in flight, as they come, and whole ones; then one at a time.
        constexpr int U = 4;
        typedef T raw __attribute__((ext_vector_type(8), aligned(sizeof(T))));
        int v = t;
        for (; (v + (U - 1) * LP_THREADS + 1) * 8 <= have; v += LP_THREADS * U) {
            raw r[U];
#pragma unroll
            for (int u = 0; u < U; ++u) r[u] = *(const raw*)(x + (v + u * LP_THREADS) * 8);
#pragma unroll
            for (int u = 0; u < U; ++u) {
                float e[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) e[i] = (float)r[u][i];
                take(e, v + u * LP_THREADS);
            }
        }
        for (; v < vecs; v += LP_THREADS) {
            float e[8];
            lp_load(x + v * 8, have - v * 8, e);
            take(e, v);
        }
#pragma unroll
        for (int d = 32; d > 0; d >>= 1) {
            const LpSums o{__shfl_xor(sum.c, d, 64), __shfl_xor(sum.l, d, 64), __shfl_xor(sum.s, d, 64)};
            lp_add(sum, o);
        }
        __syncthreads();  // the row before is done with LDS
        if ((t & 63) == 0) of_wave[t >> 6] = sum;
        if (TOP) {
            // of all its logits that equal `best`, a thread's have this index at most
            bound[t] = t < vecs ? lp_order(best, from + best_at * 8 + 7) : 0;
            if (t == 0) {
                least = 0;
                chosen_n = 0;
            }
        }
        __syncthreads();
        sum = of_wave[0];
        for (int w = 1; w < LP_THREADS / 64; ++w) lp_add(sum, of_wave[w]);
        LpRow of{};
        if (a.parts == 1)
            of = lp_finish(a, row, sum, t == 0);
        else if (t == 0)
            a.sums[item] = sum;
        if constexpr (TOP) {
            if (a.top <= LP_FEW) {
                // The largest of four threads' each, by one wave.
                if (t < 64) {
                    const lp_key k = max(max(bound[t], bound[64 + t]), max(bound[128 + t], bound[192 + t]));
                    if (lp_rank(k) == a.top - 1 && k != 0) least = k;
                }
            } else {
                int rank = 0;
#pragma unroll 16
                for (int o = 0; o < LP_THREADS; ++o) rank += bound[o] > bound[t];
                if (rank == a.top - 1 && bound[t] != 0) least = bound[t];
            }
            __syncthreads();
            // threads that hold a logit at or above `least`
            if (t < vecs && lp_order(best, from + best_at * 8) >= least)
                chosen[atomicAdd(&chosen_n, 1)] = t;
            __syncthreads();
            const int turns = (vecs + LP_THREADS - 1) / LP_THREADS, pairs = chosen_n * turns;
            // their logits at or above `low`: counted, and kept as far as there is room
            auto gather = [&](lp_key low) {
                __syncthreads();
                if (t == 0) found_n = 0;
                __syncthreads();
                for (int p = t; p < pairs; p += LP_THREADS) {
                    const int at = (chosen[p % chosen_n] + p / chosen_n * LP_THREADS) * 8;
                    if (at >= have) continue;
                    float e[8];
                    lp_load(x + at, have - at, e);
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const lp_key k = lp_order(e[i], from + at + i);
                        if (at + i < have && k >= low) {
                            const int place = atomicAdd(&found_n, 1);
                            if (place < LP_CAP) found[place] = k;
                        }
                    }
                }
                __syncthreads();
                return found_n;
            };
            lp_key low = least, high = ~0ull, under = low;
            int count = gather(low);
            const int want = min(a.top, have);
            // Too many only where a row's large logits lie on few threads (all in one
            // stretch, or in ascending order): the bound between is halved until they fit,
            // 64 times at most, as the keys differ.
            for (int i = 0; i < 64 && (count > LP_CAP || count < want); ++i) {
                if (count > LP_CAP)
                    under = low;
                else
                    high = low;
                low = under + (high - under) / 2;
                count = gather(low);
            }
            count = min(count, LP_CAP);
            for (int i = t; i < count; i += LP_THREADS) {
                const lp_key k = found[i];
                int before = 0;
#pragma unroll 8
                for (int o = 0; o < count; ++o) before += found[o] > k;
                if (before < a.top) {
                    if (a.parts == 1)
                        lp_alternative(a, row, before, k, of);
                    else
                        a.keys[item * a.top + before] = k;
                }
            }
            if (a.parts > 1)
                for (int i = count + t; i < a.top; i += LP_THREADS) a.keys[item * a.top + i] = 0;
        }
    }
}

// A row from its parts.  With q = top / parts, rounded up, the lists' q-th keys
// are ranked: the (top / q)-th largest of them, rounded up, has top keys at or above
// it, and only those that are there are ranked among each other.
template <class T>
__global__ __launch_bounds__(LP_THREADS) void logp_join(LpArgs<T> a)
{
    __shared__ lp_key found[LP_LISTS], least;
    __shared__ int found_n;
    const int t = threadIdx.x, lane = t & 63, lists = a.parts * a.top;
    const int q = a.top > 0 ? (a.top + a.parts - 1) / a.parts : 1, r = (a.top + q - 1) / q;
    for (int row = blockIdx.x; row < a.m; row += gridDim.x) {
        const size_t first = (size_t)row * a.parts;
        const lp_key* keys = a.keys + first * a.top;
        lp_key mine[LP_LISTS / LP_THREADS], head = 0;
        LpSums sum{LP_LOWEST, 0.0f, 0.0f};
        if (lane < a.parts) sum = a.sums[first + lane];
        if (t < a.parts && a.top > 0) head = keys[t * a.top + q - 1];
#pragma unroll
        for (int i = 0; i < LP_LISTS / LP_THREADS; ++i) {
            mine[i] = 0;
            if (t + i * LP_THREADS < lists) mine[i] = keys[t + i * LP_THREADS];
        }
#pragma unroll
        for (int d = 32; d > 0; d >>= 1) {
            const LpSums o{__shfl_xor(sum.c, d, 64), __shfl_xor(sum.l, d, 64), __shfl_xor(sum.s, d, 64)};
            lp_add(sum, o);
        }
        const LpRow of = lp_finish(a, row, sum, t == 0);
        if (a.top == 0) continue;
        __syncthreads();  // the row before is done with LDS
        if (t < 64) {
            const bool it = lp_rank(head) == r - 1 && head != 0, any = __ballot(it) != 0;
            if (t == 0) found_n = 0;
            if (it || (t == 0 && !any)) least = it ? head : 1;
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < LP_LISTS / LP_THREADS; ++i)
            if (mine[i] >= least) found[atomicAdd(&found_n, 1)] = mine[i];
        __syncthreads();
        const int count = found_n;
        for (int i = t; i < count; i += LP_THREADS) {
            const lp_key k = found[i];
            int before = 0;
#pragma unroll 8
            for (int o = 0; o < count; ++o) before += found[o] > k;
            if (before < a.top) lp_alternative(a, row, before, k, of);
        }
    }
}

}  // namespace xsymv
