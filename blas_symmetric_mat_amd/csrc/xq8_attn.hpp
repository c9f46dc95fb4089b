// xq8_attn.hpp -- attention over a cache of 8-bit rows in pages.
//
//   s_t = scale * ks_t * sum_d q_d kc_td,  m = max_t s_t,  l = sum_t e^(s_t - m)
//   out = sum_t e^(s_t - m) vs_t vc_t / l,  lse = m + log l
//
// Codes are whole numbers up to 127, which half precision holds exactly: both
// products run on the 16 x 16 x 32 half-precision matrix instructions with sums
// in 32 bits, the keys' scales applied to the scores, the values' scales to the
// weights.  q is brought to half precision by a power of two a row (bfloat16 loses
// nothing by it; float is two numbers, 22 bits); weights e^(s - m) vs are rounded
// to 11 bits (float: two numbers again).  Half's results, of 11 bits themselves, are off
// by 3.0e-4 of their size for that (two rows over 131072 tokens), where their own
// rounding alone is 2.0e-4, and bfloat16's by 1.7e-3 either way.  Two numbers for half
// as well take a third longer in wide jobs (4 x 1024 rows behind 8192 tokens 926 us for
// 695) and 1 % in narrow ones, of which not the one without the other: a row's bytes do
// not depend on how many rows its sequence has.
//
// The score product is taken transposed (tokens are the instruction's rows, rows of
// q its columns), so that each lane's results are scores of one row of q, and are,
// rounded, the operand of the second product as they stand: nothing crosses lanes
// between the two.  Of the running maximum only what is needed is done: a row's
// reference m follows a score that is more than a factor of two above it, which
// after a few tokens is rare, and sums stay in the lanes until the end.
//
// Work is cut into jobs: a block of rows of q (those of one sequence, or of a group
// that shares tokens) with one head's keys over the tokens they see.  Every worker
// takes an equal piece of the jobs' costs, so that lengths may differ as they like:
// a piece may begin and end inside a job, whose parts q8_attn_join adds
// (xq8_attn_plan.hpp).  Each workgroup sums the costs itself, which takes less than a
// launch.
//
//   narrow jobs (up to 16 rows of q: single tokens): a wave takes 32 tokens at a
//     time, whose codes come from memory to the registers that the instruction reads
//     them from.  Waves work by themselves.  Bound by the cache's bytes: two rows of
//     32 heads on 8, 131072 tokens each (406 MB), in 78 us, 5.2 TB/s (the call took
//     152 where a workgroup shared such a job, 120 with a wave each, 88 without a
//     launch for wide jobs and with sixteen waves in the join).
//   wide jobs (up to 256 rows: a group's tokens, prompts): each wave of a workgroup
//     has 16 or 32 rows and every token; the waves make operands of 16 tokens each
//     and share them through LDS, so that codes are converted once for all rows.
//     4 x 1024 rows of 32 heads behind 8192 shared tokens in 0.67 ms, 680 T/s.  The vector
//     ALU is busy 59 % of the time and the matrix cores 28 % (in runs of 0.72 ms, with
//     counters): neither is full, as one follows on the other's results and a SIMD has two
//     waves to overlap.  With 128 rows on four waves it was 895 us; wide and narrow jobs in
//     one kernel, 1475.
#pragma once

#include <hip/hip_runtime.h>

#include "xq8_attn_plan.hpp"
#include "xq8_rows.hpp"

namespace xsymv {

typedef _Float16 at_h2 __attribute__((ext_vector_type(2)));
typedef _Float16 at_h8 __attribute__((ext_vector_type(8)));
typedef float at_f2 __attribute__((ext_vector_type(2)));
typedef float at_f4 __attribute__((ext_vector_type(4)));
typedef int at_i4 __attribute__((ext_vector_type(4)));

template <class T>
struct AttnArgs {
    AtPlan p;
    const T* q;
    T* out;
    float* lse;
    const signed char *k, *v;
    const float *ks, *vs;
    float scale;  // times log2(e): scores are kept in units of log 2
    int ldq, ldk, ldv, ldo;
    float* slabs;  // parts of jobs (see AtPlan)
};

constexpr float AT_LN2 = 0.6931471805599453f;
constexpr float AT_LOWEST = -3.4028234663852886e38f;
// Weights are at most 2 (the reference follows beyond that) times 1 (the values'
// scale over the largest so far), times this: half precision's range is used down
// to 2^-39 of the largest.
constexpr float AT_UP = 16384.0f, AT_DOWN = 1.0f / 16384.0f;

// Codes of one dword, as half-precision numbers: with the sign's bit turned over a
// code is c + 128, which under the exponent byte 0x64 stands for 1024 + c + 128.
__device__ __forceinline__ int at_turn(int x) { return x ^ (int)0x80808080; }
__device__ __forceinline__ at_h2 at_codes(int bits)
{
    at_h2 h;
    __builtin_memcpy(&h, &bits, 4);
    return h - (at_h2){1152.0f, 1152.0f};
}
// Bytes 0, 1 (or 2, 3) of a turned dword.
__device__ __forceinline__ at_h2 at_low(int x)
{
    return at_codes(__builtin_amdgcn_perm(0x64646464, x, 0x04010400));
}
__device__ __forceinline__ at_h2 at_high(int x)
{
    return at_codes(__builtin_amdgcn_perm(0x64646464, x, 0x04030402));
}
// Byte B of two turned dwords.
template <int B>
__device__ __forceinline__ at_h2 at_pair(int x, int y)
{
    constexpr unsigned sel = 0x0c000c00u | (unsigned)B | (unsigned)(4 + B) << 16;
    return at_codes(__builtin_amdgcn_perm(y, x, sel) | 0x64006400);
}
// Eight codes of a row, turned.
__device__ __forceinline__ at_h8 at_eight(int x, int y)
{
    const at_h2 a = at_low(x), b = at_high(x), c = at_low(y), d = at_high(y);
    return (at_h8){a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

// Where a lane's pieces of a row lie.  Keys: HD / 64 pieces of 16 codes, of which
// a row's last is its last sixteen codes (q holds zeros where two pieces overlap).
// Values: HD / 16 codes, the last ones again (results that two lanes hold are the
// same numbers).
template <int HD>
struct AtLanes {
    static constexpr int NK = HD / 64, CB = HD / 16;
    int n, g;          // lane % 16, lane / 16
    int koff[NK];      // of the keys' pieces
    int voff;          // of the values' piece
    __device__ AtLanes(int hd) : AtLanes(hd, threadIdx.x & 63) {}
    __device__ AtLanes(int hd, int lane)
    {
        n = lane & 15;
        g = lane >> 4;
#pragma unroll
        for (int j = 0; j < NK; ++j) {
            const int at = j * 64 + g * 16;
            koff[j] = at >= hd ? 0 : min(at, hd - 16);
        }
        voff = at_value(n, hd);
    }
    // first code of lane x's piece of the values
    static __device__ __forceinline__ int at_value(int x, int hd) { return min(x * CB, hd - CB); }
};

template <int N>
__device__ __forceinline__ void at_load(const signed char* p, int (&x)[N])
{
    typedef int vec __attribute__((ext_vector_type(N), aligned(1)));
    const vec v = *(const vec*)p;
#pragma unroll
    for (int w = 0; w < N; ++w) x[w] = v[w];
}
template <>
__device__ __forceinline__ void at_load<1>(const signed char* p, int (&x)[1])
{
    typedef int one __attribute__((aligned(1)));
    x[0] = *(const one*)p;
}

// A lane's keys of one token, and its values of one.
template <int HD>
__device__ __forceinline__ void at_keys(const signed char* row, const AtLanes<HD>& a,
                                        int (&x)[AtLanes<HD>::NK][4])
{
#pragma unroll
    for (int j = 0; j < AtLanes<HD>::NK; ++j) at_load(row + a.koff[j], x[j]);
}
template <int HD>
__device__ __forceinline__ void at_values(const signed char* row, const AtLanes<HD>& a,
                                          int (&x)[AtLanes<HD>::CB / 4])
{
    at_load(row + a.voff, x);
}

// A tile of 16 rows of q as the score product's operand, for lane (n, g): row n's
// numbers that belong to its codes.  SPLIT: as the sum of two.
template <class T, int HD>
struct AtQuery {
    static constexpr int NF = HD / 32;
    static constexpr bool SPLIT = std::is_same<T, float>::value;
    at_h8 hi[NF], lo[SPLIT ? NF : 1];
    float unit;   // score = sum of products * key's scale * unit, which is above zero
    float reach;  // 1 / unit
    typedef T raw __attribute__((ext_vector_type(8), aligned(sizeof(T))));
    raw in[NF];
    // on their way
    __device__ __forceinline__ void fetch(const T* row, bool some, const AtLanes<HD>& a, int hd)
    {
#pragma unroll
        for (int f = 0; f < NF; ++f) {
            in[f] = raw{};
            if (some && f / 2 * 64 + a.g * 16 < hd) in[f] = *(const raw*)(row + a.koff[f / 2] + (f & 1) * 8);
        }
    }
    __device__ __forceinline__ void convert(const AtLanes<HD>& a, int hd, float scale)
    {
        float v[NF][8], most = 0.0f;
#pragma unroll
        for (int f = 0; f < NF; ++f) {
            const int from = a.koff[f / 2] + (f & 1) * 8, at = f / 2 * 64 + a.g * 16;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                v[f][e] = from + e < at ? 0.0f : (float)in[f][e];
                most = __builtin_elementwise_maximum(most, __builtin_fabsf(v[f][e]));
            }
        }
        most = __builtin_elementwise_maximum(most, __shfl_xor(most, 16, 64));
        most = __builtin_elementwise_maximum(most, __shfl_xor(most, 32, 64));
        int e = 0;
        if (!std::is_same<T, q8half>::value && most > 0.0f && most < INFINITY)
            // the largest between 2^14 and 2^15
            e = min(max(14 + 127 - (int)(__float_as_uint(most) >> 23), -126), 126);
        // less where the unit would be below 2^-120: its inverse is a number
        e = min(e, (int)(__float_as_uint(fabsf(scale)) >> 23) - 127 + 120);
        float up = __uint_as_float((unsigned)(127 + e) << 23);
        const float down = __uint_as_float((unsigned)(127 - e) << 23);
        // a negative scale is q's sign; zero is a number that makes all scores as good as it
        unit = fmaxf(fabsf(scale) * down, 0x1p-120f);
        reach = 1.0f / unit;
        if (scale < 0.0f) up = -up;
        if (scale == 0.0f) up = 0.0f;
#pragma unroll
        for (int f = 0; f < NF; ++f)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float x = v[f][e] * up;
                hi[f][e] = (_Float16)x;
                if constexpr (SPLIT) lo[f][e] = (_Float16)(x - (float)hi[f][e]);
            }
    }
};

// Results so far of 16 rows of q, in the lanes of their columns: the reference m as a
// score before its row's unit, l, the sum of the weights of a lane's tokens, and out
// in units of the row's AtUnit / 2^14.
template <int HD>
struct AtRows {
    static constexpr int CB = HD / 16;
    float m, l;
    at_f4 o[CB];  // o[jd][i]: row n's code voff(4 g + i) + jd
    __device__ __forceinline__ void clear()
    {
        m = AT_LOWEST;
        l = 0.0f;
#pragma unroll
        for (int j = 0; j < CB; ++j) o[j] = (at_f4){0.0f, 0.0f, 0.0f, 0.0f};
    }
    __device__ __forceinline__ void times(float f)
    {
#pragma unroll
        for (int j = 0; j < CB; ++j) o[j] *= f;
    }
    __device__ __forceinline__ void whole()  // l of all the row's tokens
    {
        l += __shfl_xor(l, 16, 64);
        l += __shfl_xor(l, 32, 64);
    }
};

// The reference follows where a lane's largest score is more than a factor of two of
// weight above it.
template <int HD>
__device__ __forceinline__ bool at_above(const AtRows<HD>& r, float most, float reach) { return most > r.m + reach; }
template <int HD>
__device__ __forceinline__ void at_follow(AtRows<HD>& r, float most, float unit)
{
    most = fmaxf(most, __shfl_xor(most, 16, 64));
    most = fmaxf(most, __shfl_xor(most, 32, 64));
    const float to = fmaxf(most, r.m), f = __builtin_amdgcn_exp2f((r.m - to) * unit);
    r.m = to;
    r.l *= f;
    r.times(f);
}
template <int N>
__device__ __forceinline__ float at_largest(const float (&x)[N])
{
    float most = x[0];
#pragma unroll
    for (int i = 1; i < N; ++i) most = fmaxf(most, x[i]);
    return most;
}
// Scores to weights e^(s - m).  A row that has seen no token yet has its reference at
// the lowest number, which a unit above 1 would take to -infinity, and the weight of a
// token that it does not see to that of infinity minus infinity.
template <int N, int HD>
__device__ __forceinline__ void at_weigh(AtRows<HD>& r, float (&x)[N], float unit)
{
    const float m = fmaxf(r.m * unit, AT_LOWEST);
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = __builtin_amdgcn_exp2f(__builtin_fmaf(x[i], unit, -m));
    // (in pairs: half the additions wait for the sum)
#pragma unroll
    for (int i = 0; i < N; i += 2) r.l += x[i] + x[i + 1];
}

// Which of 64 tokens a row sees: those that are there (`ok`) and lie before `limit`;
// bit 0 is a lane's first token, 4 g.
__device__ __forceinline__ unsigned long long at_seen(unsigned long long ok, int limit, int g)
{
    const int n = min(max(limit, 0), 64);
    return (n == 64 ? ok : ok & ((1ull << n) - 1)) >> (4 * g);
}

constexpr float AT_NONE = 0x1p120f;  // values' scales from here on count as no numbers

// The largest values' scale so far, as a power of two, of the tokens that a row sees:
// others may have scales beside which its own would be nothing in half precision.  Rows
// have it in common up to the step in which the first of them has its last token, and
// steps from there on are taken apart.
struct AtUnit {
    float unit = 0x1p-100f;
    __device__ __forceinline__ bool above(float v) const { return fabsf(v) > unit && fabsf(v) < AT_NONE; }
    // raised to hold `most`; the factor for what was summed in the old one
    __device__ __forceinline__ float raise(float most)
    {
        const float was = unit;
        // (the next power of two)
        if (most > unit) unit = __uint_as_float(((__float_as_uint(most) >> 23) + 1) << 23);
        return was / unit;
    }
    // The largest of the wave's scales, where one is above it.
    __device__ __forceinline__ float largest(float v) const
    {
        float most = above(v) ? fabsf(v) : unit;
#pragma unroll
        for (int d = 32; d > 0; d >>= 1) most = fmaxf(most, __shfl_xor(most, d, 64));
        return __uint_as_float(__builtin_amdgcn_readfirstlane(__float_as_uint(most)));
    }
    __device__ __forceinline__ float up() const { return AT_UP / unit; }
    // A scale for the weights.  One above the unit is no number or not to be seen, and
    // becomes the largest number: times a weight of zero, a row's that does not see the
    // token, it is nothing, and no 16-bit number in a row that does.
    __device__ __forceinline__ float scaled(float v, float up) const { return fabsf(v) <= unit ? v * up : -AT_LOWEST; }
};

// Tokens a to b - 1 of 64.
__device__ __forceinline__ unsigned long long at_stretch(int a, int b)
{
    return (~0ull << a) & (~0ull >> (64 - b));
}

template <class H8>
__device__ __forceinline__ at_f4 at_product(H8 a, H8 b, at_f4 c)
{
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
}

// Eight weights as the second product's operand.
__device__ __forceinline__ at_h8 at_round(const float (&w)[8])
{
    at_h8 h;
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
        const at_h2 p = __builtin_convertvector((at_f2){w[i], w[i + 1]}, at_h2);
        h[i] = p[0];
        h[i + 1] = p[1];
    }
    return h;
}
__device__ __forceinline__ at_h8 at_rest(const float (&w)[8], at_h8 h)
{
    float r[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) r[i] = w[i] - (float)h[i];
    return at_round(r);
}

// Values of eight tokens as operands of the second product: code B of dword W.
template <int W, int B, int N>
__device__ __forceinline__ at_h8 at_column(const int (&v)[8][N])
{
    const at_h2 a = at_pair<B>(v[0][W], v[1][W]), b = at_pair<B>(v[2][W], v[3][W]);
    const at_h2 c = at_pair<B>(v[4][W], v[5][W]), d = at_pair<B>(v[6][W], v[7][W]);
    return (at_h8){a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

// A barrier for what is in LDS: loads and stores of memory go on.
__device__ __forceinline__ void at_barrier()
{
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}

// A row's results to out and lse.
template <class T>
__device__ __forceinline__ void at_lse(const AttnArgs<T>& a, size_t row, int head, float m, float l)
{
    if (a.lse != nullptr) a.lse[row * a.p.heads + head] = l == 0.0f ? -INFINITY : m * AT_LN2 + logf(l);
}

// Where in a slab lane (n, g)'s results of registers 4 j to 4 j + 3, place i, are: a
// wave's stores of one i and j lie side by side, and of those a row's 64 bytes do.
// (With rows one after the other a lane's 128 bytes lie together, and a store of 64
// lanes touches as many lines: 64 rows of 32 heads over 16384 shared tokens took 85 us
// in all, now 80.)
__device__ __forceinline__ int at_part_of(int i, int j, int v, int n, int g)
{
    return 2 * AT_NARROW + ((i * v + j) * AT_NARROW + n) * 16 + g * 4;
}
template <bool ALL, int HD>
__device__ __forceinline__ void at_keep(const AtRows<HD>& r, const AtLanes<HD>& at, float* slab, float f, int n,
                                        int hd)
{
    constexpr int V = HD / 64;
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < V; ++j) {
            if (!ALL && (4 * at.g + i) * AtRows<HD>::CB >= hd) continue;  // the last codes again
            at_f4 v;
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] = r.o[4 * j + e][i] * f;
            *(at_f4*)(slab + at_part_of(i, j, V, n, at.g)) = v;
        }
}

// One lane's codes of a row of results, times f.
template <int HD, class O>
__device__ __forceinline__ void at_write(const AtRows<HD>& r, const AtLanes<HD>& at, O* to, float f, int hd)
{
    constexpr int CB = HD / 16;
    typedef O vec __attribute__((ext_vector_type(CB), aligned(sizeof(O))));
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        vec v;
#pragma unroll
        for (int j = 0; j < CB; ++j) v[j] = (O)(r.o[j][i] * f);
        *(vec*)(to + AtLanes<HD>::at_value(4 * at.g + i, hd)) = v;
    }
}

// A tile of 16 rows, of which the lanes' is the job's row n, to out or to its part.
template <class T, int HD>
__device__ __forceinline__ void at_finish(const AttnArgs<T>& a, const AtJob& job, AtLanes<HD> at, AtRows<HD>& r,
                                          float row_unit, float unit, int n, float* slab)
{
    // (places of results are computed here, not kept in registers while jobs run)
    asm volatile("" : "+v"(at.g));
    const int hd = a.p.hd;
    r.whole();
    r.m = r.l == 0.0f ? AT_LOWEST : r.m * row_unit;
    if (n >= job.rows) return;
    const float f = r.l == 0.0f ? 0.0f : unit * AT_DOWN;
    if (slab != nullptr) {
        float* part = slab + (size_t)(n / AT_NARROW) * at_slab(hd);
        const int m = n % AT_NARROW;
        if (at.g == 0) {
            part[2 * m] = r.m;
            part[2 * m + 1] = r.l;
        }
        if (hd == HD)
            at_keep<true>(r, at, part, f, m, hd);
        else
            at_keep<false>(r, at, part, f, m, hd);
    } else {
        size_t row;
        const int head = job.place(a.p, n, row);
        if (at.g == 0) at_lse(a, row, head, r.m, r.l);
        at_write(r, at, a.out + row * a.ldo + (size_t)head * hd, r.l == 0.0f ? 0.0f : f / r.l, hd);
    }
}

// ------------------------------------------------------------------- narrow
// Rows of the cache, and scales, of a wave's 32 tokens.
struct AtTokens {
    int row[32];
    float ks[32], vs[32];
};

template <class T, int HD>
struct AtNarrow {
    static constexpr int NK = HD / 64, CB = HD / 16, NV = CB / 4, STEP = AT_TILE;
    static constexpr bool SPLIT = AtQuery<T, HD>::SPLIT;
    struct Lds {
        AtTokens tokens[4][2];
    };
    struct Codes {  // of one step
        int k[2][NK][4], v[8][NV];
        float ks, vs;
        unsigned long long ok;  // tokens (bits 0 to 31) that are there
    };

    const AttnArgs<T>& a;
    const AtJob& job;
    const AtLanes<HD>& at;
    AtTokens (&lds)[2];
    const int* pages;  // the sequence's row of the table
    int lane, limit, least;
    AtQuery<T, HD> q;
    AtRows<HD> r;
    AtUnit unit;

    __device__ __forceinline__ int page_of(int t) const
    {
        // (unsigned: two steps behind the last token may pass the largest int)
        return lane < STEP && (unsigned)t < (unsigned)job.end ? pages[a.p.by_page.of(t)] : -1;
    }
    // rows of the step's tokens to LDS, and their codes and scales on their way
    __device__ __forceinline__ void fetch(Codes& c, AtTokens& tok, int base, int page)
    {
        const int t = base + lane;
        int row = -1;
        if (lane < STEP && t < job.end && (unsigned)page < (unsigned)a.p.pages)
            row = (page * a.p.kvheads + job.head) * a.p.ps + t - a.p.by_page.of(t) * a.p.ps;
        c.ok = __ballot(row >= 0);
        c.ks = c.vs = 0.0f;
        if (row >= 0) {
            c.ks = a.ks[row];
            c.vs = a.vs[row];
        }
        if (lane < STEP) tok.row[lane] = max(row, 0);
        at_wave_sync();
#pragma unroll
        for (int i = 0; i < 2; ++i)
            at_keys<HD>(a.k + (size_t)tok.row[16 * i + at.n] * a.ldk, at, c.k[i]);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            at_values<HD>(a.v + (size_t)tok.row[i / 4 * 16 + 4 * at.g + i % 4] * a.ldv, at, c.v[i]);
    }
    // Apart: a row's unit by the values' scales that it sees, and these in it.
    __device__ __forceinline__ void scale(float (&w)[8], unsigned mask)
    {
        float most = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i)
            most = mask >> (i / 4 * 16 + i % 4) & 1 && unit.above(w[i]) ? fmaxf(most, fabsf(w[i])) : most;
        if (__ballot(most > 0.0f) != 0) {
            most = fmaxf(most, __shfl_xor(most, 16, 64));
            most = fmaxf(most, __shfl_xor(most, 32, 64));
            r.times(unit.raise(most));
        }
        const float up = unit.up();
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i] = unit.scaled(w[i], up);
    }
    __device__ __forceinline__ void compute(Codes& c, AtTokens& tok, int base)
    {
        const bool apart = base + STEP > least;
        if (!apart && __ballot(unit.above(c.vs)) != 0) r.times(unit.raise(unit.largest(c.vs)));
        if (lane < STEP) {
            tok.ks[lane] = c.ks;
            tok.vs[lane] = apart ? c.vs : unit.scaled(c.vs, unit.up());
        }
        at_wave_sync();
        float x[8], w[8];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            at_f4 s = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int j = 0; j < NK; ++j)
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    const at_h8 k = at_eight(at_turn(c.k[i][j][2 * half]), at_turn(c.k[i][j][2 * half + 1]));
                    s = at_product(k, q.hi[2 * j + half], s);
                    if constexpr (SPLIT) s = at_product(k, q.lo[2 * j + half], s);
                }
            const at_f4 ks = *(const at_f4*)&tok.ks[16 * i + 4 * at.g];
            const at_f4 vs = *(const at_f4*)&tok.vs[16 * i + 4 * at.g];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                x[4 * i + e] = s[e] * ks[e];
                w[4 * i + e] = vs[e];
            }
        }
        if (__builtin_expect((unsigned)c.ok != ~0u || apart, 0)) {
            const unsigned mask = (unsigned)at_seen(c.ok, limit - base, at.g);
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = mask >> (i / 4 * 16 + i % 4) & 1 ? x[i] : -INFINITY;
            if (__builtin_expect(apart, 0)) scale(w, mask);
        }
        const float most = at_largest(x);
        if (__ballot(at_above(r, most, q.reach)) != 0) at_follow(r, most, q.unit);
        at_weigh(r, x, q.unit);
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i] *= x[i];
        const at_h8 p = at_round(w);
        at_h8 rest;
        if constexpr (SPLIT) rest = at_rest(w, p);
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
            for (int d = 0; d < NV; ++d) c.v[i][d] = at_turn(c.v[i][d]);
        auto add = [&](int j, at_h8 v) {
            r.o[j] = at_product(v, p, r.o[j]);
            if constexpr (SPLIT) r.o[j] = at_product(v, rest, r.o[j]);
        };
        at_each<NV>([&](auto W) {
            constexpr int d = decltype(W)::value;
            add(4 * d + 0, at_column<d, 0>(c.v));
            add(4 * d + 1, at_column<d, 1>(c.v));
            add(4 * d + 2, at_column<d, 2>(c.v));
            add(4 * d + 3, at_column<d, 3>(c.v));
        });
    }
    // The job's tokens from `from` to `to`.
    __device__ __forceinline__ void run(int from, int to, float* slab)
    {
        r.clear();
        const int count = (to - from + STEP - 1) / STEP;
        Codes c[2];
        const int page = page_of(from + lane);
        int later = page_of(from + STEP + lane);
        size_t row = 0;
        const bool some = at.n < job.rows;
        const int head = job.place(a.p, some ? at.n : 0, row);
        q.fetch(a.q + row * a.ldq + (size_t)head * a.p.hd, some, at, a.p.hd);
        limit = some ? job.limit(a.p, at.n) : 0x7fffffff;
        if (count > 0) fetch(c[0], lds[0], from, page);
        q.convert(at, a.p.hd, a.scale);
        least = at_least(limit);
        if (least >= job.end) least = 0x7fffffff;  // rows differ in no step
        auto step = [&](Codes& now, Codes& next, AtTokens& tn, AtTokens& tx, int s) {
            const int base = from + s * STEP;
            if (s + 1 < count) {
                fetch(next, tx, base + STEP, later);
                later = page_of(base + 2 * STEP + lane);
            }
            compute(now, tn, base);
        };
        for (int s = 0; s < count; s += 2) {
            step(c[0], c[1], lds[0], lds[1], s);
            if (s + 1 < count) step(c[1], c[0], lds[1], lds[0], s + 1);
        }
        at_finish(a, job, at, r, q.unit, unit.unit, at.n, slab);
    }
};

// --------------------------------------------------------------------- wide
template <class T, int HD>
struct AtWide {
    static constexpr int NK = HD / 64, NF = HD / 32, CB = HD / 16, NV = CB / 4;
    static constexpr bool SPLIT = AtQuery<T, HD>::SPLIT;
    // Eight waves on a compute unit, as one workgroup: as two of four, each wave converts
    // twice as much for its rows.  Two tiles of rows a wave where registers hold them, one
    // where not (float's two numbers over 64 codes, others over 128), and over 128 codes
    // LDS for one buffer.  4 x 1024 rows behind 8192 tokens, with four waves of two tiles
    // and as it is: bfloat16 of 128 codes 895 us and 669, of 256 4521 and 1570; float of
    // 64 codes 1234 and 655, of 128 1827 and 1185 (two tiles on eight waves: spilled).
    static constexpr int WAVES = 8, STEP = 16 * WAVES;
    static constexpr int TILES = HD <= (SPLIT ? 64 : 128) ? 2 : 1, BUFFERS = HD <= 128 ? 2 : 1, ROWS = STEP * TILES;
    struct Step {
        at_h8 k[WAVES][NF][64];      // keys of 16 tokens each, as the lanes read them
        at_h8 v[WAVES / 2][CB][64];  // values of 32 tokens each
        float ks[STEP], vs[STEP];
        float top[WAVES];            // of each wave's tokens, the largest values' scale; below
                                     // zero where one is no number
        unsigned short ok[WAVES];    // tokens that are there
    };
    struct Lds {
        Step step[BUFFERS];
        float unit[ROWS];  // of rows from the first step that is apart on
        int limit[ROWS];
    };
    struct Codes {  // a wave's 16 tokens of one step
        int k[NK][4], v[4][NV];
        float ks, vs;
        int ok;
    };

    const AttnArgs<T>& a;
    const AtJob& job;
    const AtLanes<HD>& at;
    Lds& lds;
    const int* pages;
    int lane, wave;
    int tiles;       // of 16 rows, a wave's: 1 or 2
    int first;       // the wave's first row
    AtQuery<T, HD> q[TILES];
    AtRows<HD> r[TILES];
    AtUnit unit;
    int least, most;

    __device__ __forceinline__ int page_of(int t) const
    {
        return (unsigned)t < (unsigned)job.end ? pages[a.p.by_page.of(t)] : -1;
    }

    __device__ __forceinline__ void fetch(Codes& c, int base, int page)
    {
        // (Places in rows are computed here: kept in registers, they took those of other
        // numbers, which then had to be read back from memory in each step: 728 us for
        // 4 x 1024 rows behind 8192 tokens where it is 670.)
        int x = lane;
        asm volatile("" : "+v"(x));
        const AtLanes<HD> here(a.p.hd, x);
        const int t = base + wave * 16 + here.n;
        int row = -1;
        if (t < job.end && (unsigned)page < (unsigned)a.p.pages)
            row = (page * a.p.kvheads + job.head) * a.p.ps + t - a.p.by_page.of(t) * a.p.ps;
        c.ok = row >= 0;
        c.ks = c.vs = 0.0f;
        if (row >= 0) {
            c.ks = a.ks[row];
            c.vs = a.vs[row];
        }
        row = max(row, 0);
        at_keys<HD>(a.k + (size_t)row * a.ldk, here, c.k);
#pragma unroll
        for (int i = 0; i < 4; ++i)
            at_values<HD>(a.v + (size_t)__shfl(row, 4 * here.g + i, 64) * a.ldv, here, c.v[i]);
    }
    __device__ __forceinline__ void share(Codes& c, Step& s)
    {
#pragma unroll
        for (int j = 0; j < NK; ++j)
#pragma unroll
            for (int half = 0; half < 2; ++half)
                s.k[wave][2 * j + half][lane] = at_eight(at_turn(c.k[j][2 * half]), at_turn(c.k[j][2 * half + 1]));
        typedef _Float16 h4 __attribute__((ext_vector_type(4)));
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int d = 0; d < NV; ++d) c.v[i][d] = at_turn(c.v[i][d]);
        auto put = [&](int j, at_h2 x, at_h2 y) {
            h4* to = reinterpret_cast<h4*>(&s.v[wave >> 1][j][lane]) + (wave & 1);
            *to = (h4){x[0], x[1], y[0], y[1]};
        };
        at_each<NV>([&](auto W) {
            constexpr int d = decltype(W)::value;
            put(4 * d + 0, at_pair<0>(c.v[0][d], c.v[1][d]), at_pair<0>(c.v[2][d], c.v[3][d]));
            put(4 * d + 1, at_pair<1>(c.v[0][d], c.v[1][d]), at_pair<1>(c.v[2][d], c.v[3][d]));
            put(4 * d + 2, at_pair<2>(c.v[0][d], c.v[1][d]), at_pair<2>(c.v[2][d], c.v[3][d]));
            put(4 * d + 3, at_pair<3>(c.v[0][d], c.v[1][d]), at_pair<3>(c.v[2][d], c.v[3][d]));
        });
        const unsigned long long ok = __ballot(c.ok);
        if (lane < 16) {
            s.ks[wave * 16 + lane] = c.ks;
            s.vs[wave * 16 + lane] = c.vs;
        }
        const bool number = fabsf(c.vs) < AT_NONE;
        float top = number ? fabsf(c.vs) : 0.0f;
#pragma unroll
        for (int d = 8; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor(top, d, 64));
        if (__ballot(!number) != 0) top = -fmaxf(top, 0x1p-126f);
        if (lane == 0) {
            s.ok[wave] = (unsigned short)ok;
            s.top[wave] = top;
        }
    }
    __device__ __forceinline__ int row_of(int i) const { return first + 16 * i + at.n; }
    // The first of 64 tokens from `a` on whose scale is above the unit.
    __device__ __forceinline__ int first_above(float v, int a) const
    {
        const unsigned long long m = __ballot(unit.above(v)) >> a;
        return m == 0 ? 64 : a + __builtin_ctzll(m);
    }
    // 64 tokens, `half` of a step's, from `a` on; the end of those that were taken
    template <int N, bool APART>
    __device__ __forceinline__ int compute(const Step& s, int half, int base, int a)
    {
        bool odd = false;
        int b = 64;
        unsigned long long stretch = ~0ull;
        if constexpr (APART) {
            // Apart: by stretches, of which each begins with a token that raises the unit, so
            // that rows whose tokens all lie before it keep theirs.  (A unit for each row
            // besides the two tiles' results does not fit the registers.)
            const float v = s.vs[64 * half + lane];
            b = first_above(v, a);
            if (b == a) {
                const float f = unit.raise(__uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(fabsf(v)), a)));
#pragma unroll
                for (int i = 0; i < N; ++i) {
                    const bool sees = lds.limit[row_of(i)] > base + a;
                    r[i].times(sees ? f : 1.0f);
                    if (sees) lds.unit[row_of(i)] = unit.unit;
                }
                b = first_above(v, a);
            }
            stretch = at_stretch(a, b);
            odd = b - a < 64;
        }
        float x[N][16];
        at_f4 vs[4];
#pragma unroll
        for (int sub = 0; sub < 4; ++sub) {
            at_f4 acc[N];
#pragma unroll
            for (int i = 0; i < N; ++i) acc[i] = (at_f4){0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int f = 0; f < NF; ++f) {
                const at_h8 k = s.k[4 * half + sub][f][lane];
#pragma unroll
                for (int i = 0; i < N; ++i) {
                    acc[i] = at_product(k, q[i].hi[f], acc[i]);
                    if constexpr (SPLIT) acc[i] = at_product(k, q[i].lo[f], acc[i]);
                }
            }
            const at_f4 ks = *(const at_f4*)&s.ks[64 * half + 16 * sub + 4 * at.g];
            vs[sub] = *(const at_f4*)&s.vs[64 * half + 16 * sub + 4 * at.g];
#pragma unroll
            for (int i = 0; i < N; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) x[i][4 * sub + e] = acc[i][e] * ks[e];
        }
        const float top = s.top[4 * half + (lane & 3)];
        odd |= __ballot(top < 0.0f) != 0;
        unsigned long long ok;
        __builtin_memcpy(&ok, s.ok + 4 * half, 8);
        ok &= stretch;
        if (!APART && __ballot(unit.above(top)) != 0) {
            const float f = unit.raise(unit.largest(top));
#pragma unroll
            for (int i = 0; i < N; ++i) r[i].times(f);
        }
        if (ok != ~0ull || APART) {
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const unsigned long long mask =
                    APART ? at_seen(ok, lds.limit[row_of(i)] - base, at.g) : ok >> (4 * at.g);
#pragma unroll
                for (int e = 0; e < 16; ++e) x[i][e] = mask >> (e / 4 * 16 + e % 4) & 1 ? x[i][e] : -INFINITY;
            }
        }
        float most[N];
        bool above = false;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            most[i] = at_largest(x[i]);
            above |= at_above(r[i], most[i], q[i].reach);
        }
        if (__ballot(above) != 0)
#pragma unroll
            for (int i = 0; i < N; ++i) at_follow(r[i], most[i], q[i].unit);
        const float up = unit.up();
        if (!odd) {
#pragma unroll
            for (int sub = 0; sub < 4; ++sub) vs[sub] *= up;
        } else {
#pragma unroll
            for (int sub = 0; sub < 4; ++sub)
#pragma unroll
                for (int e = 0; e < 4; ++e) vs[sub][e] = unit.scaled(vs[sub][e], up);
        }
        at_h8 p[N][2], rest[N][SPLIT ? 2 : 1];
#pragma unroll
        for (int i = 0; i < N; ++i) {
            at_weigh(r[i], x[i], q[i].unit);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                float w[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) w[e] = x[i][8 * h + e] * vs[2 * h + e / 4][e % 4];
                p[i][h] = at_round(w);
                if constexpr (SPLIT) rest[i][h] = at_rest(w, p[i][h]);
            }
        }
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int j = 0; j < CB; ++j) {
                const at_h8 c = s.v[2 * half + h][j][lane];
#pragma unroll
                for (int i = 0; i < N; ++i) {
                    r[i].o[j] = at_product(c, p[i][h], r[i].o[j]);
                    if constexpr (SPLIT) r[i].o[j] = at_product(c, rest[i][h], r[i].o[j]);
                }
            }
        return b;
    }
    // Steps from `base` up to `stop`.
    template <bool APART>
    __device__ __forceinline__ void steps(Codes& c, int& base, int stop, int to, int& p, int& later)
    {
        for (; base < stop; base += STEP) {
            share(c, lds.step[p]);
            at_barrier();
            if (base + STEP < to) {
                fetch(c, base + STEP, later);
                later = page_of(base + 2 * STEP + wave * 16 + at.n);
            }
#pragma unroll 1
            for (int half = 0, a = 0; half < WAVES / 4 && base + 64 * half < min(most, to);) {
                if (tiles == 2) {
                    if constexpr (TILES > 1) a = compute<2, APART>(lds.step[p], half, base + 64 * half, a);
                } else {
                    a = compute<1, APART>(lds.step[p], half, base + 64 * half, a);
                }
                half += a == 64;
                a &= 63;
            }
            if (BUFFERS > 1)
                p ^= 1;
            else
                at_barrier();
        }
    }
    __device__ __forceinline__ void run(int from, int to, float* slab)
    {
        // few rows are dealt 16 to a wave, so that all waves have some
        tiles = TILES > 1 && job.rows > STEP ? 2 : 1;
        first = wave * 16 * tiles;
        const int mine = wave * 16 + at.n, page = page_of(from + mine);
        int later = page_of(from + STEP + mine), limit[TILES];
#pragma unroll
        for (int i = 0; i < TILES; ++i) {
            const int n = first + 16 * i + at.n;
            const bool some = i < tiles && n < job.rows;
            size_t row = 0;
            const int head = job.place(a.p, some ? n : 0, row);
            q[i].fetch(a.q + row * a.ldq + (size_t)head * a.p.hd, some, at, a.p.hd);
            limit[i] = some ? job.limit(a.p, n) : 0x7fffffff;
            if (i < tiles) lds.limit[n] = limit[i];
            r[i].clear();
        }
        Codes c;
        if (from < to) fetch(c, from, page);
        least = 0x7fffffff;
        most = 0;
#pragma unroll
        for (int i = 0; i < TILES; ++i) {
            q[i].convert(at, a.p.hd, a.scale);
            least = min(least, at_least(limit[i]));
            most = max(most, at_most(limit[i] == 0x7fffffff ? 0 : limit[i]));
        }
        if (least >= to) least = 0x7fffffff;  // rows differ in no step
        // (a loop for either kind of step: what the second one takes costs the first none of
        // its registers)
        int p = 0, base = from;
        steps<false>(c, base, min(to, from + (max(least, from) - from) / STEP * STEP), to, p, later);
#pragma unroll
        for (int i = 0; i < TILES; ++i)
            if (i < tiles) lds.unit[row_of(i)] = unit.unit;
        steps<true>(c, base, to, to, p, later);
        at_finish(a, job, at, r[0], q[0].unit, lds.unit[row_of(0)], first + at.n, slab);
        if constexpr (TILES > 1)
            if (tiles == 2) at_finish(a, job, at, r[1], q[1].unit, lds.unit[row_of(1)], first + 16 + at.n, slab);
        at_barrier();
    }
};

// Waves of narrow jobs that a SIMD has room for: wide heads and float's two numbers take the registers
// of two.
template <class T, int HD>
constexpr int at_resident = HD <= 128 && !std::is_same<T, float>::value ? 2 : 1;

// Workgroups b, b + 8, ... are of one die: their pieces lie side by side.
__device__ __forceinline__ int at_worker(const AtPlan& p)
{
    return (int)blockIdx.x % 8 * (p.grid / 8) + (int)blockIdx.x / 8;
}

template <class T, int HD>
__global__ __launch_bounds__((64 * AtWide<T, HD>::WAVES)) void q8_attn_wide(AttnArgs<T> a)
{
    __shared__ union {
        AtScan<AT_WIDE_JOBS> scan;  // until the cursor is there
        typename AtWide<T, HD>::Lds wide;
    } lds;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const AtLanes<HD> at(a.p.hd);
    const AtLines<AT_WIDE_JOBS> lines(a.p, lds.scan);
    AtCursor<AT_WIDE_JOBS> cursor(a.p, lds.scan, lines, at_worker(a.p), a.p.grid);
    __syncthreads();
    AtJob job;
    int from, to, slab;
    while (cursor.next(a.p, job, from, to, slab)) {
        float* part = slab < 0 ? nullptr : a.slabs + (size_t)slab * at_slab(a.p.hd);
        AtWide<T, HD> w{a, job, at, lds.wide, a.p.table + (size_t)job.table * a.p.ldt, lane, wave};
        w.run(from, to, part);
    }
}

template <class T, int HD, AtKind KIND>
__global__ __launch_bounds__(256, (at_resident<T, HD>)) void q8_attn_narrow(AttnArgs<T> a)
{
    __shared__ union {
        AtScan<KIND> scan;  // until the cursor is there
        typename AtNarrow<T, HD>::Lds narrow;
    } lds;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const AtLanes<HD> at(a.p.hd);
    const AtLines<KIND> lines(a.p, lds.scan);
    AtCursor<KIND> cursor(a.p, lds.scan, lines, at_worker(a.p) * 4 + wave, a.p.grid * 4);
    __syncthreads();
    AtJob job;
    int from, to, slab;
    while (cursor.next(a.p, job, from, to, slab)) {
        float* part = slab < 0 ? nullptr : a.slabs + (size_t)slab * at_slab(a.p.hd);
        AtNarrow<T, HD> w{a, job, at, lds.narrow.tokens[wave], a.p.table + (size_t)job.table * a.p.ldt, lane};
        w.run(from, to, part);
    }
}

// Adds the parts of rows' results.  LANES lanes have a row and head, four of its codes
// each in the slabs' order, and with more than one of WAVES all waves of a workgroup
// share its parts.
template <class T, int LANES, int WAVES>
__global__ __launch_bounds__((WAVES > 4 ? 64 * WAVES : 256)) void q8_attn_join(AttnArgs<T> a)
{
    constexpr int U = 4, ITEMS = 64 / LANES * (WAVES > 1 ? 1 : 4), HD = 4 * LANES, V = HD / 64;
    __shared__ float sums[WAVES][64][6];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, hd = a.p.hd;
    const int at_g = threadIdx.x % 4, at_i = threadIdx.x % LANES / 4 / V, at_j = threadIdx.x % LANES / 4 % V;
    const int d = AtLanes<HD>::at_value(4 * at_g + at_i, hd) + 4 * at_j;
    const bool own_codes = (4 * at_g + at_i) * (HD / 16) < hd;
    const long long all = (long long)a.p.rows * a.p.heads;
    const long long item = (long long)blockIdx.x * ITEMS + (WAVES > 1 ? lane : (int)threadIdx.x) / LANES;
    int2 own{0, 0}, shared{0, 0};
    size_t row = 0;
    if (item < all) {
        own = a.p.own[item];
        if (a.p.groups > 0) shared = a.p.shared_parts[item];
        row = item / a.p.heads;
        // rows outside the sequences hold what an earlier call left there
        if (a.p.start != nullptr &&
            ((long long)row < a.p.start[0] || (long long)row >= a.p.start[a.p.seqs]))
            own.y = 0;
    }
    if (!(own.y >> 24 & 1)) shared.y = 0;
    float m = AT_LOWEST, l = 0.0f, o[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    auto add = [&](int2 where) {
        const int count = where.y & 0xffff, n = where.y >> 16 & 15;
        for (int base = WAVES > 1 ? wave : 0; base < count; base += WAVES * U) {
            float pm[U], pl[U], v[U][4];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int i = base + u * WAVES;
                pm[u] = AT_LOWEST;
                pl[u] = v[u][0] = v[u][1] = v[u][2] = v[u][3] = 0.0f;
                if (i < count) {
                    const long long at = min(max(at_part(a.p, where, i), 0ll), (long long)a.p.slabs - 1);
                    const float* s = a.slabs + at * at_slab(hd);
                    pm[u] = s[2 * n];
                    pl[u] = s[2 * n + 1];
                    if (!own_codes) continue;
                    const at_f4 x = *(const at_f4*)(s + at_part_of(at_i, at_j, V, n, at_g));
#pragma unroll
                    for (int e = 0; e < 4; ++e) v[u][e] = x[e];
                }
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const float to = fmaxf(m, pm[u]), f = __builtin_amdgcn_exp2f(m - to);
                // (a part without tokens, or none: what its place holds does not count)
                const float g = pl[u] == 0.0f ? 0.0f : __builtin_amdgcn_exp2f(pm[u] - to);
                m = to;
                l = l * f + pl[u] * g;
#pragma unroll
                for (int e = 0; e < 4; ++e) o[e] = o[e] * f + (pl[u] == 0.0f ? 0.0f : v[u][e] * g);
            }
        }
    };
    add(own);
    add(shared);
    if constexpr (WAVES > 1) {
        float(&mine)[6] = sums[wave][lane];
#pragma unroll
        for (int e = 0; e < 4; ++e) mine[e] = o[e];
        mine[4] = m;
        mine[5] = l;
        __syncthreads();
        if (wave != 0) return;
        for (int w = 1; w < WAVES; ++w) {
            const float(&p)[6] = sums[w][lane];
            const float to = fmaxf(m, p[4]), f = __builtin_amdgcn_exp2f(m - to), g = __builtin_amdgcn_exp2f(p[4] - to);
            m = to;
            l = l * f + p[5] * g;
#pragma unroll
            for (int e = 0; e < 4; ++e) o[e] = o[e] * f + p[e] * g;
        }
    }
    if (own.y == 0) return;
    const int head = (int)(item - (long long)row * a.p.heads);
    if (threadIdx.x % LANES == 0) at_lse(a, row, head, m, l);
    if (!own_codes) return;
    T* out = a.out + row * a.ldo + (size_t)head * hd + d;
    typedef T vec __attribute__((ext_vector_type(4), aligned(sizeof(T))));
    vec x;
#pragma unroll
    for (int e = 0; e < 4; ++e) x[e] = (T)(l == 0.0f ? 0.0f : o[e] / l);
    *(vec*)out = x;
}

}  // namespace xsymv
