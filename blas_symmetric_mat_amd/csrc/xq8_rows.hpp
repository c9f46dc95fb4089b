// xq8_rows.hpp -- kernels on rows held in 8 bits: the norm with the
// residual's addition, the gated activation, and a cache's store and read.
//
// A row of n numbers v_j is held as n signed codes and one 32-bit scale:
//
//   a = max(max_j |v_j|, 2^-100)
//   code_j = round_half_even(v_j * (127 / a)),  scale = a / 127
//   value_j = code_j * scale
//
// 2^-100 keeps 127 / a and a / 127 normal numbers for a row of zeros.  The
// maximum is the one that a NaN passes through (and, between threads, that of
// the bit patterns as unsigned integers, which orders them the same way, with
// infinities and NaN on top): a row that holds an infinity or a NaN gets a
// scale that is not finite, and so NaN for every value, and no other row is
// touched.
//
// Every kernel is one pass over memory: TPR threads share a row and keep it
// in registers (J chunks of 8 elements each) between the row's sums and the
// codes.  What bounds them is HBM; the arithmetic (in 32 bits, the norm's sum
// of squares in 64) hides behind the loads.
#pragma once

#include <hip/hip_runtime.h>

namespace xsymv {

using q8half = _Float16;
using q8bf16 = __bf16;

constexpr float Q8_FLOOR = 0x1p-100f;
constexpr int Q8_CHUNK = 8;  // elements a thread takes at once: 16 bytes of a 16-bit type

// ------------------------------------------------------------------ chunks
// Chunks are read and written where they lie: gfx950 takes 16-byte global
// accesses at any address, so odd strides cost partial lines but no other path.
// ONCE: the rows are not wanted in the caches after this (a non-temporal
// access).
template <bool ONCE = false, class T>
__device__ __forceinline__ void q8_load(const T* p, int have, float (&v)[Q8_CHUNK])
{
    typedef T vec __attribute__((ext_vector_type(Q8_CHUNK), aligned(sizeof(T))));
    if (have >= Q8_CHUNK) {
        vec t;
        if constexpr (ONCE)
            t = __builtin_nontemporal_load((const vec*)p);
        else
            t = *(const vec*)p;
#pragma unroll
        for (int e = 0; e < Q8_CHUNK; ++e) v[e] = (float)t[e];
    } else {
#pragma unroll
        for (int e = 0; e < Q8_CHUNK; ++e) v[e] = e < have ? (float)p[e] : 0.0f;
    }
}

template <bool ONCE = false, class T>
__device__ __forceinline__ void q8_store(T* p, int have, const float (&v)[Q8_CHUNK])
{
    typedef T vec __attribute__((ext_vector_type(Q8_CHUNK), aligned(sizeof(T))));
    if (have >= Q8_CHUNK) {
        vec t;
#pragma unroll
        for (int e = 0; e < Q8_CHUNK; ++e) t[e] = (T)v[e];
        if constexpr (ONCE)
            __builtin_nontemporal_store(t, (vec*)p);
        else
            *(vec*)p = t;
    } else {
#pragma unroll
        for (int e = 0; e < Q8_CHUNK; ++e)
            if (e < have) p[e] = (T)v[e];
    }
}

// Codes of a chunk.  Adding 1.5 * 2^23 to |t| <= 128 leaves t rounded half to
// even in the low bits, whose last byte is the code in two's complement.  The
// product with `inv` is rounded before: rows of 16-bit numbers have many
// products half way between two codes, which inv's own rounding would push to
// one side (131072 rows of 128 half-precision numbers: 2.6e-4 from a 64-bit
// quantisation's values, 3.9e-4 with a fused product, 1 % faster).
__device__ __forceinline__ void q8_store_codes(signed char* p, int have, const float (&v)[Q8_CHUNK],
                                               float inv)
{
    unsigned b[Q8_CHUNK];
#pragma unroll
    for (int e = 0; e < Q8_CHUNK; ++e) b[e] = __float_as_uint(v[e] * inv + 12582912.0f);
    if (have >= Q8_CHUNK) {
        unsigned w[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const unsigned lo = __builtin_amdgcn_perm(b[4 * i + 1], b[4 * i], 0x0c0c0400u);
            const unsigned hi = __builtin_amdgcn_perm(b[4 * i + 3], b[4 * i + 2], 0x04000c0cu);
            w[i] = lo | hi;
        }
        __builtin_memcpy(p, w, 8);
    } else {
#pragma unroll
        for (int e = 0; e < Q8_CHUNK; ++e)
            if (e < have) p[e] = (signed char)b[e];
    }
}

// -------------------------------------------------------------- reductions
// Over the TPR threads of a row: lane exchanges within a wave, then (TPR >
// 64) the results of the row's waves through LDS, read by all in the same
// order.  The LDS words alternate between `par` 0 and 1 from one
// row to the next, so one barrier per reduction suffices.
template <int TPR>
__device__ __forceinline__ unsigned q8_row_max(unsigned v, unsigned (&buf)[2][16], int par)
{
#pragma unroll
    for (int s = (TPR < 64 ? TPR : 64) / 2; s > 0; s >>= 1) {
        const unsigned o = __shfl_xor(v, s);
        v = v > o ? v : o;
    }
    if constexpr (TPR > 64) {
        if ((threadIdx.x & 63) == 0) buf[par][threadIdx.x >> 6] = v;
        __syncthreads();
        const int first = threadIdx.x / TPR * (TPR / 64);
#pragma unroll
        for (int i = 0; i < TPR / 64; ++i) {
            const unsigned o = buf[par][first + i];
            v = v > o ? v : o;
        }
    }
    return v;
}

template <int TPR>
__device__ __forceinline__ double q8_row_sum(double v, double (&buf)[2][16], int par)
{
#pragma unroll
    for (int s = (TPR < 64 ? TPR : 64) / 2; s > 0; s >>= 1) v += __shfl_xor(v, s);
    if constexpr (TPR > 64) {
        if ((threadIdx.x & 63) == 0) buf[par][threadIdx.x >> 6] = v;
        __syncthreads();
        const int first = threadIdx.x / TPR * (TPR / 64);
        v = buf[par][first];
#pragma unroll
        for (int i = 1; i < TPR / 64; ++i) v += buf[par][first + i];
    }
    return v;
}

// The larger of m and a chunk's magnitudes, or a NaN (two elements an
// instruction, where the bit patterns would take four).
__device__ __forceinline__ float q8_chunk_max(const float (&v)[Q8_CHUNK], float m)
{
#pragma unroll
    for (int e = 0; e < Q8_CHUNK; e += 2) {
        const float o = __builtin_elementwise_maximum(__builtin_fabsf(v[e]), __builtin_fabsf(v[e + 1]));
        m = __builtin_elementwise_maximum(m, o);
    }
    return m;
}

// a / 127 and 127 / a for 2^-100 <= a, each rounded once: the quotient by a
// rounded reciprocal is corrected by its exact remainder (Markstein's method),
// which has been compared with the division for all 2^23 significands and a
// reciprocal off by one unit either way.  Quotients and reciprocals are normal
// numbers (of a / 128 the reciprocal is one for every a).  The remainder
// a - 127 q of a scale can be subnormal for a below 2^-97; it is exact there as
// well, and then less than the 2^-124 it would take to change q (compared for
// all significands, the subnormal remainders kept or zero).  An infinity or NaN
// gives NaN.
// (The divisions were a sixth of a short row's instructions.)
__device__ __forceinline__ float q8_scale_of(float a)
{
    const float q = a * (1.0f / 127.0f);
    return __builtin_fmaf(__builtin_fmaf(-q, 127.0f, a), 1.0f / 127.0f, q);
}

__device__ __forceinline__ float q8_inverse_of(float a)
{
    const float t = a * 0x1p-7f, c = 127.0f / 128.0f;
    float y = __builtin_amdgcn_rcpf(t);
    y = __builtin_fmaf(__builtin_fmaf(-t, y, 1.0f), y, y);
    const float q = c * y;
    return __builtin_fmaf(__builtin_fmaf(-q, t, c), y, q);
}

// --------------------------------------------------------------- operators
// An operator gives: the row's destination (negative: the row is left out),
// a chunk of it (`first`), and, for the norm, the chunk after the row's sum
// of squares is known (`second`); `again` is `first` without its side effects.

// h = x + r rounded to R's type (which is what is kept and what is
// normalised), v = h / sqrt(mean(h^2) + eps) * w.  r may be null (h = x), h
// may be null (not kept), or r or x itself: an element is then read and written
// by the same thread alone.  The sum of squares is taken in 64 bits, which a row of the
// largest 32-bit numbers cannot overflow, and costs nothing beside the loads.
template <class T, class R, class W>
struct Q8Norm {
    static constexpr bool NORM = true;
    const T* x;
    const R* r;
    R* h;
    const W* w;
    long long ldx, ldr, ldh;
    double eps;
    int m, n;

    __device__ __forceinline__ long long dest(long long row) const { return row; }
    __host__ __device__ __forceinline__ bool in_place() const
    {
        return h != nullptr &&
               ((const void*)h == (const void*)r || (const void*)h == (const void*)x);
    }
    __device__ __forceinline__ void sum(long long row, int c, int have, float (&v)[Q8_CHUNK]) const
    {
        q8_load(x + row * ldx + c, have, v);
        if (r != nullptr) {
            float t[Q8_CHUNK];
            q8_load(r + row * ldr + c, have, t);
#pragma unroll
            for (int e = 0; e < Q8_CHUNK; ++e) v[e] += t[e];
        }
#pragma unroll
        for (int e = 0; e < Q8_CHUNK; ++e) v[e] = (float)(R)v[e];
    }
    // (the first `again` elements are another chunk's too, and counted there)
    __device__ __forceinline__ void first(long long row, int c, int have, int again,
                                          float (&v)[Q8_CHUNK], double& ss) const
    {
        sum(row, c, have, v);
        if (h != nullptr) q8_store(h + row * ldh + c, have, v);
        if (again == 0) {
#pragma unroll
            for (int e = 0; e < Q8_CHUNK; ++e) ss = __builtin_fma((double)v[e], (double)v[e], ss);
        } else {
#pragma unroll
            for (int e = 1; e < Q8_CHUNK; ++e)
                if (e >= again) ss = __builtin_fma((double)v[e], (double)v[e], ss);
        }
    }
    // a row too long for the registers: what was kept is read back (r or x may
    // have been overwritten by it)
    __device__ __forceinline__ void again(long long row, int c, int have, float (&v)[Q8_CHUNK]) const
    {
        if (h != nullptr)
            q8_load(h + row * ldh + c, have, v);
        else
            sum(row, c, have, v);
    }
    // 1 / sqrt(mean(h^2) + eps) as lift * f: it reaches from 2^-128 (a row of the
    // largest 32-bit numbers) to 2^165 (one of the smallest, where eps is 0), and
    // the power of two in front keeps f and h * lift normal numbers.
    struct Factor {
        float lift, f;
    };
    __device__ __forceinline__ Factor factor(double ss) const
    {
        const double d = 1.0 / sqrt(ss / n + eps);
        const float lift = d > 0x1p100 ? 0x1p64f : d < 0x1p-100 ? 0x1p-64f : 1.0f;
        return Factor{lift, (float)(d / lift)};
    }
    __device__ __forceinline__ void second(int c, int have, float (&v)[Q8_CHUNK], Factor k) const
    {
        float t[Q8_CHUNK];
        q8_load(w + c, have, t);
#pragma unroll
        for (int e = 0; e < Q8_CHUNK; ++e) v[e] = v[e] * k.lift * k.f * t[e];
    }
};

// v = g / (1 + exp(-g)) * u.  With z = exp(-|g|), which does not overflow,
// 1 / (1 + exp(-g)) is 1 / (1 + z) for g >= 0 and z / (1 + z) below.  z is taken
// as the square of h = exp(-|g| / 2), and h multiplies g and u below zero: the
// hardware's 2^t gives zero for results below 2^-126, which z is from g = -87.4
// on, but a row whose gates are all there has codes all the same (g = -88, u =
// 60000: 2^-104.6, 5 codes of a row at the floor).  Where h is
// zero, below g = -174, |g| z |u| < 2^-116 is less than half a code of any row.
// (z by itself: 4096 x 14336 52.4 us, so 53.1.)
// The hardware's 2^t and reciprocal (1 ulp each) serve: |g| log2(e) is rounded,
// its constant as well, so v is off by up to (2 |g| + 11) 2^-24 of itself for g
// < 0, the growing part of it z's alone.
template <class T>
struct Q8Glu {
    static constexpr bool NORM = false;
    struct Factor {};
    const T* g;
    const T* u;
    long long ldg, ldu;
    int m, n;

    __device__ __forceinline__ long long dest(long long row) const { return row; }
    __device__ __forceinline__ bool in_place() const { return false; }
    __device__ __forceinline__ void first(long long row, int c, int have, int, float (&v)[Q8_CHUNK],
                                          double&) const
    {
        float t[Q8_CHUNK];
        q8_load<true>(g + row * ldg + c, have, v);
        q8_load<true>(u + row * ldu + c, have, t);
#pragma unroll
        for (int e = 0; e < Q8_CHUNK; ++e) {
            const float h = __builtin_amdgcn_exp2f(-0.72134752f * __builtin_fabsf(v[e]));
            const float s = v[e] < 0.0f ? h : 1.0f;
            v[e] = v[e] * s * __builtin_amdgcn_rcpf(__builtin_fmaf(h, h, 1.0f)) * (t[e] * s);
        }
    }
    __device__ __forceinline__ void again(long long row, int c, int have, float (&v)[Q8_CHUNK]) const
    {
        double none = 0.0;
        first(row, c, have, 0, v, none);
    }
};

// v = x's row, written to row slot[i] of the cache (i itself without slots);
// a slot outside [0, cap) leaves the row out.
template <class T>
struct Q8Store {
    static constexpr bool NORM = false;
    struct Factor {};
    const T* x;
    const int* slot;
    long long ldx;
    int m, n, cap;

    __device__ __forceinline__ long long dest(long long row) const
    {
        const int s = slot != nullptr ? slot[row] : row;
        return s >= 0 && s < cap ? s : -1;
    }
    __device__ __forceinline__ bool in_place() const { return false; }
    __device__ __forceinline__ void first(long long row, int c, int have, int, float (&v)[Q8_CHUNK],
                                          double&) const
    {
        q8_load(x + row * ldx + c, have, v);
    }
    __device__ __forceinline__ void again(long long row, int c, int have, float (&v)[Q8_CHUNK]) const
    {
        q8_load(x + row * ldx + c, have, v);
    }
};

// Where chunks start at the latest: a row's last chunk is its last
// eight elements, some of them the chunk before's as well (their results are
// the same, whoever stores them), so that it is read and written at once; one
// element at a time it cost rows of 255 and 1564 elements 40 % more time.
// Not where an output takes an input's place: there an element belongs to one
// thread.
__host__ __device__ __forceinline__ int q8_last_column(int n, bool alone)
{
    return !alone && n >= Q8_CHUNK ? n - Q8_CHUNK : 0x7fffffff;
}

template <class OP>
struct Q8RowArgs {
    OP op;
    signed char* q;
    float* scale;
    long long ldq;
};

// One row per TPR threads; a workgroup of max(256, TPR) threads.  J chunks
// of the row in a thread's registers; J = 0: a row longer than 8 chunks of
// 1024 threads, whose elements are formed again for each of its sums.
// Two chunks a thread fit 64 registers, which lets a compute unit run two
// workgroups of 1024 threads: one's loads are on their way while the other
// waits for its row's sums.
template <class OP, int TPR, int J>
__global__ __launch_bounds__(TPR > 256 ? TPR : 256, TPR == 1024 && J == 2 ? 8 : 4) void q8_rows(
    Q8RowArgs<OP> a)
{
    constexpr int THREADS = TPR > 256 ? TPR : 256;
    constexpr int RPB = THREADS / TPR;  // rows per workgroup
    // chunks of a thread before the one that can be the row's last (a row takes
    // the smallest capacity that holds it; the largest one may be half empty)
    constexpr int LAST = J == 8 ? 4 : J - 1;
    __shared__ double sbuf[2][16];
    __shared__ unsigned mbuf[2][16];
    const OP& op = a.op;
    const int n = op.n;
    const int t = threadIdx.x % TPR;
    int par = 0;
    const int edge = q8_last_column(n, op.in_place());
    for (long long base = (long long)blockIdx.x * RPB; base < op.m;
         base += (long long)gridDim.x * RPB) {
        const long long row = base + threadIdx.x / TPR;
        const bool mine = row < op.m;
        // (a row left out is formed all the same, so that its loads need not
        // wait for the slot's)
        const long long dst = mine ? op.dest(row) : -1;
        const int have = mine ? n : 0;
        double ss = 0.0;
        float big = 0.0f;
        if constexpr (J > 0) {
            float v[J][Q8_CHUNK];
#pragma unroll
            for (int j = 0; j < J; ++j) {
                const int c = (t + j * TPR) * Q8_CHUNK, at = j < LAST ? c : min(c, edge);
                if (c < have) {
                    op.first(row, at, n - at, c - at, v[j], ss);
                } else {
#pragma unroll
                    for (int e = 0; e < Q8_CHUNK; ++e) v[j][e] = 0.0f;
                }
            }
            if constexpr (OP::NORM) {
                const auto f = op.factor(q8_row_sum<TPR>(ss, sbuf, par));
#pragma unroll
                for (int j = 0; j < J; ++j) {
                    const int c = (t + j * TPR) * Q8_CHUNK, at = j < LAST ? c : min(c, edge);
                    if (c < have) op.second(at, n - at, v[j], f);
                }
            }
#pragma unroll
            for (int j = 0; j < J; ++j) big = q8_chunk_max(v[j], big);
            const unsigned mx = q8_row_max<TPR>(__float_as_uint(big) & 0x7fffffffu, mbuf, par);
            par ^= 1;
            const float top = mx > __float_as_uint(Q8_FLOOR) ? __uint_as_float(mx) : Q8_FLOOR;
            if (dst < 0) continue;
            if (t == 0) a.scale[dst] = q8_scale_of(top);
            const float inv = q8_inverse_of(top);
#pragma unroll
            for (int j = 0; j < J; ++j) {
                const int c = (t + j * TPR) * Q8_CHUNK, at = j < LAST ? c : min(c, edge);
                if (c < n) q8_store_codes(a.q + dst * a.ldq + at, n - at, v[j], inv);
            }
        } else {
            typename OP::Factor f{};
            float v[Q8_CHUNK];
            if constexpr (OP::NORM) {
                for (long long c = t * Q8_CHUNK; c < n; c += TPR * Q8_CHUNK) {
                    const int at = min((int)c, edge);
                    op.first(row, at, n - at, (int)c - at, v, ss);
                }
                f = op.factor(q8_row_sum<TPR>(ss, sbuf, par));
            }
            for (long long c = t * Q8_CHUNK; c < n; c += TPR * Q8_CHUNK) {
                const int at = min((int)c, edge);
                op.again(row, at, n - at, v);
                if constexpr (OP::NORM) op.second(at, n - at, v, f);
                big = q8_chunk_max(v, big);
            }
            const unsigned mx = q8_row_max<TPR>(__float_as_uint(big) & 0x7fffffffu, mbuf, par);
            par ^= 1;
            const float top = mx > __float_as_uint(Q8_FLOOR) ? __uint_as_float(mx) : Q8_FLOOR;
            if (dst < 0) continue;
            if (t == 0) a.scale[dst] = q8_scale_of(top);
            const float inv = q8_inverse_of(top);
            for (long long c = t * Q8_CHUNK; c < n; c += TPR * Q8_CHUNK) {
                const int at = min((int)c, edge);
                op.again(row, at, n - at, v);
                if constexpr (OP::NORM) op.second(at, n - at, v, f);
                q8_store_codes(a.q + dst * a.ldq + at, n - at, v, inv);
            }
        }
    }
}

// -------------------------------------------------------------------- read
// out_i = code_j * scale of cache row slot[i] (i itself without slots); a
// slot outside [0, cap) gives a row of zeros.
template <class T>
struct Q8ReadArgs {
    const signed char* q;
    const float* scale;
    const int* slot;
    T* out;
    long long ldq, ldo;
    int m, n, cap;
};

// TPR threads a row, a chunk each; of a longer row, 256 chunks to a workgroup
// (blockIdx.y), so that a few long rows are as many loads in flight as many
// short ones.
template <class T, int TPR>
__global__ __launch_bounds__(256) void q8_read(Q8ReadArgs<T> a)
{
    constexpr int RPB = 256 / TPR;
    const int edge = q8_last_column(a.n, false);
    const long long first = ((long long)blockIdx.y * TPR + threadIdx.x % TPR) * Q8_CHUNK;
    for (long long row = (long long)blockIdx.x * RPB + threadIdx.x / TPR; row < a.m;
         row += (long long)gridDim.x * RPB) {
        const int s = a.slot != nullptr ? a.slot[row] : (int)row;
        const bool in = s >= 0 && s < a.cap;
        const float f = in ? a.scale[s] : 0.0f;
        for (long long c = first; c < a.n; c += (long long)gridDim.y * TPR * Q8_CHUNK) {
            const int at = min((int)c, edge);
            float v[Q8_CHUNK];
            if (in) {
                q8_load(a.q + s * a.ldq + at, a.n - at, v);
#pragma unroll
                for (int e = 0; e < Q8_CHUNK; ++e) v[e] *= f;
            } else {
#pragma unroll
                for (int e = 0; e < Q8_CHUNK; ++e) v[e] = 0.0f;
            }
            q8_store<true>(a.out + row * a.ldo + at, a.n - at, v);
        }
    }
}

}  // namespace xsymv
