// xq8_gemm.hpp -- the product of rows in 8 bits:
//
//   C[i, j] = (sum_l A[i, l] * W[j, l]) * sa[i] * sw[j] + bias[j]
//
// A is m x k and W n x k, signed 8-bit codes in rows (the format of
// xq8_rows.hpp), sa and sw their scales.  The sum is exact in 32-bit integers
// for k <= 131071 (128 * 128 * k < 2^31), so no order of it changes a bit;
// it is then rounded to 32-bit floating point once, and each product and the
// sum with the bias rounds once more there.
//
// The products run on the matrix cores (16 x 16 x 64 integer
// multiply-accumulate): lane l holds 16 bytes of row l % 16 of each operand,
// the 16-byte piece l / 16 of a 64-byte step, and receives column l % 16,
// rows 4 * (l / 16) .. + 3 of the result.  W is the first operand, so a lane
// receives four neighbouring elements of a row of C.  Which byte of a step
// meets which multiplier does not matter as long as both operands agree.
//
// Bytes past k are loaded as zeros (in both operands), rows past m or n are
// the last row again, whose results are not stored: no access leaves the
// operands.
#pragma once

#include <hip/hip_runtime.h>

#include "xq8_rows.hpp"

namespace xsymv {

typedef int q8v4 __attribute__((ext_vector_type(4)));

constexpr int Q8_MAX_K = 131071;

template <class T>
struct Q8GemmArgs {
    const signed char* a;
    const signed char* w;
    const float* sa;
    const float* sw;
    const float* bias;
    T* c;
    long long lda, ldw, ldc;
    int m, n, k;
};

// 16 bytes at p, of which `have` (any value) lie within the row.
__device__ __forceinline__ q8v4 q8_load16(const signed char* p, int have)
{
    q8v4 v = {0, 0, 0, 0};
    if (have >= 16) {
        __builtin_memcpy(&v, p, 16);
    } else if (have > 0) {
#pragma unroll
        for (int i = 0; i < 16; ++i)
            if (i < have) v[i >> 2] |= (int)(unsigned char)p[i] << (8 * (i & 3));
    }
    return v;
}

// Four neighbouring elements of row i from column j on.
template <class T>
__device__ __forceinline__ void q8_finish(const Q8GemmArgs<T>& g, int i, int j, q8v4 sum)
{
    typedef T vec __attribute__((ext_vector_type(4)));
    if (i >= g.m || j >= g.n) return;
    const float si = g.sa[i];
    vec t;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const int jj = j + e < g.n ? j + e : g.n - 1;
        float v = (float)sum[e] * si * g.sw[jj];
        if (g.bias != nullptr) v += g.bias[jj];
        t[e] = (T)v;
    }
    T* p = g.c + i * g.ldc + j;
    if (j + 4 <= g.n) {
        __builtin_memcpy(p, &t, sizeof(t));
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (j + e < g.n) p[e] = t[e];
    }
}

// Few rows: the bytes of W bound the product, and W is used once per
// workgroup, so it goes from memory to registers without LDS.  A workgroup of
// WK waves makes a block of 16 MT rows of C by 16 NT columns; the waves take
// the 256-byte steps of k in turn and add their sums through LDS.
template <class T, int MT, int NT, int WK>
__global__ __launch_bounds__(64 * WK) void q8_gemm_stream(Q8GemmArgs<T> g)
{
    constexpr int U = 4;  // 64-byte steps a wave loads at once
    __shared__ int red[WK > 1 ? WK : 1][MT * NT][4][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int mblocks = (g.m + 16 * MT - 1) / (16 * MT);
    const int i0 = (int)(blockIdx.x % mblocks) * 16 * MT;
    const int j0 = (int)(blockIdx.x / mblocks) * 16 * NT;
    const int r = lane & 15, piece = (lane >> 4) * 16;
    const signed char* pa[MT];
    const signed char* pw[NT];
#pragma unroll
    for (int i = 0; i < MT; ++i) {
        const int row = i0 + 16 * i + r;
        pa[i] = g.a + (row < g.m ? row : g.m - 1) * g.lda + piece;
    }
#pragma unroll
    for (int j = 0; j < NT; ++j) {
        const int row = j0 + 16 * j + r;
        pw[j] = g.w + (row < g.n ? row : g.n - 1) * g.ldw + piece;
    }
    q8v4 acc[MT][NT];
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j) acc[i][j] = q8v4{0, 0, 0, 0};

    for (int k0 = wave * 64 * U; k0 < g.k; k0 += WK * 64 * U) {
        q8v4 va[U][MT], vw[U][NT];
        if (k0 + 64 * U <= g.k) {
#pragma unroll
            for (int u = 0; u < U; ++u) {
#pragma unroll
                for (int j = 0; j < NT; ++j) __builtin_memcpy(&vw[u][j], pw[j] + k0 + 64 * u, 16);
#pragma unroll
                for (int i = 0; i < MT; ++i) __builtin_memcpy(&va[u][i], pa[i] + k0 + 64 * u, 16);
            }
        } else {
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int have = g.k - k0 - 64 * u - piece;
#pragma unroll
                for (int j = 0; j < NT; ++j) vw[u][j] = q8_load16(pw[j] + k0 + 64 * u, have);
#pragma unroll
                for (int i = 0; i < MT; ++i) va[u][i] = q8_load16(pa[i] + k0 + 64 * u, have);
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int i = 0; i < MT; ++i)
#pragma unroll
                for (int j = 0; j < NT; ++j)
                    acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(vw[u][j], va[u][i], acc[i][j],
                                                                      0, 0, 0);
    }
    if constexpr (WK > 1) {
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) red[wave][i * NT + j][e][lane] = acc[i][j][e];
        __syncthreads();
        for (int tile = wave; tile < MT * NT; tile += WK) {
            q8v4 sum = {0, 0, 0, 0};
#pragma unroll
            for (int w = 0; w < WK; ++w)
#pragma unroll
                for (int e = 0; e < 4; ++e) sum[e] += red[w][tile][e][lane];
            q8_finish(g, i0 + 16 * (tile / NT) + r, j0 + 16 * (tile % NT) + piece / 4, sum);
        }
    } else {
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int j = 0; j < NT; ++j)
                q8_finish(g, i0 + 16 * i + r, j0 + 16 * j + piece / 4, acc[i][j]);
    }
}

}  // namespace xsymv
