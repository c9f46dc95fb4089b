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

#include <type_traits>

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

// 16 bytes at p, of which `have` (any value) lie within the row; the bytes
// past it are read from the row's last instead, and zeroed.
__device__ __forceinline__ q8v4 q8_load16(const signed char* p, int have)
{
    q8v4 v = {0, 0, 0, 0};
    if (have >= 16) {
        __builtin_memcpy(&v, p, 16);
    } else if (have > 0) {
        unsigned char b[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) b[i] = (unsigned char)p[i < have ? i : have - 1];
#pragma unroll
        for (int i = 0; i < 16; ++i) v[i >> 2] |= (i < have ? (int)b[i] : 0) << (8 * (i & 3));
    }
    return v;
}

// A lane's results: rows i + 16 f, four neighbouring columns from j + 16 h on.
// The scales are loaded ahead of the products (rows and columns past the last
// take the last's, and are not stored).
template <class T, int FM, int FN>
__device__ __forceinline__ void q8_finish(const Q8GemmArgs<T>& g, int i, int j,
                                          const q8v4 (&sum)[FM][FN])
{
    typedef T vec __attribute__((ext_vector_type(4)));
    float si[FM], sj[FN][4], bj[FN][4];
#pragma unroll
    for (int f = 0; f < FM; ++f) si[f] = g.sa[i + 16 * f < g.m ? i + 16 * f : g.m - 1];
#pragma unroll
    for (int h = 0; h < FN; ++h)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int c = j + 16 * h + e;
            sj[h][e] = g.sw[c < g.n ? c : g.n - 1];
        }
    if (g.bias != nullptr) {
#pragma unroll
        for (int h = 0; h < FN; ++h)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int c = j + 16 * h + e;
                bj[h][e] = g.bias[c < g.n ? c : g.n - 1];
            }
    } else {
#pragma unroll
        for (int h = 0; h < FN; ++h)
#pragma unroll
            for (int e = 0; e < 4; ++e) bj[h][e] = -0.0f;  // v + -0 is v
    }
#pragma unroll
    for (int f = 0; f < FM; ++f) {
        if (i + 16 * f >= g.m) break;
        T* row = g.c + (i + 16 * f) * g.ldc;
#pragma unroll
        for (int h = 0; h < FN; ++h) {
            const int c = j + 16 * h;
            vec t;
#pragma unroll
            for (int e = 0; e < 4; ++e) t[e] = (T)((float)sum[f][h][e] * si[f] * sj[h][e] + bj[h][e]);
            if (c + 4 <= g.n) {
                __builtin_memcpy(row + c, &t, sizeof(t));
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (c + e < g.n) row[c + e] = t[e];
            }
        }
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
            q8v4 sum[1][1] = {{{0, 0, 0, 0}}};
#pragma unroll
            for (int w = 0; w < WK; ++w)
#pragma unroll
                for (int e = 0; e < 4; ++e) sum[0][0][e] += red[w][tile][e][lane];
            q8_finish<T, 1, 1>(g, i0 + 16 * (tile / NT) + r, j0 + 16 * (tile % NT) + piece / 4, sum);
        }
    } else {
        q8_finish<T, MT, NT>(g, i0 + r, j0 + piece / 4, acc);
    }
}

// ------------------------------------------------------- many rows: tiles
// A workgroup of WM x WN waves makes a BM x BN tile of C, 128 bytes of k at a
// time through LDS, where the tile's rows lie 128 bytes apart with their
// eight 16-byte pieces permuted by the row (piece c at c ^ (row / 2) % 8), so
// that the 16 rows a wave reads at once fall on different banks.  Two
// buffers; one barrier per 128 bytes:
//
//   read the second half of step t     | multiply the first half
//   barrier: step t + 1 has arrived, and nobody reads step t's buffer again
//   fetch step t + 2 into that buffer, read the first half of step t + 1
//                                      | multiply the second half of step t
//
// so the loads from memory have a whole step to arrive and the reads from LDS
// half a step, behind the other half's multiplications.
//
// DMA: the loads go from memory to LDS by themselves (rows at multiples of 16
// bytes); the wait for them is the one before the barrier.  Otherwise they go
// through registers, 16 bytes at any address, and are written to LDS before
// the next barrier.  A k that is no multiple of 128 has its last, partial step
// taken first, through registers in either case, its bytes past k being zeros.

// Waits for everything this wave has in flight, then for the other waves.
__device__ __forceinline__ void q8_sync()
{
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
}

// 16 bytes of each lane from rsrc's base + voff + soff to LDS address `lds`
// plus 16 times the lane.  Nothing is returned; q8_sync waits for it.
__device__ __forceinline__ void q8_fetch(unsigned lds, unsigned voff, q8v4 rsrc, unsigned soff)
{
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds"
                 :
                 : "s"(__builtin_amdgcn_readfirstlane((int)lds)), "v"(voff), "s"(rsrc),
                   "s"(__builtin_amdgcn_readfirstlane((int)soff))
                 : "memory", "m0");
}

__device__ __forceinline__ q8v4 q8_rsrc(const signed char* p, unsigned bytes)
{
    const unsigned long long a = (unsigned long long)p;
    return q8v4{__builtin_amdgcn_readfirstlane((int)a),
                __builtin_amdgcn_readfirstlane((int)(a >> 32) & 0xffff),
                __builtin_amdgcn_readfirstlane((int)bytes), 0x00020000};
}

// Work item `id` of `mt` x `nt` tiles: the chip's eight dies take workgroups
// in turn and have a cache each, so a die gets a run of consecutive tiles,
// and tiles are numbered in bands of 8 rows of tiles, column by column: the
// 32 tiles a die works on at a time share 8 blocks of A and 4 of W.
__device__ __forceinline__ void q8_tile(unsigned id, unsigned mt, unsigned nt, unsigned& ti,
                                        unsigned& tj)
{
    const unsigned total = mt * nt, die = id % 8, per = total / 8, more = total % 8;
    const unsigned k = die * per + (die < more ? die : more) + id / 8;
    const unsigned band = k / (8 * nt), rows = mt - 8 * band < 8 ? mt - 8 * band : 8;
    const unsigned in = k - band * 8 * nt;
    ti = 8 * band + in % rows;
    tj = in / rows;
}

template <class T, int BM, int BN, int WM, int WN, bool DMA>
__global__ __launch_bounds__(64 * WM * WN) void q8_gemm_tile(Q8GemmArgs<T> g)
{
    constexpr int BK = 128, WAVES = WM * WN;
    constexpr int FM = BM / WM / 16, FN = BN / WN / 16;    // 16 x 16 results of a wave
    constexpr int LA = BM / 8 / WAVES, LW = BN / 8 / WAVES;  // 1 KB loads of a wave and step
    constexpr int BUF = (BM + BN) * BK;
    static_assert(LA * 8 * WAVES == BM && LW * 8 * WAVES == BN, "whole loads");
    __shared__ __attribute__((aligned(1024))) signed char lds[2][BUF];

    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    unsigned ti, tj;
    q8_tile(blockIdx.x, (g.m + BM - 1) / BM, (g.n + BN - 1) / BN, ti, tj);
    const int i0 = ti * BM, j0 = tj * BN;
    const int steps = (g.k + BK - 1) / BK, part = g.k % BK != 0;

    // loads: 8 rows of 128 bytes each, lane l row l / 8, its piece where the
    // permutation puts it
    const int lrow = wave * 8 + (lane >> 3);  // row of load 0; load i: + 8 * WAVES * i
    const int lpiece = ((lane & 7) ^ ((lrow >> 1) & 7)) * 16;
    const signed char* ga = g.a + i0 * g.lda;
    const signed char* gw = g.w + j0 * g.ldw;
    const int ma = g.m - 1 - i0, mw = g.n - 1 - j0;  // last rows
    // a tile's rows lie within 32-bit offsets where DMA is chosen
    typename std::conditional<DMA, unsigned, long long>::type oa[LA], ow[LW];
#pragma unroll
    for (int i = 0; i < LA; ++i) {
        const int row = lrow + 8 * WAVES * i;
        oa[i] = (row < ma ? row : ma) * g.lda + lpiece;
    }
#pragma unroll
    for (int i = 0; i < LW; ++i) {
        const int row = lrow + 8 * WAVES * i;
        ow[i] = (row < mw ? row : mw) * g.ldw + lpiece;
    }
    const q8v4 ra = q8_rsrc(ga, 0xffffffffu), rw = q8_rsrc(gw, 0xffffffffu);
    const unsigned base = (unsigned)(unsigned long long)(__attribute__((address_space(3))) void*)lds;
    q8v4 st[DMA ? 1 : LA + LW];
    int held = -1;  // the step whose bytes wait in st

    auto put = [&](int t) {  // registers to LDS
        if constexpr (!DMA) {
            if (held < 0) return;
#pragma unroll
            for (int i = 0; i < LA; ++i)
                *(q8v4*)&lds[t & 1][(wave + WAVES * i) * 1024 + lane * 16] = st[i];
#pragma unroll
            for (int i = 0; i < LW; ++i)
                *(q8v4*)&lds[t & 1][BM * BK + (wave + WAVES * i) * 1024 + lane * 16] = st[LA + i];
            held = -1;
        }
    };
    // step t starts at byte (t - part) * BK of k; a partial step is taken first
    auto fetch = [&](int t) {
        if (t >= steps) return;
        const int k0 = (t - part) * BK;
        if constexpr (DMA) {
            const unsigned to = base + (t & 1) * BUF + wave * 1024;
#pragma unroll
            for (int i = 0; i < LA; ++i) q8_fetch(to + WAVES * 1024 * i, oa[i], ra, k0);
#pragma unroll
            for (int i = 0; i < LW; ++i) q8_fetch(to + BM * BK + WAVES * 1024 * i, ow[i], rw, k0);
        } else {
#pragma unroll
            for (int i = 0; i < LA; ++i) __builtin_memcpy(&st[i], ga + oa[i] + k0, 16);
#pragma unroll
            for (int i = 0; i < LW; ++i) __builtin_memcpy(&st[LA + i], gw + ow[i] + k0, 16);
            held = t;
        }
    };

    // reads: lane l takes row l % 16 of a block of 16, piece 4 h + l / 16 of half h
    const int wm = wave / WN, wn = wave % WN;
    const int perm = (((lane >> 4) ^ ((lane >> 1) & 7)) * 16) + (lane & 15) * BK;
    const int fa = wm * FM * 16 * BK, fw = BM * BK + wn * FN * 16 * BK;
    q8v4 xa[2][FM], xw[2][FN], acc[FM][FN];
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j) acc[i][j] = q8v4{0, 0, 0, 0};
    auto read = [&](int t, int h) {
        const signed char* p = &lds[t & 1][perm ^ (h * 64)];
#pragma unroll
        for (int j = 0; j < FN; ++j) xw[h][j] = *(const q8v4*)(p + fw + j * 16 * BK);
#pragma unroll
        for (int i = 0; i < FM; ++i) xa[h][i] = *(const q8v4*)(p + fa + i * 16 * BK);
    };
    auto multiply = [&](int h) {
#pragma unroll
        for (int i = 0; i < FM; ++i)
#pragma unroll
            for (int j = 0; j < FN; ++j)
                acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(xw[h][j], xa[h][i], acc[i][j], 0,
                                                                  0, 0);
    };

    if (steps > 0) {
        if (part) {
            const int k0 = g.k / BK * BK, have = g.k - k0 - lpiece;
#pragma unroll
            for (int i = 0; i < LA; ++i)
                *(q8v4*)&lds[0][(wave + WAVES * i) * 1024 + lane * 16] =
                    q8_load16(ga + oa[i] + k0, have);
#pragma unroll
            for (int i = 0; i < LW; ++i)
                *(q8v4*)&lds[0][BM * BK + (wave + WAVES * i) * 1024 + lane * 16] =
                    q8_load16(gw + ow[i] + k0, have);
        } else {
            fetch(0);
            put(0);
        }
        q8_sync();
        fetch(1);
        read(0, 0);
        for (int t = 0; t < steps; ++t) {
            read(t, 1);
            __builtin_amdgcn_sched_barrier(0);
            multiply(0);
            __builtin_amdgcn_sched_barrier(0);
            put(t + 1);
            q8_sync();
            fetch(t + 2);
            if (t + 1 < steps) read(t + 1, 0);
            __builtin_amdgcn_sched_barrier(0);
            multiply(1);
            __builtin_amdgcn_sched_barrier(0);
        }
    }
    q8_finish<T, FM, FN>(g, i0 + wm * FM * 16 + (lane & 15), j0 + wn * FN * 16 + (lane >> 4) * 4, acc);
}

}  // namespace xsymv
