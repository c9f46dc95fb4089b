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
// Bytes past k count as zeros, rows past m or n are the last row again, whose
// results are not stored: no access leaves the operands.
//
// Three kinds of kernel make it, each at the sizes where it measured fastest:
// tiles of 16 to 256 rows of both operands through LDS, whose waves share what
// is loaded; for few results a ring of buffers for each wave, which waits for
// no other wave; and for up to 16 of the shortest rows at odd strides straight
// loads to registers, which have nothing to set up.  Where there are fewer
// tiles than the chip holds at once, k is split into shares, whose sums are
// added by another launch.
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
    // k in `splits` shares of `per` of the kernel's steps, their sums in `part`
    // (one share: straight to C); the stream kernel takes k whole
    int* part;
    int splits, per;
};

// Row length of the shares' sums.
__host__ __device__ inline long long q8_part_ld(int n) { return ((long long)n + 3) / 4 * 4; }

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

// The scales (and bias) of a lane's results: rows i + 16 f, four neighbouring
// columns from j + 16 h on.  Rows and columns past the last take the last's,
// and are not stored.  The ring loads them before its sums (1 x 4096 x 4096
// 5.8 -> 5.6 us); the tiles after, since the registers they would hold cost
// them more (128 x 128 at k = 128, odd strides: 20.7 us after, 25.2 before).
template <class T, int FM, int FN>
struct Q8Scales {
    float si[FM], sj[FN][4], bj[FN][4];

    __device__ __forceinline__ void load(const Q8GemmArgs<T>& g, int i, int j)
    {
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
    }
};

template <class T, int FM, int FN>
__device__ __forceinline__ void q8_finish(const Q8GemmArgs<T>& g, int i, int j,
                                          const Q8Scales<T, FM, FN>& s, const q8v4 (&sum)[FM][FN])
{
    typedef T vec __attribute__((ext_vector_type(4)));
#pragma unroll
    for (int f = 0; f < FM; ++f) {
        if (i + 16 * f >= g.m) break;
        T* row = g.c + (i + 16 * f) * g.ldc;
#pragma unroll
        for (int h = 0; h < FN; ++h) {
            const int c = j + 16 * h;
            vec t;
#pragma unroll
            for (int e = 0; e < 4; ++e)
                t[e] = (T)((float)sum[f][h][e] * s.si[f] * s.sj[h][e] + s.bj[h][e]);
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

template <class T, int FM, int FN>
__device__ __forceinline__ void q8_finish(const Q8GemmArgs<T>& g, int i, int j,
                                          const q8v4 (&sum)[FM][FN])
{
    Q8Scales<T, FM, FN> s;
    s.load(g, i, j);
    q8_finish(g, i, j, s, sum);
}

// The same results as a share's sums.
template <class T, int FM, int FN>
__device__ __forceinline__ void q8_partial(const Q8GemmArgs<T>& g, unsigned share, int i, int j,
                                           const q8v4 (&sum)[FM][FN])
{
    const long long ldp = q8_part_ld(g.n);
    int* sums = g.part + share * (g.m * ldp);
#pragma unroll
    for (int f = 0; f < FM; ++f) {
        if (i + 16 * f >= g.m) break;
#pragma unroll
        for (int h = 0; h < FN; ++h)
            if (j + 16 * h < g.n) *(q8v4*)(sums + (i + 16 * f) * ldp + j + 16 * h) = sum[f][h];
    }
}

// ------------------------------------------------ few rows: straight to registers
// Rows at any address, 16 x 16 results a workgroup: the eight waves take the
// 256-byte steps of k in turn, load both operands' 16-byte pieces where the
// multiplier wants them, and add their sums through LDS.  A load brings 64
// bytes of each of 16 rows, so lines are fetched in halves and long rows take
// twice as long as with the ring (16 x 1024 x 8192 at odd strides 21.6 us, the
// ring 8.3); with nothing to set up, short ones are quicker (1 x 1024 x 256
// 3.2 us, the ring 3.8).
constexpr int Q8_WAVES = 8;  // of a workgroup

template <class T>
__global__ __launch_bounds__(64 * Q8_WAVES) void q8_gemm_stream(Q8GemmArgs<T> g)
{
    constexpr int U = 4;  // 64-byte steps a wave loads at once
    __shared__ q8v4 red[Q8_WAVES][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int mblocks = (g.m + 15) / 16;
    const int i0 = (int)(blockIdx.x % mblocks) * 16, j0 = (int)(blockIdx.x / mblocks) * 16;
    const int r = lane & 15, piece = (lane >> 4) * 16;
    const signed char* pa = g.a + (i0 + r < g.m ? i0 + r : g.m - 1) * g.lda + piece;
    const signed char* pw = g.w + (j0 + r < g.n ? j0 + r : g.n - 1) * g.ldw + piece;
    q8v4 acc = {0, 0, 0, 0};
    for (int k0 = wave * 64 * U; k0 < g.k; k0 += Q8_WAVES * 64 * U) {
        q8v4 va[U], vw[U];
        if (k0 + 64 * U <= g.k) {
#pragma unroll
            for (int u = 0; u < U; ++u) {
                __builtin_memcpy(&vw[u], pw + k0 + 64 * u, 16);
                __builtin_memcpy(&va[u], pa + k0 + 64 * u, 16);
            }
        } else {
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int have = g.k - k0 - 64 * u - piece;
                vw[u] = q8_load16(pw + k0 + 64 * u, have);
                va[u] = q8_load16(pa + k0 + 64 * u, have);
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
            acc = __builtin_amdgcn_mfma_i32_16x16x64_i8(vw[u], va[u], acc, 0, 0, 0);
    }
    red[wave][lane] = acc;
    __syncthreads();
    if (wave != 0) return;
    q8v4 sum[1][1] = {{{0, 0, 0, 0}}};
#pragma unroll
    for (int w = 0; w < Q8_WAVES; ++w) sum[0][0] += red[w][lane];
    q8_finish<T, 1, 1>(g, i0 + r, j0 + piece / 4, sum);
}

// ------------------------------------------------------------------- tiles
// A workgroup of WM x WN waves makes a BM x BN tile of C, 128 Q bytes of k at
// a time through LDS, in S buffers, with one barrier a step:
//
//   multiply all but the last 64 bytes of step t, reading the next 64 meanwhile
//   barrier: step t + 1 has arrived, and nobody reads step t's buffer again
//   multiply the last 64, reading the first 64 of step t + 1 and fetching
//   step t + S into the buffer meanwhile
//
// so the loads from memory have S - 1 steps to arrive and the reads from LDS
// the time of a piece's multiplications.  Loads and reads are issued between
// the multiplications, a few at a time: issued together they hold up the
// wave's multiplications until the memory pipeline has taken them all.
//
// What bounds a full compute unit is LDS, at 128 bytes a cycle: a step of 128
// bytes of k takes 1024 cycles of reads and writes and 512 of multiplications
// in a 128 x 128 tile of eight waves, 1408 and 1024 in 256 x 128, 2048 and 2048
// in 256 x 256.  The steps that fit best over many sizes are 0.48, 0.69 and 1.27
// us; the last is 1.6 in 4096 x 28672 x 8192 (740 us, 448 steps one after the
// other), where the multiplications leave a clock of 1.9 GHz.  The loads could bring
// twice the bytes (125 GB/s a compute unit from the die's cache).  Four waves
// of larger parts read less but wait more: 2048 x 8192 x 8192 by 128 x 128
// tiles of four waves 196 us, of eight 163, by 256 x 128 of eight 131.
//
// How the rows come to LDS (HOW):
//
// Q8_LINES  rows at multiples of 16 bytes.  The loads go from memory to LDS by
//           themselves, and the wait for them is the one before the barrier.
//           A row's step is 128 Q bytes of LDS with its 16-byte pieces
//           permuted by the row, so that the 16 rows a wave reads at once fall
//           on different banks.
// Q8_ANY    rows at any stride, the first at a multiple of 16 bytes.  The same
//           loads take the 8 Q + 1 aligned pieces that hold a row's step (an
//           odd number of pieces, which spreads the rows over the banks as
//           well); the reads take the three words of 8 bytes that hold a piece
//           of the row, and its bytes are shifted out of them before they are
//           multiplied.  (LDS reads 16 bytes at once at any address too, but
//           several times slower, and in words of 4 bytes it takes five reads.)
//           Memory delivers 64 bytes at a time, so a row's step that
//           starts anywhere costs one delivery more: Q = 2 where LDS has room.
// Q8_REGS   anything else: through registers, 16 bytes at any address, written
//           to LDS before the next barrier; S = 2.
//
// No load leaves the operands.  Where a step reaches past k, the loads take
// what lies there, the row's gap or the next row, and the multiplier's first
// half (A's bytes) is zeroed past k.  In the operand's last row a piece that
// reaches past its end takes the last whole piece instead; if such a piece
// still holds the row's last bytes, they are written over it one by one before
// they are read (patch).
enum { Q8_REGS = 0, Q8_LINES = 1, Q8_ANY = 2 };

// Waits until at most N of this wave's loads are on their way and its reads
// and writes of LDS are done, then for the other waves.
template <int N>
__device__ __forceinline__ void q8_sync()
{
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(N) : "memory");
}

// 16 bytes of each lane from rsrc's base + voff + soff to LDS address `lds`
// plus 16 times the lane.  Nothing is returned; q8_sync waits for it.
__device__ __forceinline__ void q8_fetch(unsigned lds, unsigned voff, q8v4 rsrc, unsigned soff = 0)
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

// The tile (and share of k) of workgroup blockIdx.x: the chip's eight dies
// take workgroups in turn and have a cache each, so a die gets a run of
// consecutive tiles, and the tiles of a share are numbered in bands of 8 rows
// of tiles, column by column: the 32 tiles a die works on at a time read 8
// blocks of A and 4 of W.
__device__ __forceinline__ void q8_tile(unsigned mt, unsigned nt, unsigned& ti, unsigned& tj,
                                        unsigned& share)
{
    const unsigned die = blockIdx.x % 8, per = gridDim.x / 8, more = gridDim.x % 8;
    unsigned k = die * per + (die < more ? die : more) + blockIdx.x / 8;
    share = k / (mt * nt);
    k -= share * (mt * nt);
    const unsigned band = k / (8 * nt), rows = mt - 8 * band < 8 ? mt - 8 * band : 8;
    const unsigned in = k - band * 8 * nt;
    ti = 8 * band + in % rows;
    tj = in / rows;
}

// 16 bytes of a row in LDS, `at` (plus `k` into the step), as Q8_LINES lays
// them out; with Q8_ANY the three words of 8 bytes that hold them where the
// row starts at byte `shift` of its first piece, and then (q8_bytes) the bytes.
template <int HOW, class V>
__device__ __forceinline__ void q8_read(V& x, const signed char* p, int at, int k, int shift)
{
    if constexpr (HOW == Q8_ANY) {
        typedef int two __attribute__((ext_vector_type(2)));
        typedef const volatile __attribute__((address_space(3))) two word;
        word* v = (word*)(p + at + k + (shift & 8));
#pragma unroll
        for (int e = 0; e < 3; ++e) {
            const two y = v[e];
            x[2 * e] = y.x;
            x[2 * e + 1] = y.y;
        }
    } else {
        x = *(const V*)(p + (at ^ k));
    }
}

template <int HOW, class V>
__device__ __forceinline__ q8v4 q8_bytes(const V& x, int shift)
{
    if constexpr (HOW == Q8_ANY) {
        const int odd = -(shift >> 2 & 1);  // all bits where they start in the second half
        int y[5];
        q8v4 v;
#pragma unroll
        for (int e = 0; e < 5; ++e) y[e] = (x[e + 1] & odd) | (x[e] & ~odd);
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = __builtin_amdgcn_alignbyte(y[e + 1], y[e], shift & 3);
        return v;
    } else {
        return x;
    }
}

template <class T, int BM, int BN, int WM, int WN, int Q, int S, int HOW>
__global__ __launch_bounds__(64 * WM * WN) void q8_gemm_tile(Q8GemmArgs<T> g)
{
    constexpr bool DMA = HOW != Q8_REGS;
    constexpr int BK = 128 * Q, WAVES = WM * WN, CH = 8 * Q + (HOW == Q8_ANY ? 1 : 0);
    constexpr int PITCH = 16 * CH, H = 2 * Q;            // bytes of LDS a row, pieces of 64 a step
    constexpr int FM = BM / WM / 16, FN = BN / WN / 16;  // 16 x 16 results of a wave
    constexpr int R = FM + FN;                           // reads of a wave and 64 bytes
    // loads of 64 pieces, a wave each: A's, then W's (the last may reach past
    // the block's rows), P to a wave (the last ones may be done twice)
    constexpr int CA = (BM * CH + 63) / 64, CW = (BN * CH + 63) / 64;
    constexpr int P = (CA + CW + WAVES - 1) / WAVES;
    constexpr int BUF = (CA + CW) * 1024, OW = CA * 1024;
    static_assert(DMA ? S >= 2 && (S - 1) * P < 64 : S == 2, "the counter of outstanding loads");
    __shared__ __attribute__((aligned(1024))) signed char lds[S * BUF];

    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    unsigned ti, tj, share;
    q8_tile((g.m + BM - 1) / BM, (g.n + BN - 1) / BN, ti, tj, share);
    const int i0 = ti * BM, j0 = tj * BN;
    // this share's steps: t0 and the `steps` - 1 after it
    const int all = (g.k + BK - 1) / BK, t0 = (int)share * g.per;
    const int steps = all - t0 < g.per ? all - t0 : g.per;

    const signed char* ga = g.a + i0 * g.lda;
    const signed char* gw = g.w + j0 * g.ldw;
    const int ma = g.m - 1 - i0, mw = g.n - 1 - j0;  // last rows
    const int sha = HOW == Q8_ANY ? (int)((size_t)ga & 15) : 0;
    const int shw = HOW == Q8_ANY ? (int)((size_t)gw & 15) : 0;
    const q8v4 ra = q8_rsrc(ga - sha, 0xffffffffu), rw = q8_rsrc(gw - shw, 0xffffffffu);
    // the operands' ends, from the bases of ra and rw, and their last whole pieces
    const long long enda = ma * g.lda + sha + g.k, endw = mw * g.ldw + shw + g.k;
    const unsigned lasta = (unsigned)(enda < 1ll << 32 ? enda - 16 : 0xfffffff0ll) & ~15u;
    const unsigned lastw = (unsigned)(endw < 1ll << 32 ? endw - 16 : 0xfffffff0ll) & ~15u;
    auto turned = [](int row) { return Q == 1 ? (row >> 1) & 7 : row & 15; };

    // a tile's rows lie within 32-bit offsets where the loads need them to
    typename std::conditional<DMA, unsigned, long long>::type off[P];
    int in[DMA ? 1 : P];  // the byte of the step a load starts at
    auto load_id = [&](int p) {
        const int id = p * WAVES + wave;
        return (CA + CW) % WAVES == 0 || id < CA + CW ? id : CA + CW - 1;
    };
    auto of_w = [&](int p) { return CA % WAVES == 0 ? p >= CA / WAVES : load_id(p) >= CA; };
#pragma unroll
    for (int p = 0; p < P; ++p) {
        const bool w = of_w(p);
        const int piece = (load_id(p) - (w ? CA : 0)) * 64 + lane;
        const int r = piece / CH, c = piece % CH, last = w ? mw : ma;
        const long long o = (r < last ? r : last) * (w ? g.ldw : g.lda);
        if constexpr (HOW == Q8_ANY)
            off[p] = (unsigned)((o + (w ? shw : sha)) & ~15ll) + 16 * c;
        else
            off[p] = o + 16 * (c ^ turned(r));
        if constexpr (!DMA) in[p] = 16 * (c ^ turned(r));
    }
    const unsigned base = (unsigned)(unsigned long long)(__attribute__((address_space(3))) void*)lds;
    q8v4 st[DMA ? 1 : P];

    auto fetch = [&](int t, int p) {  // load p of the share's step t
        const int k0 = (t0 + t) * BK;
        if constexpr (DMA) {
            const unsigned o = off[p] + k0, last = of_w(p) ? lastw : lasta;
            q8_fetch(base + (unsigned)(t % S) * BUF + load_id(p) * 1024, o < last ? o : last,
                     of_w(p) ? rw : ra);
        } else {
            const signed char* v = (of_w(p) ? gw : ga) + off[p] + k0;
            if (k0 + BK <= g.k)
                __builtin_memcpy(&st[p], v, 16);
            else
                st[p] = q8_load16(v, g.k - k0 - in[p]);
        }
    };
    auto put = [&](int t) {  // the loads of step t, in registers, to LDS
        if constexpr (!DMA) {
#pragma unroll
            for (int p = 0; p < P; ++p)
                *(q8v4*)&lds[(t % S) * BUF + load_id(p) * 1024 + lane * 16] = st[p];
        }
    };

    // the last bytes of an operand's last row, where no whole piece holds them:
    // lanes 0 to 15 those of A, 16 to 31 those of W, if step t covers them (the
    // last step, or with Q8_ANY the last piece of the one before, which may be
    // another share's last)
    const bool frayed = DMA && ((ma < BM && (enda & 15) != 0) || (mw < BN && (endw & 15) != 0)) &&
                        t0 + steps + 1 >= all;
    auto patch = [&](int t) {
        if (wave == 0 && lane < 32) {
            const bool w = lane >= 16;
            const int r = w ? mw : ma, e = lane & 15;
            const long long end = w ? endw : enda, piece = end & ~15ll;
            const long long row = (r * (w ? g.ldw : g.lda) + (w ? shw : sha)) & ~15ll;
            const long long c = (piece - row) / 16 - (long long)(t0 + t) * (8 * Q);
            if (r < (w ? BN : BM) && c >= 0 && c < CH && e < (int)(end - piece)) {
                const signed char v = ((w ? gw - shw : ga - sha) + piece)[e];
                const int at = HOW == Q8_ANY ? (int)c : (int)c ^ turned(r);
                lds[(t % S) * BUF + (w ? OW : 0) + r * PITCH + 16 * at + e] = v;
            }
        }
        q8_sync<63>();
    };

    // reads: lane l takes row l % 16 of a block of 16, 16 bytes l / 16 of 64
    constexpr int WORDS = HOW == Q8_ANY ? 8 : 4;  // (six of the eight are used)
    typedef int words __attribute__((ext_vector_type(WORDS)));
    const int wm = wave / WN, wn = wave % WN, r16 = lane & 15, quad = lane >> 4;
    const int fa = wm * FM * 16 * PITCH, fw = OW + wn * FN * 16 * PITCH;
    // the byte of a piece that a row starts at is the same for rows 16 apart
    const int sa = HOW == Q8_ANY ? (int)((size_t)(ga + r16 * g.lda) & 15) : 0;
    const int sw = HOW == Q8_ANY ? (int)((size_t)(gw + r16 * g.ldw) & 15) : 0;
    const int pl = r16 * PITCH + (HOW == Q8_ANY ? quad : quad ^ turned(r16)) * 16;
    words xa[2][FM], xw[2][FN];
    q8v4 acc[FM][FN], bw[FN];
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j) acc[i][j] = q8v4{0, 0, 0, 0};
    auto read = [&](int t, int h, int q) {
        const signed char* p = lds + (t % S) * BUF;
        p += q < FN ? fw + q * 16 * PITCH : fa + (q - FN) * 16 * PITCH;
        q8_read<HOW>(q < FN ? xw[h & 1][q] : xa[h & 1][q - FN], p, pl, h * 64, q < FN ? sw : sa);
    };
    auto multiply = [&](int h, int i, int have) {  // `have` bytes of the step before k
        if (i == 0) {
#pragma unroll
            for (int j = 0; j < FN; ++j) bw[j] = q8_bytes<HOW>(xw[h & 1][j], sw);
        }
        q8v4 ba = q8_bytes<HOW>(xa[h & 1][i], sa);
        if (have < BK) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int b = have - 64 * h - 16 * quad - 4 * e;
                ba[e] &= b >= 4 ? -1 : b <= 0 ? 0 : (1 << (8 * b)) - 1;
            }
        }
#pragma unroll
        for (int j = 0; j < FN; ++j)
            acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(bw[j], ba, acc[i][j], 0, 0, 0);
        __builtin_amdgcn_sched_barrier(0);
    };
    // a step, with another (NEXT) or S others (MORE) after it
    auto step = [&](int t, auto next, auto more) {
        constexpr bool NEXT = decltype(next)::value, MORE = decltype(more)::value;
        const int have = NEXT ? BK : g.k - (t0 + t) * BK;
#pragma unroll
        for (int h = 0; h < H - 1; ++h)
#pragma unroll
            for (int i = 0; i < FM; ++i) {
#pragma unroll
                for (int q = i * R / FM; q < (i + 1) * R / FM; ++q) read(t, h + 1, q);
                multiply(h, i, have);
            }
        if constexpr (NEXT) {
            put(t + 1);
            if (DMA && (MORE || t + S == steps))
                q8_sync<DMA ? (S - 2) * P : 0>();
            else
                q8_sync<0>();
            if (frayed && t + 3 >= steps) patch(t + 1);
        }
#pragma unroll
        for (int i = 0; i < FM; ++i) {
            if constexpr (NEXT) {
#pragma unroll
                for (int q = i * R / FM; q < (i + 1) * R / FM; ++q) read(t + 1, 0, q);
            }
            if constexpr (MORE) {
#pragma unroll
                for (int p = i * P / FM; p < (i + 1) * P / FM; ++p) fetch(t + S, p);
            }
            multiply(H - 1, i, have);
        }
    };

    if (steps > 0) {
#pragma unroll
        for (int t = 0; t < S; ++t) {
            if (t < steps) {
#pragma unroll
                for (int p = 0; p < P; ++p) fetch(t, p);
                if (t == 0) put(0);
            }
        }
        if (DMA && steps >= S)
            q8_sync<DMA ? (S - 1) * P : 0>();
        else
            q8_sync<0>();
        if (frayed && steps <= 2) patch(0);
#pragma unroll
        for (int q = 0; q < R; ++q) read(0, 0, q);
        int t = 0;
        for (; t + S < steps; ++t) step(t, std::true_type{}, std::true_type{});
        for (; t + 1 < steps; ++t) step(t, std::true_type{}, std::false_type{});
        step(t, std::false_type{}, std::false_type{});
    }
    const int ci = i0 + wm * FM * 16 + r16, cj = j0 + wn * FN * 16 + quad * 4;
    if (g.splits == 1)
        q8_finish<T, FM, FN>(g, ci, cj, acc);
    else
        q8_partial<T, FM, FN>(g, share, ci, cj, acc);
}

// Adds the shares' sums, whole numbers, and finishes as the tiles do: a
// thread four neighbouring elements of C.
template <class T>
__global__ __launch_bounds__(256) void q8_gemm_join(Q8GemmArgs<T> g)
{
    const long long ldp = q8_part_ld(g.n), quads = ldp / 4, total = g.m * quads;
    for (long long q = blockIdx.x * 256ll + threadIdx.x; q < total; q += gridDim.x * 256ll) {
        const long long i = q / quads;
        const int j = (int)(q - i * quads) * 4;
        q8v4 sum[1][1] = {{{0, 0, 0, 0}}};
#pragma unroll 4
        for (int h = 0; h < g.splits; ++h)
            sum[0][0] += *(const q8v4*)(g.part + h * (g.m * ldp) + i * ldp + j);
        q8_finish<T, 1, 1>(g, (int)i, j, sum);
    }
}

// ------------------------------------------------- few results: a ring a wave
// Where few rows of A meet W, loads in flight and whole lines count; where
// there are few results, the time to start, wait and add up.  A workgroup makes
// 16 F x 16 F results; its WK waves take the 128-byte steps of the share of k
// in turn, each with a ring of S buffers in LDS of its own, laid out as in the
// tiles; the loads go to LDS by themselves (HOW: Q8_LINES or Q8_ANY), S - 1
// steps ahead of the step that is multiplied.  No wave waits for another until
// the sums are added.  The end of k goes straight from memory to the
// multiplier's layout, with zeros past k; with Q8_ANY the whole steps end 16
// bytes or more before k, so that the ninth piece of the last one lies within
// the row.
//
// F = 1, WK = 8 (S = 3, or 2 with Q8_ANY): 16 x 4096 x 4096 6.1 us, the tile of
// 16 x 64 10.0; 16 x 8192 x 28672 41 us, 5.7 TB/s, where 6.6 is what reading
// alone reaches; at odd strides 16 x 1024 x 4096 7.5 us, the tile with 16 shares
// of k 9.4.  (At 28672 columns of 8192 the tile reads W faster: 43 us, the ring
// 51.)  F = 2, WK = 4: 256 x 1024 x 2048 4.8 us, the 64 x 64 tile with shares
// 8.4, F = 1 more than one round; at odd strides 6.9 and 10.6.
template <int N>
__device__ __forceinline__ void q8_wait_loads()
{
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}

template <class T, int F, int WK, int S, int HOW>
__global__ __launch_bounds__(64 * WK) void q8_gemm_ring(Q8GemmArgs<T> g)
{
    // CB loads of 64 pieces for 16 rows (with Q8_ANY the last one reaches past
    // them), F times of W and then of A
    constexpr int BK = 128, CH = HOW == Q8_ANY ? 9 : 8, CB = (16 * CH + 63) / 64;
    constexpr int BLOCK = CB * 1024, LOADS = 2 * F * CB, SLOT = LOADS * 1024;
    static_assert((S - 1) * LOADS < 64, "the counter of outstanding loads");
    static_assert(WK >= F * F, "a wave for each 16 x 16 results");
    __shared__ __attribute__((aligned(1024))) signed char lds[WK][S * SLOT];

    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    unsigned ti, tj, share;
    q8_tile((g.m + 16 * F - 1) / (16 * F), (g.n + 16 * F - 1) / (16 * F), ti, tj, share);
    const int i0 = (int)ti * 16 * F, j0 = (int)tj * 16 * F;
    // this share's whole steps, t0 and on; the rest of k is the first share's
    const int all = HOW == Q8_ANY ? (g.k - 16) / BK : g.k / BK, t0 = (int)share * g.per;
    const int steps = all - t0 < g.per ? all - t0 : g.per;
    const int mine = (steps - wave + WK - 1) / WK;  // steps wave, wave + WK, ...
    // rows at a multiple of 4096 bytes lie on the same memory channels, column
    // by column, so there each workgroup of a die starts at another step
    // (16 x 8192 x 28672: 47 -> 41 us; at other strides it costs 2 %)
    const int turn =
        g.ldw % 4096 == 0 && mine > 0 ? (int)((blockIdx.x / 8) % (unsigned)mine) : 0;
    const signed char* ga = g.a + i0 * g.lda;
    const signed char* gw = g.w + j0 * g.ldw;
    const int ma = g.m - 1 - i0, mw = g.n - 1 - j0;
    const int sha = HOW == Q8_ANY ? (int)((size_t)ga & 15) : 0;
    const int shw = HOW == Q8_ANY ? (int)((size_t)gw & 15) : 0;

    unsigned oa[F * CB], ow[F * CB];
    auto offset = [&](int i, int last, long long ld, int sh) {  // load i of an operand's rows
        const int piece = i % CB * 64 + lane, c = piece % CH, row = i / CB * 16 + piece / CH;
        const unsigned o = (unsigned)((row < last ? row : last) * ld + sh);
        return HOW == Q8_ANY ? (o & ~15u) + 16 * c : o + 16 * (c ^ ((row >> 1) & 7));
    };
#pragma unroll
    for (int i = 0; i < F * CB; ++i) {
        oa[i] = offset(i, ma, g.lda, sha);
        ow[i] = offset(i, mw, g.ldw, shw);
    }
    const q8v4 ra = q8_rsrc(ga - sha, 0xffffffffu), rw = q8_rsrc(gw - shw, 0xffffffffu);
    signed char* ring = lds[wave];
    const unsigned base =
        (unsigned)(unsigned long long)(__attribute__((address_space(3))) void*)ring;
    auto fetch = [&](int t) {  // this wave's t-th step
        int turned = t + turn;
        turned -= turned >= mine ? mine : 0;
        const unsigned to = base + (unsigned)(t % S) * SLOT;
        const unsigned k0 = (unsigned)(t0 + turned * WK + wave) * BK;
#pragma unroll
        for (int i = 0; i < F * CB; ++i) q8_fetch(to + 1024 * i, ow[i], rw, k0);
#pragma unroll
        for (int i = 0; i < F * CB; ++i) q8_fetch(to + F * BLOCK + 1024 * i, oa[i], ra, k0);
    };
    // (each of the first F * F waves finishes 16 x 16 of the results)
    const int r = lane & 15, piece = lane >> 4;
    const int ci = i0 + 16 * (wave / F) + r, cj = j0 + 16 * (wave % F) + 4 * piece;
    Q8Scales<T, 1, 1> scales;
    if (wave < F * F && g.splits == 1) scales.load(g, ci, cj);
    for (int t = 0; t < S - 1 && t < mine; ++t) fetch(t);

    q8v4 acc[F][F];
#pragma unroll
    for (int i = 0; i < F; ++i)
#pragma unroll
        for (int j = 0; j < F; ++j) acc[i][j] = q8v4{0, 0, 0, 0};
    auto multiply = [&](const q8v4(&xa)[F], const q8v4(&xw)[F]) {
#pragma unroll
        for (int i = 0; i < F; ++i)
#pragma unroll
            for (int j = 0; j < F; ++j)
                acc[i][j] =
                    __builtin_amdgcn_mfma_i32_16x16x64_i8(xw[j], xa[i], acc[i][j], 0, 0, 0);
    };
    if (share == 0 && wave == WK - 1) {
#pragma unroll 1
        for (int k0 = all * BK; k0 < g.k; k0 += 64) {
            const int at = k0 + 16 * piece;
            q8v4 xa[F], xw[F];
#pragma unroll
            for (int f = 0; f < F; ++f) {
                const int row = 16 * f + r;
                xw[f] = q8_load16(gw + (row < mw ? row : mw) * g.ldw + at, g.k - at);
                xa[f] = q8_load16(ga + (row < ma ? row : ma) * g.lda + at, g.k - at);
            }
            multiply(xa, xw);
        }
    }

    // the byte of a piece that a row starts at is the same for rows 16 apart
    typedef int words __attribute__((ext_vector_type(HOW == Q8_ANY ? 8 : 4)));
    const int sa = HOW == Q8_ANY ? (int)((size_t)(ga + r * g.lda) & 15) : 0;
    const int sw = HOW == Q8_ANY ? (int)((size_t)(gw + r * g.ldw) & 15) : 0;
    const int pl = r * 16 * CH + (HOW == Q8_ANY ? piece : piece ^ ((r >> 1) & 7)) * 16;
    for (int t = 0; t < mine; ++t) {
        if (t + S - 1 < mine) {
            fetch(t + S - 1);  // into the buffer of step t - 1, which has been read
            q8_wait_loads<(S - 1) * LOADS>();
        } else {
            q8_wait_loads<0>();
        }
        const signed char* p = ring + (t % S) * SLOT;
        words wa[2][F], ww[2][F];
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int f = 0; f < F; ++f) {
                q8_read<HOW>(ww[h][f], p + f * BLOCK, pl, h * 64, sw);
                q8_read<HOW>(wa[h][f], p + (F + f) * BLOCK, pl, h * 64, sa);
            }
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            q8v4 xa[F], xw[F];
#pragma unroll
            for (int f = 0; f < F; ++f) {
                xw[f] = q8_bytes<HOW>(ww[h][f], sw);
                xa[f] = q8_bytes<HOW>(wa[h][f], sa);
            }
            multiply(xa, xw);
        }
    }
    // the waves' sums, in their rings, which nothing is on its way to
    q8v4* sums = (q8v4*)ring;
#pragma unroll
    for (int i = 0; i < F; ++i)
#pragma unroll
        for (int j = 0; j < F; ++j) sums[(i * F + j) * 64 + lane] = acc[i][j];
    __syncthreads();
    if (wave >= F * F) return;
    q8v4 sum[1][1] = {{{0, 0, 0, 0}}};
#pragma unroll
    for (int w = 0; w < WK; ++w) sum[0][0] += ((const q8v4*)lds[w])[wave * 64 + lane];
    if (g.splits == 1)
        q8_finish(g, ci, cj, scales, sum);
    else
        q8_partial<T, 1, 1>(g, share, ci, cj, sum);
}

// ------------------------------------------------------------------ copies
// Rows of A and of W to strides of whole lines, 16 bytes a lane from any
// address; a row's last 16 bytes are written again by their own lane (k >= 16).
struct Q8CopyArgs {
    const signed char* a;
    const signed char* w;
    signed char* ca;
    signed char* cw;
    long long lda, ldw, ldc;
    int m, n, k;
};

static __global__ __launch_bounds__(256) void q8_gemm_copy(Q8CopyArgs g)
{
    const long long rows = (long long)g.m + g.n;
    for (long long r = blockIdx.x * 4ll + (threadIdx.x >> 6); r < rows; r += gridDim.x * 4ll) {
        const signed char* from = r < g.m ? g.a + r * g.lda : g.w + (r - g.m) * g.ldw;
        signed char* to = r < g.m ? g.ca + r * g.ldc : g.cw + (r - g.m) * g.ldc;
        for (int c = (threadIdx.x & 63) * 16; c < g.k; c += 1024) {
            const int at = c < g.k - 16 ? c : g.k - 16;
            q8v4 v;
            __builtin_memcpy(&v, from + at, 16);
            __builtin_memcpy(to + at, &v, 16);
        }
    }
}

}  // namespace xsymv
