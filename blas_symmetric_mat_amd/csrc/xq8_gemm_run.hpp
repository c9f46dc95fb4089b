// xq8_gemm_run.hpp -- a call of the product of rows in 8 bits: checks, the
// choice of a kernel, its launch (kernels: xq8_gemm.hpp; the choice:
// xq8_gemm.hip).  The precision units xq8_gemm_[shb].hip compile it.
#pragma once

#include "xsymv_host.hpp"
#include "xq8_gemm.hpp"
#include "xq8_host.hpp"

namespace xsymv {

enum Q8Kernel {
    Q8_RING,
    Q8_RING32,
    Q8_STREAM,
    Q8_TILE16,
    Q8_TILE32,
    Q8_TILE64,
    Q8_TILE64_SHORT,  // two buffers: more workgroups a compute unit, for few steps
    Q8_TILE128X64,
    Q8_TILE128,
    Q8_TILE128_SHORT,
    Q8_TILE256X128,
    Q8_TILE256
};

struct Q8Plan {
    Q8Kernel kernel;
    int how, splits, per;  // how the rows are read; shares of k, steps in each
    unsigned groups;       // workgroups
    size_t part;           // bytes of workspace, for the shares' sums
    int ldc;               // rows copied to this stride first (0: read where they lie)
    size_t copy;           // bytes of workspace, for the copies
};

// Stride of copied rows: whole lines, and not a multiple of 4096 bytes, which
// would put every row's beginning on the same memory channels.
inline int q8_copy_ld(int k)
{
    const int ld = (k + 127) / 128 * 128;
    return ld % 4096 == 0 ? ld + 128 : ld;
}

// The kernel for m x n x k with rows read as `how`; `cut`: they do not start at
// multiples of 128 bytes, so that a step's bytes lie on more lines; `whole`: of
// the plans that take no workspace, k in one share and the rows where they lie.
Q8Plan q8_plan(int how, bool cut, bool whole, int m, int n, int k);

// Rows and columns of one launch at most.
constexpr int Q8_BLOCK = 1 << 24;

template <class T>
using Q8GemmKernel = void (*)(Q8GemmArgs<T>);

// The kernel of a plan and its threads.  LDS allows two workgroups a compute
// unit up to 80 KB each, else one with more buffers.
template <class T>
Q8GemmKernel<T> q8_kernel(const Q8Plan& p, int& threads)
{
    threads = 512;
    if (p.kernel == Q8_RING)
        return p.how == Q8_LINES ? &q8_gemm_ring<T, 1, 8, 3, Q8_LINES>
                                 : &q8_gemm_ring<T, 1, 8, 2, Q8_ANY>;
    if (p.kernel == Q8_STREAM) return &q8_gemm_stream<T>;
    if (p.how == Q8_LINES) {
        switch (p.kernel) {
        case Q8_TILE128X64: return &q8_gemm_tile<T, 128, 64, 4, 2, 2, 3, Q8_LINES>;
        case Q8_TILE128: return &q8_gemm_tile<T, 128, 128, 2, 4, 1, 4, Q8_LINES>;
        case Q8_TILE128_SHORT: return &q8_gemm_tile<T, 128, 128, 2, 4, 1, 2, Q8_LINES>;
        case Q8_TILE256X128: return &q8_gemm_tile<T, 256, 128, 4, 2, 1, 3, Q8_LINES>;
        case Q8_TILE256: return &q8_gemm_tile<T, 256, 256, 2, 4, 1, 2, Q8_LINES>;
        default: break;
        }
        threads = 256;
        switch (p.kernel) {
        case Q8_RING32: return &q8_gemm_ring<T, 2, 4, 3, Q8_LINES>;
        case Q8_TILE16: return &q8_gemm_tile<T, 16, 64, 1, 4, 2, 3, Q8_LINES>;
        case Q8_TILE32: return &q8_gemm_tile<T, 32, 64, 2, 2, 2, 3, Q8_LINES>;
        case Q8_TILE64_SHORT: return &q8_gemm_tile<T, 64, 64, 2, 2, 1, 2, Q8_LINES>;
        default: return &q8_gemm_tile<T, 64, 64, 2, 2, 1, 4, Q8_LINES>;
        }
    }
    if (p.how == Q8_ANY) {
        switch (p.kernel) {
        case Q8_TILE128: return &q8_gemm_tile<T, 128, 128, 2, 4, 2, 2, Q8_ANY>;
        case Q8_TILE128_SHORT: return &q8_gemm_tile<T, 128, 128, 2, 4, 1, 2, Q8_ANY>;
        case Q8_TILE256X128: return &q8_gemm_tile<T, 256, 128, 4, 2, 1, 2, Q8_ANY>;
        case Q8_TILE256: return &q8_gemm_tile<T, 256, 256, 2, 4, 1, 2, Q8_ANY>;
        default: break;
        }
        threads = 256;
        switch (p.kernel) {
        case Q8_RING32: return &q8_gemm_ring<T, 2, 4, 2, Q8_ANY>;
        case Q8_TILE16: return &q8_gemm_tile<T, 16, 64, 1, 4, 2, 3, Q8_ANY>;
        case Q8_TILE32: return &q8_gemm_tile<T, 32, 64, 2, 2, 2, 3, Q8_ANY>;
        case Q8_TILE64_SHORT: return &q8_gemm_tile<T, 64, 64, 2, 2, 1, 2, Q8_ANY>;
        default: return &q8_gemm_tile<T, 64, 64, 2, 2, 2, 2, Q8_ANY>;
        }
    }
    if (p.kernel == Q8_TILE256X128) return &q8_gemm_tile<T, 256, 128, 4, 2, 1, 2, Q8_REGS>;
    threads = 256;
    if (p.kernel == Q8_TILE16) return &q8_gemm_tile<T, 16, 64, 1, 4, 1, 2, Q8_REGS>;
    return &q8_gemm_tile<T, 64, 64, 2, 2, 1, 2, Q8_REGS>;
}

// How the rows of both operands can be read (see xq8_gemm.hpp): the loads to
// LDS want 16 bytes of a row at least, a first row at a multiple of 16 bytes
// and a tile's rows within 32-bit offsets; whole lines want every row there.
inline int q8_how(int k, const signed char* a, int lda, const signed char* w, int ldw)
{
    const size_t starts = reinterpret_cast<size_t>(a) | reinterpret_cast<size_t>(w);
    if (k < 16 || starts % 16 != 0 || lda > 1 << 23 || ldw > 1 << 23) return Q8_REGS;
    return lda % 16 == 0 && ldw % 16 == 0 ? Q8_LINES : Q8_ANY;
}

template <class T>
int gemm_block(Q8GemmArgs<T> g, int lda, int ldw, hipStream_t stream)
{
    const int how = q8_how(g.k, g.a, lda, g.w, ldw);
    const size_t starts = reinterpret_cast<size_t>(g.a) | reinterpret_cast<size_t>(g.w);
    const bool cut = how == Q8_LINES && (starts | (size_t)(lda | ldw)) % 128 != 0;
    Q8Plan p = q8_plan(how, cut, false, g.m, g.n, g.k);
    auto fits = [&] { return p.groups != 0; };  // else more than a launch holds
    if (!fits()) return ERR_HIP + (int)hipErrorInvalidValue;
    int threads = 0;
    auto straight = [&] {  // without a workspace
        g.splits = 1;
        g.per = p.per;
        const Q8GemmKernel<T> kernel = q8_kernel<T>(p, threads);
        return q8_launch(kernel, p.groups, threads, stream, g);
    };
    if (p.copy + p.part == 0) return straight();

    int dev = 0;
    XSYMV_HIP(hipGetDevice(&dev));
    DeviceState* ds = device_state(dev);
    std::lock_guard<std::mutex> lk(device_mutex(ds));
    void* ws = nullptr;
    // Where the workspace cannot be had, because the device has no memory left
    // or a capture forbids to allocate it, the product is made without: slower,
    // and to the same bytes.
    int rc = ERR_HIP + (int)hipErrorOutOfMemory;
    if (!workspace_barred(ds, stream, p.copy + p.part)) {
        rc = get_workspace(ds, stream, p.copy + p.part, &ws);
        if (rc == ERR_HIP + (int)hipErrorOutOfMemory) (void)hipGetLastError();  // dealt with
    }
    if (rc == ERR_HIP + (int)hipErrorOutOfMemory) {
        p = q8_plan(how, cut, true, g.m, g.n, g.k);
        return fits() ? straight() : rc;
    }
    if (rc) return rc;
    g.splits = p.splits;
    g.per = p.per;
    const Q8GemmKernel<T> kernel = q8_kernel<T>(p, threads);
    TimedCall tc{};
    const int timing = timing_enabled();
    if (timing) {
        XSYMV_HIP(timed_call_create(tc, timing, p.splits > 1));
    }
    hipEvent_t start = tc.e0;  // the call's first kernel
    if (p.ldc != 0) {
        signed char* ca = static_cast<signed char*>(ws);
        const Q8CopyArgs c{g.a, g.w, ca, ca + (size_t)g.m * p.ldc, g.lda, g.ldw, p.ldc, g.m, g.n, g.k};
        const unsigned groups = (unsigned)std::min(((long long)g.m + g.n + 3) / 4, 1ll << 20);
        XSYMV_HIP(launch_k(&q8_gemm_copy, dim3(groups), dim3(256), stream, c, start, nullptr));
        start = nullptr;
        g.a = c.ca;
        g.w = c.cw;
        g.lda = g.ldw = p.ldc;
    }
    g.part = reinterpret_cast<int*>(static_cast<char*>(ws) + p.copy);
    XSYMV_HIP(launch_k(kernel, dim3(p.groups), dim3(threads), stream, g, start, tc.e1));
    if (p.splits > 1) {
        const long long quads = (long long)g.m * (q8_part_ld(g.n) / 4);
        XSYMV_HIP(launch_k(&q8_gemm_join<T>, dim3((unsigned)std::min((quads + 255) / 256, 2048ll)),
                           dim3(256), stream, g, nullptr, tc.e2));
    }
    if (timing) timing_push(tc);
    return 0;
}

template <class T>
int gemm_run(int m, int n, int k, const signed char* a, int lda, const float* sa,
             const signed char* w, int ldw, const float* sw, const float* bias, T* c, int ldc,
             hipStream_t stream)
{
    if (m < 0) return -1;
    if (n < 0) return -2;
    if (k < 0 || k > Q8_MAX_K) return -3;
    const bool some = m > 0 && n > 0;
    if (some && k > 0 && a == nullptr) return -4;
    if (lda < std::max(1, k)) return -5;
    if (some && sa == nullptr) return -6;
    if (some && k > 0 && w == nullptr) return -7;
    if (ldw < std::max(1, k)) return -8;
    if (some && sw == nullptr) return -9;
    if (some && c == nullptr) return -11;
    if (ldc < std::max(1, n)) return -12;
    for (int i = 0; some && i < m;) {
        const int rows = std::min(m - i, Q8_BLOCK);
        for (int j = 0; j < n;) {
            const int cols = std::min(n - j, Q8_BLOCK);
            const Q8GemmArgs<T> g{a + (size_t)i * lda,  w + (size_t)j * ldw, sa + i,
                                  sw + j,               bias ? bias + j : nullptr,
                                  c + (size_t)i * ldc + j, lda, ldw, ldc, rows, cols, k,
                                  nullptr,              1,                1};
            const int rc = gemm_block(g, lda, ldw, stream);
            if (rc) return rc;
            j += cols;
        }
        i += rows;
    }
    return 0;
}

}  // namespace xsymv

#define XSYMV_Q8_GEMM(L, CT, T)                                                                   \
    extern "C" int xsymv_q8gemm_##L(int m, int n, int k, const signed char* a, int lda,           \
                                    const float* sa, const signed char* w, int ldw,               \
                                    const float* sw, const float* bias, CT* c, int ldc,           \
                                    void* stream)                                                 \
    {                                                                                             \
        return xsymv::q8_guard([&] {                                                              \
            return xsymv::gemm_run<T>(m, n, k, a, lda, sa, w, ldw, sw, bias,                      \
                                      reinterpret_cast<T*>(c), ldc, (hipStream_t)stream);         \
        });                                                                                       \
    }
