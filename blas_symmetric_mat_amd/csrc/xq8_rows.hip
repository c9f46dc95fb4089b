// xq8_rows.hip -- entry points of the operators on rows in 8 bits: norm,
// gated activation, cache store and read (kernels: xq8_rows.hpp).
#include "xsymv_host.hpp"
#include "xq8_host.hpp"
#include "xq8_rows.hpp"

#include <cmath>

namespace xsymv {
namespace {

// Workgroups for twice the threads that the chip holds at once (256 compute
// units of 2048), which take the rows in turn: a workgroup for every few rows
// cost the start of each (store of 65536 x 512 24.7 us, 22.1 so; activation of
// 4096 x 14336 55.8 and 54.3; norm of 8192 x 4096, bfloat16, 53.7 and 51.4), and
// with no more than the chip holds a norm's loads wait for its sums (58.5).
// Norms of one chunk a thread do best with four times as many (200000 x 128:
// every row its own 42.0 us, twice 40.5, four times 38.9).
template <class OP, int TPR, int J>
int rows_launch(const Q8RowArgs<OP>& a, hipStream_t stream)
{
    constexpr int threads = TPR > 256 ? TPR : 256;
    constexpr unsigned most = (OP::NORM && J == 1 ? 4 : 2) * (256 * 2048 / threads);
    const unsigned grid = std::min(q8_grid(a.op.m, threads / TPR), most);
    return q8_launch(&q8_rows<OP, TPR, J>, grid, threads, stream, a);
}

// Threads per row and chunks per thread by the row's length alone: of the
// compiled capacities (TPR * J chunks) the smallest that holds the row.  Two
// or three chunks a thread were the fastest for long rows of every length
// (norm of 4096 x 8192, bfloat16 with a 32-bit residual: 256 threads of four
// 80 us, 512 of two 72, 1024 of one 87), the sums' waits being shared by more
// loads; a capacity that is half empty costs up to 30 % (norm of 3000 x 9000:
// 1024 threads of two 74 us, 512 of three 56).
template <class OP, int TPR, int J, int... NEXT>
int rows_fit(int chunks, const Q8RowArgs<OP>& a, hipStream_t stream)
{
    if constexpr (sizeof...(NEXT) > 0)
        if (chunks > TPR * J) return rows_fit<OP, NEXT...>(chunks, a, stream);
    return rows_launch<OP, TPR, J>(a, stream);
}

template <class OP>
int rows_run(const Q8RowArgs<OP>& a, hipStream_t stream)
{
    const int chunks = (int)(((long long)a.op.n + Q8_CHUNK - 1) / Q8_CHUNK);
    return rows_fit<OP, 8, 1, 16, 1, 32, 1, 64, 1, 32, 3, 64, 2, 64, 3, 256, 1, 256, 2, 256, 3, 512,
                    2, 512, 3, 1024, 2, 1024, 3, 1024, 4, 1024, 8, 1024, 0>(chunks, a, stream);
}

template <class T, class R, class W>
int norm_typed(int m, int n, const T* x, int ldx, const void* r, int ldr, const void* w, float eps,
               void* h, int ldh, signed char* q, int ldq, float* scale, hipStream_t stream)
{
    const Q8Norm<T, R, W> op{x,   static_cast<const R*>(r), static_cast<R*>(h),
                             static_cast<const W*>(w), ldx, ldr, ldh, (double)eps, m, n};
    return rows_run(Q8RowArgs<Q8Norm<T, R, W>>{op, q, scale, ldq}, stream);
}

template <class T>
int norm_run(int m, int n, const T* x, int ldx, char rtype, const void* r, int ldr, char wtype,
             const void* w, float eps, void* h, int ldh, signed char* q, int ldq, float* scale,
             hipStream_t stream)
{
    const int rt = q8_type<T>(rtype), wt = q8_type<T>(wtype);
    if (m < 0) return -1;
    if (n < 0) return -2;
    const bool some = m > 0 && n > 0;
    if (some && x == nullptr) return -3;
    if (ldx < std::max(1, n)) return -4;
    if (rt < 0) return -5;
    if (r != nullptr && ldr < std::max(1, n)) return -7;
    if (wt < 0) return -8;
    if (some && w == nullptr) return -9;
    if (!(eps >= 0.0f) || std::isinf(eps)) return -10;
    if (h != nullptr && (ldh < std::max(1, n) || (h == r && ldh != ldr))) return -12;
    if (some && q == nullptr) return -13;
    if (ldq < std::max(1, n)) return -14;
    if (some && scale == nullptr) return -15;
    if (!some) return 0;
    // (after the others: it is about two arguments together)
    if (h == x && rt != 0) return -11;
    if (h == x && ldh != ldx) return -12;
    if (rt == 0 && wt == 0)
        return norm_typed<T, T, T>(m, n, x, ldx, r, ldr, w, eps, h, ldh, q, ldq, scale, stream);
    if constexpr (!std::is_same<T, float>::value) {
        if (rt == 0)
            return norm_typed<T, T, float>(m, n, x, ldx, r, ldr, w, eps, h, ldh, q, ldq, scale,
                                           stream);
        if (wt == 0)
            return norm_typed<T, float, T>(m, n, x, ldx, r, ldr, w, eps, h, ldh, q, ldq, scale,
                                           stream);
    }
    return norm_typed<T, float, float>(m, n, x, ldx, r, ldr, w, eps, h, ldh, q, ldq, scale, stream);
}

template <class T>
int glu_run(int m, int n, const T* g, int ldg, const T* u, int ldu, signed char* q, int ldq,
            float* scale, hipStream_t stream)
{
    if (m < 0) return -1;
    if (n < 0) return -2;
    const bool some = m > 0 && n > 0;
    if (some && g == nullptr) return -3;
    if (ldg < std::max(1, n)) return -4;
    if (some && u == nullptr) return -5;
    if (ldu < std::max(1, n)) return -6;
    if (some && q == nullptr) return -7;
    if (ldq < std::max(1, n)) return -8;
    if (some && scale == nullptr) return -9;
    if (!some) return 0;
    return rows_run(Q8RowArgs<Q8Glu<T>>{Q8Glu<T>{g, u, ldg, ldu, m, n}, q, scale, ldq}, stream);
}

template <class T>
int store_run(int m, int n, const T* x, int ldx, const int* slot, int cap, signed char* q, int ldq,
              float* scale, hipStream_t stream)
{
    if (m < 0) return -1;
    if (n < 0) return -2;
    const bool some = m > 0 && n > 0;
    if (some && x == nullptr) return -3;
    if (ldx < std::max(1, n)) return -4;
    if (cap < 0 || (slot == nullptr && cap < m)) return -6;
    if (some && cap > 0 && q == nullptr) return -7;
    if (ldq < std::max(1, n)) return -8;
    if (some && cap > 0 && scale == nullptr) return -9;
    if (!some || cap == 0) return 0;
    return rows_run(Q8RowArgs<Q8Store<T>>{Q8Store<T>{x, slot, ldx, m, n, cap}, q, scale, ldq},
                    stream);
}

template <class T, int TPR>
int read_launch(const Q8ReadArgs<T>& a, hipStream_t stream)
{
    // 2^20 workgroups at most, which loop over the rest
    const long long parts = ((long long)a.n + TPR * Q8_CHUNK - 1) / (TPR * Q8_CHUNK);
    const unsigned rows = q8_grid(a.m, 256 / TPR);
    const dim3 grid(rows, (unsigned)std::min(parts, std::max(1ll, (1ll << 16) / rows)));
    return q8_launch(&q8_read<T, TPR>, grid, 256, stream, a);
}

template <class T>
int read_run(int m, int n, const signed char* q, int ldq, const float* scale, const int* slot,
             int cap, T* out, int ldo, hipStream_t stream)
{
    if (m < 0) return -1;
    if (n < 0) return -2;
    const bool some = m > 0 && n > 0;
    if (some && cap > 0 && q == nullptr) return -3;
    if (ldq < std::max(1, n)) return -4;
    if (some && cap > 0 && scale == nullptr) return -5;
    if (cap < 0 || (slot == nullptr && cap < m)) return -7;
    if (some && out == nullptr) return -8;
    if (ldo < std::max(1, n)) return -9;
    if (!some) return 0;
    const Q8ReadArgs<T> a{q, scale, slot, out, ldq, ldo, m, n, cap};
    if (n <= 64) return read_launch<T, 8>(a, stream);
    if (n <= 128) return read_launch<T, 16>(a, stream);
    if (n <= 256) return read_launch<T, 32>(a, stream);
    if (n <= 512) return read_launch<T, 64>(a, stream);
    return read_launch<T, 256>(a, stream);
}

}  // namespace
}  // namespace xsymv

#define XSYMV_Q8_ROWS(L, CT, T)                                                                    \
    extern "C" int xsymv_q8norm_##L(int m, int n, const CT* x, int ldx, char rtype, const void* r, \
                                    int ldr, char wtype, const void* w, float eps, void* h,        \
                                    int ldh, signed char* q, int ldq, float* scale, void* stream)  \
    {                                                                                              \
        return xsymv::q8_guard([&] {                                                               \
            return xsymv::norm_run<T>(m, n, reinterpret_cast<const T*>(x), ldx, rtype, r, ldr,     \
                                      wtype, w, eps, h, ldh, q, ldq, scale, (hipStream_t)stream);  \
        });                                                                                        \
    }                                                                                              \
    extern "C" int xsymv_q8glu_##L(int m, int n, const CT* g, int ldg, const CT* u, int ldu,       \
                                   signed char* q, int ldq, float* scale, void* stream)            \
    {                                                                                              \
        return xsymv::q8_guard([&] {                                                               \
            return xsymv::glu_run<T>(m, n, reinterpret_cast<const T*>(g), ldg,                     \
                                     reinterpret_cast<const T*>(u), ldu, q, ldq, scale,            \
                                     (hipStream_t)stream);                                         \
        });                                                                                        \
    }                                                                                              \
    extern "C" int xsymv_q8store_##L(int m, int n, const CT* x, int ldx, const int* slot, int cap, \
                                     signed char* q, int ldq, float* scale, void* stream)          \
    {                                                                                              \
        return xsymv::q8_guard([&] {                                                               \
            return xsymv::store_run<T>(m, n, reinterpret_cast<const T*>(x), ldx, slot, cap, q,     \
                                       ldq, scale, (hipStream_t)stream);                           \
        });                                                                                        \
    }                                                                                              \
    extern "C" int xsymv_q8read_##L(int m, int n, const signed char* q, int ldq,                   \
                                    const float* scale, const int* slot, int cap, CT* out,         \
                                    int ldo, void* stream)                                         \
    {                                                                                              \
        return xsymv::q8_guard([&] {                                                               \
            return xsymv::read_run<T>(m, n, q, ldq, scale, slot, cap, reinterpret_cast<T*>(out),   \
                                      ldo, (hipStream_t)stream);                                   \
        });                                                                                        \
    }

XSYMV_Q8_ROWS(s, float, float)
XSYMV_Q8_ROWS(h, xhalf, xsymv::q8half)
XSYMV_Q8_ROWS(b, xbfloat16, xsymv::q8bf16)
