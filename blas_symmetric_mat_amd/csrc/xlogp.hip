// xlogp.hip -- entry points of the log probabilities (kernels: xlogp.hpp).
#include "xlogp.hpp"
#include "xq8_host.hpp"

namespace xsymv {
namespace {

// Workgroups that share a row: where the rows alone do not give every compute
// unit a few, a row goes to more of them, of a load a thread at least.
int logp_parts(int m, int n, int top)
{
    long long p = std::min<long long>(1024 / std::max(m, 1), ((long long)n + 2047) / 2048);
    p = std::min<long long>(p, LP_PARTS);
    if (top > 0) p = std::min<long long>(p, LP_LISTS / top);
    return (int)std::max(p, 1ll);
}

size_t logp_bytes(int m, int parts, int top)
{
    if (parts == 1) return 0;
    return align_up((size_t)m * parts * sizeof(LpSums)) + align_up((size_t)m * parts * top * sizeof(lp_key));
}

template <class T>
int logp_launch(LpArgs<T> a, int parts, void* ws, hipStream_t stream, const TimedCall& tc)
{
    // (a row without logits is one part too)
    a.each = (int)std::max(8ll, (((long long)a.n + parts - 1) / parts + 7) / 8 * 8);
    a.parts = (int)std::max(1ll, ((long long)a.n + a.each - 1) / a.each);
    a.sums = static_cast<LpSums*>(ws);
    a.keys = reinterpret_cast<lp_key*>(static_cast<char*>(ws) + align_up((size_t)a.m * parts * sizeof(LpSums)));
    const unsigned grid = (unsigned)std::min((long long)a.m * a.parts, 1ll << 20);
    const bool join = a.parts > 1;
    XSYMV_HIP(launch_k(a.top > 0 ? &logp_rows<T, true> : &logp_rows<T, false>, dim3(grid), dim3(LP_THREADS),
                       stream, a, tc.e0, tc.e1));
    if (join) XSYMV_HIP(launch_k(&logp_join<T>, dim3((unsigned)a.m), dim3(LP_THREADS), stream, a, nullptr, tc.e2));
    return 0;
}

template <class T>
int logp_run(int m, int n, const T* x, int ldx, const int* token, float* logp, float* entropy, float* lse,
             int top, int* index, float* value, int ldt, hipStream_t stream)
{
    if (m < 0) return -1;
    if (n < 0 || n > LP_MOST) return -2;
    const bool some = m > 0;
    if (some && n > 0 && x == nullptr) return -3;
    if (ldx < std::max(1, n)) return -4;
    if (some && token != nullptr && logp == nullptr) return -6;
    if (top < 0 || top > LP_TOP || (some && top > n)) return -9;
    if (some && top > 0 && index == nullptr) return -10;
    if (ldt < top) return -12;
    if (!some) return 0;
    const LpArgs<T> a{x, token, logp, entropy, lse, index, value, m, n, ldx, top, ldt, 1, n, nullptr, nullptr};
    int parts = logp_parts(m, n, top);
    const size_t bytes = logp_bytes(m, parts, top);
    return q8_with_workspace(bytes, parts > 1, stream, [&](void* ws, const TimedCall& tc) {
        return logp_launch(a, ws ? parts : 1, ws, stream, tc);
    });
}

}  // namespace
}  // namespace xsymv

extern "C" size_t xsymv_logp_workspace_bytes(int m, int n, int top)
{
    using namespace xsymv;
    if (m <= 0 || n <= 0 || n > LP_MOST || top < 0 || top > LP_TOP) return 0;
    return logp_bytes(m, logp_parts(m, n, top), top);
}

#define XSYMV_LOGP(L, CT, T)                                                                             \
    extern "C" int xsymv_logp_##L(int m, int n, const CT* x, int ldx, const int* token, float* logp,     \
                                  float* entropy, float* lse, int top, int* index, float* value,         \
                                  int ldt, void* stream)                                                 \
    {                                                                                                    \
        return xsymv::q8_guard([&] {                                                                     \
            return xsymv::logp_run<T>(m, n, reinterpret_cast<const T*>(x), ldx, token, logp, entropy,    \
                                      lse, top, index, value, ldt, (hipStream_t)stream);                 \
        });                                                                                              \
    }

XSYMV_LOGP(s, float, float)
XSYMV_LOGP(h, xhalf, xsymv::q8half)
XSYMV_LOGP(b, xbfloat16, xsymv::q8bf16)
