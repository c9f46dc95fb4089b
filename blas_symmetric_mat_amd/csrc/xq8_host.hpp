// xq8_host.hpp -- host side shared by the operators on rows in 8 bits.
#pragma once

#include "xsymv_host.hpp"
#include "xq8_rows.hpp"

#include <new>

namespace xsymv {

// Type letter of an argument beside one of type T: 0 T's own, 1 float (where
// T is another type), -1 neither.
template <class T>
int q8_type(char c)
{
    const char own = std::is_same<T, float>::value ? 's' : std::is_same<T, q8half>::value ? 'h' : 'b';
    if (c >= 'A' && c <= 'Z') c = (char)(c - 'A' + 'a');
    return c == own ? 0 : c == 's' ? 1 : -1;
}

// Workgroups for m rows, `per` to a workgroup; at most 2^20, which loop over
// the rest (a launch's threads are counted in 32 bits).
inline unsigned q8_grid(int m, int per)
{
    return (unsigned)std::min(((long long)m + per - 1) / per, 1ll << 20);
}

// A call of one kernel, with its timing record where timing is on.
template <class A>
int q8_launch(void (*k)(A), dim3 grid, unsigned threads, hipStream_t stream, const A& a)
{
    TimedCall tc{};
    const int timing = timing_enabled();
    if (timing) {
        XSYMV_HIP(timed_call_create(tc, timing, false));
    }
    XSYMV_HIP(launch_k(k, grid, dim3(threads), stream, a, tc.e0, tc.e1));
    if (timing) timing_push(tc);
    return 0;
}

// No exception leaves a C entry point.
template <class F>
int q8_guard(F&& f)
{
    try {
        return f();
    } catch (const std::bad_alloc&) {
        return ERR_HIP + (int)hipErrorOutOfMemory;
    } catch (...) {
        return ERR_HIP + (int)hipErrorUnknown;
    }
}

}  // namespace xsymv
