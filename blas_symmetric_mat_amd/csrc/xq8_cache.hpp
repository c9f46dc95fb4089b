// xq8_cache.hpp -- a cache of 8-bit rows in pages, as the kernels see it.
#pragma once

#include <hip/hip_runtime.h>

namespace xsymv {

struct PgCache {
    int* len;
    int* table;
    int* refs;
    int seqs, ldt, pages, ps;
    // tokens of sequence s, as far as its row of the table can hold them
    __device__ __forceinline__ int length(int s) const
    {
        int n;
        return length(s, n);
    }
    // (n: what len holds)
    __device__ __forceinline__ int length(int s, int& n) const
    {
        const long long room = (long long)ldt * ps;
        n = __hip_atomic_load(&len[s], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        return n < 0 ? 0 : n > room ? (int)room : n;
    }
    __device__ __forceinline__ int* row(int s) const { return table + (size_t)s * ldt; }
    __device__ __forceinline__ bool is_page(int p) const { return (unsigned)p < (unsigned)pages; }
    __device__ __forceinline__ bool is_seq(int s) const { return (unsigned)s < (unsigned)seqs; }
};

// Sequence of row r of the calls that take `start`, -1 for none: the last one
// that begins at or before it, if it does not end there.
__device__ __forceinline__ int pg_sequence(const int* start, int seqs, int r)
{
    if (start == nullptr) return r < seqs ? r : -1;
    int lo = 0, hi = seqs;
    while (lo < hi) {
        const int mid = lo + (hi - lo) / 2;
        if (start[mid + 1] <= r)
            lo = mid + 1;
        else
            hi = mid;
    }
    return lo < seqs && start[lo] <= r ? lo : -1;
}

}  // namespace xsymv
