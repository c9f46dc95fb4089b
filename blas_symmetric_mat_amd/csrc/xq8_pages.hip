// xq8_pages.hip -- entry points of the calls on the pages of a cache of 8-bit
// rows (kernels: xq8_pages.hpp).
#include "xq8_pages.hpp"
#include "xq8_host.hpp"

namespace xsymv {
namespace {

// A call of two kernels, the first one of one workgroup: one timing record.
template <class A>
int launch_two(void (*first)(A), void (*second)(A), unsigned grid, hipStream_t stream, const A& a)
{
    TimedCall tc{};
    const int timing = timing_enabled();
    if (timing) XSYMV_HIP(timed_call_create(tc, timing));
    XSYMV_HIP(launch_k(first, dim3(1), dim3(PG_THREADS), stream, a, tc.e0, tc.e1));
    XSYMV_HIP(launch_k(second, dim3(grid), dim3(256), stream, a, nullptr, tc.e2));
    if (timing) timing_push(tc);
    return 0;
}

// Rows of a cache count in an int, as slots do.
bool too_many(int pages, int kvheads, int ps)
{
    return (long long)pages * ps > 0x7fffffffll || (long long)pages * ps * kvheads > 0x7fffffffll;
}

int grow_run(int n, const int* seq, const int* add, int seqs, int* len, int* table, int ldt, int pages,
             int ps, int* refs, int* got, hipStream_t stream)
{
    if (n < 0 || n > PG_MOST) return -1;
    const bool some = n > 0, any = some && seqs > 0;
    if (some && seq == nullptr) return -2;
    if (some && add == nullptr) return -3;
    if (seqs < 0) return -4;
    if (any && len == nullptr) return -5;
    if (any && ldt > 0 && table == nullptr) return -6;
    if (ldt < 0) return -7;
    if (pages < 0) return -8;
    if (ps < 1) return -9;
    if (any && pages > 0 && refs == nullptr) return -10;
    if (some && got == nullptr) return -11;
    if (!some) return 0;
    const PgGrowArgs a{{len, table, refs, seqs, ldt, pages, ps}, seq, add, got, n};
    return q8_launch(&q8_pages_grow, 1, PG_THREADS, stream, a);
}

int slots_run(int rows, int kvheads, const int* start, int seqs, const int* len, const int* table, int ldt,
              int pages, int ps, int* slot, hipStream_t stream)
{
    if (rows < 0) return -1;
    if (kvheads < 1) return -2;
    if (seqs < 0 || (start == nullptr && seqs != rows)) return -4;
    const bool some = rows > 0 && seqs > 0;
    if (some && len == nullptr) return -5;
    if (some && ldt > 0 && table == nullptr) return -6;
    if (ldt < 0) return -7;
    if (pages < 0 || (ps >= 1 && too_many(pages, kvheads, ps))) return -8;
    if (ps < 1) return -9;
    if (some && slot == nullptr) return -10;
    if (!some) return 0;
    const PgSlotArgs a{{const_cast<int*>(len), const_cast<int*>(table), nullptr, seqs, ldt, pages, ps},
                       start, slot, rows, kvheads};
    const long long groups = ((long long)rows * kvheads + 255) / 256;
    return q8_launch(&q8_pages_slots, (unsigned)std::min(groups, 4096ll), 256, stream, a);
}

int fork_run(int n, const int* parent, const int* child, int seqs, int* len, int* table, int ldt, int pages,
             int ps, int* refs, int* src, int* dst, hipStream_t stream)
{
    if (n < 0 || n > PG_MOST) return -1;
    const bool some = n > 0, any = some && seqs > 0;
    if (some && parent == nullptr) return -2;
    if (some && child == nullptr) return -3;
    if (seqs < 0) return -4;
    if (any && len == nullptr) return -5;
    if (any && ldt > 0 && table == nullptr) return -6;
    if (ldt < 0) return -7;
    if (pages < 0) return -8;
    if (ps < 1) return -9;
    if (any && pages > 0 && refs == nullptr) return -10;
    if (some && src == nullptr) return -11;
    if (some && dst == nullptr) return -12;
    if (!some) return 0;
    PgForkArgs a{{len, table, refs, seqs, ldt, pages, ps}, parent, child, src, dst, n, 0};
    // Few entries are written by the workgroup that gave out the pages, which
    // saves the second launch; what a single workgroup writes is bound by its own
    // latency, a table's row at a time.
    a.whole = n <= 16 && (long long)n * ldt <= 16 * PG_THREADS;
    if (a.whole) return q8_launch(&q8_pages_fork, 1, PG_THREADS, stream, a);
    return launch_two(&q8_pages_fork, &q8_pages_inherit, (unsigned)n, stream, a);
}

int free_run(int n, const int* seq, int seqs, int* len, int* table, int ldt, int pages, int ps, int* refs,
             hipStream_t stream)
{
    if (n < 0) return -1;
    const bool some = n > 0, any = some && seqs > 0;
    if (some && seq == nullptr) return -2;
    if (seqs < 0) return -3;
    if (any && len == nullptr) return -4;
    if (any && ldt > 0 && table == nullptr) return -5;
    if (ldt < 0) return -6;
    if (pages < 0) return -7;
    if (ps < 1) return -8;
    if (any && pages > 0 && refs == nullptr) return -9;
    if (!any) return 0;
    const PgFreeArgs a{{len, table, refs, seqs, ldt, pages, ps}, seq, n};
    return q8_launch(&q8_pages_free, q8_grid(n, 1), 256, stream, a);
}

int compact_run(int seqs, const int* table, int ldt, int* out, int ldo, int pages, const int* refs, int* rout,
                int* src, int* dst, int* live, hipStream_t stream)
{
    if (seqs < 0) return -1;
    const bool some = seqs > 0 && ldt > 0;
    if (some && table == nullptr) return -2;
    if (ldt < 0) return -3;
    if (some && out == nullptr) return -4;
    if (ldo < ldt || (out == table && out != nullptr && ldo != ldt)) return -5;
    if (pages < 0) return -6;
    if (pages > 0 && refs == nullptr) return -7;
    if (pages > 0 && rout == nullptr) return -8;
    if (pages > 1 && src == nullptr) return -9;
    if (pages > 1 && dst == nullptr) return -10;
    if (live == nullptr) return -11;
    const PgCompactArgs a{table, refs, out, rout, src, dst, live, seqs, ldt, ldo, pages};
    const long long all = (long long)seqs * ldt + pages;
    if (all == 0) return q8_launch(&q8_pages_plan, 1, PG_THREADS, stream, a);
    return launch_two(&q8_pages_plan, &q8_pages_rename, (unsigned)std::min((all + 255) / 256, 4096ll), stream, a);
}

int copy_run(int n, const int* src, const int* dst, int pages, int rows, int hd, signed char* k, int ldk,
             float* ks, signed char* v, int ldv, float* vs, int layers, int stride, hipStream_t stream)
{
    if (n < 0) return -1;
    if (n > 0 && src == nullptr) return -2;
    if (n > 0 && dst == nullptr) return -3;
    if (pages < 0 || (long long)pages * std::max(rows, 0) > 0x7fffffffll) return -4;
    if (rows < 0) return -5;
    if (hd < 0) return -6;
    const bool some = n > 0 && pages > 0 && rows > 0 && layers > 0;
    if (some && hd > 0 && k == nullptr) return -7;
    if (ldk < std::max(1, hd)) return -8;
    if (some && ks == nullptr) return -9;
    if (v != nullptr && ldv < std::max(1, hd)) return -11;
    if (some && v != nullptr && vs == nullptr) return -12;
    if (layers < 0) return -13;
    if (layers > 1 && (long long)stride < (long long)pages * rows) return -14;
    if (!some) return 0;
    PgCopyArgs a{src, dst, k, v, ks, vs, n, pages, rows, hd, ldk, ldv, layers, stride, 1};
    const bool run = ldk == hd && (v == nullptr || ldv == hd);
    const long long pieces = run ? ((long long)rows * hd + PG_PIECE - 1) / PG_PIECE
                                 : ((long long)rows + PG_ROWS - 1) / PG_ROWS;
    a.pieces = (int)std::max(1ll, pieces);
    const long long all = (long long)n * (v != nullptr ? 2 : 1) * layers * a.pieces;
    return q8_launch(&q8_pages_copy, (unsigned)std::min(all, 1ll << 16), 256, stream, a);
}

}  // namespace
}  // namespace xsymv

extern "C" int xsymv_q8pages_grow(int n, const int* seq, const int* add, int seqs, int* len, int* table,
                                  int ldt, int pages, int ps, int* refs, int* got, void* stream)
{
    return xsymv::q8_guard([&] {
        return xsymv::grow_run(n, seq, add, seqs, len, table, ldt, pages, ps, refs, got,
                               (hipStream_t)stream);
    });
}

extern "C" int xsymv_q8pages_slots(int rows, int kvheads, const int* start, int seqs, const int* len,
                                   const int* table, int ldt, int pages, int ps, int* slot, void* stream)
{
    return xsymv::q8_guard([&] {
        return xsymv::slots_run(rows, kvheads, start, seqs, len, table, ldt, pages, ps, slot,
                                (hipStream_t)stream);
    });
}

extern "C" int xsymv_q8pages_fork(int n, const int* parent, const int* child, int seqs, int* len, int* table,
                                  int ldt, int pages, int ps, int* refs, int* src, int* dst, void* stream)
{
    return xsymv::q8_guard([&] {
        return xsymv::fork_run(n, parent, child, seqs, len, table, ldt, pages, ps, refs, src, dst,
                               (hipStream_t)stream);
    });
}

extern "C" int xsymv_q8pages_free(int n, const int* seq, int seqs, int* len, int* table, int ldt, int pages,
                                  int ps, int* refs, void* stream)
{
    return xsymv::q8_guard([&] {
        return xsymv::free_run(n, seq, seqs, len, table, ldt, pages, ps, refs, (hipStream_t)stream);
    });
}

extern "C" int xsymv_q8pages_compact(int seqs, const int* table, int ldt, int* out, int ldo, int pages,
                                     const int* refs, int* rout, int* src, int* dst, int* live, void* stream)
{
    return xsymv::q8_guard([&] {
        return xsymv::compact_run(seqs, table, ldt, out, ldo, pages, refs, rout, src, dst, live,
                                  (hipStream_t)stream);
    });
}

extern "C" int xsymv_q8pages_copy(int n, const int* src, const int* dst, int pages, int rows, int hd,
                                  signed char* k, int ldk, float* ks, signed char* v, int ldv, float* vs,
                                  int layers, int stride, void* stream)
{
    return xsymv::q8_guard([&] {
        return xsymv::copy_run(n, src, dst, pages, rows, hd, k, ldk, ks, v, ldv, vs, layers, stride,
                               (hipStream_t)stream);
    });
}
