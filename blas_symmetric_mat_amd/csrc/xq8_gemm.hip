// xq8_gemm.hip -- the product of rows in 8 bits: which kernel makes a call
// (see xq8_gemm_run.hpp), and the workspace query.
#include "xq8_gemm_run.hpp"

namespace xsymv {
namespace {

// What ranks the kernels: a model of a call's time fitted to measurements on
// MI355X over a grid of sizes (m 1 to 8000, n and k 128 to 28672, every number
// of shares; tuned/mi355x_q8gemm.json holds what is within 1.5 times of each
// size's fastest).  `launch`, and for every
// round of workgroups that the chip holds at once `round` plus, for each of the
// share's steps, `alone` where a compute unit runs one workgroup, `full` where
// it runs all it can and between them otherwise; but no less than W's bytes take
// at `rate` TB/s.  The constants are those that choose best and fit, not times
// of parts that were measured by themselves, and the estimates are no times to
// quote: half of them are within 8 % of the measured ones, nine in ten within
// 20 %, and the largest products take longer for the bytes of A and C, which are
// not in it (8000 x 8192 x 1024 in 256 x 256 tiles 94 us, estimated 65).  The
// choice is 1 % slower on average than the fastest kernel measured (2 % for up
// to 16 rows, 4 % where those lie at odd strides; at worst 2 times, at sizes of
// a few microseconds).  The rings are chosen at 400 of the grid's 1070 sizes of
// whole lines and 200 of 630 at odd strides, and are 1.16 (up to 16 rows) to 1.37 times faster there than
// the next kernel.  The 64-row tile alone, at its best number of shares, would
// be 1.07 (m = 65 to 128) to 1.36 times (m > 512) slower than the tiles together,
// and without shares of k up to 5 times.
struct Cost {
    float launch, alone, full, round, rate;
};
struct Kernel {
    Q8Kernel id;
    int bm, bn, waves;  // its tile, and waves a workgroup
    int step, turn;     // bytes of k a step; steps that waves take side by side
    int together;       // workgroups a compute unit runs at once
    int from, to;       // rows it is meant for
    float cut;          // factor of a step where rows cut lines (Q8_LINES)
    Cost cost;
};

constexpr int ANY_M = 1 << 30;
const Kernel LINES[] = {
    {Q8_RING, 16, 16, 8, 128, 8, 1, 1, ANY_M, 1.15f, {2.04f, 0.44f, 0.44f, 1.17f, 5.32f}},
    {Q8_RING32, 32, 32, 4, 128, 4, 1, 17, ANY_M, 1.25f, {1.97f, 0.34f, 0.34f, 1.34f, 3.21f}},
    {Q8_TILE16, 16, 64, 4, 256, 1, 2, 1, 16, 1.12f, {2.99f, 0.37f, 1.16f, 0.48f, 6.44f}},
    {Q8_TILE32, 32, 64, 4, 256, 1, 2, 1, 64, 1.15f, {2.27f, 0.33f, 0.98f, 1.57f, 4.87f}},
    {Q8_TILE64, 64, 64, 4, 128, 1, 2, 17, ANY_M, 1.35f, {2.30f, 0.24f, 0.53f, 1.69f, 5.92f}},
    {Q8_TILE64_SHORT, 64, 64, 4, 128, 1, 4, 17, ANY_M, 1.15f, {2.76f, 0.45f, 1.04f, 0.76f, 4.37f}},
    {Q8_TILE128X64, 128, 64, 8, 256, 1, 1, 65, ANY_M, 1.20f, {1.78f, 0.64f, 0.64f, 3.06f, 4.81f}},
    {Q8_TILE128, 128, 128, 8, 128, 1, 1, 65, ANY_M, 1.37f, {1.47f, 0.48f, 0.48f, 4.01f, 5.60f}},
    {Q8_TILE128_SHORT, 128, 128, 8, 128, 1, 2, 65, ANY_M, 1.20f, {2.96f, 0.73f, 1.23f, 1.97f, 4.07f}},
    {Q8_TILE256X128, 256, 128, 8, 128, 1, 1, 65, ANY_M, 1.27f, {1.60f, 0.69f, 0.69f, 5.62f, 4.68f}},
    {Q8_TILE256, 256, 256, 8, 128, 1, 1, 65, ANY_M, 1.19f, {4.15f, 1.27f, 1.27f, 4.95f, 3.96f}},
};
const Kernel ANY[] = {
    {Q8_RING, 16, 16, 8, 128, 8, 1, 1, ANY_M, 1.0f, {2.38f, 0.61f, 0.61f, 1.73f, 3.69f}},
    {Q8_RING32, 32, 32, 4, 128, 4, 1, 17, ANY_M, 1.0f, {1.64f, 0.65f, 0.65f, 2.44f, 1.88f}},
    {Q8_STREAM, 16, 16, 8, 256, 8, 4, 1, 16, 1.0f, {0.98f, 3.25f, 2.58f, 0.49f, 1.61f}},
    {Q8_TILE16, 16, 64, 4, 256, 1, 2, 1, 16, 1.0f, {4.15f, 0.47f, 1.05f, 0.14f, 7.60f}},
    {Q8_TILE32, 32, 64, 4, 256, 1, 2, 1, 64, 1.0f, {2.39f, 0.74f, 1.37f, 1.80f, 5.59f}},
    {Q8_TILE64, 64, 64, 4, 256, 1, 2, 17, ANY_M, 1.0f, {3.36f, 0.77f, 1.28f, 2.19f, 5.35f}},
    {Q8_TILE64_SHORT, 64, 64, 4, 128, 1, 4, 17, ANY_M, 1.0f, {2.39f, 0.78f, 1.60f, 1.59f, 3.38f}},
    {Q8_TILE128, 128, 128, 8, 256, 1, 1, 65, ANY_M, 1.0f, {2.02f, 1.81f, 1.81f, 4.45f, 3.39f}},
    {Q8_TILE128_SHORT, 128, 128, 8, 128, 1, 2, 65, ANY_M, 1.0f, {2.66f, 0.97f, 2.05f, 3.25f, 2.66f}},
    {Q8_TILE256X128, 256, 128, 8, 128, 1, 1, 65, ANY_M, 1.0f, {0.26f, 1.37f, 1.37f, 7.04f, 2.26f}},
    {Q8_TILE256, 256, 256, 8, 128, 1, 1, 65, ANY_M, 1.0f, {4.15f, 1.56f, 1.56f, 7.54f, 3.18f}},
};
const Kernel REGS[] = {
    {Q8_STREAM, 16, 16, 8, 256, 8, 4, 1, 16, 1.0f, {0.47f, 3.66f, 2.70f, 0.03f, 1.80f}},
    {Q8_TILE16, 16, 64, 4, 128, 1, 4, 1, 16, 1.0f, {3.16f, 0.67f, 1.62f, 0.01f, 3.78f}},
    {Q8_TILE64, 64, 64, 4, 128, 1, 2, 17, ANY_M, 1.0f, {2.85f, 0.70f, 0.92f, 0.92f, 3.23f}},
    {Q8_TILE256X128, 256, 128, 8, 128, 1, 1, 65, ANY_M, 1.0f, {1.49f, 1.65f, 1.65f, 4.84f, 1.94f}},
};

// Adding the shares: a launch, and their sums written and read.
constexpr float JOIN_LAUNCH = 2.9f, JOIN_MILLION = 1.26f;
// Copying rows to whole lines: a launch, and each byte read and written (what
// was copied last is still cached when it is read, hence the rate).
constexpr double COPY_LAUNCH = 2.9, COPY_BYTE = 2.0 / 6.5e6;
constexpr size_t MAX_COPY = (size_t)1 << 30;
constexpr int CUS = 256;
constexpr long long MAX_PART = 1ll << 28;  // bytes of the shares' sums

double cost_of(const Kernel& c, bool cut, int m, int n, int k, int splits, Q8Plan& p)
{
    const int steps = std::max(1, (k + c.step - 1) / c.step);
    p.kernel = c.id;
    p.per = (steps + splits - 1) / splits;
    p.splits = (steps + p.per - 1) / p.per;
    const long long groups = (((long long)m + c.bm - 1) / c.bm) *
                             (((long long)n + c.bn - 1) / c.bn) * p.splits;
    p.groups = (unsigned)groups;
    p.part = p.splits > 1 ? (size_t)p.splits * m * q8_part_ld(n) * sizeof(int) : 0;
    if (groups * c.waves * 64 >= 1ll << 31 || (p.splits > 1 && (long long)p.part > MAX_PART))
        return -1.0;  // a launch's threads are counted in 32 bits
    const float taken = (float)((p.per + c.turn - 1) / c.turn) * (cut ? c.cut : 1.0f);
    const long long slots = (long long)CUS * c.together, full = groups / slots, rest = groups % slots;
    double t = (double)full * (taken * (c.together > 1 ? c.cost.full : c.cost.alone) + c.cost.round);
    if (rest > 0) {
        const int load = (int)((rest + CUS - 1) / CUS);  // workgroups of the fullest compute unit
        const float more = c.together > 1 ? (float)(load - 1) / (c.together - 1) : 0.0f;
        t += taken * (c.cost.alone + (c.cost.full - c.cost.alone) * more) + c.cost.round;
    }
    t = c.cost.launch + std::max(t, (double)n * k / c.cost.rate * 1e-6);
    if (p.splits > 1) t += JOIN_LAUNCH + JOIN_MILLION * 1e-6 * m * n * p.splits;
    return t;
}

template <int N>
Q8Plan cheapest(const Kernel (&list)[N], bool cut, bool whole, int m, int n, int k, double& low)
{
    Q8Plan best{};
    low = -1.0;
    for (const Kernel& c : list) {
        if (m < c.from || m > c.to) continue;
        for (int splits = 1; splits <= (whole || c.id == Q8_STREAM ? 1 : 16); ++splits) {
            if (splits > 1 && k / 256 < splits) break;
            Q8Plan p{};
            const double t = cost_of(c, cut, m, n, k, splits, p);
            if (t >= 0.0 && (low < 0.0 || t < low)) {
                low = t;
                best = p;
            }
        }
    }
    return best;
}

}  // namespace

Q8Plan q8_plan(int how, bool cut, bool whole, int m, int n, int k)
{
    // the last sizes' choices: some hundred estimates take as long as a launch
    struct Known {
        int how, m, n, k;
        bool cut, whole;
        Q8Plan plan;
    };
    static thread_local Known known[64] = {};
    const unsigned key = ((unsigned)m * 31u + (unsigned)n) * 31u + (unsigned)k * 7u + (unsigned)how;
    Known& e = known[key % 64];
    if (e.m == m && e.n == n && e.k == k && e.how == how && e.cut == cut && e.whole == whole && m > 0)
        return e.plan;
    double cost = 0.0;
    Q8Plan p = how == Q8_LINES ? cheapest(LINES, cut, whole, m, n, k, cost)
               : how == Q8_ANY ? cheapest(ANY, false, whole, m, n, k, cost)
                               : cheapest(REGS, false, whole, m, n, k, cost);
    p.how = how;
    if ((how != Q8_LINES || cut) && k >= 16 && !whole) {
        // many rows: each is read often, and from whole lines a third faster
        // than at odd strides (4096 x 28672 x 8192: 1124 us where they lie,
        // 832 with the copy; 100 x 28672 x 8192: 73 and 142 us), a tenth
        // faster than where they cut lines (896 and 843; 1024 x 8192 x 4096:
        // 48 and 50 us)
        const size_t copy = align_up(((size_t)m + n) * q8_copy_ld(k));
        double lines = 0.0;
        Q8Plan c = cheapest(LINES, false, false, m, n, k, lines);
        if (copy <= MAX_COPY && c.groups != 0 &&
            (p.groups == 0 || lines + COPY_LAUNCH + COPY_BYTE * k * ((double)m + n) < cost)) {
            p = c;
            p.how = Q8_LINES;
            p.ldc = q8_copy_ld(k);
            p.copy = copy;
        }
    }
    e = Known{how, m, n, k, cut, whole, p};
    return p;
}

}  // namespace xsymv

extern "C" size_t xsymv_q8gemm_workspace_bytes(int m, int n, int k)
{
    using namespace xsymv;
    if (m <= 0 || n <= 0 || k <= 0 || k > Q8_MAX_K) return 0;
    size_t most = 0;
    // a call of more rows or columns is made in blocks of these (and what is left)
    for (int rows : {std::min(m, Q8_BLOCK), m % Q8_BLOCK})
        for (int cols : {std::min(n, Q8_BLOCK), n % Q8_BLOCK})
            for (int how : {Q8_REGS, Q8_LINES, Q8_ANY})
                for (bool cut : {false, true})
                    if (rows > 0 && cols > 0) {
                        const Q8Plan p = q8_plan(how, cut, false, rows, cols, k);
                        most = std::max(most, p.copy + p.part);
                    }
    return most;
}
