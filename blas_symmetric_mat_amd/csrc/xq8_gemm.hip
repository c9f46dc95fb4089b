// xq8_gemm.hip -- the product of rows in 8 bits: which kernel makes a call
// (see xq8_gemm_run.hpp), and the workspace query.
#include "xq8_gemm_run.hpp"

namespace xsymv {
namespace {

// What a kernel costs, in microseconds, as measured on MI355X over a grid of
// sizes (m 1 to 4096, n and k 256 to 28672, every number of shares) and
// fitted: `launch`, and for every round of workgroups that the chip holds at
// once `round` plus, for each of the share's steps, `alone` where a compute
// unit runs one workgroup and `pair` where it runs two; but no less than W's
// bytes take at `rate` TB/s.  Over that grid the kernel this chooses is 1 %
// slower on average than the fastest one measured (at worst 1.6 times, at
// sizes of a few microseconds).  The 64-row tile alone, at its best number of
// shares, would be 1.07 (m = 65 to 128) to 1.36 times (m > 512) slower, and
// without shares of k up to 5 times.
struct Cost {
    float launch, alone, pair, round, rate;
};
struct Kernel {
    Q8Kernel id;
    int bm, bn, waves;  // its tile, and waves a workgroup
    int step, turn;     // bytes of k a step; steps that waves take side by side
    int together;       // workgroups a compute unit runs at once
    int from, to;       // rows it is meant for
    Cost cost;
};

constexpr int ANY_M = 1 << 30;
const Kernel LINES[] = {
    {Q8_RING, 16, 16, 8, 128, 8, 1, 1, 16, {1.86f, 0.49f, 0.49f, 1.45f, 5.54f}},
    {Q8_TILE16, 16, 64, 4, 256, 1, 2, 1, 16, {3.05f, 0.37f, 1.22f, 0.01f, 5.98f}},
    {Q8_TILE32, 32, 64, 4, 256, 1, 2, 1, 64, {2.98f, 0.44f, 0.96f, 0.29f, 5.63f}},
    {Q8_TILE64, 64, 64, 4, 128, 1, 2, 17, ANY_M, {2.98f, 0.23f, 0.48f, 1.29f, 5.33f}},
    {Q8_TILE128X64, 128, 64, 8, 256, 1, 1, 65, ANY_M, {1.83f, 0.66f, 0.66f, 2.69f, 5.54f}},
    {Q8_TILE128, 128, 128, 8, 128, 1, 1, 65, ANY_M, {1.58f, 0.51f, 0.51f, 3.49f, 5.99f}},
    {Q8_TILE256X128, 256, 128, 8, 128, 1, 1, 65, ANY_M, {2.01f, 0.69f, 0.69f, 4.87f, 4.79f}},
    {Q8_TILE256, 256, 256, 8, 128, 1, 1, 65, ANY_M, {1.32f, 1.21f, 1.21f, 8.06f, 3.91f}},
};
const Kernel ANY[] = {
    {Q8_STREAM, 16, 16, 8, 256, 8, 4, 1, 16, {0.41f, 3.12f, 3.10f, 0.76f, 1.60f}},
    {Q8_TILE16, 16, 64, 4, 256, 1, 2, 1, 16, {3.59f, 0.46f, 1.01f, 0.24f, 7.99f}},
    {Q8_TILE32, 32, 64, 4, 256, 1, 2, 1, 64, {2.25f, 0.75f, 1.32f, 1.88f, 5.54f}},
    {Q8_TILE64, 64, 64, 4, 256, 1, 2, 17, ANY_M, {3.44f, 0.74f, 1.25f, 1.99f, 5.64f}},
    {Q8_TILE128, 128, 128, 8, 256, 1, 1, 65, ANY_M, {2.12f, 1.60f, 1.60f, 5.09f, 3.85f}},
    {Q8_TILE256X128, 256, 128, 8, 128, 1, 1, 65, ANY_M, {3.23f, 1.23f, 1.23f, 3.82f, 2.46f}},
    {Q8_TILE256, 256, 256, 8, 128, 1, 1, 65, ANY_M, {4.40f, 1.23f, 1.23f, 7.34f, 3.96f}},
};
const Kernel REGS[] = {
    {Q8_STREAM, 16, 16, 8, 256, 8, 4, 1, 16, {0.31f, 3.84f, 3.82f, 0.01f, 1.91f}},
    {Q8_TILE16, 16, 64, 4, 128, 1, 4, 1, 16, {2.54f, 0.81f, 0.98f, 0.01f, 3.82f}},
    {Q8_TILE64, 64, 64, 4, 128, 1, 2, 17, ANY_M, {3.28f, 0.84f, 1.00f, 0.02f, 4.10f}},
    {Q8_TILE256X128, 256, 128, 8, 128, 1, 1, 65, ANY_M, {2.46f, 1.86f, 1.86f, 2.94f, 2.14f}},
};

// Adding the shares: a launch, and their sums written and read.
constexpr float JOIN_LAUNCH = 3.0f, JOIN_MILLION = 1.42f;
constexpr int CUS = 256;
constexpr long long MAX_PART = 1ll << 28;  // bytes of the shares' sums

double cost_of(const Kernel& c, int m, int n, int k, int splits, Q8Plan& p)
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
    const int taken = (p.per + c.turn - 1) / c.turn;
    const long long slots = (long long)CUS * c.together, full = groups / slots, rest = groups % slots;
    double t = (double)full * (taken * (c.together > 1 ? c.cost.pair : c.cost.alone) + c.cost.round);
    if (rest > 0) t += taken * (rest <= CUS ? c.cost.alone : c.cost.pair) + c.cost.round;
    t = c.cost.launch + std::max(t, (double)n * k / c.cost.rate * 1e-6);
    if (p.splits > 1) t += JOIN_LAUNCH + JOIN_MILLION * 1e-6 * m * n * p.splits;
    return t;
}

template <int N>
Q8Plan cheapest(const Kernel (&list)[N], int m, int n, int k)
{
    Q8Plan best{};
    double low = -1.0;
    for (const Kernel& c : list) {
        if (m < c.from || m > c.to) continue;
        for (int splits = 1; splits <= (c.id == Q8_STREAM ? 1 : 16); splits *= 2) {
            if (splits > 1 && k / 256 < splits) break;
            Q8Plan p{};
            const double t = cost_of(c, m, n, k, splits, p);
            if (t >= 0.0 && (low < 0.0 || t < low)) {
                low = t;
                best = p;
            }
        }
    }
    return best;
}

}  // namespace

Q8Plan q8_plan(int how, int m, int n, int k)
{
    // the last sizes' choices: forty estimates take as long as a third of a launch
    struct Known {
        int how, m, n, k;
        Q8Plan plan;
    };
    static thread_local Known known[64] = {};
    const unsigned key = ((unsigned)m * 31u + (unsigned)n) * 31u + (unsigned)k * 7u + (unsigned)how;
    Known& e = known[key % 64];
    if (e.m == m && e.n == n && e.k == k && e.how == how && m > 0) return e.plan;
    Q8Plan p = how == Q8_LINES ? cheapest(LINES, m, n, k)
               : how == Q8_ANY ? cheapest(ANY, m, n, k)
                               : cheapest(REGS, m, n, k);
    p.how = how;
    e = Known{how, m, n, k, p};
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
                if (rows > 0 && cols > 0) most = std::max(most, q8_plan(how, rows, cols, k).part);
    return most;
}
