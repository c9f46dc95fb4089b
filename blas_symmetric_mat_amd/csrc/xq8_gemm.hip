// xq8_gemm.hip -- the product of rows in 8 bits: which kernel makes a call
// (see xq8_gemm_run.hpp), and the workspace query.
#include "xq8_gemm_run.hpp"

namespace xsymv {
namespace {

// What a kernel costs, in microseconds, as measured on MI355X over a grid of
// sizes (m 1 to 2048, n 128 to 28672, k 256 to 28672, every number of shares)
// and fitted: `launch`, and for every round of workgroups that the chip holds
// at once `round` plus, for each of the share's steps, `alone` where a
// compute unit runs one workgroup and `pair` where it runs two; but no less
// than W's bytes take at `rate` TB/s.  The estimates are within 9 to 16 % of
// the times (root mean square); the kernel they choose is, by the same
// measurement, on average 1 % slower than the fastest one (5 % at m <= 16),
// where one kernel for all sizes is up to 10 times slower.
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
    {Q8_RING, 16, 16, 8, 128, 8, 1, 1, 16, {1.79f, 0.45f, 0.45f, 1.29f, 4.9f}},
    {Q8_TILE16, 16, 64, 4, 256, 1, 2, 1, 16, {3.32f, 0.32f, 1.31f, 0.0f, 5.6f}},
    {Q8_TILE32, 32, 64, 4, 256, 1, 2, 1, 64, {2.71f, 0.39f, 0.92f, 0.94f, 5.6f}},
    {Q8_TILE64, 64, 64, 4, 128, 1, 2, 17, ANY_M, {2.60f, 0.27f, 0.50f, 1.41f, 5.2f}},
    {Q8_TILE128X64, 128, 64, 8, 256, 1, 1, 65, ANY_M, {1.72f, 0.67f, 0.67f, 2.62f, 4.2f}},
    {Q8_TILE128, 128, 128, 8, 128, 1, 1, 65, ANY_M, {1.55f, 0.47f, 0.47f, 3.63f, 4.4f}},
    {Q8_TILE256X128, 256, 128, 8, 128, 1, 1, 65, ANY_M, {2.26f, 0.64f, 0.64f, 4.43f, 3.7f}},
    {Q8_TILE256, 256, 256, 8, 128, 1, 1, 65, ANY_M, {1.43f, 1.23f, 1.23f, 6.62f, 4.1f}},
};
const Kernel ANY[] = {
    {Q8_STREAM, 16, 16, 8, 256, 8, 4, 1, 16, {0.41f, 3.70f, 4.26f, 0.0f, 2.0f}},
    {Q8_TILE16, 16, 64, 4, 256, 1, 2, 1, 16, {3.79f, 0.48f, 1.45f, 0.0f, 5.2f}},
    {Q8_TILE32, 32, 64, 4, 256, 1, 2, 1, 64, {4.18f, 0.67f, 1.43f, 0.06f, 4.8f}},
    {Q8_TILE64, 64, 64, 4, 256, 1, 2, 17, ANY_M, {3.09f, 0.89f, 1.47f, 1.42f, 4.1f}},
    {Q8_TILE128, 128, 128, 8, 256, 1, 1, 65, ANY_M, {2.31f, 1.92f, 1.92f, 3.57f, 8.0f}},
    {Q8_TILE256X128, 256, 128, 8, 128, 1, 1, 65, ANY_M, {2.40f, 1.45f, 1.45f, 4.33f, 8.0f}},
    {Q8_TILE256, 256, 256, 8, 128, 1, 1, 65, ANY_M, {1.09f, 2.04f, 2.04f, 8.95f, 8.0f}},
};
const Kernel REGS[] = {
    {Q8_STREAM, 16, 16, 8, 256, 8, 4, 1, 16, {0.48f, 3.71f, 4.26f, 0.0f, 2.0f}},
    {Q8_TILE16, 16, 64, 4, 128, 1, 4, 1, 16, {2.50f, 0.80f, 1.06f, 0.0f, 3.9f}},
    {Q8_TILE64, 64, 64, 4, 128, 1, 2, 17, ANY_M, {3.15f, 0.86f, 1.0f, 0.0f, 3.1f}},
    {Q8_TILE256X128, 256, 128, 8, 128, 1, 1, 65, ANY_M, {2.17f, 1.83f, 1.83f, 3.16f, 8.0f}},
};

// Adding the shares: a launch, and their sums written and read.
constexpr float JOIN_LAUNCH = 2.6f, JOIN_MILLION = 1.42f;
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
    Q8Plan p = how == Q8_LINES ? cheapest(LINES, m, n, k)
               : how == Q8_ANY ? cheapest(ANY, m, n, k)
                               : cheapest(REGS, m, n, k);
    p.how = how;
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
