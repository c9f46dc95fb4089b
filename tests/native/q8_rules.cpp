// Host program: the rules of the row kernels (xq8_rows.hpp) that depend on
// which of a norm's arguments are given and which are the same.  Prints a line
// for each case: the arguments, whether elements belong to one thread alone,
// and where the last chunk of 100 elements starts.
#include <cstdio>

#include "../../blas_symmetric_mat_amd/csrc/xq8_rows.hpp"

using namespace xsymv;

template <class R>
static void norm(const char* name, const float* x, const R* r, R* h)
{
    Q8Norm<float, R, float> op{};
    op.x = x;
    op.r = r;
    op.h = h;
    op.n = 100;
    std::printf("%s %d %d\n", name, (int)op.in_place(), q8_last_column(op.n, op.in_place()));
}

int main()
{
    float a[2], b[2], c[2];
    norm<float>("apart", a, b, c);
    norm<float>("h_is_r", a, b, b);
    norm<float>("h_is_x", a, b, a);
    norm<float>("h_is_x_alone", a, nullptr, a);
    norm<float>("all_one", a, a, a);
    norm<float>("no_r", a, nullptr, c);
    norm<float>("no_h", a, b, nullptr);
    norm<float>("neither", a, nullptr, nullptr);
    return 0;
}
