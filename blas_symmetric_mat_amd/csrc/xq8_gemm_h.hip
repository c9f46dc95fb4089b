// The product of rows in 8 bits, results in half precision.
#include "xq8_gemm_run.hpp"

XSYMV_Q8_GEMM(h, xhalf, xsymv::q8half)
