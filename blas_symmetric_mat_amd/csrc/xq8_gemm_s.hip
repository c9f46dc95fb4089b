// The product of rows in 8 bits, results in float.
#include "xq8_gemm_run.hpp"

XSYMV_Q8_GEMM(s, float, float)
