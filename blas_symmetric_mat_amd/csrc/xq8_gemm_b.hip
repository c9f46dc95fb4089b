// The product of rows in 8 bits, results in bfloat16.
#include "xq8_gemm_run.hpp"

XSYMV_Q8_GEMM(b, xbfloat16, xsymv::q8bf16)
