// xq8_attn_b.hip -- the attention over a cache of 8-bit rows for bfloat16 rows.
#include "xq8_attn_run.hpp"

XSYMV_Q8_ATTN(b, xbfloat16, xsymv::q8bf16)
