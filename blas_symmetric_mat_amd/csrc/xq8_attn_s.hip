// xq8_attn_s.hip -- the attention over a cache of 8-bit rows for float rows.
#include "xq8_attn_run.hpp"

XSYMV_Q8_ATTN(s, float, float)
