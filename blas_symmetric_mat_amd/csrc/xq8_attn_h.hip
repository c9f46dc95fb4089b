// xq8_attn_h.hip -- the attention over a cache of 8-bit rows for half rows.
#include "xq8_attn_run.hpp"

XSYMV_Q8_ATTN(h, xhalf, xsymv::q8half)
