// xq8_attn.hip -- the attention's workspace query.
#include "xq8_host.hpp"

extern "C" size_t xsymv_q8attn_workspace_bytes(int rows, int heads, int kvheads, int hd, int seqs, int groups)
{
    (void)rows, (void)heads, (void)kvheads, (void)hd, (void)seqs, (void)groups;
    return 0;
}
