// xq8_attn.hip -- the attention's workspace query.
#include "xq8_attn_run.hpp"

extern "C" size_t xsymv_q8attn_workspace_bytes(int rows, int heads, int kvheads, int hd, int seqs, int groups)
{
    using namespace xsymv;
    if (rows <= 0 || kvheads < 1 || heads < 1 || heads % kvheads != 0 || hd < AT_LOW || hd > AT_HD || seqs < 0 ||
        groups < 0)
        return 0;
    return AttnSpace(rows, heads, kvheads, hd, seqs, groups, false).bytes;
}
