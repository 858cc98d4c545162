// attn_rows_tree.hip -- instantiations of k_attn_rows (attn_rows.h) for trees of
// drafted tokens.  Kept apart so that the sources compile in parallel.
#include "attn_rows.h"

namespace fc {

hipError_t run_attn_rows_tree(int dtype, const AttnArgs& a, hipStream_t st)
{
    return dtype == DT_F16 ? rows_by_d<half_t, true>(a, st) : rows_by_d<bf16_t, true>(a, st);
}

}  // namespace fc
