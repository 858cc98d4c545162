// attn_tile_tree.hip -- instantiations of k_attn_tile (attn_tile.h) for trees of
// drafted tokens.
#include "attn_tile.h"

namespace fc {

hipError_t run_attn_tile_tree(int dtype, const AttnArgs& a, hipStream_t st)
{
    const hipError_t e = dtype == DT_F16 ? tile_by_d<half_t, true>(a, st) : tile_by_d<bf16_t, true>(a, st);
    if (e != hipSuccess || !a.even) return e;
    return dtype == DT_F16 ? launch_tree_join<half_t>(a, st) : launch_tree_join<bf16_t>(a, st);
}

}  // namespace fc
