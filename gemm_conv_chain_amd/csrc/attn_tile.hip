// attn_tile.hip -- instantiations of k_attn_tile (attn_tile.h) for new tokens in
// causal order or all seen.
#include "attn_tile.h"

namespace fc {

hipError_t run_attn_tile(int dtype, const AttnArgs& a, hipStream_t st)
{
    return dtype == DT_F16 ? tile_by_d<half_t, false>(a, st) : tile_by_d<bf16_t, false>(a, st);
}

}  // namespace fc
