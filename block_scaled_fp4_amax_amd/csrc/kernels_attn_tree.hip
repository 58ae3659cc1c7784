// kernels_attn_tree.hip -- fp4_attn_tree: attn_kernels.h's kernels with a mask of the drafted keys.
// plan_attn_tree (kernels_attn.hip) plans these calls.
#include "attn_kernels.h"

namespace fp4q {

hipError_t launch_attn_tree(int bias, const AttnArgs& a, hipStream_t s)
{
    if (bias == 0) return launch_bias<0, true>(a, s);
    if (bias == 7) return launch_bias<7, true>(a, s);
    return launch_bias<15, true>(a, s);
}

}  // namespace fp4q
