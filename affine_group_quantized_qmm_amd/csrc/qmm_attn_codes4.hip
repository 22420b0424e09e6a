// Attention over a paged cache of 4-bit codes: the launches. The kernels are in
// qmm_attn_codes.hpp.
#include "qmm_attn_codes.hpp"

namespace qmm {

hipError_t launch_attention_codes4(const AttnArgs &a, const AttnPlan &p, int D, hipStream_t stream)
{
    return launch_dim<4>(a, p, D, stream);
}

}  // namespace qmm
