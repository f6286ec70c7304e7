// ibp_attention_bf16.hip -- attention over pages of bf16 numbers.
#include "ibp_attention.hpp"

namespace ibp {

hipError_t launch_attention_bf16(const AttnArgs& a, const AttnPlan& p, uint32_t head_dim, uint32_t page_tokens,
                                 bool tree, uint32_t lds, hipStream_t s) {
    return launch_attention_e<Bf16>(a, p, head_dim, page_tokens, tree, lds, s);
}

}  // namespace ibp
