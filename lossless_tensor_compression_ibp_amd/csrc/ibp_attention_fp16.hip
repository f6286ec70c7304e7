// ibp_attention_fp16.hip -- attention over pages of fp16 numbers.
#include "ibp_attention.hpp"

namespace ibp {

hipError_t launch_attention_fp16(const AttnArgs& a, const AttnPlan& p, uint32_t head_dim, uint32_t page_tokens,
                                 bool tree, uint32_t lds, hipStream_t s) {
    return launch_attention_e<Fp16>(a, p, head_dim, page_tokens, tree, lds, s);
}

}  // namespace ibp
