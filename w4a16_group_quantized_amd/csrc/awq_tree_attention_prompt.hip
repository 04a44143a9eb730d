// awq_tree_attention for many rows: see awq_attention_prompt.h.
#include "awq_attention_prompt.h"

namespace awq {

hipError_t launch_tree_attention_prefill(const AttnArgs &p, int head_dim, bool bf16, int row_tiles, bool flat, hipStream_t s) {
    return launch_prompt_rows<true>(p, head_dim, bf16, row_tiles, flat, s);
}

}  // namespace awq
