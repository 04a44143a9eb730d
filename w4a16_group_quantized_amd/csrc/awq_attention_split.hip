// awq_attention for few rows: see awq_attention_split.h.
#include "awq_attention_split.h"

namespace awq {

hipError_t launch_attention_split(const AttnArgs &p, int head_dim, bool bf16, bool wide, int row_tiles, hipStream_t s) {
    return launch_split_rows<false>(p, head_dim, bf16, wide, row_tiles, s);
}

}  // namespace awq
