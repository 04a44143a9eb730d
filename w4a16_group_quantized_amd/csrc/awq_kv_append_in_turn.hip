// awq_kv_append_at where the axes take the frequencies in turn; see awq_kv_append_kernels.h.
#include "awq_kv_append_kernels.h"

namespace awq {

hipError_t launch_append_in_turn(const AppendArgs &p, int head_dim, bool adjacent, bool bf16, int max_q, hipStream_t s) {
    return launch_append<kInTurn>(p, head_dim, adjacent, bf16, max_q, s);
}

}  // namespace awq
