// awq_kv_append_at: awq_kv_append with given rotary positions; see awq_kv_append_kernels.h.
#include "awq_kv_append_kernels.h"

namespace awq {

hipError_t launch_kv_append_at(const KvView &c, int head_dim, const uint16_t *q, long long q_stride,
                               const uint16_t *k, long long k_stride, const uint16_t *v,
                               long long v_stride, uint16_t *q_out, int q_heads, const float *rope,
                               int rope_positions, int rot, bool adjacent, const int32_t *positions,
                               int axes, const AxisMap &map, bool bf16, int max_q, hipStream_t s) {
    const AppendArgs p{c, q, k, v, q_stride, k_stride, v_stride, q_out, rope, rope_positions, rot, q_heads, positions, axes, map};
    if (map.in_turn(rot / 2)) return launch_append_in_turn(p, head_dim, adjacent, bf16, max_q, s);
    return launch_append<kSections>(p, head_dim, adjacent, bf16, max_q, s);
}

}  // namespace awq
