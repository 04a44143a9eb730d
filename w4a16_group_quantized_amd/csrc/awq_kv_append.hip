// awq_kv_append: see awq_kv_append_kernels.h.
#include "awq_kv_append_kernels.h"

namespace awq {

bool kv_head_dim_supported(int head_dim) { return head_dim == 64 || head_dim == 128 || head_dim == 256; }

hipError_t launch_kv_append(const KvView &c, int head_dim, const uint16_t *q, long long q_stride,
                            const uint16_t *k, long long k_stride, const uint16_t *v,
                            long long v_stride, uint16_t *q_out, int q_heads, const float *rope,
                            int rope_positions, int rot, bool adjacent, bool bf16, int max_q,
                            hipStream_t s) {
    const AppendArgs p{c, q, k, v, q_stride, k_stride, v_stride, q_out, rope, rope_positions, rot, q_heads, nullptr, 0, {}};
    return launch_append<0>(p, head_dim, adjacent, bf16, max_q, s);
}

}  // namespace awq
