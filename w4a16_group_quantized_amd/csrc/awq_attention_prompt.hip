// awq_attention for many rows: see awq_attention_prompt.h.
#include <algorithm>

#include "awq_attention_prompt.h"

namespace awq {

int prefill_row_tiles(int seqs, int rows, int kv_heads, int group, int head_dim, int max_q, int few, bool flat) {
    const int each = rows_of(head_dim);
    if (flat)                                  // all that there can be
        return (int)((long long)rows * group / each + std::min<long long>(seqs, (long long)rows * group / few));
    const long long tiles = ((long long)max_q * group + each - 1) / each;
    const long long pairs = (long long)kv_heads * seqs;                          // below 2^20
    return (int)std::max<long long>(1, std::min<long long>(tiles, ((1 << 24) - 1) / (kMostSplits * pairs)));
}

// Chunks of the keys where row tiles are too few to fill the GPU (two workgroups to a CU).
int prefill_splits(int seqs, int kv_heads, int row_tiles, bool flat, long long key_tiles) {
    const long long groups = std::max<long long>(1, (long long)(flat ? 1 : seqs) * kv_heads * row_tiles);
    return (int)std::max<long long>(1, std::min<long long>({512 / groups, key_tiles / kLeastChunk, kMostSplits}));
}

// Trees: workgroups of a kv head, two to a CU in all, or where keys are not cut, one to a row tile;
// and chunks that a row tile has room for, twice what it has on average, since sequences are not
// equally long.
TreePlan tree_plan(int seqs, int kv_heads, int row_tiles, bool flat, long long key_tiles) {
    const long long groups = std::max<long long>(1, (long long)(flat ? 1 : seqs) * row_tiles);   // of a kv head
    const long long all = groups * kv_heads;
    TreePlan t{(int)std::min<long long>(groups, (1 << 24) / kv_heads), 1};
    if (key_tiles >= 2 * kLeastChunk && all < kManyTreeTiles) {
        t.shares = std::max(1, kTreeSlots / kv_heads);
        t.room = (int)std::max<long long>(3, std::min<long long>({2 * kTreeSlots / all + 1, key_tiles / kLeastChunk + 1, kMostSplits + 1}));
    }
    return t;
}

hipError_t launch_attention_prefill(const AttnArgs &p, int head_dim, bool bf16, int row_tiles, bool flat, hipStream_t s) {
    return launch_prompt_rows<false>(p, head_dim, bf16, row_tiles, flat, s);
}

}  // namespace awq
