// awq_tree_rows: from the parents of drafted rows, the rows that each sees (itself and its
// ancestors), as bits, and its position, the tokens before the tree plus its depth.
//
// A thread follows one row's parents for one word of bits; parents go to LDS first, since
// that chain of reads is all that takes time.  Bound: latency.
#include <algorithm>

#include "awq_internal.h"
#include "awq_kv.h"

namespace awq {
namespace {

constexpr int kThreads = 256;
constexpr int kHeld = 4096;                // parents that LDS holds; of longer trees they are read where they are

__global__ void __launch_bounds__(kThreads) tree_rows_kernel(const int32_t *parents, KvView c, uint32_t *mask, int words,
                                                              int32_t *positions) {
    __shared__ int32_t held[kHeld];
    const int b = blockIdx.y;
    const int a = min(max(c.q_starts[b], 0), c.rows), n = max(min(max(c.q_starts[b + 1], 0), c.rows) - a, 0);
    if ((long long)blockIdx.x * kThreads >= (long long)n * words) return;
    const int32_t *up = parents + a;
    const int first = max(c.kv_lens[b], 0) - n;
    for (int t = threadIdx.x; t < min(n, kHeld); t += kThreads) held[t] = up[t];
    __syncthreads();
    for (long long i = (long long)blockIdx.x * kThreads + threadIdx.x; i < (long long)n * words; i += (long long)gridDim.x * kThreads) {
        const int t = (int)(i / words), w = (int)(i % words);
        uint32_t bits = 0;
        int depth = 0;
        for (int u = t;;) {
            if (u >> 5 == w) bits |= 1u << (u & 31);
            if (u >> 5 < w) break;             // (parents come before their children)
            const int next = u < kHeld ? held[u] : up[u];
            if (next < 0 || next >= u) break;
            u = next;
            ++depth;
        }
        mask[(long long)(a + t) * words + w] = bits;
        if (w == 0 && positions != nullptr) positions[a + t] = first + depth;
    }
}

}  // namespace

hipError_t launch_tree_rows(const int32_t *parents, const KvView &c, int max_q, uint32_t *mask, int words, int32_t *positions, hipStream_t s) {
    const long long items = (long long)max_q * words;
    const int grid = (int)std::min<long long>((items + kThreads - 1) / kThreads, 4096);
    tree_rows_kernel<<<dim3(grid, c.seqs), kThreads, 0, s>>>(parents, c, mask, words, positions);
    return hipGetLastError();
}

}  // namespace awq
