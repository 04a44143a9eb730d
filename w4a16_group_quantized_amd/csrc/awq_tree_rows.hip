// awq_tree_rows: from the parents of drafted rows, the rows that each sees (itself and its
// ancestors), as bits, and its position, the tokens before the tree plus its depth.
//
// Rows are taken in blocks of 64, a wave each.  Within its block a row's ancestors come from six
// rounds in which each row adds what its ancestor so far has seen and goes on to that one's
// (bits of the block, and the last ancestor's parent, which is in an earlier block or none).  Then
// a row's bits in any block are those of the first ancestor that it has there, found by
// going from block to block.  So chains take hardly longer than bushy trees (256 trees of 512 rows: 13.5 us,
// as chains 17; with a thread going from parent to parent for each word 20 and 400).
// Bound: latency.
#include <algorithm>

#include "awq_internal.h"
#include "awq_kv.h"

namespace awq {
namespace {

constexpr int kThreads = 256;

// kHeld: rows that LDS holds (of larger trees the others go from parent to parent): 1024, or 4096 where
// there may be more; workgroups of the first are eight to a CU (256 trees of 512 rows 20 -> 13.5 us).
template <int kHeld>
__global__ void __launch_bounds__(kThreads) tree_rows_kernel(const int32_t *parents, KvView c, uint32_t *mask, int words,
                                                              int32_t *positions) {
    __shared__ uint64_t seen[kHeld];       // of its block's rows
    __shared__ int16_t next[kHeld];        // where its ancestors go on in an earlier block, or -1
    const int b = blockIdx.y, lane = threadIdx.x & 63;
    const int a = min(max(c.q_starts[b], 0), c.rows), n = max(min(max(c.q_starts[b + 1], 0), c.rows) - a, 0);
    const uint32_t items = (uint32_t)n * (uint32_t)words;      // below 2^31
    if (blockIdx.x * kThreads >= items) return;
    const int32_t *up = parents + a;
    const int first = max(c.kv_lens[b], 0) - n, held = min(n, kHeld);
    int ahead = up[min((int)threadIdx.x, n - 1)];
    for (int t0 = threadIdx.x & ~63; t0 < held; t0 += kThreads) {
        const int t = t0 + lane, above = ahead;
        ahead = up[min(t + kThreads, n - 1)];
        int at = above >= 0 && above < t ? above : -1;
        uint64_t bits = 1ull << lane;
#pragma unroll
        for (int k = 0; k < 6; ++k) {
            if (!__any(at >= t0)) break;
            const int from = at >= t0 ? at - t0 : lane;
            const uint64_t other = __shfl(bits, from);
            const int further = __shfl(at, from);
            if (at >= t0) {
                bits |= other;
                at = further;
            }
        }
        if (t < held) {
            seen[t] = bits;
            next[t] = (int16_t)at;
        }
    }
    __syncthreads();
    for (uint32_t i = blockIdx.x * kThreads + threadIdx.x; i < items; i += gridDim.x * kThreads) {
        const int t = (int)(i / (uint32_t)words), w = (int)(i - t * (uint32_t)words);
        uint32_t bits = 0;
        int u = t;
        if (n > kHeld) {
            for (; u >= kHeld && u >> 5 >= w; u = up[u] >= 0 && up[u] < u ? up[u] : -1)
                if (u >> 5 == w) bits |= 1u << (u & 31);
            if (u >= kHeld) u = -1;
        }
        while (u >= 0 && u >> 6 > w >> 1) u = next[u];
        if (u >= 0 && u >> 6 == w >> 1) bits |= (uint32_t)(seen[u] >> (w & 1 ? 32 : 0));
        mask[(long long)(a + t) * words + w] = bits;
        if (w == 0 && positions != nullptr) {
            int depth = -1;
            u = t;
            if (n > kHeld)
                for (; u >= kHeld; u = up[u] >= 0 && up[u] < u ? up[u] : -1) ++depth;
            for (; u >= 0; u = next[u]) depth += __builtin_popcountll(seen[u]);
            positions[a + t] = first + depth;
        }
    }
}

}  // namespace

hipError_t launch_tree_rows(const int32_t *parents, const KvView &c, int max_q, uint32_t *mask, int words, int32_t *positions, hipStream_t s) {
    const long long items = (long long)max_q * words;
    // two words to a thread: with eight, one tree of 512 rows takes 11.9 us for 6.6, 256 of them the same
    // (a launch has less than 2^32 threads; the kernel steps on)
    const long long most = std::min(4096, std::max(1, (1 << 23) / c.seqs));
    const dim3 grid((unsigned)std::min((items + 2 * kThreads - 1) / (2 * kThreads), most), c.seqs);
    if (max_q <= 1024)
        tree_rows_kernel<1024><<<grid, kThreads, 0, s>>>(parents, c, mask, words, positions);
    else
        tree_rows_kernel<4096><<<grid, kThreads, 0, s>>>(parents, c, mask, words, positions);
    return hipGetLastError();
}

}  // namespace awq
