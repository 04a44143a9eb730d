// awq_kv_fork: the page table of the next step out of the present one, and awq_kv_copy: pages
// from one cache to another, or within one.
//
// awq_kv_fork.  The table itself is all the state there is: a page is free if no sequence of
// the new table has it (and the caller does not hold it), and shared if two have it, so two
// bits of each page say what there is to know.  mark_kernel writes the rows that go on and sets the
// bits, give_kernel (one workgroup) numbers the pages that sequences need, in their order, and
// hands out the free ones from the lowest: sums in a fixed order, so the result does not depend on
// when which wave runs.  Bound: latency.
#include <algorithm>

#include "awq_internal.h"
#include "awq_kv.h"

namespace awq {
namespace {

constexpr int kThreads = 256, kGivers = 1024;

struct ForkArgs {
    const int32_t *table, *lens, *from, *grow;
    const uint8_t *held;                       // [pages] or null
    int32_t *table_out, *lens_out, *copies, *missing;
    int seqs, new_seqs, width, log2_page, pages;
    uint32_t *once, *twice;                    // bits of pages in use; in use more than once
    int32_t *offset, *list;                    // [new_seqs]: pages given before a sequence's; free pages
    int room;                                  // of list
};

__global__ void __launch_bounds__(kThreads) clear_kernel(ForkArgs p) {
    const int w = blockIdx.x * kThreads + threadIdx.x;
    if (w >= (p.pages + 31) / 32) return;
    uint32_t bits = 0;
    if (p.held != nullptr)
        for (int k = 0; k < 32 && 32 * w + k < p.pages; ++k) bits |= (p.held[32 * w + k] != 0 ? 1u : 0u) << k;
    p.once[w] = p.twice[w] = bits;
}

// What sequence b goes on with, and what it grows to, in tokens.
struct Growth {
    int from, len, want, have;                 // have: pages that it goes on with
};
__device__ __forceinline__ Growth growth(const ForkArgs &p, int b) {
    Growth g;
    const int cap = p.width << p.log2_page;
    g.from = p.from[b];
    const bool some = g.from >= 0 && g.from < p.seqs;
    if (!some) g.from = -1;
    g.len = some ? min(max(p.lens[g.from], 0), cap) : 0;
    const int more = max(p.grow[b], 0);
    g.want = more < cap - g.len ? g.len + more : cap;
    g.have = (g.len + (1 << p.log2_page) - 1) >> p.log2_page;
    return g;
}

__global__ void __launch_bounds__(kThreads) mark_kernel(ForkArgs p) {
    const int b = blockIdx.y;
    const Growth g = growth(p, b);
    if (blockIdx.x == 0 && threadIdx.x == 0) p.lens_out[b] = g.len;
    for (int j = blockIdx.x * kThreads + threadIdx.x; j < p.width; j += gridDim.x * kThreads) {
        int id = -1;
        if (j < g.have) {
            id = p.table[(long long)g.from * p.width + j];
            if (id < 0 || id >= p.pages) id = -1;
        }
        p.table_out[(long long)b * p.width + j] = id;
        if (id >= 0) {
            const uint32_t bit = 1u << (id & 31);
            if (atomicOr(p.once + id / 32, bit) & bit) atomicOr(p.twice + id / 32, bit);
        }
    }
}

// The sum over the threads before this one, and over all.
__device__ __forceinline__ int before(int x, int &all, int (&sums)[kGivers / 64]) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    int upto = x;
#pragma unroll
    for (int k = 1; k < 64; k <<= 1) {
        const int other = __shfl_up(upto, k);
        upto += lane >= k ? other : 0;
    }
    __syncthreads();                           // sums of the call before are read
    if (lane == 63) sums[wave] = upto;
    __syncthreads();
    int ahead = 0;
    all = 0;
    for (int w = 0; w < kGivers / 64; ++w) {
        ahead += w < wave ? sums[w] : 0;
        all += sums[w];
    }
    return ahead + upto - x;
}

__global__ void __launch_bounds__(kGivers) give_kernel(ForkArgs p) {
    __shared__ int sums[kGivers / 64];
    const int tid = threadIdx.x;
    // pages that each sequence needs: behind its last one, and in place of that if others have it
    int total = 0;
    for (int b0 = 0; b0 < p.new_seqs; b0 += kGivers) {
        const int b = b0 + tid;
        int need = 0;
        bool copy = false;
        if (b < p.new_seqs) {
            const Growth g = growth(p, b);
            need = ((g.want + (1 << p.log2_page) - 1) >> p.log2_page) - g.have;
            if (g.want > g.len && (g.len & ((1 << p.log2_page) - 1)) != 0) {
                const int id = p.table_out[(long long)b * p.width + g.have - 1];
                copy = id >= 0 && (p.twice[id / 32] >> (id & 31) & 1);
            }
            need += copy;
        }
        int all;
        const int at = before(need, all, sums);
        if (b < p.new_seqs) {
            p.offset[b] = total + at;
            p.copies[2 * b] = copy ? 0 : -1;   // (its page comes below)
            p.copies[2 * b + 1] = -1;
        }
        total += all;                          // below 2^31: at most a table
    }
    // the free pages, from the lowest
    const int words = (p.pages + 31) / 32, most = min(total, p.room);
    int found = 0;
    for (int w0 = 0; w0 < words && found < most; w0 += kGivers) {
        const int w = w0 + tid;
        uint32_t open = w < words ? ~p.once[w] : 0u;
        if (w == words - 1 && (p.pages & 31)) open &= (1u << (p.pages & 31)) - 1u;
        int all;
        int at = found + before(__builtin_popcount(open), all, sums);
        for (; open != 0 && at < most; open &= open - 1) p.list[at++] = 32 * w + __builtin_ctz(open);
        found += all;
    }
    __syncthreads();
    // a wave to a sequence
    int lost = 0;
    for (int b = tid >> 6; b < p.new_seqs; b += kGivers / 64) {
        const Growth g = growth(p, b);
        const bool copy = p.copies[2 * b] == 0;
        const int j0 = g.have - copy, need = ((g.want + (1 << p.log2_page) - 1) >> p.log2_page) - j0, at = p.offset[b];
        const bool given = (long long)at + need <= found;
        int32_t *row = p.table_out + (long long)b * p.width + j0;
        if (copy && (tid & 63) == 0) {
            p.copies[2 * b] = given ? row[0] : -1;
            p.copies[2 * b + 1] = given ? p.list[at] : -1;
        }
        for (int i = tid & 63; i < need; i += 64) row[i] = given ? p.list[at + i] : -1;
        lost += given || (tid & 63) ? 0 : need;
    }
    int all;
    before(lost, all, sums);
    if (tid == 0) p.missing[0] = all;
}

// Pages' codes and scales.  A workgroup takes 16 KiB of a page's keys or values.
// Bound: HBM, or the launch.
struct CopyArgs {
    const int32_t *pairs;
    const uint8_t *k, *v;
    uint8_t *ko, *vo;
    const float *ks, *vs;
    float *kso, *vso;
    int from_pages, to_pages, heads;
    long long slab;                            // bytes of a page's keys
};
constexpr int kPiece = 16384;

__global__ void __launch_bounds__(kThreads) copy_kernel(CopyArgs p) {
    const int n = blockIdx.x;
    const int src = p.pairs[2 * n], dst = p.pairs[2 * n + 1];
    if (src < 0 || src >= p.from_pages || dst < 0 || dst >= p.to_pages) return;
    const bool values = blockIdx.z != 0;
    const uint8_t *from = (values ? p.v : p.k) + src * p.slab;
    uint8_t *to = (values ? p.vo : p.ko) + dst * p.slab;
    for (long long at = (long long)blockIdx.y * kPiece + 16 * threadIdx.x; at < p.slab; at += (long long)gridDim.y * kPiece) {
        uint4 r[kPiece / 16 / kThreads];
#pragma unroll
        for (int i = 0; i < kPiece / 16 / kThreads; ++i)
            if (at + 16 * kThreads * i < p.slab) r[i] = *reinterpret_cast<const uint4 *>(from + at + 16 * kThreads * i);
#pragma unroll
        for (int i = 0; i < kPiece / 16 / kThreads; ++i)
            if (at + 16 * kThreads * i < p.slab) *reinterpret_cast<uint4 *>(to + at + 16 * kThreads * i) = r[i];
    }
    if (blockIdx.y == 0)
        for (int h = threadIdx.x; h < p.heads; h += kThreads)
            (values ? p.vso : p.kso)[(long long)dst * p.heads + h] = (values ? p.vs : p.ks)[(long long)src * p.heads + h];
}

long long list_room(int new_seqs, int width, int pages) { return std::min<long long>((long long)new_seqs * width, pages); }

}  // namespace

size_t kv_fork_workspace(int new_seqs, int width, int pages) {
    return 4 * (2 * (((size_t)pages + 31) / 32) + new_seqs + list_room(new_seqs, width, pages));
}

hipError_t launch_kv_fork(const int32_t *from, const int32_t *grow, int new_seqs, const uint8_t *held, const KvView &c,
                          int32_t *table_out, int32_t *lens_out, int32_t *copies, int32_t *missing, void *workspace, hipStream_t s) {
    const int words = (c.pages + 31) / 32;
    uint32_t *once = (uint32_t *)workspace;
    int32_t *offset = (int32_t *)(once + 2 * (size_t)words);
    const ForkArgs p{c.page_table, c.kv_lens, from, grow, held, table_out, lens_out, copies, missing, c.seqs, new_seqs, c.table_width,
                     c.log2_page, c.pages, once, once + words, offset, offset + new_seqs, (int)list_room(new_seqs, c.table_width, c.pages)};
    clear_kernel<<<(words + kThreads - 1) / kThreads, kThreads, 0, s>>>(p);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    mark_kernel<<<dim3(std::min((c.table_width + kThreads - 1) / kThreads, 1024), new_seqs), kThreads, 0, s>>>(p);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
    give_kernel<<<1, kGivers, 0, s>>>(p);
    return hipGetLastError();
}

hipError_t launch_kv_copy(const int32_t *pairs, int n, const KvView &from, const KvView &to, int head_dim, hipStream_t s) {
    const long long slab = (long long)from.kv_heads * head_dim << from.log2_page;
    const CopyArgs p{pairs, from.k, from.v, to.k, to.v, from.k_scales, from.v_scales, to.k_scales, to.v_scales,
                     from.pages, to.pages, from.kv_heads, slab};
    // (a launch has less than 2^32 threads; the kernel steps on)
    const long long pieces = std::min<long long>((slab + kPiece - 1) / kPiece, std::max(1, (1 << 22) / n));
    copy_kernel<<<dim3(n, (unsigned)std::min<long long>(pieces, 65535), 2), kThreads, 0, s>>>(p);
    return hipGetLastError();
}

}  // namespace awq
