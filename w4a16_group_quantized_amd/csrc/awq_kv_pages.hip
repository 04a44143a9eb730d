// awq_kv_fork: the page table of the next step out of the present one, and awq_kv_copy: pages
// from one cache to another, or within one.
//
// awq_kv_fork.  The table itself is all the state there is: a page is free if no sequence of
// the new table has it (and the caller does not hold it), and shared if two have it, so two
// bits of each page say what there is to know.  Rows that go on are written and their bits set;
// then the pages that sequences need are numbered, in the sequences' order, and the free ones handed
// out from the lowest: sums in a fixed order, so the result does not depend on when which wave
// runs.  Bound: latency.
//   fork_kernel does it all in one workgroup, with the bits in LDS, where the table is small.
//   clear_kernel, mark_kernel and give_kernel (one workgroup) do it for any table, with
//   the bits in the workspace.  Either, in us: 64 sequences by 64 places 7.2 / 10.1, by 256 11.1 /
//   12.7, by 512 16.6 / 14.1, by 2048 48.5 / 16.7; 1000 by 32 17.1 / 16.3.
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
    int32_t *offset, *first, *list;            // [new_seqs]: pages given before a sequence's, and its place for them; free pages
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

__device__ __forceinline__ int pages_for(const ForkArgs &p, int tokens) { return (tokens + (1 << p.log2_page) - 1) >> p.log2_page; }

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
    g.have = pages_for(p, g.len);
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

// The last page that a sequence goes on with, if it is to be replaced: it is in part full, to be
// grown into, and shared; else -1.  twice: the bits.
__device__ __forceinline__ int replaced(const ForkArgs &p, const Growth &g, int last, const uint32_t *twice) {
    const bool part = g.want > g.len && (g.len & ((1 << p.log2_page) - 1)) != 0;
    return part && last >= 0 && (twice[last / 32] >> (last & 31) & 1) ? last : -1;
}
// The last of the n ascending numbers that is at most k (the first is).
__device__ __forceinline__ int last_at_most(const int32_t *x, int n, int k) {
    int lo = 0, hi = n - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) / 2;
        if (x[mid] <= k)
            lo = mid;
        else
            hi = mid - 1;
    }
    return lo;
}

__global__ void __launch_bounds__(kGivers) give_kernel(ForkArgs p) {
    __shared__ int sums[kGivers / 64];
    const int tid = threadIdx.x;
    // pages that each sequence needs: behind its last one, and in place of that if others have it
    int total = 0;
    for (int b0 = 0; b0 < p.new_seqs; b0 += kGivers) {
        const int b = b0 + tid;
        int need = 0, last = -1, first = 0;
        if (b < p.new_seqs) {
            const Growth g = growth(p, b);
            last = replaced(p, g, g.have > 0 ? p.table_out[(long long)b * p.width + g.have - 1] : -1, p.twice);
            first = g.have - (last >= 0);
            need = pages_for(p, g.want) - first;
        }
        int all;
        const int at = before(need, all, sums);
        if (b < p.new_seqs) {
            p.offset[b] = total + at;
            p.first[b] = first;
            p.copies[2 * b] = last;            // (if its pages are there: below)
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
    for (int k = tid; k < total; k += kGivers) {
        const int b = last_at_most(p.offset, p.new_seqs, k), all = b + 1 < p.new_seqs ? p.offset[b + 1] : total;
        p.table_out[(long long)b * p.width + p.first[b] + k - p.offset[b]] = all <= found ? p.list[k] : -1;
    }
    int lost = 0;
    for (int b = tid; b < p.new_seqs; b += kGivers) {
        const int at = p.offset[b], all = b + 1 < p.new_seqs ? p.offset[b + 1] : total;
        const bool given = all <= found, copy = given && p.copies[2 * b] >= 0;
        if (!copy) p.copies[2 * b] = -1;
        p.copies[2 * b + 1] = copy ? p.list[at] : -1;
        lost += given ? 0 : all - at;
    }
    int all;
    before(lost, all, sums);
    if (tid == 0) p.missing[0] = all;
}

// Calls that one workgroup takes: sequences, pages and entries of the new table.
constexpr int kSmallSeqs = kGivers, kSmallPages = 1 << 17;
constexpr long long kSmallTable = 20000;

__global__ void __launch_bounds__(kGivers) fork_kernel(ForkArgs p) {
    constexpr int kWords = kSmallPages / 32, kEach = kWords / kGivers;
    __shared__ uint32_t once[kWords], twice[kWords];
    __shared__ int ahead[kWords], sums[kGivers / 64];          // free pages before a word's
    __shared__ int from[kSmallSeqs], have[kSmallSeqs], first[kSmallSeqs], offset[kSmallSeqs];
    const int tid = threadIdx.x, words = (p.pages + 31) / 32;
    Growth g{-1, 0, 0, 0};
    if (tid < p.new_seqs) {
        g = growth(p, tid);
        p.lens_out[tid] = g.len;
        from[tid] = g.from;
        have[tid] = g.have;
    }
    for (int w = tid; w < words; w += kGivers) {
        uint32_t bits = 0;
        if (p.held != nullptr)
            for (int k = 0; k < 32 && 32 * w + k < p.pages; ++k) bits |= (p.held[32 * w + k] != 0 ? 1u : 0u) << k;
        once[w] = twice[w] = bits;
    }
    __syncthreads();
    const int entries = p.new_seqs * p.width;
    for (int i0 = tid; i0 < entries; i0 += 4 * kGivers) {
        int id[4];
#pragma unroll
        for (int n = 0; n < 4; ++n) {
            const int i = min(i0 + n * kGivers, entries - 1), b = i / p.width, j = i - b * p.width;
            id[n] = -1;
            if (j < have[b]) id[n] = p.table[(long long)from[b] * p.width + j];
        }
#pragma unroll
        for (int n = 0; n < 4; ++n) {
            const int i = i0 + n * kGivers;
            if (i >= entries) continue;
            if (id[n] < 0 || id[n] >= p.pages) id[n] = -1;
            p.table_out[i] = id[n];
            if (id[n] >= 0) {
                const uint32_t bit = 1u << (id[n] & 31);
                if (atomicOr(once + id[n] / 32, bit) & bit) atomicOr(twice + id[n] / 32, bit);
            }
        }
    }
    __syncthreads();
    // pages that each sequence needs
    int last = -1, need = 0, total, free;
    if (tid < p.new_seqs && g.have > 0) {
        last = p.table[(long long)g.from * p.width + g.have - 1];
        if (last >= p.pages) last = -1;
    }
    last = replaced(p, g, last, twice);
    if (tid < p.new_seqs) need = pages_for(p, g.want) - g.have + (last >= 0);
    const int at = before(need, total, sums);
    if (tid < p.new_seqs) {
        offset[tid] = at;
        first[tid] = g.have - (last >= 0);
    }
    // the free pages before each word's
    int open[kEach], mine = 0;
#pragma unroll
    for (int n = 0; n < kEach; ++n) {
        const int w = kEach * tid + n;
        uint32_t bits = w < words ? ~once[w] : 0u;
        if (w == words - 1 && (p.pages & 31)) bits &= (1u << (p.pages & 31)) - 1u;
        open[n] = mine;
        mine += __builtin_popcount(bits);
    }
    const int base = before(mine, free, sums);
#pragma unroll
    for (int n = 0; n < kEach; ++n) ahead[kEach * tid + n] = base + open[n];
    __syncthreads();
    // the k-th of them
    const auto page = [&](int k) {
        const int lo = last_at_most(ahead, words, k);
        uint32_t bits = ~once[lo];
        for (int n = k - ahead[lo]; n > 0; --n) bits &= bits - 1;
        return 32 * lo + (int)__builtin_ctz(bits);
    };
    for (int k = tid; k < total; k += kGivers) {
        const int lo = last_at_most(offset, p.new_seqs, k);      // (with none to itself, a sequence is not the last)
        const int all = lo + 1 < p.new_seqs ? offset[lo + 1] : total;
        p.table_out[(long long)lo * p.width + first[lo] + k - offset[lo]] = all <= free ? page(k) : -1;
    }
    const bool given = at + need <= free;
    if (tid < p.new_seqs) {
        const bool copy = last >= 0 && given;
        p.copies[2 * tid] = copy ? last : -1;
        p.copies[2 * tid + 1] = copy ? page(at) : -1;
    }
    int lost;
    before(given ? 0 : need, lost, sums);
    if (tid == 0) p.missing[0] = lost;
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
    typedef uint32_t words_t __attribute__((ext_vector_type(4)));
    constexpr int kStep = 16 * kThreads;
    static_assert(kPiece == 4 * kStep, "four loads on the way");
    for (long long at = (long long)blockIdx.y * kPiece + 16 * threadIdx.x; at < p.slab; at += (long long)gridDim.y * kPiece) {
        // (no condition around the loads, which would be a wait: behind the end the last again)
        const auto load = [&](int i) { return *reinterpret_cast<const words_t *>(from + min(at + i * kStep, p.slab - 16)); };
        const auto store = [&](int i, words_t r) {
            if (at + i * kStep < p.slab) *reinterpret_cast<words_t *>(to + at + i * kStep) = r;
        };
        const words_t r0 = load(0), r1 = load(1), r2 = load(2), r3 = load(3);
        store(0, r0);
        store(1, r1);
        store(2, r2);
        store(3, r3);
    }
    if (blockIdx.y == 0)
        for (int h = threadIdx.x; h < p.heads; h += kThreads)
            (values ? p.vso : p.kso)[(long long)dst * p.heads + h] = (values ? p.vs : p.ks)[(long long)src * p.heads + h];
}

long long list_room(int new_seqs, int width, int pages) { return std::min<long long>((long long)new_seqs * width, pages); }

bool small_fork(int new_seqs, int width, int pages) {
    return new_seqs <= kSmallSeqs && pages <= kSmallPages && (long long)new_seqs * width <= kSmallTable;
}

}  // namespace

size_t kv_fork_workspace(int new_seqs, int width, int pages) {
    if (small_fork(new_seqs, width, pages)) return 0;
    return 4 * (2 * (((size_t)pages + 31) / 32) + 2 * (size_t)new_seqs + list_room(new_seqs, width, pages));
}

hipError_t launch_kv_fork(const int32_t *from, const int32_t *grow, int new_seqs, const uint8_t *held, const KvView &c,
                          int32_t *table_out, int32_t *lens_out, int32_t *copies, int32_t *missing, void *workspace, hipStream_t s) {
    if (small_fork(new_seqs, c.table_width, c.pages)) {
        const ForkArgs p{c.page_table, c.kv_lens, from, grow, held, table_out, lens_out, copies, missing, c.seqs, new_seqs, c.table_width,
                         c.log2_page, c.pages, nullptr, nullptr, nullptr, nullptr, nullptr, 0};
        fork_kernel<<<1, kGivers, 0, s>>>(p);
        return hipGetLastError();
    }
    const int words = (c.pages + 31) / 32;
    uint32_t *once = (uint32_t *)workspace;
    int32_t *offset = (int32_t *)(once + 2 * (size_t)words);
    const ForkArgs p{c.page_table, c.kv_lens, from, grow, held, table_out, lens_out, copies, missing, c.seqs, new_seqs, c.table_width,
                     c.log2_page, c.pages, once, once + words, offset, offset + new_seqs, offset + 2 * new_seqs, (int)list_room(new_seqs, c.table_width, c.pages)};
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
