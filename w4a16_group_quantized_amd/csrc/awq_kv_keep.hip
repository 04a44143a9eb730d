// awq_kv_keep: compaction.  Of a sequence's rows, its last tokens, the kept ones move together,
// in place: token first + i becomes the token that was first + kept[i].
//
//   scale   of a page that tokens come to: the largest of the scales of the pages that its
//           tokens (those that come, and those before them that stay) were in
//   codes   c as it is where the scales are alike, else e4m3_rne(c * (old / new)): scales that are
//           powers of two only shift the exponent, exact but for codes that become subnormal
//
// kept ascends, so a token never moves up: what a place takes lies there or behind it.  So if
// places are taken from the first, what is read for some of them may be read before or after
// earlier ones are written, and must be read before they are.
//
// few_kernel (few kept rows, a matter of latency): one workgroup owns a (sequence, kv head) and
// takes the pages one after the other, each in pieces that are read, then (after a barrier)
// written.
//
// many_kernel: keys, and each element's row of the values, do not meet, so waves share a sequence
// and kv head by pieces of the elements, each through all of its tokens: 16 elements of the keys, or 4
// rows of the values, and all of a block of 256 tokens on the way before the first is written.  A
// value's codes lie side by side by token, so what a block needs of a row is runs of sixteen codes: these
// are loaded, and each lane takes a word's four out of LDS (half of 8 x 8192 tokens: byte after byte
// from HBM 93 us, so 69); where tokens are of more runs than LDS holds, fewer than a quarter or so of
// them, byte by byte.  The scales are what waves share: only the codes move, and a second launch
// goes over the scales alone.
//
// Nobody else writes a sequence's slabs or scales: the same bits each time.
// Bound: latency of a block (kept, page, scales, codes: four loads in a row), blocks one after the other.
// Half of 8 x 8192 tokens of 8 heads of 128: codes 52 us, scales 7.6, 61 in a graph (2.2 TB/s) and 71 called one after
// the other (1.9); 25 of them without any codes' loads and stores; asking for a block's codes before the last
// block's are written: 65 in a graph.
#include <algorithm>

#include "awq_internal.h"
#include "awq_kv.h"

namespace awq {
namespace {

constexpr int kFewThreads = 256, kMaxPage = 256, kAtOnce = 4;
constexpr int kThreads = 256, kScaleThreads = 1024;
constexpr int kBlock = 256;                // tokens on the way: whole pages; of the scales' launch
constexpr int kScaleBlock = 2048;
constexpr int kLeastPage = 16;
constexpr int kKeyWidth = 16, kRows = 4;   // elements of a piece of the keys; rows of a piece of the values
constexpr int kRuns = 64;                  // runs of sixteen slots that a block's tokens may come from, for LDS to hold them
constexpr int kStays = -2;

struct KeepArgs {
    KvView c;
    const int32_t *kept, *counts;
    int32_t *lens_out;
    int width;
};

// Four codes under another scale: times f, which is at most 1.
__device__ __forceinline__ uint32_t rescaled(uint32_t w, float f) {
    if (f == 1.0f) return w;
    float x[4];
    from_e4m3x4(w, x);
    return to_e4m3x4(x[0] * f, x[1] * f, x[2] * f, x[3] * f);
}

template <int D>
__global__ void __launch_bounds__(kFewThreads) few_kernel(KeepArgs p) {
    constexpr int U = D / 16;                  // 16-byte pieces of a key
    __shared__ int m_s, id_s[kMaxPage], slot_s[kMaxPage];
    __shared__ float fk_s[kMaxPage], fv_s[kMaxPage], red[2][kFewThreads / 64];
    const KvView &c = p.c;
    const int tid = threadIdx.x, h = blockIdx.x, b = blockIdx.y;
    const Seq s = load_seq(c, b);
    const int P = 1 << c.log2_page, first = s.first();
    const int32_t *kept = p.kept + (long long)b * p.width;
    const int32_t *table = c.page_table + (long long)b * c.table_width;
    // the kept rows: up to the first that is not behind the one before it, or is none
    const int most = first < 0 ? 0 : min(max(p.counts[b], 0), min(s.n, p.width));
    if (tid == 0) m_s = most;
    __syncthreads();
    for (int i = tid; i < most; i += kFewThreads) {
        const int k = kept[i];
        if (k <= (i > 0 ? kept[i - 1] : -1) || k >= s.n) atomicMin(&m_s, i);
    }
    __syncthreads();
    const int m = m_s;
    if (h == 0 && tid == 0) p.lens_out[b] = first < 0 ? s.len : first + m;
    const long long slab = (long long)P * D;
    for (int j = first >> c.log2_page; (j << c.log2_page) < first + m; ++j) {
        const int base = j << c.log2_page, lo = max(first, base), hi = min(first + m, base + P);
        const int count = hi - lo, held = lo - base, i0 = lo - first;
        if (count <= 0 || kept[i0 + count - 1] == i0 + count - 1) continue;        // all are where they belong
        const int id = table[j];
        if (id < 0 || id >= c.pages) continue;                                      // names no page: nothing comes
        const long long ph = (long long)id * c.kv_heads + h;
        const float ks0 = c.k_scales[ph], vs0 = c.v_scales[ph];
        // by slot of the page: where its token comes from, and the scales there
        float ka = held > 0 ? ks0 : 0.0f, va = held > 0 ? vs0 : 0.0f;
        float ks_own = 0.0f, vs_own = 0.0f;
        if (tid < held + count) {
            const int tok = tid < held ? base + tid : first + kept[i0 + tid - held];
            int from = table[tok >> c.log2_page];
            if (from < 0 || from >= c.pages) from = -1;
            id_s[tid] = from;
            slot_s[tid] = tok & (P - 1);
            if (from >= 0) {
                ks_own = c.k_scales[(long long)from * c.kv_heads + h];
                vs_own = c.v_scales[(long long)from * c.kv_heads + h];
                ka = fmaxf(ka, ks_own);
                va = fmaxf(va, vs_own);
            }
        }
        for (int k = 32; k > 0; k >>= 1) {
            ka = fmaxf(ka, __shfl_xor(ka, k));
            va = fmaxf(va, __shfl_xor(va, k));
        }
        if ((tid & 63) == 0) {
            red[0][tid >> 6] = ka;
            red[1][tid >> 6] = va;
        }
        __syncthreads();
        ka = fmaxf(fmaxf(red[0][0], red[0][1]), fmaxf(red[0][2], red[0][3]));
        va = fmaxf(fmaxf(red[1][0], red[1][1]), fmaxf(red[1][2], red[1][3]));
        if (tid < held + count) {
            fk_s[tid] = ks_own == ka ? 1.0f : ks_own / ka;
            fv_s[tid] = vs_own == va ? 1.0f : vs_own / va;
        }
        __syncthreads();
        if (tid == 0 && ka > 0.0f) {           // (none: no token has a page)
            c.k_scales[ph] = ka;
            c.v_scales[ph] = va;
        }
        uint8_t *kslab = c.k + ph * slab, *vslab = c.v + ph * slab;
        // tokens that stay
        if (held > 0 && ka != ks0) {
            const float f = ks0 / ka;
            for (int i = tid; i < held * (D / 4); i += kFewThreads) {
                uint32_t *w = reinterpret_cast<uint32_t *>(kslab) + i;
                *w = rescaled(*w, f);
            }
        }
        const int w0 = held >> 2, w1 = (held + count + 3) >> 2, words = w1 - w0;
        if (w0 > 0 && va != vs0) {
            const float f = vs0 / va;
            for (int i = tid; i < w0 * D; i += kFewThreads) {
                uint32_t *w = reinterpret_cast<uint32_t *>(vslab + (i / w0) * P) + i % w0;
                *w = rescaled(*w, f);
            }
        }
        // keys that come, token after token
        for (int x0 = 0; x0 < count * U; x0 += kAtOnce * kFewThreads) {
            uint4 r[kAtOnce];
#pragma unroll
            for (int n = 0; n < kAtOnce; ++n) {
                const int x = x0 + n * kFewThreads + tid, t = held + x / U;
                if (x >= count * U) continue;
                const int from = id_s[t];
                r[n] = make_uint4(0x7F7F7F7Fu, 0x7F7F7F7Fu, 0x7F7F7F7Fu, 0x7F7F7F7Fu);
                if (from >= 0) {
                    const float f = fk_s[t];
                    const uint4 u = *reinterpret_cast<const uint4 *>(c.k + ((long long)from * c.kv_heads + h) * slab + slot_s[t] * D + 16 * (x % U));
                    r[n] = make_uint4(rescaled(u.x, f), rescaled(u.y, f), rescaled(u.z, f), rescaled(u.w, f));
                }
            }
            __syncthreads();
#pragma unroll
            for (int n = 0; n < kAtOnce; ++n) {
                const int x = x0 + n * kFewThreads + tid;
                if (x < count * U) *reinterpret_cast<uint4 *>(kslab + (held + x / U) * D + 16 * (x % U)) = r[n];
            }
        }
        // values, element after element: four slots to a word
        for (int x0 = 0; x0 < words * D; x0 += kAtOnce * kFewThreads) {
            uint32_t r[kAtOnce];
#pragma unroll
            for (int n = 0; n < kAtOnce; ++n) {
                const int x = x0 + n * kFewThreads + tid, d = x / words, w = w0 + x % words;
                if (x >= words * D) continue;
                uint32_t now = held + count < 4 * w + 4 ? reinterpret_cast<const uint32_t *>(vslab + d * P)[w] : 0u;     // (slots behind stay)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int t = 4 * w + e;
                    if (t >= held + count) continue;
                    const int from = id_s[t];
                    const uint32_t code = from < 0 ? 0u : c.v[((long long)from * c.kv_heads + h) * slab + d * P + slot_s[t]];
                    now = (now & ~(0xFFu << (8 * e))) | (rescaled(code, fv_s[t]) & 0xFFu) << (8 * e);
                }
                r[n] = now;
            }
            __syncthreads();
#pragma unroll
            for (int n = 0; n < kAtOnce; ++n) {
                const int x = x0 + n * kFewThreads + tid;
                if (x < words * D) reinterpret_cast<uint32_t *>(vslab + (x / words) * P)[w0 + x % words] = r[n];
            }
        }
        __syncthreads();                       // what the page's tokens came from is read no more
    }
}

// Four rows' codes, one byte of each in a lane, as words of four lanes' bytes: lane 4 i + e gets
// row e's word of the lanes 4 i .. 4 i + 3.
__device__ __forceinline__ uint32_t words_of(const uint32_t (&r)[4]) {
    const int at = threadIdx.x & 3;
    uint32_t out = 0;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        int x = (int)(r[e] << (8 * at));
        x |= __builtin_amdgcn_mov_dpp(x, 0xB1, 0xF, 0xF, false);       // lanes 1, 0, 3, 2
        x |= __builtin_amdgcn_mov_dpp(x, 0x4E, 0xF, 0xF, false);       // lanes 2, 3, 0, 1
        out = at == e ? (uint32_t)x : out;
    }
    return out;
}

// The largest of sixteen lanes' numbers, none below 0.
__device__ __forceinline__ float most_of_16(float x) {
    int y = __builtin_bit_cast(int, x);
    y = max(y, __builtin_amdgcn_update_dpp(y, y, 0x128, 0xF, 0xF, false));     // eight lanes on, of sixteen
    y = max(y, __builtin_amdgcn_update_dpp(y, y, 0x124, 0xF, 0xF, false));     // four
    y = max(y, __builtin_amdgcn_update_dpp(y, y, 0x122, 0xF, 0xF, false));
    y = max(y, __builtin_amdgcn_update_dpp(y, y, 0x121, 0xF, 0xF, false));
    return __builtin_bit_cast(float, y);
}

// All waves' reads and writes of LDS are done; those of HBM go on.
__device__ __forceinline__ void lds_barrier() {
    __builtin_amdgcn_s_waitcnt(0xC07F);
    asm volatile("s_barrier" ::: "memory");
}

constexpr int pieces_of(int head_dim) { return head_dim / kKeyWidth + head_dim / kRows; }

// SCALES: only these, and the lengths; otherwise only the codes, a piece to a wave: gridDim.y
// workgroups share a sequence and kv head.
template <int D, int kThreads, int kBlock, bool SCALES>
__global__ void __launch_bounds__(kThreads, SCALES ? 4 : 3) many_kernel(KeepArgs p) {
    constexpr int kWaves = kThreads / 64;
    constexpr int kGroups = kBlock / 64, kEach = kBlock / kThreads, kPages = kBlock / kLeastPage;
    // by place in the block: the page that its token comes from (-1: none, kStays: nothing is written),
    // the slot there, what its codes are multiplied by
    __shared__ __align__(16) int from[kBlock];
    __shared__ int slot[kBlock], to[2][kPages], limits[2];
    __shared__ __align__(16) float fk[kBlock], fv[kBlock];
    // runs of sixteen slots that tokens come from: number of a group's, page, first slot, the values' codes;
    // and where in these a token's are
    __shared__ int runs[kGroups], run_page[kRuns], run_slot[kRuns];
    __shared__ __align__(8) uint16_t code_at[kBlock];
    __shared__ uint4 codes[kWaves][kRows][kRuns];
    __shared__ uint32_t most[2][2][kPages];    // scales as bits (they are positive)
    // (most and to, of this block and the next, which a wave may begin while others are at this one)
    const KvView &c = p.c;
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int h = blockIdx.x % c.kv_heads, b = blockIdx.x / c.kv_heads;
    const Seq s = load_seq(c, b);
    const int lp = c.log2_page, P = 1 << lp, first = s.first();
    const int32_t *kept = p.kept + (long long)b * p.width;
    const int32_t *table = c.page_table + (long long)b * c.table_width;
    // the kept rows: up to the first that is not behind the one before it, or is none; and from
    // where on they are not in place
    const int listed = first < 0 ? 0 : min(max(p.counts[b], 0), min(s.n, p.width));
    if (tid < 2) limits[tid] = listed;
    if (tid < 2 * kPages) most[0][tid / kPages][tid % kPages] = 0u;
    __syncthreads();
    int bad = listed, moved = listed;
    for (int i0 = tid; i0 < listed; i0 += 8 * kThreads) {
        int k[8], last[8];                     // (all on the way at once)
#pragma unroll
        for (int n = 0; n < 8; ++n) {
            const int i = min(i0 + n * kThreads, listed - 1);
            k[n] = kept[i];
            last[n] = kept[max(i - 1, 0)];
        }
#pragma unroll
        for (int n = 0; n < 8; ++n) {
            const int i = min(i0 + n * kThreads, listed - 1);
            if (k[n] <= (i > 0 ? last[n] : -1) || k[n] >= s.n) bad = min(bad, i);
            if (k[n] != i) moved = min(moved, i);
        }
    }
    for (int k = 32; k > 0; k >>= 1) {
        bad = min(bad, __shfl_xor(bad, k));
        moved = min(moved, __shfl_xor(moved, k));
    }
    if (lane == 0) {
        atomicMin(&limits[0], bad);
        atomicMin(&limits[1], moved);
    }
    __syncthreads();
    const int m = limits[0], end = first + m, begin = first + limits[1];
    if (SCALES && h == 0 && tid == 0) p.lens_out[b] = first < 0 ? s.len : end;
    if (begin >= end) return;
    const long long slab = (long long)P * D;
    const int start = begin >> lp << lp;

    // A block's tokens, their pages and these pages' scales are asked for three, two and one block
    // ahead: each is found by the one before.  (What is loaded is looked at when it is used, and
    // loads have no conditions around them: either would be a wait.)
    int tok1[kEach], tok2[kEach], tok3[kEach], id1[kEach], id2[kEach], own1, own2;
    float ks1[kEach], vs1[kEach];
    const auto ask_tokens = [&](int base, int (&row)[kEach]) {
#pragma unroll
        for (int n = 0; n < kEach; ++n) row[n] = kept[min(max(base + n * kThreads + tid - first, 0), m - 1)];
    };
    const auto token = [&](int base, int n, int row) {     // of a place; -1: it has none
        const int place = base + n * kThreads + tid;
        return place >= end ? -1 : place < first ? place : first + row;
    };
    const auto ask_pages = [&](int base, const int (&row)[kEach], int (&id)[kEach], int &own) {
#pragma unroll
        for (int n = 0; n < kEach; ++n) id[n] = table[max(token(base, n, row[n]), 0) >> lp];
        own = table[min(base + (tid << lp), end - 1) >> lp];
    };
    const auto page = [&](int base, int n, int row, int id) { return token(base, n, row) >= 0 && id >= 0 && id < c.pages ? id : -1; };
    const auto ask_scales = [&](int base, const int (&row)[kEach], const int (&id)[kEach], float (&ks)[kEach], float (&vs)[kEach]) {
#pragma unroll
        for (int n = 0; n < kEach; ++n) {
            const long long at = (long long)max(page(base, n, row[n], id[n]), 0) * c.kv_heads + h;
            ks[n] = c.k_scales[at];
            vs[n] = c.v_scales[at];
        }
    };
    ask_tokens(start, tok1);
    ask_tokens(start + kBlock, tok2);
    ask_tokens(start + 2 * kBlock, tok3);
    ask_pages(start, tok1, id1, own1);
    ask_pages(start + kBlock, tok2, id2, own2);
    ask_scales(start, tok1, id1, ks1, vs1);
    for (int base = start, odd = 0; base < end; base += kBlock, odd ^= 1) {
        // the largest scales of each page's tokens, sixteen of them to an atomic
        uint64_t begins[kEach] = {};           // lanes whose token is the first of a run
        int all_runs = 0;
#pragma unroll
        for (int n = 0; n < kEach; ++n) {
            const int id = page(base, n, tok1[n], id1[n]);
            ks1[n] = id < 0 ? 0.0f : ks1[n];
            vs1[n] = id < 0 ? 0.0f : vs1[n];
            id1[n] = id;
            const float ka = most_of_16(ks1[n]), va = most_of_16(vs1[n]);
            const int x = n * kThreads + tid;
            if constexpr (!SCALES) {
                const int run = token(base, n, tok1[n]) >> 4, last = __shfl_up(run, 1);
                begins[n] = __ballot(run >= 0 && (lane == 0 || last != run));
                if (lane == 0) runs[n * kWaves + wave] = __builtin_popcountll(begins[n]);
            }
            if ((lane & 15) == 0) {
                atomicMax(&most[odd][0][x >> lp], __builtin_bit_cast(uint32_t, ka));
                atomicMax(&most[odd][1][x >> lp], __builtin_bit_cast(uint32_t, va));
            }
        }
        if (tid < kBlock >> lp) to[odd][tid] = base + (tid << lp) >= end || own1 < 0 || own1 >= c.pages ? -1 : own1;
        lds_barrier();                       // (and every wave is done with the block before)
        if (tid < 2 * kPages) most[odd ^ 1][tid / kPages][tid % kPages] = 0u;
        if constexpr (!SCALES) {
#pragma unroll
            for (int n = 0; n < kEach; ++n) {
                const int x = n * kThreads + tid, place = base + x, tok = token(base, n, tok1[n]);
                const float ka = __builtin_bit_cast(float, most[odd][0][x >> lp]), va = __builtin_bit_cast(float, most[odd][1][x >> lp]);
                const float a = ks1[n] == ka ? 1.0f : ks1[n] / ka, v = vs1[n] == va ? 1.0f : vs1[n] / va;
                const bool stays = tok < 0 || to[odd][x >> lp] < 0 || (tok == place && a == 1.0f && v == 1.0f);
                from[x] = stays ? kStays : id1[n];
                slot[x] = tok & (P - 1);
                fk[x] = a;
                fv[x] = v;
                // (the sum of the runs of all groups in all_runs)
                int run = __builtin_popcountll(begins[n] & (2ull << lane) - 1) - 1;
                all_runs = 0;
#pragma unroll
                for (int g = 0; g < kGroups; ++g) {
                    run += g < n * kWaves + wave ? runs[g] : 0;
                    all_runs += runs[g];
                }
                code_at[x] = (uint16_t)(16 * max(run, 0) + (tok & 15));
                if ((begins[n] >> lane & 1) && run < kRuns) {
                    run_page[run] = max(id1[n], 0);
                    run_slot[run] = tok & (P - 1) & ~15;
                }
            }
            lds_barrier();
        }
#pragma unroll
        for (int n = 0; n < kEach; ++n) {
            tok1[n] = tok2[n];
            tok2[n] = tok3[n];
            id1[n] = id2[n];
        }
        own1 = own2;
        ask_scales(base + kBlock, tok1, id1, ks1, vs1);
        ask_pages(base + 2 * kBlock, tok2, id2, own2);
        ask_tokens(base + 3 * kBlock, tok3);
        if constexpr (SCALES) {
            // (later blocks' are of later pages)
            if (tid < kBlock >> lp && to[odd][tid] >= 0 && most[odd][0][tid] != 0u) {
                c.k_scales[(long long)to[odd][tid] * c.kv_heads + h] = __builtin_bit_cast(float, most[odd][0][tid]);
                c.v_scales[(long long)to[odd][tid] * c.kv_heads + h] = __builtin_bit_cast(float, most[odd][1][tid]);
            }
            lds_barrier();
            continue;
        }
        const int piece = blockIdx.y * kWaves + wave;
        if (piece >= pieces_of(D)) continue;
        if (piece < D / kKeyWidth) {
            const int at = piece * kKeyWidth;
            uint4 r[kGroups];
#pragma unroll
            for (int n = 0; n < kGroups; ++n) {
                const int x = 64 * n + lane;
                r[n] = *reinterpret_cast<const uint4 *>(c.k + ((long long)max(from[x], 0) * c.kv_heads + h) * slab + slot[x] * D + at);
            }
#pragma unroll
            for (int n = 0; n < kGroups; ++n) {
                const int x = 64 * n + lane, id = from[x];
                if (id != kStays) {
                    const float f = fk[x];
                    const uint32_t none = 0x7F7F7F7Fu;
                    *reinterpret_cast<uint4 *>(c.k + ((long long)to[odd][x >> lp] * c.kv_heads + h) * slab + (x & (P - 1)) * D + at) =
                        id < 0 ? make_uint4(none, none, none, none)
                               : make_uint4(rescaled(r[n].x, f), rescaled(r[n].y, f), rescaled(r[n].z, f), rescaled(r[n].w, f));
                }
            }
        } else if (all_runs <= kRuns) {
            // The runs' codes to LDS, from which a lane takes the four of a word.
            const int d = (piece - D / kKeyWidth) * kRows;
            uint4 r[kRuns / 64][kRows];
#pragma unroll
            for (int n = 0; n < kRuns / 64; ++n) {
                const int run = min(64 * n + lane, all_runs - 1);
                const uint8_t *v = c.v + ((long long)run_page[run] * c.kv_heads + h) * slab + d * P + run_slot[run];
#pragma unroll
                for (int e = 0; e < kRows; ++e) r[n][e] = *reinterpret_cast<const uint4 *>(v + e * P);
            }
#pragma unroll
            for (int n = 0; n < kRuns / 64; ++n)
#pragma unroll
                for (int e = 0; e < kRows; ++e) codes[wave][e][64 * n + lane] = r[n][e];
            __builtin_amdgcn_wave_barrier();
#pragma unroll
            for (int n = 0; n < kBlock / 256; ++n) {
                const int x = 256 * n + 4 * lane;
                const int4 id = *reinterpret_cast<const int4 *>(from + x);
                const float4 f = *reinterpret_cast<const float4 *>(fv + x);
                const ushort4 at = *reinterpret_cast<const ushort4 *>(code_at + x);
                const bool put[4] = {id.x != kStays, id.y != kStays, id.z != kStays, id.w != kStays};
                const uint32_t same = (f.x == 1.0f ? 0xFFu : 0u) | (f.y == 1.0f ? 0xFF00u : 0u) | (f.z == 1.0f ? 0xFF0000u : 0u) | (f.w == 1.0f ? 0xFF000000u : 0u);
                const uint32_t live = (id.x < 0 ? 0u : 0xFFu) | (id.y < 0 ? 0u : 0xFF00u) | (id.z < 0 ? 0u : 0xFF0000u) | (id.w < 0 ? 0u : 0xFF000000u);
                uint8_t *v = c.v + ((long long)to[odd][x >> lp] * c.kv_heads + h) * slab + d * P + (x & (P - 1));
                const uint8_t *bytes = reinterpret_cast<const uint8_t *>(codes[wave]);
#pragma unroll
                for (int e = 0; e < kRows; ++e) {
                    const uint8_t *row = bytes + e * 16 * kRuns;
                    uint32_t w = row[at.x] | row[at.y] << 8 | row[at.z] << 16 | (uint32_t)row[at.w] << 24;
                    if (same != 0xFFFFFFFFu) {
                        float y[4];
                        from_e4m3x4(w, y);
                        w = (w & same) | (to_e4m3x4(y[0] * f.x, y[1] * f.y, y[2] * f.z, y[3] * f.w) & ~same);
                    }
                    w &= live;
                    if (put[0] & put[1] & put[2] & put[3]) {
                        *reinterpret_cast<uint32_t *>(v + e * P) = w;
                    } else {
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            if (put[k]) v[e * P + k] = (uint8_t)(w >> (8 * k));
                    }
                }
            }
            __builtin_amdgcn_wave_barrier();
        } else {
            const int d = (piece - D / kKeyWidth) * kRows;
            uint32_t r[kGroups][kRows];
#pragma unroll
            for (int n = 0; n < kGroups; ++n) {
                const int x = 64 * n + lane;
                const uint8_t *v = c.v + ((long long)max(from[x], 0) * c.kv_heads + h) * slab + d * P + slot[x];
#pragma unroll
                for (int e = 0; e < kRows; ++e) r[n][e] = v[e * P];
            }
#pragma unroll
            for (int n = 0; n < kGroups; ++n) {
                const int x = 64 * n + lane, id = from[x];
                const bool put = id != kStays;
                const float f = fv[x];
                uint8_t *v = c.v + ((long long)to[odd][x >> lp] * c.kv_heads + h) * slab + d * P + (x & (P - 1));
#pragma unroll
                for (int e = 0; e < kRows; ++e) r[n][e] = id < 0 ? 0u : rescaled(r[n][e], f) & 0xFFu;
                // four places to a word, where all four are written (pages are of whole words)
                const uint32_t four = (uint32_t)(__ballot(put) >> (lane & ~3)) & 15u;
                const uint32_t w = words_of(r[n]);
                if (four == 15u) {
                    *reinterpret_cast<uint32_t *>(v - (lane & 3) + (lane & 3) * P) = w;
                } else if (put) {
#pragma unroll
                    for (int e = 0; e < kRows; ++e) v[e * P] = (uint8_t)r[n][e];
                }
            }
        }
    }
}

// Kept rows of a sequence from which many waves share it (half of 8 x 8192 tokens of 8 heads 845 -> 61 us;
// 4 of 16 rows of 32 sequences 9.9 / 7.6), and the sequences times heads up to which its launch, of
// up to 20 workgroups for each, has less than 2^32 threads.
constexpr int kMany = 64, kManyPairs = 1 << 19;

template <int D>
void launch(const KeepArgs &p, hipStream_t s) {
    const int pairs = p.c.kv_heads * p.c.seqs;
    if (p.width <= kMany || pairs > kManyPairs) {
        few_kernel<D><<<dim3(p.c.kv_heads, p.c.seqs), kFewThreads, 0, s>>>(p);
        return;
    }
    constexpr int kWaves = kThreads / 64;
    many_kernel<D, kThreads, kBlock, false><<<dim3(pairs, (pieces_of(D) + kWaves - 1) / kWaves), kThreads, 0, s>>>(p);
    many_kernel<D, kScaleThreads, kScaleBlock, true><<<pairs, kScaleThreads, 0, s>>>(p);
}

}  // namespace

hipError_t launch_kv_keep(const KvView &c, int head_dim, const int32_t *kept, int width, const int32_t *counts, int32_t *lens_out, hipStream_t s) {
    const KeepArgs p{c, kept, counts, lens_out, width};
    switch (head_dim) {
    case 64: launch<64>(p, s); break;
    case 128: launch<128>(p, s); break;
    case 256: launch<256>(p, s); break;
    default: return hipErrorInvalidValue;
    }
    return hipGetLastError();
}

}  // namespace awq
