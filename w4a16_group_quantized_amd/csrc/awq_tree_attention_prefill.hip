// awq_tree_attention for many rows: see awq_attention_split.h for the formula and the transposed
// products, and awq_attention_prefill.hip for the tiles in LDS and how keys are dealt to the
// products; the arithmetic of a row is the same here, weights of two halves in it.
//
// What differs: all rows of a tree see the same tiles of keys, so workgroups go over several row tiles,
// in equal shares of all the work (TreeShare); and which of a tile's keys a row sees is bits, from the
// mask's words, needed for the tiles at the tree (and at a window's border) alone.
//
// Bound: vector and matrix instructions, one after the other: 390 or so of a wave for 32 rows by 64 keys of 128
// elements beside 48 products, which hold the vector port up for 11 cycles each.  16 trees of up to 64 rows
// over up to 8191 keys, 32 heads on 8: 170 to 187 us (74 at the rate of a large matrix product); one of 48 rows, 64
// heads on 8, over 131000 keys: 318 to 343 us (172).  Eight waves in two groups, one at its products
// while the other is at its weights: 279 us where this took 257 (16 trees of 64 rows over 8192 keys, then).
#include <algorithm>

#include "awq_attention.h"
#include "awq_internal.h"
#include "awq_tree_share.h"

namespace awq {
namespace {

constexpr int kWaveRows = 32;
// Least tiles of a chunk and of a workgroup's share; most chunks of a row tile.
constexpr int kLeastChunk = 6, kLeastShare = 8, kMostSplits = 32;
constexpr int kTreeWaves = 2048, kManyTreeTiles = 2048;                // waves that the GPU holds; row tiles from which keys are not cut
constexpr float kWeightBits = 11.0f, kSlack = 4.0f;

constexpr bool in_pairs(int head_dim) { return head_dim > 128; }
constexpr int rows_of(int head_dim, int waves) { return kWaveRows * (in_pairs(head_dim) ? waves / 2 : waves); }
// Waves of a workgroup: four share a tile's keys and values, or two where that leaves fewer rows of
// the longest sequence's row tiles empty (which four, in the same time, make up for where these are a
// fifth): 16 trees over 8k keys, four / two: 64 rows times heads 127 / 97 us, 160 211 / 196, 256 240 / 264.
int waves_of(int head_dim, long long rows) {
    return !in_pairs(head_dim) && 6 * ((rows + 63) / 64 * 64) < 5 * ((rows + 127) / 128 * 128) ? 2 : 4;
}

// Drafted trees: how workgroups share the work of a kv head.  All rows of a tree see the same
// tiles of keys, so the work is a line of units, a row tile's tile of keys each: row tiles one after
// the other, with all of their tiles.  Workgroup k takes the units [k each, (k + 1) each), so
// that all take the same time, whatever the lengths of the sequences: a part of a row tile's keys, or all
// of some, or both.  A border less than kLeastChunk tiles from the border of a row tile moves there.
// 16 trees of 32 to 64 rows over 4k to 8k keys: a grid over sequences, row tiles and chunks 211 us, this 199.  Units are of
// 2^shift tiles, so that there are no more than 2^30.
struct TreeShare {
    int seq, row_tile, start, count, chunk, chunks;    // a piece: tiles start .. start + count - 1
    int number, at, end, each, shift;
    // of the lane's one of the first 64 sequences
    Seq own;
    int own_upto, own_units;

    // A row tile of the line: its sequence, number there, first unit and units.
    struct RowTile {
        int seq, number, first, units;
    };
    // Row tiles of a sequence, and the tiles of keys that each sees.
    static __device__ __forceinline__ int row_tiles(const AttnArgs &p, int rows, int b, int &tiles) {
        Seq s;
        return row_tiles(p, rows, b, tiles, s);
    }
    static __device__ __forceinline__ int row_tiles(const AttnArgs &p, int rows, int b, int &tiles, Seq &s) {
        tiles = 0;
        s = Seq{};
        if (b >= p.c.seqs) return 0;
        s = load_seq(p.c, b);
        const int total = s.n * p.group;
        if (total == 0 || total < p.few) return 0;
        tiles = max(1, visible_tiles(p, first_place<true>(s, 0), s.len - 1, s.len).count());
        return (total + rows - 1) / rows;
    }
    __device__ __forceinline__ int units_of(int tiles) const { return (tiles + (1 << shift) - 1) >> shift; }
    static __device__ __forceinline__ int sum_up(int x) {
        const int lane = threadIdx.x & 63;
#pragma unroll
        for (int k = 1; k < 64; k <<= 1) {
            const int other = __shfl_up(x, k);
            x += lane >= k ? other : 0;
        }
        return x;
    }
    // The lane's one of 64 sequences: the units up to it, and those of its row tiles each.
    struct Lane {
        int upto, units;
    };
    __device__ __forceinline__ Lane lane_of(int n, int tiles) const { return {sum_up(n * units_of(tiles)), units_of(tiles)}; }
    __device__ __forceinline__ Lane lane_from(const AttnArgs &p, int rows, int from) const {
        int tiles;
        const int n = row_tiles(p, rows, from + (int)(threadIdx.x & 63), tiles);
        return lane_of(n, tiles);
    }
    // The row tile that unit u (there is one) is in; l: of the first 64 sequences.
    __device__ __forceinline__ RowTile find(const AttnArgs &p, int rows, Lane l, int u) const {
        int before = 0, from = 0;
        while (u >= before + __builtin_amdgcn_readlane(l.upto, 63)) {
            before += __builtin_amdgcn_readlane(l.upto, 63);
            from += 64;
            l = lane_from(p, rows, from);
        }
        const int at_lane = (int)__builtin_ctzll(__ballot(before + l.upto > u));
        RowTile r;
        r.seq = from + at_lane;
        r.units = __builtin_amdgcn_readlane(l.units, at_lane);
        const int start_of = before + (at_lane > 0 ? __builtin_amdgcn_readlane(l.upto, at_lane > 0 ? at_lane - 1 : 0) : 0);
        r.number = __builtin_amdgcn_readfirstlane((uint32_t)(u - start_of) / (uint32_t)r.units);
        r.first = start_of + r.number * r.units;
        return r;
    }
    // (in units) how near a border may be to that of a row tile
    __device__ __forceinline__ int least(const AttnArgs &p, int all) const { return p.splits > 1 ? units_of(kLeastChunk) : all; }
    __device__ __forceinline__ int border(const AttnArgs &p, int rows, const Lane &l, int u, int all) const {
        if (u >= all) return all;
        const RowTile r = find(p, rows, l, u);
        const int far = least(p, r.units);
        return u - r.first < far ? r.first : r.first + r.units - u < far ? r.first + r.units : u;
    }
    __device__ __forceinline__ void begin(const AttnArgs &p, int rows, int k) {
        const int lane = threadIdx.x & 63;
        number = k;
        int tiles, most;
        const int n = row_tiles(p, rows, lane, tiles, own);
        most = tiles;
        float about = (float)n * (float)tiles;
        for (int from = 64; from < p.c.seqs; from += 64) {
            int other;
            const int m = row_tiles(p, rows, from + lane, other);
            most = max(most, other);
            about += (float)m * (float)other;
        }
#pragma unroll
        for (int i = 32; i > 0; i >>= 1) {
            about += __shfl_xor(about, i);
            most = max(most, __shfl_xor(most, i));
        }
        // (rounding tiles up to units at most doubles what is no more than 2^29)
        shift = __builtin_amdgcn_readfirstlane(max((int)(__builtin_bit_cast(uint32_t, about) >> 23) - 127 - 28, 0));
        const Lane l = lane_of(n, tiles);
        own_upto = l.upto;
        own_units = l.units;
        int all = __builtin_amdgcn_readlane(l.upto, 63);
        for (int from = 64; from < p.c.seqs; from += 64) {
            int other;
            const int m = row_tiles(p, rows, from + lane, other);
            all += __builtin_amdgcn_readlane(sum_up(m * units_of(other)), 63);
        }
        // a row tile has room for p.splits chunks
        each = __builtin_amdgcn_readfirstlane(share_units(all, p.most, units_of(kLeastShare), units_of(most), p.splits));
        at = __builtin_amdgcn_readfirstlane(border(p, rows, l, share_border(k, each, all), all));
        end = __builtin_amdgcn_readfirstlane(border(p, rows, l, share_border(k + 1, each, all), all));
    }
    // (What is not used while tiles are multiplied is kept in vector registers meanwhile, where there are some.)
    __device__ __forceinline__ void keep() {
        asm volatile("" : "+v"(at), "+v"(end), "+v"(each), "+v"(number), "+v"(shift), "+v"(chunk), "+v"(chunks));
    }
    __device__ __forceinline__ bool next(const AttnArgs &p, int rows, bool kept) {
        at = __builtin_amdgcn_readfirstlane(at);
        end = __builtin_amdgcn_readfirstlane(end);
        each = __builtin_amdgcn_readfirstlane(each);
        number = __builtin_amdgcn_readfirstlane(number);
        shift = __builtin_amdgcn_readfirstlane(shift);
        if (at >= end) return false;
        // (loads that are in front of all others of a piece: 16 trees of up to 64 rows over up to 2k keys 67.9 -> 65.9 us)
        const RowTile r = find(p, rows, kept ? Lane{own_upto, own_units} : lane_from(p, rows, 0), at);
        const int stop = min(end, r.first + r.units);
        seq = r.seq;
        row_tile = r.number;
        start = (at - r.first) << shift;
        count = ((stop - r.first) << shift) - start;   // (the last unit may be short: the caller's to cut)
        // borders inside of the row tile: of workgroups lo .. hi
        const int far = least(p, r.units);
        const int lo = first_share_from(r.first + far, each), hi = last_share_upto(r.first + r.units - far, each);
        chunks = max(hi - lo + 1, 0) + 1;
        chunk = start == 0 ? 0 : number - lo + 1;
        at = stop;
        if (kept) keep();
        return true;
    }
    __device__ __forceinline__ Seq sequence(const AttnArgs &p, bool kept) const {
        if (!kept || seq >= 64) return load_seq(p.c, seq);
        Seq s;
        s.row0 = __builtin_amdgcn_readlane(own.row0, seq);
        s.n = __builtin_amdgcn_readlane(own.n, seq);
        s.len = __builtin_amdgcn_readlane(own.len, seq);
        return s;
    }
};

// BIG: pages of at least a tile, so that a tile's page and scales are the same for all lanes.
template <typename T, int D, bool BIG, int W>
__global__ void __launch_bounds__(64 * W, 2) tree_kernel(AttnArgs p) {
    constexpr int kC = D / 16;                 // pieces of a key
    constexpr int kP = D / 32;                 // pairs of pieces of a key; 32-element blocks of a value
    constexpr bool kPairs = in_pairs(D);
    constexpr int kRows = rows_of(D, W);          // rows of a workgroup
    constexpr int kO = kPairs ? kP / 2 : kP;   // 32-element blocks of a value that a wave sums up
    constexpr int kLoads = D / 16 / W;         // loads of a wave for the keys of a tile, and for the values
    // (with pairs) A wave's weights, written by it and read by its partner; and, between that
    // reading and the next writing, what the partner has to tell it: a maximum or a sum.
    __shared__ uint4 weights[W][4][64];
    __shared__ uint4 kbuf0[kTile * kC], vbuf0[kTile * kC], kbuf1[kTile * kC], vbuf1[kTile * kC];
    const KvView &c = p.c;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int m = lane & 31, hf = lane >> 5;
    // with pairs: which 32 keys of a tile, and which half of the outputs, are the wave's
    const int side = kPairs ? wave & 1 : 0, row_wave = kPairs ? wave >> 1 : wave;
    const int h = blockIdx.x % c.kv_heads;
    const int P = 1 << c.log2_page;
    const int gv = (lane & 3) ^ ((lane >> 3) & 3);         // sixteen-key group whose values this lane loads
    const long long slab = (long long)P * D;

    // where this lane's pieces of a tile lie in its page or pages, and which of the wave's two
    // sixteen-key groups the keys' are of
    uint32_t koff[kLoads], voff[kLoads];
    bool kodd[kLoads];
#pragma unroll
    for (int n = 0; n < kLoads; ++n) {
        const int at = (wave * kLoads + n) * 64 + lane, row = at / kC, mm = row & 31;
        const int key = (row & 32) + 16 * ((mm >> 2) & 1) + 4 * (mm >> 3) + (mm & 3);
        const int pc = kC >= 8 ? (at % kC) ^ (row & 7) : (at % kC) ^ ((row >> 1) & 3);
        koff[n] = (key & (P - 1)) * D + 16 * pc;
        kodd[n] = (mm >> 2) & 1;
        voff[n] = ((wave * kLoads + n) * 16 + (lane >> 2)) * P + ((16 * gv) & (P - 1));
    }

    TreeShare share;
    share.begin(p, kRows, blockIdx.x / c.kv_heads);
    while (share.next(p, kRows, !kPairs)) {
        const Seq s = share.sequence(p, !kPairs);
        const int total = s.n * p.group;
        const int32_t *table = c.page_table + (long long)share.seq * c.table_width;
        const int r0 = share.row_tile * kRows, r1 = min(r0 + kRows, total) - 1;
        const Tiles tiles = visible_tiles(p, first_place<true>(s, 0), s.len - 1, s.len);
        const int start = share.start, count = min(share.count, max(1, tiles.count()) - start);
        // the wave's rows, and the lane's
        const int w0 = min(r0 + row_wave * kWaveRows, r1), w1 = min(w0 + kWaveRows - 1, r1);
        const bool idle = r0 + row_wave * kWaveRows > r1;
        const int lo = first_place<true>(s, 0), hi = s.len - 1;
        const int r = min(w0 + m, r1);
        const int token = r / p.group, head = h * p.group + r % p.group;
        const TreeSight sight(p, s, token);
        int seen_from = 0;                     // keys that no window hides from one of the wave's rows
        if (p.window > 0) {
            seen_from = sight.far + 1;
#pragma unroll
            for (int k = 16; k > 0; k >>= 1) seen_from = max(seen_from, __shfl_xor(seen_from, k));
            seen_from = __builtin_amdgcn_readfirstlane(seen_from);
        }
        const uint16_t *qrow = p.q + (long long)(s.row0 + token) * p.q_stride + head * D + 16 * hf;
        float up = p.scale < 0.0f ? -1.0f : 1.0f, down = fabsf(p.scale);
        if constexpr (!__is_same(T, half_t)) {
            float big = 0.0f;
#pragma unroll
            for (int i = 0; i < kP; ++i)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float x[8];
                    load8<T>(qrow + 32 * i + 8 * e, x);
#pragma unroll
                    for (int u = 0; u < 8; ++u) big = fmaxf(big, fabsf(x[u]));
                }
            big = half_max(big);
            const int e = min(max((int)(__builtin_bit_cast(uint32_t, big) >> 23) - 127, -100), 126);
            up *= pow2(min(14 - e, 127));
            down *= pow2(max(e - 14, -126));
        }
        half8_t qf[kP][2];
#pragma unroll
        for (int i = 0; i < kP; ++i)
#pragma unroll
            for (int e = 0; e < 2; ++e) qf[i][e] = as_row_half<T>(qrow + 32 * i + 8 * e, up);

        float mx = kEmpty, l = 0.0f;
        OutUnit unit;                          // the scale of the values that o counts in
        float16_t o[kO];
#pragma unroll
        for (int i = 0; i < kO; ++i) o[i] = float16_t{};

        // Page numbers run two tiles ahead and scales one, a sixteen-key group to a lane
        // (group g in lane g): page_of() asks, issue() loads a tile's codes and scales.
        int next_id = 0;
        float ks_l = 1.0f, vs_l = 0.0f;
        uint64_t has = 0;
        auto page_of = [&](int i) {
            const int j = tiles.at(start + min(i, count - 1)) * kTile + (BIG ? 0 : 16 * gv);
            return j < s.len ? table[j >> c.log2_page] : -1;
        };
        const uint8_t *v_from = nullptr;       // the next tile's values, as this lane loads them
        auto issue_keys = [&](int i, uint4 *kb) {
            const int j0 = tiles.at(start + i) * kTile;
            const int want = BIG ? __builtin_amdgcn_readfirstlane(next_id) : next_id;
            const bool ok = (uint32_t)want < (uint32_t)c.pages;
            const int id = ok ? want : 0;
            has = BIG ? (ok ? 15 : 0) : __ballot(ok);
            const long long ph = (long long)id * c.kv_heads + h;
            ks_l = c.k_scales[ph];             // (of page 0 where there is none: used for no key)
            vs_l = c.v_scales[ph];
            const int in_page = j0 & (P - 1);
            v_from = c.v + ph * slab + in_page;
            if constexpr (BIG) {
                const uint8_t *kp = c.k + ph * slab + in_page * D;
#pragma unroll
                for (int n = 0; n < kLoads; ++n) to_lds16(kp + koff[n], kb + (wave * kLoads + n) * 64);
                return;
            }
            const int id0 = __builtin_amdgcn_readlane(id, wave * (4 / W) & 2), id1 = __builtin_amdgcn_readlane(id, (wave * (4 / W) & 2) + 1);
            const long long page0 = ((long long)id0 * c.kv_heads + h) * slab, page1 = ((long long)id1 * c.kv_heads + h) * slab;
#pragma unroll
            for (int n = 0; n < kLoads; ++n)
                to_lds16(c.k + (kodd[n] ? page1 : page0) + in_page * D + koff[n], kb + (wave * kLoads + n) * 64);
        };
        auto issue_values = [&](uint4 *vb) {
#pragma unroll
            for (int n = 0; n < kLoads; ++n) to_lds16(v_from + voff[n], vb + (wave * kLoads + n) * 64);
        };

        // Codes of slots that hold no token may be anything, NaN among it: those of the values
        // become zero before a tile that has such slots is used.
        auto live_keys = [&](int j0, int grp, uint64_t ok) {
            return (ok >> grp) & 1 ? min(max(s.len - j0 - 16 * grp, 0), 16) : 0;
        };
        const auto tell = [&](float x) { reinterpret_cast<uint32_t *>(weights[wave ^ 1])[lane] = __builtin_bit_cast(uint32_t, x); };
        const auto told = [&]() { return __builtin_bit_cast(float, reinterpret_cast<const uint32_t *>(weights[wave])[lane]); };
        auto clear_dead = [&](int j0, uint4 *vb, uint64_t ok) {
#pragma unroll
            for (int n = 0; n < kLoads; ++n) {
                const int at = n * 64 * W + threadIdx.x;
                uint32_t keep[4];
                live_bytes(live_keys(j0, (at & 3) ^ ((at >> 3) & 3), ok), keep);
                uint4 v = vb[at];
                vb[at] = make_uint4(v.x & keep[0], v.y & keep[1], v.z & keep[2], v.w & keep[3]);
            }
            __builtin_amdgcn_s_waitcnt(0xC07F);
            barrier_no_fence();
        };

        if constexpr (kPairs) {
            // the scores of a tile: the wave's 32 keys
            float16_t acc;
            float ks = 1.0f, vmost = kNone, vown = kNone, vother = kNone, top = 0.0f;   // (of the values' scales, logarithms)
            auto scores = [&](int j0, const uint4 *kb, float ksl, float vsl, uint64_t ok) {
                acc = float16_t{};
                uint4 k0 = kb[piece<kC>(32 * side + m, hf)];
#pragma unroll
                for (int e = 0; e < kP; ++e) {
                    const uint4 a0 = k0;
                    if (e + 1 < kP) k0 = kb[piece<kC>(32 * side + m, 2 * e + 2 + hf)];
                    acc = __builtin_amdgcn_mfma_f32_32x32x16_f16(e4m3x8_to_half(a0.x, a0.y), qf[e][0], acc, 0, 0, 0);
                    acc = __builtin_amdgcn_mfma_f32_32x32x16_f16(e4m3x8_to_half(a0.z, a0.w), qf[e][1], acc, 0, 0, 0);
                }
                settle(acc);
                // (every row of the wave sees every key of most tiles)
                if ((ok & 15) != 15 || j0 + kTile > lo + 1 ||
                    (j0 < seen_from && j0 + kTile > p.sinks)) {
                    const int jg = j0 + 32 * side + 16 * hf;
                    const int live = live_keys(j0, 2 * side + hf, ok);
                    const uint32_t see = sight.sixteen(args_again(), jg, live);
#pragma unroll
                    for (int e = 0; e < 16; ++e) acc[e] = see >> e & 1 ? acc[e] : -__builtin_inff();
                }
                const float vlog = __builtin_amdgcn_logf(vsl);
                float vs[4];
#pragma unroll
                for (int g = 0; g < (BIG ? 1 : 4); ++g) vs[g] = (ok >> g) & 1 ? lane_value(vlog, g) : kNone;
                const float k_lo = lane_value(ksl, BIG ? 0 : 2 * side), k_hi = BIG ? k_lo : lane_value(ksl, 2 * side + 1);
                // never 0, which would turn a hidden key's -inf into NaN; and where there is no page
                // the scale may be anything, but no key is seen
                ks = fminf(fmaxf((hf ? k_hi : k_lo) * down, 0x1p-126f), 0x1p126f);
                vmost = BIG ? vs[0] : fmaxf(fmaxf(vs[0], vs[1]), fmaxf(vs[2], vs[3]));
                vown = BIG ? vs[0] : side ? (hf ? vs[3] : vs[2]) : (hf ? vs[1] : vs[0]);
                vother = BIG ? vs[0] : side ? (hf ? vs[1] : vs[0]) : (hf ? vs[3] : vs[2]);
                float a = max3(acc[0], acc[1], acc[2]);
#pragma unroll
                for (int e = 3; e < 15; e += 2) a = max3(a, acc[e], acc[e + 1]);
                top = max3(a, a, acc[15]) * ks;
                tell(top);                     // of sixteen keys
            };
            // the weights, of the maximum of both waves
            half8_t w[4];                      // leading parts, remainders
            auto weigh = [&]() {
                const float other = told(), now = half_max(fmaxf(top, other)), to = fmaxf(mx, now);
                const float need = BIG ? vmost + (now - to) : half_max(fmaxf(vown + (top - to), vother + (other - to)));
                if (__any(now - mx > kSlack || unit.moves(need, vmost))) {     // rare
                    const float turn = unit.move(need, vmost, mx - to);
                    l *= __builtin_amdgcn_exp2f(mx - to);
                    mx = to;
#pragma unroll
                    for (int e = 0; e < kO; ++e) o[e] *= turn;
                }
                const float to_unit = vown > kNone ? vown - unit.at : 0.0f;    // (no weight where there is no page)
                float shift = mx;
                if (__any(fabsf(mx) >= kFar)) {
#pragma clang fp contract(off)   // the products as the maximum was taken of them
#pragma unroll
                    for (int e = 0; e < 16; ++e) acc[e] = acc[e] * ks - mx;
                    ks = 1.0f;
                    shift = 0.0f;
                }
                const float base = kWeightBits + to_unit - shift;
                float back = __builtin_amdgcn_exp2f(-to_unit);
                if (__any(to_unit < kLeastToUnit)) {
#pragma unroll
                    for (int e = 0; e < 16; ++e) l += __builtin_amdgcn_exp2f(__builtin_fmaf(acc[e], ks, kWeightBits - shift));
                    back = 0.0f;
                }
                float sum = 0.0f;
                uint32_t lead[8], rest[8];
#pragma unroll
                for (int e = 0; e < 16; e += 2) {
                    const float f = __builtin_amdgcn_exp2f(__builtin_fmaf(acc[e], ks, base));
                    const float g = __builtin_amdgcn_exp2f(__builtin_fmaf(acc[e + 1], ks, base));
                    sum += f;
                    sum += g;
                    lead_and_rest(f, g, lead[e / 2], rest[e / 2]);
                }
                settle(rest);
                l += sum * back;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    w[e] = halves8((e < 2 ? lead : rest) + 4 * (e & 1));
                    weights[wave][e][lane] = __builtin_bit_cast(uint4, w[e]);
                }
            };
            // the wave's own 32 keys first, then its partner's, for which its own weights' registers are free
            auto add_values = [&](const uint4 *vb) {
                const int row = 32 * kO * side + m;
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const int at = 2 * (u ? side ^ 1 : side) + hf;
                    uint4 v = vb[piece<4>(row, at)];
                    if (u) {
#pragma unroll
                        for (int e = 0; e < 4; ++e) w[e] = __builtin_bit_cast(half8_t, weights[wave ^ 1][e][lane]);
                    }
#pragma unroll
                    for (int e = 0; e < kO; ++e) {
                        const uint4 codes = v;
                        if (e + 1 < kO) v = vb[piece<4>(row + 32 * e + 32, at)];
                        add_products(o[e], codes, w);
                    }
                }
            };

            if (count > 0) {
                next_id = page_of(0);
                issue_keys(0, kbuf0);
                next_id = page_of(1);
                issue_values(vbuf0);
                bool before = false, dead = false;         // of the tile before: whether it is the wave's; slots of no token
                int j_before = 0;
                uint64_t ok_before = 0;
                // A tile's scores beside the sums of the tile before, then its weights.  Keys are loaded a
                // tile ahead, values as the keys' tile begins its weights.
                auto step = [&](int i, const uint4 *kb, uint4 *vb, uint4 *kn, uint4 *vn) {
                    // this wave's loads of the keys of tile i, and of the values of tile i - 1, are in LDS,
                    // its reads and writes of LDS done
                    __builtin_amdgcn_s_waitcnt(0xC07F);
                    wait_vmcnt<kLoads>();
                    barrier_no_fence();            // and everyone's
                    const float ksl = ks_l, vsl = vs_l;
                    const uint64_t ok = has;
                    if (dead) clear_dead(j_before, vn, ok_before);
                    // (unconditionally, the last tile again behind it: around a condition the compiler
                    // waits for all loads)
                    issue_keys(min(i + 1, count - 1), kn);
                    next_id = page_of(i + 2);
                    const int j0 = tiles.at(start + i) * kTile;
                    const bool mine = !idle && j0 <= hi;
                    __builtin_amdgcn_s_setprio(1);     // products before the other workgroup's weights: 1%
                    if (before) add_values(vn);
                    if (mine) scores(j0, kb, ksl, vsl, ok);
                    __builtin_amdgcn_s_waitcnt(0xC07F);
                    __builtin_amdgcn_s_setprio(0);
                    barrier_no_fence();            // the maxima are there; the values of tile i - 1 are done with
                    issue_values(vn);
                    if (mine) weigh();
                    before = mine;
                    dead = (ok & 15) != 15 || j0 + kTile > s.len;
                    j_before = j0;
                    ok_before = ok;
                };
                for (int i = 0; i < count; i += 2) {
                    step(i, kbuf0, vbuf0, kbuf1, vbuf1);
                    if (i + 1 < count) step(i + 1, kbuf1, vbuf1, kbuf0, vbuf0);
                }
                uint4 *last = count & 1 ? vbuf0 : vbuf1;
                __builtin_amdgcn_s_waitcnt(0xC07F);
                wait_vmcnt<0>();
                barrier_no_fence();
                if (dead) clear_dead(j_before, last, ok_before);
                if (before) add_values(last);
            }
        } else {
            auto multiply = [&](int j0, const uint4 *kb, const uint4 *vb, float ksl, float vsl, uint64_t ok) {
                // the pieces of the next products are read while these run; the barriers keep the
                // compiler from reading all of them at once, for which there are no registers (beside the
                // values' products, where there are, barriers took 2%)
                float16_t acc[2] = {};
                uint4 k0 = kb[piece<kC>(m, hf)], k1 = kb[piece<kC>(32 + m, hf)];
#pragma unroll
                for (int e = 0; e < kP; ++e) {
                    const uint4 a0 = k0, a1 = k1;
                    if (e + 1 < kP) {
                        k0 = kb[piece<kC>(m, 2 * e + 2 + hf)];
                        k1 = kb[piece<kC>(32 + m, 2 * e + 2 + hf)];
                    }
                    acc[0] = __builtin_amdgcn_mfma_f32_32x32x16_f16(e4m3x8_to_half(a0.x, a0.y), qf[e][0], acc[0], 0, 0, 0);
                    acc[1] = __builtin_amdgcn_mfma_f32_32x32x16_f16(e4m3x8_to_half(a1.x, a1.y), qf[e][0], acc[1], 0, 0, 0);
                    acc[0] = __builtin_amdgcn_mfma_f32_32x32x16_f16(e4m3x8_to_half(a0.z, a0.w), qf[e][1], acc[0], 0, 0, 0);
                    acc[1] = __builtin_amdgcn_mfma_f32_32x32x16_f16(e4m3x8_to_half(a1.z, a1.w), qf[e][1], acc[1], 0, 0, 0);
                    __builtin_amdgcn_sched_barrier(0);
                }
                settle(acc[0], acc[1]);
                // (every row of the wave sees every key of most tiles)
                if ((ok & 15) != 15 || j0 + kTile > lo + 1 ||
                    (j0 < seen_from && j0 + kTile > p.sinks)) {
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        const int jg = j0 + 32 * u + 16 * hf;
                        const int live = live_keys(j0, 2 * u + hf, ok);
                        const uint32_t see = sight.sixteen(args_again(), jg, live);
#pragma unroll
                        for (int e = 0; e < 16; ++e) acc[u][e] = see >> e & 1 ? acc[u][e] : -__builtin_inff();
                    }
                }
                // (read here, they are there when the weights are: 1 to 2%)
                uint4 v0 = vb[piece<4>(m, hf)], v1 = vb[piece<4>(m, 2 + hf)];
                // The scales (of the values their logarithms) of the tile's four groups of sixteen keys, with
                // BIG all the same, and, of the lane's two groups, the keys' scale and what the values' is
                // to the outputs' unit.
                const float vlog = __builtin_amdgcn_logf(vsl);
                float ks[2], top[2], vs[4], to_unit[2];
#pragma unroll
                for (int g = 0; g < (BIG ? 1 : 4); ++g) vs[g] = (ok >> g) & 1 ? lane_value(vlog, g) : kNone;
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const float a = lane_value(ksl, BIG ? 0 : 2 * u), d = BIG ? a : lane_value(ksl, 2 * u + 1);
                    // never 0, which would turn a hidden key's -inf into NaN; and where there is no page
                    // the scale may be anything, but no key is seen
                    ks[u] = fminf(fmaxf((hf ? d : a) * down, 0x1p-126f), 0x1p126f);
                    float t = max3(acc[u][0], acc[u][1], acc[u][2]);
#pragma unroll
                    for (int e = 3; e < 15; e += 2) t = max3(t, acc[u][e], acc[u][e + 1]);
                    top[u] = max3(t, t, acc[u][15]) * ks[u];
                }
                const float now = half_max(fmaxf(top[0], top[1])), to = fmaxf(mx, now);
                const float most = BIG ? vs[0] : fmaxf(fmaxf(vs[0], vs[1]), fmaxf(vs[2], vs[3]));
                const float need = BIG ? most + (now - to)
                                       : half_max(fmaxf((hf ? vs[1] : vs[0]) + (top[0] - to), (hf ? vs[3] : vs[2]) + (top[1] - to)));
                if (__any(now - mx > kSlack || unit.moves(need, most))) {      // rare
                    const float turn = unit.move(need, most, mx - to);
                    l *= __builtin_amdgcn_exp2f(mx - to);
                    mx = to;
#pragma unroll
                    for (int e = 0; e < kO; ++e) o[e] *= turn;
                }
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const float v = BIG ? vs[0] : hf ? vs[2 * u + 1] : vs[2 * u];
                    to_unit[u] = v > kNone ? v - unit.at : 0.0f;           // (no weight where there is no page)
                }
                float shift = mx;
                if (__any(fabsf(mx) >= kFar)) {
#pragma clang fp contract(off)   // the products as the maximum was taken of them
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
#pragma unroll
                        for (int e = 0; e < 16; ++e) acc[u][e] = acc[u][e] * ks[u] - mx;
                        ks[u] = 1.0f;
                    }
                    shift = 0.0f;
                }
                float back[2] = {__builtin_amdgcn_exp2f(-to_unit[0]), __builtin_amdgcn_exp2f(-to_unit[1])};
                if (__any(fminf(to_unit[0], to_unit[1]) < kLeastToUnit)) {
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
#pragma unroll
                        for (int e = 0; e < 16; ++e) l += __builtin_amdgcn_exp2f(__builtin_fmaf(acc[u][e], ks[u], kWeightBits - shift));
                        back[u] = 0.0f;
                    }
                }
                half8_t w[2][4];               // leading parts, remainders
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const float base = kWeightBits + to_unit[u] - shift;
                    float sum = 0.0f;
                    uint32_t lead[8], rest[8];
#pragma unroll
                    for (int e = 0; e < 16; e += 2) {
                        const float f = __builtin_amdgcn_exp2f(__builtin_fmaf(acc[u][e], ks[u], base));
                        const float g = __builtin_amdgcn_exp2f(__builtin_fmaf(acc[u][e + 1], ks[u], base));
                        sum += f;
                        sum += g;
                        lead_and_rest(f, g, lead[e / 2], rest[e / 2]);
                    }
                    settle(rest);
                    l += sum * back[u];
#pragma unroll
                    for (int e = 0; e < 4; ++e) w[u][e] = halves8((e < 2 ? lead : rest) + 4 * (e & 1));
                }
#pragma unroll
                for (int e = 0; e < kP; ++e) {
                    const uint4 a0 = v0, a1 = v1;
                    if (e + 1 < kP) {
                        v0 = vb[piece<4>(32 * e + 32 + m, hf)];
                        v1 = vb[piece<4>(32 * e + 32 + m, 2 + hf)];
                    }
                    add_products(o[e], a0, w[0]);
                    add_products(o[e], a1, w[1]);
                }
            };

            if (count > 0) {
                next_id = page_of(0);
                issue_keys(0, kbuf0);
                issue_values(vbuf0);
                next_id = page_of(1);
                auto step = [&](int i, const uint4 *kb, uint4 *vb, uint4 *kn, uint4 *vn) {
                    // this wave's loads of tile i are in LDS, its reads of tile i - 1 done
                    __builtin_amdgcn_s_waitcnt(0xC07F);
                    wait_vmcnt<0>();
                    barrier_no_fence();            // everyone's are, and tile i - 1 is done with
                    const float ksl = ks_l, vsl = vs_l;
                    const uint64_t ok = has;
                    if (i + 1 < count) {
                        issue_keys(i + 1, kn);
                        issue_values(vn);
                        next_id = page_of(i + 2);
                    }
                    const int j0 = tiles.at(start + i) * kTile;
                    if ((ok & 15) != 15 || j0 + kTile > s.len) clear_dead(j0, vb, ok);
                    if (!idle && j0 <= hi) multiply(j0, kb, vb, ksl, vsl, ok);
                };
                for (int i = 0; i < count; i += 2) {
                    step(i, kbuf0, vbuf0, kbuf1, vbuf1);
                    if (i + 1 < count) step(i + 1, kbuf1, vbuf1, kbuf0, vbuf0);
                }
            }
        }
        l = half_sum(l);
        if constexpr (kPairs) {
            tell(l);
            __syncthreads();
            l += told();
        }
        if (!idle && w0 + m <= r1) {
            // over the sum first: outputs that are no larger than the values are
            const ArgsAgain args = args_again();
            const long long at = (long long)(s.row0 + token) * args->q_heads + head;
            const float inv = l > 0.0f || !(l == l) ? 1.0f / l : 0.0f, scale = __builtin_amdgcn_exp2f(unit.at);
#pragma unroll
            for (int e = 0; e < kO; ++e) o[e] = o[e] * inv * scale;
            if (share.chunks > 1) {
                float *dst = args->part + (at * args->splits + share.chunk) * kPart<D> + 32 * kO * side + 4 * hf;
#pragma unroll
                for (int e = 0; e < kO; ++e)
#pragma unroll
                    for (int u = 0; u < 4; ++u)
                        *reinterpret_cast<float4_t *>(dst + 32 * e + 8 * u) =
                            float4_t{o[e][4 * u], o[e][4 * u + 1], o[e][4 * u + 2], o[e][4 * u + 3]};
                if (hf == 0 && side == 0) {
                    dst[D] = mx;
                    dst[D + 1] = l;
                    dst[D + 2] = (float)share.chunks;
                }
            } else {
                if (args->part != nullptr && hf == 0 && side == 0) args->part[at * args->splits * kPart<D> + D + 2] = 1.0f;
                uint16_t *dst = args->out + at * D + 32 * kO * side + 4 * hf;
#pragma unroll
                for (int e = 0; e < kO; ++e)
#pragma unroll
                    for (int u = 0; u < 4; ++u) {
                        uint2 y;
                        y.x = (uint32_t)from_float<T>(o[e][4 * u]) | ((uint32_t)from_float<T>(o[e][4 * u + 1]) << 16);
                        y.y = (uint32_t)from_float<T>(o[e][4 * u + 2]) | ((uint32_t)from_float<T>(o[e][4 * u + 3]) << 16);
                        *reinterpret_cast<uint2 *>(dst + 32 * e + 8 * u) = y;
                    }
            }
        }
        __syncthreads();                       // the buffers are free again
    }
}

template <typename T, int D, int W>
void launch_page(const AttnArgs &p, hipStream_t s) {
    const int grid = p.c.kv_heads * p.most;
    if ((1 << p.c.log2_page) >= kTile)
        tree_kernel<T, D, true, W><<<grid, 64 * W, 0, s>>>(p);
    else
        tree_kernel<T, D, false, W><<<grid, 64 * W, 0, s>>>(p);
}

template <typename T>
hipError_t launch_dim(const AttnArgs &p, int D, int waves, hipStream_t s) {
    switch (D) {
    case 64: waves == 2 ? launch_page<T, 64, 2>(p, s) : launch_page<T, 64, 4>(p, s); break;
    case 128: waves == 2 ? launch_page<T, 128, 2>(p, s) : launch_page<T, 128, 4>(p, s); break;
    case 256: launch_page<T, 256, 4>(p, s); break;
    default: return hipErrorInvalidValue;
    }
    return hipGetLastError();
}

}  // namespace

// Workgroups of a kv head: as many as the GPU holds, or where keys are not cut, one to a row tile;
// and chunks that a row tile has room for, twice what it has on average, since sequences are not
// equally long.
TreePlan tree_plan(int seqs, int rows, int kv_heads, int group, int head_dim, int max_q, bool mixed, int few, long long key_tiles) {
    int waves = waves_of(head_dim, (long long)max_q * group);
    // row tiles of a kv head: all that there can be, or of sequences of max_q rows
    const auto row_tiles = [&]() {
        const int each = rows_of(head_dim, waves);
        return std::max<long long>(1, mixed ? (long long)rows * group / each + std::min<long long>(seqs, (long long)rows * group / few)
                                            : ((long long)max_q * group + each - 1) / each * seqs);
    };
    const auto cut = [&]() {
        const long long all = row_tiles() * kv_heads;
        return key_tiles >= (all < kTreeFullTiles ? 2 * kLeastChunk : kTreeCutTiles) && all < kManyTreeTiles;
    };
    // (where keys are not cut, sequences of fewer rows than the longest gain nothing from two waves: 32 trees of up
    // to 40 rows of 32 heads on 8 over up to 1000 keys 73 us, with four 57)
    if (waves == 2 && (long long)max_q * group > 64 && !cut()) waves = 4;
    const int slots = kTreeWaves / waves;
    const long long groups = row_tiles(), all = groups * kv_heads;
    TreePlan t{(int)std::min<long long>(groups, ((1 << 24) - 1) / kv_heads), 1, waves};
    if (cut()) {
        t.shares = std::max(1, slots / kv_heads);
        t.room = (int)std::max<long long>(3, std::min<long long>({2 * slots / all + 1, key_tiles / kLeastChunk + 1, kMostSplits + 1}));
    }
    return t;
}

hipError_t launch_tree_attention_prefill(const AttnArgs &p, int head_dim, bool bf16, int waves, hipStream_t s) {
    return bf16 ? launch_dim<bhalf_t>(p, head_dim, waves, s) : launch_dim<half_t>(p, head_dim, waves, s);
}

}  // namespace awq
