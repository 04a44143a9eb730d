// awq_attention for many rows (prompts, chunks of prompts): see
// awq_attention.hip for the formula and the transposed products.
//
// A workgroup of four waves takes 128 rows (64 with heads of 256; row r of a kv head: token r / group,
// head r % group) of one kv head and one sequence, 32 to a wave, and goes once
// over the keys in tiles of 64, held in LDS as codes: 64 D bytes of keys and as
// many of values, loaded straight into LDS, the next tile while this one is
// multiplied (two buffers, one barrier a tile).  Products are
// v_mfma_f32_32x32x16_f16: S^T = K Q^T leaves a lane with one row and 32 scores,
// O^T = V^T P^T takes them as they lie.  LDS row m of a half tile holds key
// 16 (m / 4 % 2) + 4 (m / 8) + m % 4, so that lane half hf ends up with the
// sixteen consecutive keys 16 hf .. 16 hf + 15 of it, one 16-byte piece of a row
// of V^T.  Pieces are stored xor-swizzled by their row, which spreads eight rows over the
// banks; rows r and r + 8 meet (half of the LDS cycles with 128 elements are such conflicts,
// a third with 256).
//
// Heads of 256 elements: queries, outputs and scores of 32 rows are 224 registers of
// a wave, which leaves one wave to a SIMD and nothing beside its vector instructions
// while its products run, and the other way round.  There two waves share 32 rows (a
// workgroup has 64): each has the scores of 32 of a tile's 64 keys and sums up one half
// of the outputs; the rows' maxima and the weights go from one to the other through LDS, lane
// by lane as they lie.  A tile's scores run beside the outputs of the tile before, so
// two barriers a tile do.  Two waves to a SIMD: 8192 rows under a window of 1024, 250
// -> 191 us.  With 128 elements, where two waves fit as it is, 163 against 180 us on 4096
// rows: not there.  (Both before weights were two halves.)  Four registers are spilled, six
// with pages of fewer than 64 tokens.
//
// Bound: vector and matrix instructions, one after the other: of a SIMD's cycles on 4096
// rows the first take 54%, the second 43% (1.5 times that of the formula's products, for the
// remainders), and the two waves of a SIMD hardly overlap them.
//
// Few row tiles over many keys are cut into chunks of keys, joined by combine_kernel.
//
// Weights go into the products as two halves, the leading part and its remainder
// (lead_and_rest), as in the split kernel: a query's outputs are as exact in a prompt as alone.
// Half more matrix instructions for it: 4096 rows 166 -> 214 us (640 TFLOP/s), chunks of 512
// rows on 16k contexts 700 -> 898 us, 8192 rows of 256 elements under a window 194 -> 235 us;
// with one half the error against 64 bits was 2.4e-4 where fp16's own rounding makes 1.8e-4.
// The sum takes them before the roundings.
// They are scaled by 2^11 so that small ones stay normal numbers, and the
// maximum that they refer to is moved only when a row exceeds it by 2^4, so the
// largest is 2^15, and rescaling the outputs is rare after the first tiles.  (The difference
// is compared: mx + 2^4 rounds up by half a step of 2^26 and more.)
#include <algorithm>

#include "awq_attention.h"
#include "awq_internal.h"

namespace awq {
namespace {

constexpr int kWaveRows = 32, kWaves = 4;
// Least tiles of a chunk, most chunks of a row tile.  32 rows of 32 heads over 4k, 16k and 131k
// keys, one sequence: 47 / 43 / 140 us at 16 tiles, 26 / 32 / 137 at 6, 24 / 32 / 140 at 4; 16
// sequences of 32 rows over 4k: 90 / 84 / 85.
constexpr int kLeastChunk = 6, kMostSplits = 32;
constexpr float kWeightBits = 11.0f, kSlack = 4.0f;

// Heads of 256 elements: two waves share 32 rows.  Elsewhere a wave has 32 rows to itself.
constexpr bool in_pairs(int head_dim) { return head_dim > 128; }
constexpr int rows_of(int head_dim) { return kWaveRows * (in_pairs(head_dim) ? kWaves / 2 : kWaves); }

template <int N>
__device__ __forceinline__ void wait_vmcnt() {
    __builtin_amdgcn_s_waitcnt((N & 0xF) | ((N >> 4) << 14) | (0x7 << 4) | (0xF << 8));
}
// A barrier that waits for no load in flight.
__device__ __forceinline__ void barrier_no_fence() { asm volatile("s_barrier" ::: "memory"); }
__device__ __forceinline__ void to_lds16(const void *src, uint4 *dst) {
    __builtin_amdgcn_global_load_lds(src, dst, 16, 0, 0);
}
__device__ __forceinline__ float lane_value(float x, int lane) {
    return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, x), lane));
}

// LDS piece of (row, 16-byte piece), C pieces a row.
template <int C>
__device__ __forceinline__ int piece(int row, int at) {
    return row * C + (C >= 8 ? at ^ (row & 7) : at ^ ((row >> 1) & 3));
}

// The outputs of 32 elements, and sixteen codes of each times weights w (their leading
// parts in w[0] and w[1], their remainders in w[2] and w[3]).
__device__ __forceinline__ void add_products(float16_t &o, uint4 codes, const half8_t w[4]) {
    const half8_t a = e4m3x8_to_half(codes.x, codes.y), b = e4m3x8_to_half(codes.z, codes.w);
    o = __builtin_amdgcn_mfma_f32_32x32x16_f16(a, w[0], o, 0, 0, 0);
    o = __builtin_amdgcn_mfma_f32_32x32x16_f16(a, w[2], o, 0, 0, 0);
    o = __builtin_amdgcn_mfma_f32_32x32x16_f16(b, w[1], o, 0, 0, 0);
    o = __builtin_amdgcn_mfma_f32_32x32x16_f16(b, w[3], o, 0, 0, 0);
}

// BIG: pages of at least a tile, so that a tile's page and scales are the same for
// all lanes and its addresses are scalar arithmetic (about 150 of 450 vector
// instructions a tile less).
template <typename T, int D, bool BIG>
__global__ void __launch_bounds__(64 * kWaves, 2) prefill_kernel(AttnArgs p, int tiles_per_seq) {      // 0: flat
    constexpr int kC = D / 16;                 // pieces of a key
    constexpr int kP = D / 32;                 // pairs of pieces of a key; 32-element blocks of a value
    constexpr bool kPairs = in_pairs(D);
    constexpr int kRows = rows_of(D);          // rows of a workgroup
    constexpr int kO = kPairs ? kP / 2 : kP;   // 32-element blocks of a value that a wave sums up
    constexpr int kLoads = D / 64;             // loads of a wave for the keys of a tile, and for the values
    // (with pairs) A wave's weights, written by it and read by its partner; and, between that
    // reading and the next writing, what the partner has to tell it: a maximum or a sum.
    __shared__ uint4 weights[kWaves][4][64];
    __shared__ uint4 kbuf0[kTile * kC], vbuf0[kTile * kC], kbuf1[kTile * kC], vbuf1[kTile * kC];
    const KvView &c = p.c;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int m = lane & 31, hf = lane >> 5;
    // with pairs: which 32 keys of a tile, and which half of the outputs, are the wave's
    const int side = kPairs ? wave & 1 : 0, row_wave = kPairs ? wave >> 1 : wave;
    const int h = blockIdx.x % c.kv_heads, split = blockIdx.x / c.kv_heads % p.most;
    const int slot = blockIdx.x / (c.kv_heads * p.most);
    int b, tile, tile_step = tiles_per_seq;
    if (tiles_per_seq > 0) {
        b = seq_of_rank(c, slot / tiles_per_seq);
        tile = slot % tiles_per_seq;
    } else {
        const int2 at = seq_of_piece(c, slot, [&](const Seq &s) {
            return s.n * p.group >= p.few ? (s.n * p.group + kRows - 1) / kRows : 0;
        });
        if (at.x >= c.seqs) return;
        b = at.x;
        tile = at.y;
        tile_step = 1 << 30;
    }
    const Seq s = load_seq(c, b);
    const int P = 1 << c.log2_page;
    const int total = s.n * p.group;
    const int row_tiles = (total + kRows - 1) / kRows;
    const int32_t *table = c.page_table + (long long)b * c.table_width;
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

    // the longest rows first
    for (int rt = row_tiles - 1 - tile; rt >= 0; rt -= tile_step) {
        const int r0 = rt * kRows, r1 = min(r0 + kRows, total) - 1;
        const Tiles tiles = visible_tiles(p, s.first() + r0 / p.group, s.first() + r1 / p.group, s.len);
        // this workgroup's chunk of them
        const int every = tiles.count(), chunks = max(1, min(p.most, every / kLeastChunk));
        if (split >= chunks) continue;
        const int start = (int)((long long)every * split / chunks);
        const int count = (int)((long long)every * (split + 1) / chunks) - start;
        // the wave's rows, and the lane's
        const int w0 = min(r0 + row_wave * kWaveRows, r1), w1 = min(w0 + kWaveRows - 1, r1);
        const bool idle = r0 + row_wave * kWaveRows > r1;
        const int lo = s.first() + w0 / p.group, hi = s.first() + w1 / p.group;
        const int r = min(w0 + m, r1);
        const int token = r / p.group, head = h * p.group + r % p.group;
        const int pos = s.first() + token;
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
            const int id0 = __builtin_amdgcn_readlane(id, wave & 2), id1 = __builtin_amdgcn_readlane(id, (wave & 2) + 1);
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
                const int at = n * 64 * kWaves + threadIdx.x;
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
                    (p.window > 0 && j0 <= hi - p.window && j0 + kTile > p.sinks)) {
                    const int jg = j0 + 32 * side + 16 * hf;
                    const int live = live_keys(j0, 2 * side + hf, ok);
                    const int far = p.window > 0 ? pos - p.window : -0x7FFFFFFF;      // keys up to it are out of sight
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        const int j = jg + e;
                        const bool see = (e < live) & (j <= pos) & ((j > far) | (j < p.sinks));
                        acc[e] = see ? acc[e] : -__builtin_inff();
                    }
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
                    (p.window > 0 && j0 <= hi - p.window && j0 + kTile > p.sinks)) {
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        const int jg = j0 + 32 * u + 16 * hf;
                        const int live = live_keys(j0, 2 * u + hf, ok);
                        const int far = p.window > 0 ? pos - p.window : -0x7FFFFFFF;      // keys up to it are out of sight
#pragma unroll
                        for (int e = 0; e < 16; ++e) {
                            const int j = jg + e;
                            const bool see = (e < live) & (j <= pos) & ((j > far) | (j < p.sinks));
                            acc[u][e] = see ? acc[u][e] : -__builtin_inff();
                        }
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
            const long long at = (long long)(s.row0 + token) * p.q_heads + head;
            const float inv = l > 0.0f || !(l == l) ? 1.0f / l : 0.0f, scale = __builtin_amdgcn_exp2f(unit.at);
#pragma unroll
            for (int e = 0; e < kO; ++e) o[e] = o[e] * inv * scale;
            if (chunks > 1) {
                float *dst = p.part + (at * p.splits + split) * kPart<D> + 32 * kO * side + 4 * hf;
#pragma unroll
                for (int e = 0; e < kO; ++e)
#pragma unroll
                    for (int u = 0; u < 4; ++u)
                        *reinterpret_cast<float4_t *>(dst + 32 * e + 8 * u) =
                            float4_t{o[e][4 * u], o[e][4 * u + 1], o[e][4 * u + 2], o[e][4 * u + 3]};
                if (hf == 0 && side == 0) {
                    dst[D] = mx;
                    dst[D + 1] = l;
                    dst[D + 2] = (float)chunks;
                }
            } else {
                if (p.part != nullptr && hf == 0 && side == 0) p.part[at * p.splits * kPart<D> + D + 2] = 1.0f;
                uint16_t *dst = p.out + at * D + 32 * kO * side + 4 * hf;
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

template <typename T, int D>
void launch_page(const AttnArgs &p, int grid, int tiles_per_seq, hipStream_t s) {
    if ((1 << p.c.log2_page) >= kTile)
        prefill_kernel<T, D, true><<<grid, 64 * kWaves, 0, s>>>(p, tiles_per_seq);
    else
        prefill_kernel<T, D, false><<<grid, 64 * kWaves, 0, s>>>(p, tiles_per_seq);
}

template <typename T>
hipError_t launch_dim(const AttnArgs &p, int D, int grid, int tiles_per_seq, hipStream_t s) {
    switch (D) {
    case 64: launch_page<T, 64>(p, grid, tiles_per_seq, s); break;
    case 128: launch_page<T, 128>(p, grid, tiles_per_seq, s); break;
    case 256: launch_page<T, 256>(p, grid, tiles_per_seq, s); break;
    default: return hipErrorInvalidValue;
    }
    return hipGetLastError();
}

}  // namespace

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

hipError_t launch_attention_prefill(const AttnArgs &p, int head_dim, bool bf16, int row_tiles, bool flat, hipStream_t s) {
    // The kv head fastest: with a multiple of eight of them, the row tiles that read the same
    // keys meet in one XCD's cache.  Then the row tiles of a sequence, and the sequences, the
    // longest first, so that the last workgroups to start are short (four sequences of 512 rows,
    // one of them over twice the keys of the others: 1080 -> 693 us before weights were two halves).  The kernel steps on where
    // the grid is cut.  Flat: the row tiles of the sequences that have `few` rows or more.
    const int grid = p.c.kv_heads * (flat ? 1 : p.c.seqs) * row_tiles * p.most;
    if (grid == 0) return hipSuccess;
    return bf16 ? launch_dim<bhalf_t>(p, head_dim, grid, flat ? 0 : row_tiles, s)
                : launch_dim<half_t>(p, head_dim, grid, flat ? 0 : row_tiles, s);
}

}  // namespace awq
