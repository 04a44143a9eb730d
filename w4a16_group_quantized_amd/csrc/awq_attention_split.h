// awq_attention, awq_tree_attention: attention of a ragged batch over the 8-bit paged cache.
//
//   x_j = scale * (q . k_j) * log2(e),  o = sum_j 2^(x_j - m) v_j / sum_j 2^(x_j - m)
//
// over the keys j that the row at position i sees: j <= i, j < len, and with a
// window w > 0: j > i - w or j < sinks.  k_j and v_j are e4m3 codes times the
// scale of their page and kv head; the scale of a page's keys multiplies the
// fp32 products, that of its values the weights.  One pass over the keys, with
// the running maximum m and sum of each row in fp32.
//
// split_kernel.  A workgroup of four waves (eight with heads of 64 where that
// takes the place of a cut, see plan()) takes sixteen rows (row r of a kv
// head: token r / group, head r % group) of one kv head and one sequence, over
// a chunk of the keys; the waves take its 64-key tiles in turn.  The products
// run transposed, on v_mfma_f32_16x16x32_f16: S^T = K Q^T, so a lane holds
// sixteen scores of one row, and O^T = V^T P^T, whose operand P^T is what the
// lane already holds, without a lane exchange.  For that the keys of a tile are
// dealt to the four 16-key products so that lane group g = lane / 16 ends up
// with the keys 16 g .. 16 g + 15, which are sixteen consecutive bytes of a row
// of V^T: every load is 16 bytes a lane, and 16 keys never leave a page.
// Weights go into the products as two halves, a leading part and its remainder
// (lead_and_rest): the second product is free beside the loads (16 sequences of 3 to 5
// rows with heads of 64, whose time is latency: 10.7 -> 11.4 us), and the result keeps
// fp32's quality.
// Weights are scaled by 2^14 so that the small ones stay normal fp16 numbers.
// Bound: the bytes of K and V (HBM).
//
// combine_kernel (awq_attention.hip) joins the chunks' partial results (fp32, in the
// workspace) where there is more than one chunk.
//
// TREE (awq_tree_attention): the last tokens are a drafted tree's rows; see TreeSight.
#pragma once

#include <type_traits>

#include "awq_attention.h"
#include "awq_internal.h"

namespace awq {
namespace {

constexpr int kRows = kSplitRows, kLeastChunk = kSplitLeastChunk, kWaves = 4;
constexpr float kWeightBits = 14.0f;       // weights are 2^14 times those of the formula

// Chunks for a tile: from the tiles that all sequences' rows see, for all kv heads.
// The host knows no lengths, so each wave adds them up, with more than 64 sequences four
// to a lane at a time.
template <bool TREE>
__device__ __forceinline__ float chunks_per_tile(const AttnArgs &p) {
    const KvView &c = p.c;
    float sum = 0.0f;
    const auto add = [&](const Seq &s) {
        if (s.n > 0 && s.n * p.group < p.few)
            sum += (float)visible_tiles(p, first_place<TREE>(s, 0), s.len - 1, s.len).count() * (float)((s.n * p.group + kRows - 1) / kRows);
    };
    const int lane = threadIdx.x & 63;
    if (c.seqs <= 64) {
        if (lane < c.seqs) add(load_seq(c, lane));
    } else {
        for (int b = lane; b < c.seqs; b += 256) {
            Seq s[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) s[k] = load_seq(c, min(b + 64 * k, c.seqs - 1));
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (b + 64 * k < c.seqs) add(s[k]);
        }
    }
    for (int k = 32; k > 0; k >>= 1) sum += __shfl_xor(sum, k);
    sum *= (float)c.kv_heads;
    return (float)p.target / fmaxf(sum, 1.0f);
}

// Where sixteen rows are all that a kv head has, codes are read once, and with pages of a
// tile whole 128-byte lines at a time: the caches need not keep them (32 sequences of 8k: 97
// -> 87 us; with larger pages, where two waves share the lines of the values, 25% slower, and
// with more rows, for which they are read again, 121 -> 150 us at 32, 160 -> 214 us at 44).
template <bool ONCE>
__device__ __forceinline__ uint4 load_codes(const uint8_t *p) {
    typedef uint32_t words __attribute__((ext_vector_type(4)));
    const words *w = reinterpret_cast<const words *>(p);
    const words v = ONCE ? __builtin_nontemporal_load(w) : *w;
    return make_uint4(v[0], v[1], v[2], v[3]);
}

// PAGE: pages of 64 keys (a tile), read once (kOne), of that and more (kLarge), or of fewer (kSmall).  With
// those of a tile or more, a tile's page and scales are the same for all lanes.
enum { kSmall, kOne, kLarge };
template <typename T, int D, int PAGE, int W, bool TREE>
__global__ void __launch_bounds__(64 * W, D > 128 ? 1 : D > 64 ? 2 : 4) split_kernel(AttnArgs p, int row_tiles) {
    constexpr bool BIG = PAGE != kSmall;
    constexpr int kC = D / 64;             // 64-element pieces of a key
    constexpr int kT = D / 16;             // 16-element pieces of a value
    __shared__ float red_m[W][kRows], red_l[W][kRows];
    __shared__ __align__(16) float red_o[W][kRows][D + 4];
    const KvView &c = p.c;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int m = lane & 15, g = lane >> 4;
    // Workgroups go to the XCDs in turn.  A chunk of a sequence, with all of its kv heads and row
    // tiles, stays on one XCD, so that each XCD translates the addresses of its own pages only
    // (with a head to an XCD: 97 -> 112 us on two sequences of 131k tokens).  Chunks after the
    // first come last, so that the workgroups that have none do too.
    const int slot = blockIdx.x / kXcds;
    const int unit_id = slot / (row_tiles * c.kv_heads) * kXcds + blockIdx.x % kXcds;
    const int split = unit_id / c.seqs, b = unit_id % c.seqs;
    const int h = slot / row_tiles % c.kv_heads;
    if (split >= p.most) return;
    const Seq s = load_seq(c, b);
    const int P = 1 << c.log2_page;
    const int total = s.n * p.group;
    if (total >= p.few) return;                // the prompt kernel's
    float per_tile = 0.0f;
    if (p.most > 1) {
        // With many sequences only those who may be cut ask: 1024 of 300 tokens in a call that may
        // have 64k, 760 -> 182 us (142 uncut).  With few, asking at once saves a load's time (0.6 us).
        bool ask = c.seqs < 64;
        if (!ask) {
            const int most = min(p.most, visible_tiles(p, first_place<TREE>(s, 0), s.len - 1, s.len).count() / kLeastChunk);
            if (split >= max(1, most)) return;
            ask = most > 1;
        }
        if (ask) per_tile = chunks_per_tile<TREE>(p);
    }
    for (int rt = slot % row_tiles; rt * kRows < total; rt += row_tiles) {
        const int r0 = rt * kRows, r1 = min(r0 + kRows, total) - 1;
        const int lo = first_place<TREE>(s, r0 / p.group), hi = last_place<TREE>(s, r1 / p.group);
        const Tiles tiles = visible_tiles(p, lo, hi, s.len);
        const int count = tiles.count();
        // its share of the chunks, rounded down: one more than one for each CU would share a CU
        const int chunks = __builtin_amdgcn_readfirstlane(
            max(1, min(min(p.most, count / kLeastChunk), (int)((float)count * per_tile * 1.0001f))));
        if (split >= chunks) continue;
        // Chunks begin at, and waves take, tiles by their number in the sequence modulo the waves:
        // with pages of 128 and more two tiles share each 128-byte line of the values, which two
        // waves should read at the same time (131k tokens: 112 -> 97 us).
        const int shift = tiles.b - tiles.a;
        int t0 = 0, t1 = count;
        if (chunks > 1) {
            const uint32_t each = (uint32_t)count / (uint32_t)chunks, over = count - each * chunks;
            const auto border = [&](uint32_t k) {      // count * k / chunks, in 32 bits
                const int at = (int)(each * k + over * k / (uint32_t)chunks);
                return max(0, at - ((at + shift) & (W - 1)));
            };
            t0 = split == 0 ? 0 : border(split);
            t1 = split + 1 == chunks ? count : border(split + 1);
        }
        const int first = t0 + ((wave - t0 - shift) & (W - 1));
        // this lane's row
        const int r = min(r0 + m, r1);
        const int token = r / p.group, head = h * p.group + r % p.group;
        const int pos = s.first() + token;
        const std::conditional_t<TREE, TreeSight, NoSight> sight(p, s, token);
        const uint16_t *qrow = p.q + (long long)(s.row0 + token) * p.q_stride + head * D;
        // bf16 rows are brought into fp16's range by a power of two of their own (exact but for
        // elements 2^-38 below the largest)
        float up = 1.0f, down = p.scale;
        if constexpr (!__is_same(T, half_t)) {
            float big = 0.0f;
#pragma unroll
            for (int i = 0; i < kC; ++i) {
                float x[8];
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    load8<T>(qrow + 64 * i + 16 * g + 8 * half, x);
#pragma unroll
                    for (int e = 0; e < 8; ++e) big = fmaxf(big, fabsf(x[e]));
                }
            }
            big = fmaxf(big, __shfl_xor(big, 16));
            big = fmaxf(big, __shfl_xor(big, 32));
            const int e = min(max((int)(__builtin_bit_cast(uint32_t, big) >> 23) - 127, -100), 126);
            up = pow2(min(14 - e, 127));
            down = p.scale * pow2(max(e - 14, -126));
        }
        half8_t qf[kC][2];
#pragma unroll
        for (int i = 0; i < kC; ++i)
#pragma unroll
            for (int half = 0; half < 2; ++half) qf[i][half] = as_row_half<T>(qrow + 64 * i + 16 * g + 8 * half, up);

        float mx = kEmpty, l = 0.0f;
        OutUnit unit;                                   // the scale of the values that o counts in
        float4_t o[kT];
#pragma unroll
        for (int i = 0; i < kT; ++i) o[i] = float4_t{0.0f, 0.0f, 0.0f, 0.0f};

        // A tile's page numbers are asked for two tiles ahead, its key codes and scales one, and
        // its value codes as its scores begin: something is always in flight.  (A second set of
        // registers for values a tile ahead gained nothing on short calls and lost 17% on long ones.)
        const int32_t *table = c.page_table + (long long)b * c.table_width;
        int ask_g = -1, ask_k = -1;            // page numbers of the group that the lane scores (g), and loads (m / 4)
        int live_n = 0;
        bool page_n = false;
        float ks_n = 0.0f, vs_n = 0.0f;
        const uint8_t *vp_n = nullptr;
        uint4 kc[4][kC];
        auto ask = [&](int i) {
            const int j0 = tiles.at(i) * kTile, jg = j0 + (BIG ? 0 : 16 * g), jk = j0 + 16 * (m >> 2);
            ask_g = jg < s.len ? table[jg >> c.log2_page] : -1;
            if (!BIG) ask_k = jk < s.len ? table[jk >> c.log2_page] : -1;
        };
        auto fetch = [&](int i) {
            const int j0 = tiles.at(i) * kTile, jg = j0 + 16 * g, jk = j0 + 16 * (m >> 2);
            const int want = BIG ? __builtin_amdgcn_readfirstlane(ask_g) : ask_g;
            const bool ok = (uint32_t)want < (uint32_t)c.pages;
            const int idg = ok ? want : 0, idk = BIG ? idg : (uint32_t)ask_k < (uint32_t)c.pages ? ask_k : 0;
            page_n = ok;
            live_n = ok ? min(max(s.len - jg, 0), 16) : 0;      // keys of group g that exist
            const long long pg = (long long)idg * c.kv_heads + h, pk = BIG ? pg : (long long)idk * c.kv_heads + h;
            const int at_g = BIG ? (j0 & (P - 1)) + 16 * g : jg & (P - 1), at_k = BIG ? (j0 & (P - 1)) + 16 * (m >> 2) : jk & (P - 1);
            const uint8_t *kp = c.k + pk * P * D + (uint32_t)(at_k * D + (m & 3) * D + 16 * g);
            vp_n = c.v + pg * P * D + (uint32_t)(m * P + at_g);
#pragma unroll
            for (int t = 0; t < 4; ++t)
#pragma unroll
                for (int e = 0; e < kC; ++e) kc[t][e] = load_codes<PAGE == kOne>(kp + 4 * t * D + 64 * e);
            ks_n = c.k_scales[pg];
            vs_n = c.v_scales[pg];
        };
        if (first < t1) {
            ask(first);
            fetch(first);
            ask(min(first + W, t1 - 1));
        }
        // One tile, with the next one's loads or without: a condition around the loads would make
        // the products wait for all of them.
        auto tile = [&](int i, auto more) {
            const int j0 = tiles.at(i) * kTile, jg = j0 + 16 * g;
            uint4 vc[kT];
#pragma unroll
            for (int t = 0; t < kT; ++t) vc[t] = load_codes<PAGE == kOne>(vp_n + 16 * t * P);
            __builtin_amdgcn_sched_barrier(0);         // now, not between the products
            // (a page's scales, whether or not all of its keys exist: with BIG the same in all lanes)
            float ks = page_n ? ks_n * down : 0.0f, vs = page_n ? vs_n : 0.0f;
            int live = live_n;
            // taken here, so that the next tile's can be loaded into the same registers (copies of
            // them would wait for every load)
            asm volatile("" : "+v"(ks), "+v"(vs), "+v"(live));
            float x[16];
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                float4_t acc = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                for (int e = 0; e < kC; ++e) {
                    acc = __builtin_amdgcn_mfma_f32_16x16x32_f16(e4m3x8_to_half(kc[t][e].x, kc[t][e].y), qf[e][0], acc, 0, 0, 0);
                    acc = __builtin_amdgcn_mfma_f32_16x16x32_f16(e4m3x8_to_half(kc[t][e].z, kc[t][e].w), qf[e][1], acc, 0, 0, 0);
                }
#pragma unroll
                for (int e = 0; e < 4; ++e) x[4 * t + e] = acc[e] * ks;
            }
            if constexpr (decltype(more)::value) {
                fetch(i + W);
                ask(min(i + 2 * W, t1 - 1));
                __builtin_amdgcn_sched_barrier(0);
            }
            int hidden = hi - p.window;        // keys up to it are out of sight of some of the rows
            if constexpr (TREE) hidden = sight.far;            // (of the lane's)
            const bool whole = live == 16 && j0 + kTile <= lo + 1 && (p.window <= 0 || j0 > hidden || j0 + kTile <= p.sinks);
            if (!__all(whole)) {
                if constexpr (TREE) {
                    const uint32_t see = sight.sixteen(args_again(), jg, live);
#pragma unroll
                    for (int e = 0; e < 16; ++e) x[e] = see >> e & 1 ? x[e] : -__builtin_inff();
                } else {
                    const int far = p.window > 0 ? pos - p.window : -0x7FFFFFFF;      // keys up to it are out of sight
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        const int j = jg + e;
                        const bool see = (e < live) & (j <= pos) & ((j > far) | (j < p.sinks));
                        x[e] = see ? x[e] : -__builtin_inff();
                    }
                }
                // codes of slots that hold no token may be anything, NaN among it
                uint32_t keep[4];
                live_bytes(live, keep);
#pragma unroll
                for (int t = 0; t < kT; ++t) {
                    vc[t].x &= keep[0];
                    vc[t].y &= keep[1];
                    vc[t].z &= keep[2];
                    vc[t].w &= keep[3];
                }
            }
            float top = max3(x[0], x[1], x[2]);
#pragma unroll
            for (int e = 3; e < 15; e += 2) top = max3(top, x[e], x[e + 1]);
            const float own = max3(top, top, x[15]);
            top = group_max(own);
            // What a page's scale is to the outputs' unit goes into the exponent.
            const float lv = __builtin_amdgcn_logf(vs);               // (no page: -inf)
            const float most = BIG ? lv : group_max(lv);
            const float now = fmaxf(mx, top);
            const float need = BIG ? lv + (top - now) : group_max(lv + (own - now));
            if (__any(now != mx || unit.moves(need, most))) {
                l *= __builtin_amdgcn_exp2f(mx - now);
                const float turn = unit.move(need, most, mx - now);
#pragma unroll
                for (int t = 0; t < kT; ++t) o[t] *= turn;
                mx = now;
            }
            const float to_unit = lv > kNone ? lv - unit.at : 0.0f;   // (no weight where there is no page)
            float shift = mx;
            if (__any(fabsf(mx) >= kFar)) {
#pragma unroll
                for (int e = 0; e < 16; ++e) x[e] -= mx;
                shift = 0.0f;
            }
            const float base = kWeightBits + to_unit - shift;
            float back = __builtin_amdgcn_exp2f(-to_unit);
            if (__any(to_unit < kLeastToUnit)) {
#pragma unroll
                for (int e = 0; e < 16; ++e) l += __builtin_amdgcn_exp2f(x[e] + (kWeightBits - shift));
                back = 0.0f;
            }
            float sum = 0.0f;
            uint32_t lead[8], rest[8];
#pragma unroll
            for (int e = 0; e < 16; e += 2) {
                const float a = __builtin_amdgcn_exp2f(x[e] + base), b = __builtin_amdgcn_exp2f(x[e + 1] + base);
                sum += a;
                sum += b;
                lead_and_rest(a, b, lead[e / 2], rest[e / 2]);
            }
            settle(rest);
            const half8_t ph[2] = {halves8(lead), halves8(lead + 4)}, pl[2] = {halves8(rest), halves8(rest + 4)};
            l += sum * back;
#pragma unroll
            for (int t = 0; t < kT; ++t) {
                const half8_t v0 = e4m3x8_to_half(vc[t].x, vc[t].y), v1 = e4m3x8_to_half(vc[t].z, vc[t].w);
                o[t] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v0, ph[0], o[t], 0, 0, 0);
                o[t] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v1, ph[1], o[t], 0, 0, 0);
                o[t] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v0, pl[0], o[t], 0, 0, 0);
                o[t] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v1, pl[1], o[t], 0, 0, 0);
            }
        };
        int i = first;
        for (; i + W < t1; i += W) tile(i, std::true_type{});
        if (i < t1) tile(i, std::false_type{});

        // join the four waves
        l = group_sum(l);
        if (g == 0) {
            red_m[wave][m] = mx;
            red_l[wave][m] = l;
        }
        __syncthreads();
        float all = red_m[0][m];
#pragma unroll
        for (int w = 1; w < W; ++w) all = fmaxf(all, red_m[w][m]);
        float sum = 0.0f;
#pragma unroll
        for (int w = 0; w < W; ++w) sum += red_l[w][m] * __builtin_amdgcn_exp2f(red_m[w][m] - all);
        // over the sum first: outputs that are no larger than the values are; the unit last, which
        // may be the least number
        const float inv = sum > 0.0f || !(sum == sum) ? 1.0f / sum : 0.0f;
        const float f = __builtin_amdgcn_exp2f(mx - all), scale = __builtin_amdgcn_exp2f(unit.at);
#pragma unroll
        for (int e = 0; e < kT; ++e) *reinterpret_cast<float4_t *>(&red_o[wave][m][16 * e + 4 * g]) = o[e] * inv * f * scale;
        __syncthreads();
        // (each wave its own: one after the other into the same took 0.8 us longer, 4 with 256 elements)
        const auto joined = [&](int row, int e) {
            float4_t y = *reinterpret_cast<const float4_t *>(&red_o[0][row][e]);
#pragma unroll
            for (int w = 1; w < W; ++w) y += *reinterpret_cast<const float4_t *>(&red_o[w][row][e]);
            return y;
        };
        if (chunks == 1) {
            // a row of D outputs by 16 lanes
            const int rr = threadIdx.x >> 4;
            if (rr < kRows && r0 + rr <= r1) {
                const int tok = (r0 + rr) / p.group, hd = h * p.group + (r0 + rr) % p.group;
                uint16_t *dst = p.out + ((long long)(s.row0 + tok) * p.q_heads + hd) * D;
                for (int e = (threadIdx.x & 15) * 8; e < D; e += 128) {
                    const float4_t a = joined(rr, e), b = joined(rr, e + 4);
                    const float y[8] = {a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
                    *reinterpret_cast<uint4 *>(dst + e) = pack8<T>(y);
                }
            }
        } else {
            const int rr = threadIdx.x >> 4;
            if (rr < kRows && r0 + rr <= r1) {
                const int tok = (r0 + rr) / p.group, hd = h * p.group + (r0 + rr) % p.group;
                float *dst = p.part + (((long long)(s.row0 + tok) * p.q_heads + hd) * p.splits + split) * kPart<D>;
                for (int e = (threadIdx.x & 15) * 4; e < D; e += 64)
                    *reinterpret_cast<float4_t *>(dst + e) = joined(rr, e);
                const float total_l = __shfl(sum, rr & 15), total_m = __shfl(all, rr & 15);  // lane m == rr of any group holds row rr's
                if ((threadIdx.x & 15) == 0) {
                    dst[D] = total_m;
                    dst[D + 1] = total_l;
                    dst[D + 2] = (float)chunks;
                }
            }
        }
        if (chunks == 1 && p.part != nullptr) {
            const int rr = threadIdx.x;
            if (rr < kRows && r0 + rr <= r1) {
                const int tok = (r0 + rr) / p.group, hd = h * p.group + (r0 + rr) % p.group;
                p.part[((long long)(s.row0 + tok) * p.q_heads + hd) * p.splits * kPart<D> + D + 2] = 1.0f;
            }
        }
        __syncthreads();                    // red_* are free again
    }
}

template <typename T, int D, int W, bool TREE>
void launch_split(const AttnArgs &p, int row_tiles, int grid, hipStream_t s) {
    const int page = 1 << p.c.log2_page;
    if (page == kTile && row_tiles == 1)
        split_kernel<T, D, kOne, W, TREE><<<grid, 64 * W, 0, s>>>(p, row_tiles);
    else if (page >= kTile)
        split_kernel<T, D, kLarge, W, TREE><<<grid, 64 * W, 0, s>>>(p, row_tiles);
    else
        split_kernel<T, D, kSmall, W, TREE><<<grid, 64 * W, 0, s>>>(p, row_tiles);
}

template <typename T, bool TREE>
hipError_t launch_split_dim(const AttnArgs &p, int D, bool wide, int row_tiles, int grid, hipStream_t s) {
    switch (D) {
    case 64:
        if (wide)
            launch_split<T, 64, 2 * kWaves, TREE>(p, row_tiles, grid, s);
        else
            launch_split<T, 64, kWaves, TREE>(p, row_tiles, grid, s);
        break;
    case 128: launch_split<T, 128, kWaves, TREE>(p, row_tiles, grid, s); break;
    case 256: launch_split<T, 256, kWaves, TREE>(p, row_tiles, grid, s); break;
    default: return hipErrorInvalidValue;
    }
    return hipGetLastError();
}

template <bool TREE>
hipError_t launch_split_rows(const AttnArgs &p, int head_dim, bool bf16, bool wide, int row_tiles, hipStream_t s) {
    const int units = (p.c.seqs * p.most + kXcds - 1) / kXcds * kXcds;
    const int grid = units * p.c.kv_heads * row_tiles;
    return bf16 ? launch_split_dim<bhalf_t, TREE>(p, head_dim, wide, row_tiles, grid, s)
                : launch_split_dim<half_t, TREE>(p, head_dim, wide, row_tiles, grid, s);
}

}  // namespace
}  // namespace awq
