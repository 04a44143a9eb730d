// awq_attention: attention of a ragged batch over the 8-bit paged cache.
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
// combine_kernel joins the chunks' partial results (fp32, in the workspace)
// where there is more than one chunk.
#include <algorithm>
#include <type_traits>

#include "awq_attention.h"
#include "awq_internal.h"

namespace awq {
namespace {

constexpr int kRows = 16;                  // rows of a workgroup
constexpr int kWaves = 4;
constexpr int kXcds = 8;
constexpr float kWeightBits = 14.0f;       // weights are 2^14 times those of the formula

// How a call is cut into chunks of keys, from the number of (sequence, kv head, row
// tile) groups and, on the device, from the sequences' lengths.  Measured at 32 heads
// over 8 of 128 elements, pages of 64 (us):
//   not cut / dealt to 256 / 512 / 1024 workgroups
//   1 sequence of 300: 7.3 / 10.0 / 10.0 / 10.0;  of 1000: 10.8 / 10.4 / 10.4 / 10.4
//   1 of 32k: 211 / 19.0 / 19.8 / 25.6;  8 of 4k to 8k: 57 / 34.3 / 31.3 / 37.3
//   16 of 4k to 8k: 68 / 58.1 / 46.5 / 53.1;  24 of 3k to 6k: 53.9 / 56.5 / 55.4 / 57.8
//   64 of 1k to 2k: 39.8 / 45.1 / 45.0 / 48.8
// So: few tiles take no longer than the launch that joins chunks (and the call itself,
// which is some 4 us shorter for one launch); one workgroup for
// each CU streams as fast as the memory, while sequences of different lengths need a
// finer cut; and many groups need no cut, unless sequences may be so long that one
// among short ones would be the last by far.
constexpr int kUncutTiles = 12, kManyGroups = 192, kLongTiles = 256, kLeastChunk = 4, kMaxSplits = 256;
constexpr int kJoinGroups = 8192;          // workgroups that join chunks
constexpr size_t kMixedRoom = 1u << 28;    // bytes of partial results for single tokens among prompts

// Chunks for a tile: from the tiles that all sequences' rows see, for all kv heads.
// The host knows no lengths, so each wave adds them up, with more than 64 sequences four
// to a lane at a time.
__device__ __forceinline__ float chunks_per_tile(const AttnArgs &p) {
    const KvView &c = p.c;
    float sum = 0.0f;
    const auto add = [&](const Seq &s) {
        if (s.n > 0 && s.n * p.group < p.few)
            sum += (float)visible_tiles(p, s.first(), s.len - 1, s.len).count() * (float)((s.n * p.group + kRows - 1) / kRows);
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
template <typename T, int D, int PAGE, int W>
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
            const int most = min(p.most, visible_tiles(p, s.first(), s.len - 1, s.len).count() / kLeastChunk);
            if (split >= max(1, most)) return;
            ask = most > 1;
        }
        if (ask) per_tile = chunks_per_tile(p);
    }
    for (int rt = slot % row_tiles; rt * kRows < total; rt += row_tiles) {
        const int r0 = rt * kRows, r1 = min(r0 + kRows, total) - 1;
        const int lo = s.first() + r0 / p.group, hi = s.first() + r1 / p.group;
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
            const bool whole = live == 16 && j0 + kTile <= lo + 1 &&
                               (p.window <= 0 || j0 > hi - p.window || j0 + kTile <= p.sinks);
            if (!__all(whole)) {
                const int far = p.window > 0 ? pos - p.window : -0x7FFFFFFF;      // keys up to it are out of sight
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    const int j = jg + e;
                    const bool see = (e < live) & (j <= pos) & ((j > far) | (j < p.sinks));
                    x[e] = see ? x[e] : -__builtin_inff();
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

// A workgroup joins the chunks of one (row, head) after the other: D / 4 threads to a chunk, as many
// chunks at once as that leaves room for, then the threads' sums through LDS.
// Bound: latency (a few loads in a row), and the launch.
template <typename T, int D>
__global__ void __launch_bounds__(256) combine_kernel(AttnArgs p) {
    constexpr int kLanes = D / 4, kAtOnce = 256 / kLanes;
    __shared__ float weight[kMaxSplits], red[2][4];
    __shared__ float4_t part[kAtOnce][kLanes];
    const KvView &c = p.c;
    const int tid = threadIdx.x;
    const int row0 = min(max(c.q_starts[0], 0), c.rows), row1 = min(max(c.q_starts[c.seqs], 0), c.rows);
    for (int i = row0 * p.q_heads + blockIdx.x; i < row1 * p.q_heads; i += gridDim.x) {
        const float *src = p.part + (long long)i * p.splits * kPart<D>;
        const int n = min((int)src[D + 2], p.splits);
        if (n <= 1) continue;                  // the one chunk has written its outputs
        // one chunk's maximum and sum to a thread
        float own = kEmpty, l = 0.0f;
        if (tid < n) {
            own = src[tid * kPart<D> + D];
            l = src[tid * kPart<D> + D + 1];
        }
        float mx = own;
        for (int k = 32; k > 0; k >>= 1) mx = fmaxf(mx, __shfl_xor(mx, k));
        if ((tid & 63) == 0) red[0][tid >> 6] = mx;
        __syncthreads();
        mx = fmaxf(fmaxf(red[0][0], red[0][1]), fmaxf(red[0][2], red[0][3]));
        l = tid < n ? l * __builtin_amdgcn_exp2f(own - mx) : 0.0f;
        if (tid < n) weight[tid] = l;
        for (int k = 32; k > 0; k >>= 1) l += __shfl_xor(l, k);
        if ((tid & 63) == 0) red[1][tid >> 6] = l;
        __syncthreads();
        l = (red[1][0] + red[1][1]) + (red[1][2] + red[1][3]);
        const float inv = l > 0.0f || !(l == l) ? 1.0f / l : 0.0f;
        const int lane = tid % kLanes, at = tid / kLanes;
        float4_t o = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 4
        for (int k = at; k < n; k += kAtOnce)
            o += weight[k] * inv * *reinterpret_cast<const float4_t *>(src + k * kPart<D> + 4 * lane);
        part[at][lane] = o;
        __syncthreads();
        if (at == 0) {
#pragma unroll
            for (int k = 1; k < kAtOnce; ++k) o += part[k][lane];
            uint2 y;
            y.x = (uint32_t)from_float<T>(o[0]) | ((uint32_t)from_float<T>(o[1]) << 16);
            y.y = (uint32_t)from_float<T>(o[2]) | ((uint32_t)from_float<T>(o[3]) << 16);
            *reinterpret_cast<uint2 *>(p.out + (long long)i * D + 4 * lane) = y;
        }
        __syncthreads();                       // the LDS arrays are free again
    }
}

// Rows of a sequence and kv head from which the prompt kernel takes a call, by the width of
// heads, the pairs of sequence and kv head, and the tiles of keys of all pairs.  The split kernel
// reads keys and values again for every sixteen rows; the prompt kernel is slower to start, and
// cuts a row tile into 32 chunks at most, so with few pairs most of the GPU has nothing to do.
// With fewer sequences than XCDs the split kernel's chunks leave some of these idle.
// Measured (us, split / prompt, by rows times query heads to a kv head, pages of 64):
//   heads of 128                 32        64        96       128       256       512
//   1 x 1 kv head, 16k        20/25     20/26     22/28     20/28     23/29     27/31
//   1 x 1, 131k              22/114    27/119    48/121    38/124    60/125   115/128
//   1 x 2, 131k              28/115    39/120    81/123    61/123   104/128   464/137
//   1 x 8, 500                13/21     14/21     14/22     14/23     21/24     36/24
//   1 x 8, 4000               19/24     19/25     24/27     29/28     48/32    182/45
//   1 x 8, 16k                21/26     27/28     51/32     63/33    109/47    681/72
//   1 x 8, 131k              66/118   107/124   293/132   359/137   801/222  4788/418
//   16 x 1, 4000              19/26     21/27     27/30     29/32     30/42     51/53
//   16 x 1, 16k               26/30     40/39     50/42     64/48     92/72   169/119
//   16 x 1, 131k            126/132   244/184   298/207   462/232   704/435  1366/802
//   16 x 2, 4000              21/27     30/34     30/38     30/40     51/51     92/80
//   16 x 2, 16k               40/43     64/58     91/65     94/71   170/121   326/211
//   16 x 8, 500               14/21     14/24     18/25     22/26     37/28     66/39
//   16 x 8, 4000              31/46     50/62     71/70     92/81   173/140   336/185
//   16 x 8, 16k             107/126   183/178   257/196   331/233   650/418  1278/713
//   heads of 64: 1 x 8, 500   14/17     14/17     14/18     14/18     13/19     20/19
//   1 x 8, 4000               20/20     19/22     21/23     20/23     50/25     90/35
//   1 x 8, 16k                20/23     22/24     33/26     39/28     61/37    289/55
//   1 x 8, 131k               46/90     76/97    153/99   188/100   409/150  1918/277
//   16 x 2, 4000              19/23     19/27     19/30     19/33     31/41     50/66
//   16 x 2, 16k               31/34     41/46     63/50     64/52     93/86   158/152
//   16 x 8, 4000              20/37     30/52     39/58     48/64    85/109   153/125
//   16 x 8, 16k               63/94    93/136   123/146   155/156   284/287   538/472
//   heads of 256: 1 x 2, 131k 45/126   66/132   152/135   109/133   195/147   803/208
//   1 x 8, 500                15/23     15/25     26/26     26/26     50/26     97/26
//   1 x 8, 4000               21/27     26/30     44/32     55/34     96/42    388/51
//   1 x 8, 16k                33/30     46/35     95/43    117/48    219/71  1384/117
//   16 x 1, 4000              30/29     31/32     50/37     53/40     53/49     99/74
//   16 x 2, 16k               67/55    120/78   175/105   178/113   333/201   661/376
//   16 x 8, 500               16/25     28/28     40/29     51/30     96/39    187/70
//   16 x 8, 4000              54/57    101/79   146/114   192/124   375/184   750/341
int prompt_rows(int seqs, int kv_heads, long long tiles, int head_dim) {
    static const int rows[3][2][5] = {{{80, 80, 80, 144, 512}, {96, 128, 768, 768, 768}},
                                      {{72, 72, 72, 120, 288}, {64, 96, 256, 384, 768}},
                                      {{24, 24, 24, 72, 96}, {24, 24, 40, 72, 288}}};
    const long long pairs = (long long)seqs * kv_heads, all = pairs * tiles;
    const int width = head_dim > 128 ? 2 : head_dim > 64 ? 1 : 0;
    const int at = all >= 12000 ? 0 : all >= 3000 ? 1 : all >= 1500 ? 2 : all >= 400 ? 3 : 4;
    return (int)std::max<long long>(rows[width][seqs >= kXcds][at], (width == 2 ? 320 : 640) / pairs);
}

// The grid of a call: the most chunks, whose number is found on the device, and the
// workgroups that they are dealt to.
// Where most sequences have far fewer rows than the longest, each kernel takes those that
// suit it (one sequence of 2048 rows, 63 of one, all over 4k keys: 810 us with the prompt
// kernel alone, 235 with both, before weights were two halves, 255 since; 255 of one: 1854,
// 476 and 494), and cuts them by a number of its own (one of 2048 rows and one single token
// over 131k keys: 930 -> 221 us, the prompt alone 70).
struct Plan {
    bool prompt, mixed;      // whether the prompt kernel is needed, and both are
    bool wide;               // eight waves to a workgroup
    int few, prompt_tiles, prompt_splits;
    int row_tiles, splits, target;
    int room() const { return std::max(splits, prompt_splits); }
};
Plan plan(int seqs, int rows, int kv_heads, int group, int head_dim, int max_q, int max_kv, int window, int sinks) {
    Plan pl;
    long long keys = max_kv;
    if (window > 0) keys = std::min(keys, (long long)window + max_q + std::min(sinks, max_kv) + 2 * kTile);
    const long long tiles = (keys + kTile - 1) / kTile;
    pl.few = prompt_rows(seqs, kv_heads, tiles, head_dim);
    pl.prompt = (long long)max_q * group >= pl.few;
    pl.mixed = pl.prompt && rows_differ(seqs, rows, max_q);
    pl.row_tiles = pl.target = 0;
    pl.splits = pl.prompt_splits = 1;
    pl.wide = false;
    if (pl.prompt) {
        pl.prompt_tiles = prefill_row_tiles(seqs, rows, kv_heads, group, head_dim, max_q, pl.few, pl.mixed);
        pl.prompt_splits = prefill_splits(seqs, kv_heads, pl.prompt_tiles, pl.mixed, tiles);
        if (!pl.mixed) return pl;
    }
    // (the kernel steps on where the grid is cut)
    const int units = (seqs + kXcds - 1) / kXcds * kXcds;
    const long long some = pl.mixed ? std::min((rows - max_q) / (seqs - 1) + 1, (pl.few - 1) / group + 1) : max_q;
    pl.row_tiles = (int)std::min<long long>((some * group + kRows - 1) / kRows,
                                            std::max(1, ((1 << 24) - 1) / (units * kv_heads)));
    const long long groups = (long long)seqs * kv_heads * pl.row_tiles;
    pl.target = groups <= 64 ? 256 : 512;
    // lengths may differ by much; but a workgroup that has no chunk takes its launch
    // (8 kv heads of 1024 sequences of 300 tokens: 274 us at eight chunks, 209 at four; of 4096,
    // 1126 at eight, 692 at two)
    long long want = groups >= 16384 ? 2 : groups >= 4096 ? 4 : std::max(8ll, 4 * ((pl.target + groups - 1) / groups));
    // Heads of 64 (8 kv heads; us, four waves and joined or not / eight waves and not cut):
    // 1, 16, 32, 48 sequences of 500 to 1000: 9.1 / 7.4, 11.9 / 8.2, 8.7 / 8.6, 11.6 / 12.0; of 1k to
    // 2k 9.2 / 10.2, 13.5 / 10.7, 13.3 / 12.6, 18.3 / 18.8; of 3k to 6k 10.6 / 21.8, 23.1 / 24.2,
    // 30.6 / 29.0, 43.0 / 44.7; of 250 to 500 5.9 / 5.9 at one.  With heads of 128 a CU has room for
    // eight waves, whose workgroup is no faster (1 of 1000: 12.1 / 12.3).
    pl.wide = !pl.mixed && head_dim == 64 && groups <= 256 && tiles > kUncutTiles && tiles <= std::max(24ll, groups / 2);
    if (tiles <= kUncutTiles || pl.wide || (groups >= kManyGroups && tiles <= kLongTiles)) want = 1;
    pl.splits = (int)std::max<long long>(1, std::min<long long>({want, (tiles + kLeastChunk - 1) / kLeastChunk, kMaxSplits}));
    // Partial results have room by rows, the prompts' among them.
    if (pl.mixed) {
        const size_t each = (size_t)rows * kv_heads * group * (head_dim + 4) * sizeof(float);
        pl.splits = (int)std::max<long long>(1, std::min<long long>(pl.splits, (long long)(kMixedRoom / each)));
    }
    // (a launch has less than 2^32 threads)
    const long long once = (long long)(units + kXcds) * pl.splits * kv_heads;
    pl.row_tiles = (int)std::max<long long>(1, std::min<long long>(pl.row_tiles, ((1 << 24) - 1) / once));
    return pl;
}

template <typename T, int D, int W>
void launch_split(const AttnArgs &p, int row_tiles, int grid, hipStream_t s) {
    const int page = 1 << p.c.log2_page;
    if (page == kTile && row_tiles == 1)
        split_kernel<T, D, kOne, W><<<grid, 64 * W, 0, s>>>(p, row_tiles);
    else if (page >= kTile)
        split_kernel<T, D, kLarge, W><<<grid, 64 * W, 0, s>>>(p, row_tiles);
    else
        split_kernel<T, D, kSmall, W><<<grid, 64 * W, 0, s>>>(p, row_tiles);
}

template <typename T, int D>
hipError_t launch(AttnArgs p, const Plan &pl, bool bf16, hipStream_t s) {
    hipError_t e = hipSuccess;
    if (pl.prompt) {
        p.few = pl.mixed ? pl.few : 0;
        p.most = pl.prompt_splits;
        e = launch_attention_prefill(p, D, bf16, pl.prompt_tiles, pl.mixed, s);
        if (e != hipSuccess) return e;
    }
    if (!pl.prompt || pl.mixed) {
        p.few = pl.mixed ? pl.few : 0x7FFFFFFF;
        p.most = pl.splits;
        const int units = (p.c.seqs * pl.splits + kXcds - 1) / kXcds * kXcds;
        const int grid = units * p.c.kv_heads * pl.row_tiles;
        if constexpr (D == 64) {
            if (pl.wide)
                launch_split<T, D, 2 * kWaves>(p, pl.row_tiles, grid, s);
            else
                launch_split<T, D, kWaves>(p, pl.row_tiles, grid, s);
        } else {
            launch_split<T, D, kWaves>(p, pl.row_tiles, grid, s);
        }
        e = hipGetLastError();
    }
    if (e != hipSuccess || p.part == nullptr) return e;
    combine_kernel<T, D><<<(int)std::min<long long>((long long)p.c.rows * p.q_heads, kJoinGroups), 256, 0, s>>>(p);
    return hipGetLastError();
}

template <typename T>
hipError_t launch_dim(const AttnArgs &p, int D, const Plan &pl, bool bf16, hipStream_t s) {
    switch (D) {
    case 64: return launch<T, 64>(p, pl, bf16, s);
    case 128: return launch<T, 128>(p, pl, bf16, s);
    case 256: return launch<T, 256>(p, pl, bf16, s);
    }
    return hipErrorInvalidValue;
}

}  // namespace

size_t attention_workspace(int seqs, int rows, int q_heads, int kv_heads, int head_dim, int max_q,
                           int max_kv, int window, int sinks) {
    const Plan pl = plan(seqs, rows, kv_heads, q_heads / kv_heads, head_dim, max_q, max_kv, window, sinks);
    if (pl.room() == 1) return 0;
    return (size_t)rows * q_heads * pl.room() * (head_dim + 4) * sizeof(float);
}

hipError_t launch_attention(const KvView &c, int head_dim, const uint16_t *q, long long q_stride,
                            uint16_t *out, int q_heads, bool bf16, float scale, int window, int sinks,
                            int max_q, int max_kv, void *workspace, hipStream_t s) {
    const Plan pl = plan(c.seqs, c.rows, c.kv_heads, q_heads / c.kv_heads, head_dim, max_q, max_kv, window, sinks);
    AttnArgs p{c, q, q_stride, out, pl.room() > 1 ? (float *)workspace : nullptr, q_heads,
               q_heads / c.kv_heads, scale * kLog2e, std::min(window, kWidest), sinks, 1, pl.target, pl.room(), 0};
    return bf16 ? launch_dim<bhalf_t>(p, head_dim, pl, bf16, s) : launch_dim<half_t>(p, head_dim, pl, bf16, s);
}

}  // namespace awq
