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
// split_kernel.  A workgroup of four waves takes sixteen rows (row r of a kv
// head: token r / group, head r % group) of one kv head and one sequence, over
// a chunk of the keys; the waves take its 64-key tiles in turn.  The products
// run transposed, on v_mfma_f32_16x16x32_f16: S^T = K Q^T, so a lane holds
// sixteen scores of one row, and O^T = V^T P^T, whose operand P^T is what the
// lane already holds, without a lane exchange.  For that the keys of a tile are
// dealt to the four 16-key products so that lane group g = lane / 16 ends up
// with the keys 16 g .. 16 g + 15, which are sixteen consecutive bytes of a row
// of V^T: every load is 16 bytes a lane, and 16 keys never leave a page.
// Weights are held to fp16 twice, as a leading part and its remainder: the
// second product is free beside the loads, and the result keeps fp32's quality.
// Weights are scaled by 2^14 so that the small ones stay normal fp16 numbers.
// Bound: the bytes of K and V (HBM).
//
// combine_kernel joins the chunks' partial results (fp32, in the workspace)
// where there is more than one chunk.
#include <algorithm>

#include "awq_attention.h"
#include "awq_internal.h"

namespace awq {
namespace {

constexpr int kRows = 16;                  // rows of a workgroup
constexpr int kWaves = 4;
constexpr float kWeightBits = 14.0f;       // weights are 2^14 times those of the formula

// A partial result: D outputs, then the maximum and the sum.
template <int D>
constexpr int kPart = D + 4;

template <typename T, int D>
__global__ void __launch_bounds__(64 * kWaves) split_kernel(AttnArgs p) {
    constexpr int kC = D / 64;             // 64-element pieces of a key
    constexpr int kT = D / 16;             // 16-element pieces of a value
    __shared__ float red_m[kWaves][kRows], red_l[kWaves][kRows];
    __shared__ float red_o[kRows][D + 4];
    const KvView &c = p.c;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int m = lane & 15, g = lane >> 4;
    const int split = blockIdx.x, b = blockIdx.z;
    const int h = blockIdx.y % c.kv_heads;
    const Seq s = load_seq(c, b);
    const int P = 1 << c.log2_page;
    const int total = s.n * p.group;
    const int row_tiles = gridDim.y / c.kv_heads;
    for (int rt = blockIdx.y / c.kv_heads; rt * kRows < total; rt += row_tiles) {
        const int r0 = rt * kRows, r1 = min(r0 + kRows, total) - 1;
        const int lo = s.first() + r0 / p.group, hi = s.first() + r1 / p.group;
        const Tiles tiles = visible_tiles(p, lo, hi, s.len);
        const int count = tiles.count();
        const int chunk = max(p.chunk, (count + p.splits - 1) / p.splits);
        const int t0 = split * chunk, t1 = min(count, t0 + chunk);
        if (t0 >= t1 && split > 0) continue;
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

        float mx = kEmpty, l = 0.0f, unit = 1.0f;       // unit: the scale of the values that o counts in
        float4_t o[kT];
#pragma unroll
        for (int i = 0; i < kT; ++i) o[i] = float4_t{0.0f, 0.0f, 0.0f, 0.0f};

        for (int i = t0 + wave; i < t1; i += kWaves) {
            const int j0 = tiles.at(i) * kTile;
            // the page of the sixteen keys that this lane scores (group g), and of those whose
            // codes it loads as keys (group m / 4)
            const int jg = j0 + 16 * g, jk = j0 + 16 * (m >> 2);
            int idg = 0, idk = 0;
            if (jg < s.len) idg = c.page_table[(long long)b * c.table_width + (jg >> c.log2_page)];
            if (jk < s.len) idk = c.page_table[(long long)b * c.table_width + (jk >> c.log2_page)];
            int live = min(max(s.len - jg, 0), 16);     // keys of group g that exist
            if (idg < 0 || idg >= c.pages) {
                idg = 0;
                live = 0;
            }
            if (idk < 0 || idk >= c.pages) idk = 0;
            const long long pg = (long long)idg * c.kv_heads + h;
            const uint8_t *kp = c.k + ((long long)idk * c.kv_heads + h) * P * D + (jk & (P - 1)) * D + (m & 3) * D + 16 * g;
            const uint8_t *vp = c.v + pg * P * D + m * P + (jg & (P - 1));
            uint4 kc[4][kC], vc[kT];
#pragma unroll
            for (int t = 0; t < 4; ++t)
#pragma unroll
                for (int e = 0; e < kC; ++e) kc[t][e] = *reinterpret_cast<const uint4 *>(kp + 4 * t * D + 64 * e);
#pragma unroll
            for (int t = 0; t < kT; ++t) vc[t] = *reinterpret_cast<const uint4 *>(vp + 16 * t * P);
            const float ks = live ? c.k_scales[pg] * down : 0.0f;
            float vs = live ? c.v_scales[pg] : 0.0f;

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
            const bool whole = live == 16 && j0 + kTile <= lo + 1 &&
                               (p.window <= 0 || j0 > hi - p.window || j0 + kTile <= p.sinks);
            if (!__all(whole)) {
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    const int j = jg + e;
                    const bool see = e < live && j <= pos && (p.window <= 0 || j > pos - p.window || j < p.sinks);
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
            float top = x[0];
#pragma unroll
            for (int e = 1; e < 16; ++e) top = fmaxf(top, x[e]);
            top = fmaxf(top, __shfl_xor(top, 16));
            top = fmaxf(top, __shfl_xor(top, 32));
            const float now = fmaxf(mx, top);
            // the values of this tile count in units of its largest scale
            float vmax = fmaxf(vs, __shfl_xor(vs, 16));
            vmax = fmaxf(vmax, __shfl_xor(vmax, 32));
            if (!(vmax > 0.0f)) vmax = unit;
            const float ratio = vs / vmax;
            const float alpha = __builtin_amdgcn_exp2f(mx - now);
            const float turn = alpha * (unit / vmax);
            unit = vmax;
            mx = now;
            const float base = now - kWeightBits;
            float sum = 0.0f;
            half8_t ph[2], pl[2];
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                const float w = __builtin_amdgcn_exp2f(x[e] - base);
                sum += w;
                const float wv = w * ratio;
                const half_t lead = (half_t)wv;
                ph[e >> 3][e & 7] = lead;
                pl[e >> 3][e & 7] = (half_t)(wv - (float)lead);
            }
            l = l * alpha + sum;
            if (__any(turn != 1.0f)) {
#pragma unroll
                for (int t = 0; t < kT; ++t) o[t] *= turn;
            }
#pragma unroll
            for (int t = 0; t < kT; ++t) {
                const half8_t v0 = e4m3x8_to_half(vc[t].x, vc[t].y), v1 = e4m3x8_to_half(vc[t].z, vc[t].w);
                o[t] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v0, ph[0], o[t], 0, 0, 0);
                o[t] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v1, ph[1], o[t], 0, 0, 0);
                o[t] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v0, pl[0], o[t], 0, 0, 0);
                o[t] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v1, pl[1], o[t], 0, 0, 0);
            }
        }

        // join the four waves
        l += __shfl_xor(l, 16);
        l += __shfl_xor(l, 32);
        if (g == 0) {
            red_m[wave][m] = mx;
            red_l[wave][m] = l;
        }
        __syncthreads();
        float all = red_m[0][m];
#pragma unroll
        for (int w = 1; w < kWaves; ++w) all = fmaxf(all, red_m[w][m]);
        float sum = 0.0f;
#pragma unroll
        for (int w = 0; w < kWaves; ++w) sum += red_l[w][m] * __builtin_amdgcn_exp2f(red_m[w][m] - all);
        const float f = unit * __builtin_amdgcn_exp2f(mx - all);
        for (int w = 0; w < kWaves; ++w) {
            if (wave == w) {
#pragma unroll
                for (int t = 0; t < kT; ++t) {
                    float4_t *at = reinterpret_cast<float4_t *>(&red_o[m][16 * t + 4 * g]);
                    *at = (w == 0 ? float4_t{0.0f, 0.0f, 0.0f, 0.0f} : *at) + o[t] * f;
                }
            }
            __syncthreads();
        }
        if (p.part == nullptr) {
            // a row of D outputs by 16 lanes
            const int rr = threadIdx.x >> 4;
            if (r0 + rr <= r1) {
                const float total_l = __shfl(sum, rr & 15);       // lane m == rr of any group holds row rr's sum
                const float inv = total_l > 0.0f || !(total_l == total_l) ? 1.0f / total_l : 0.0f;
                const int tok = (r0 + rr) / p.group, hd = h * p.group + (r0 + rr) % p.group;
                uint16_t *dst = p.out + ((long long)(s.row0 + tok) * p.q_heads + hd) * D;
                for (int e = (threadIdx.x & 15) * 8; e < D; e += 128) {
                    float y[8];
#pragma unroll
                    for (int u = 0; u < 8; ++u) y[u] = red_o[rr][e + u] * inv;
                    *reinterpret_cast<uint4 *>(dst + e) = pack8<T>(y);
                }
            }
        } else {
            const int rr = threadIdx.x >> 4;
            if (r0 + rr <= r1) {
                const int tok = (r0 + rr) / p.group, hd = h * p.group + (r0 + rr) % p.group;
                float *dst = p.part + (((long long)(s.row0 + tok) * p.q_heads + hd) * p.splits + split) * kPart<D>;
                for (int e = (threadIdx.x & 15) * 4; e < D; e += 64)
                    *reinterpret_cast<float4_t *>(dst + e) = *reinterpret_cast<const float4_t *>(&red_o[rr][e]);
                const float total_l = __shfl(sum, rr & 15), total_m = __shfl(all, rr & 15);
                if ((threadIdx.x & 15) == 0) {
                    dst[D] = total_m;
                    dst[D + 1] = total_l;
                }
            }
        }
        __syncthreads();                    // red_* are free again
    }
}

// One wave joins the chunks of one (row, head).
template <typename T, int D>
__global__ void __launch_bounds__(256) combine_kernel(AttnArgs p) {
    const KvView &c = p.c;
    const int lane = threadIdx.x & 63;
    const int b = blockIdx.z;
    const Seq s = load_seq(c, b);
    const int waves = gridDim.x * 4;
    for (int i = blockIdx.x * 4 + (threadIdx.x >> 6); i < s.n * p.q_heads; i += waves) {
        const int token = i / p.q_heads, head = i % p.q_heads;
        // the chunks that the split kernel made of this row's tile
        const int r = token * p.group + head % p.group;
        const int r0 = r / kRows * kRows, r1 = min(r0 + kRows, s.n * p.group) - 1;
        const Tiles tiles = visible_tiles(p, s.first() + r0 / p.group, s.first() + r1 / p.group, s.len);
        const int count = tiles.count();
        const int chunk = max(p.chunk, (count + p.splits - 1) / p.splits);
        const int n = max(1, (count + chunk - 1) / chunk);
        const float *src = p.part + ((long long)(s.row0 + token) * p.q_heads + head) * p.splits * kPart<D>;
        float mx = kEmpty;
        for (int k = 0; k < n; ++k) mx = fmaxf(mx, src[k * kPart<D> + D]);
        float o[D / 64] = {}, l = 0.0f;
        for (int k = 0; k < n; ++k) {
            const float f = __builtin_amdgcn_exp2f(src[k * kPart<D> + D] - mx);
            l += f * src[k * kPart<D> + D + 1];
#pragma unroll
            for (int e = 0; e < D / 64; ++e) o[e] += f * src[k * kPart<D> + 64 * e + lane];
        }
        const float inv = l > 0.0f || !(l == l) ? 1.0f / l : 0.0f;
        uint16_t *dst = p.out + ((long long)(s.row0 + token) * p.q_heads + head) * D;
#pragma unroll
        for (int e = 0; e < D / 64; ++e) dst[64 * e + lane] = from_float<T>(o[e] * inv);
    }
}

// How a call is cut: chunks and their least length.  Enough workgroups for the
// 256 CUs, but no chunk below eight tiles (two for each wave).
constexpr int kWantGroups = 1024, kLeastChunk = 8, kMaxSplits = 256;

struct Plan {
    int row_tiles, splits, chunk;
};
Plan plan(int seqs, int kv_heads, int group, int max_q, int max_kv, int window, int sinks) {
    Plan pl;
    // (the kernel steps on where the grid is cut)
    pl.row_tiles = (int)std::min<long long>(((long long)max_q * group + kRows - 1) / kRows, 65535 / kv_heads);
    long long keys = max_kv;
    if (window > 0) keys = std::min(keys, (long long)window + max_q + std::min(sinks, max_kv) + 2 * kTile);
    const int tiles = (int)((keys + kTile - 1) / kTile);
    const long long groups = (long long)seqs * kv_heads * pl.row_tiles;
    const int want = (int)std::min<long long>(kMaxSplits, std::max<long long>(1, kWantGroups / groups));
    pl.chunk = std::max(kLeastChunk, (tiles + want - 1) / want);
    pl.splits = std::max(1, (tiles + pl.chunk - 1) / pl.chunk);
    return pl;
}

template <typename T, int D>
hipError_t launch(AttnArgs p, const Plan &pl, int max_q, hipStream_t s) {
    const dim3 grid(pl.splits, pl.row_tiles * p.c.kv_heads, p.c.seqs);
    split_kernel<T, D><<<grid, 64 * kWaves, 0, s>>>(p);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || p.part == nullptr) return e;
    combine_kernel<T, D><<<dim3((max_q * p.q_heads + 3) / 4, 1, p.c.seqs), 256, 0, s>>>(p);
    return hipGetLastError();
}

template <typename T>
hipError_t launch_dim(const AttnArgs &p, int D, const Plan &pl, int max_q, hipStream_t s) {
    switch (D) {
    case 64: return launch<T, 64>(p, pl, max_q, s);
    case 128: return launch<T, 128>(p, pl, max_q, s);
    case 256: return launch<T, 256>(p, pl, max_q, s);
    }
    return hipErrorInvalidValue;
}

}  // namespace

// Rows of a sequence and kv head from which the prompt kernel takes the call.
constexpr int kPrefillRows = 128;
bool prefill_rows(int group, int max_q) { return (long long)max_q * group >= kPrefillRows; }

size_t attention_workspace(int seqs, int rows, int q_heads, int kv_heads, int head_dim, int max_q,
                           int max_kv, int window, int sinks) {
    if (prefill_rows(q_heads / kv_heads, max_q)) return 0;
    const Plan pl = plan(seqs, kv_heads, q_heads / kv_heads, max_q, max_kv, window, sinks);
    if (pl.splits == 1) return 0;
    return (size_t)rows * q_heads * pl.splits * (head_dim + 4) * sizeof(float);
}

hipError_t launch_attention(const KvView &c, int head_dim, const uint16_t *q, long long q_stride,
                            uint16_t *out, int q_heads, bool bf16, float scale, int window, int sinks,
                            int max_q, int max_kv, void *workspace, hipStream_t s) {
    const Plan pl = plan(c.seqs, c.kv_heads, q_heads / c.kv_heads, max_q, max_kv, window, sinks);
    AttnArgs p{c, q, q_stride, out, pl.splits > 1 ? (float *)workspace : nullptr, q_heads,
               q_heads / c.kv_heads, scale * kLog2e, window, sinks, pl.splits, pl.chunk};
    if (prefill_rows(p.group, max_q)) return launch_attention_prefill(p, head_dim, bf16, max_q, s);
    return bf16 ? launch_dim<bhalf_t>(p, head_dim, pl, max_q, s) : launch_dim<half_t>(p, head_dim, pl, max_q, s);
}

}  // namespace awq
