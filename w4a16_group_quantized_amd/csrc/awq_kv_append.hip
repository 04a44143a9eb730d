// awq_kv_append: rotates the new rows' queries and keys by their positions and
// writes the keys and values into the paged cache, as e4m3 codes under one
// power-of-two scale for each page and kv head.
//
//   rotation   a' = a cos - b sin,  b' = b cos + a sin   (fp32, each product
//              and sum rounded once) for the pairs (i, i + R/2) or (2i, 2i + 1)
//              of a head's first R elements; q is then rounded once to its type
//   scale      2^e, e the least integer >= -64 with max|x| <= 448 * 2^e over
//              the new tokens of the page and head; never below the page's
//              scale if the page holds tokens from before
//   codes      e4m3_rne(x / scale); codes held from before move from scale s to
//              s' as e4m3_rne(c * s / s').
//
// Why powers of two: an e4m3 value has the same relative step in every binade,
// so a power-of-two scale loses nothing against the quotient max|x| / 448 but
// up to one binade at the far (subnormal) end, and raising the scale of codes
// that are there only shifts their exponents: no second rounding, except of
// codes that become subnormal (below 2^-6 of 448, an error of 2^-19 of the
// page's largest value).  A quotient scale would round every held code again
// each time a page's maximum grows.
//
// A token whose key or value holds a NaN or an infinity in some head has all
// key codes of that head set to NaN, and its non-finite value elements to zero:
// a row that sees the token comes out NaN, and a row that does not see it is
// not disturbed, since values never hold a NaN.
//
// One workgroup owns one (page, kv head) and the query heads that share the
// head, for the page's new tokens: nobody else writes that slab or its scales,
// so no atomics.  Bound: HBM for prompts, launch latency for single tokens.
#include "awq_internal.h"
#include "awq_kv.h"

namespace awq {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxPage = 256;
constexpr int kMinExp = -64;

struct AppendArgs {
    KvView c;
    const uint16_t *q, *k, *v;
    long long q_stride, k_stride, v_stride;   // elements between rows
    uint16_t *q_out;
    const float *rope;                        // [positions][rot]: cos | sin
    int rope_positions, rot, q_heads;
};

// The scale of a largest magnitude: 2^e, see the top.
__device__ __forceinline__ float scale_for(float amax) {
    if (!(amax > 0.0f)) return pow2(kMinExp);
    const uint32_t u = __builtin_bit_cast(uint32_t, amax);
    // amax = m 2^x with 1 <= m < 2 (a subnormal has x = -127 here, far below kMinExp);
    // 448 = 1.75 * 2^8
    const int x = (int)(u >> 23) - 127;
    const int e = x - 8 + ((u & 0x7FFFFFu) > 0x600000u ? 1 : 0);
    return pow2(max(e, kMinExp));
}

// Sixteen elements of a head row: those of unit `u` of the D / 16 units, as two
// chunks of eight at element c0 and c1.  Rotated units in half pairing hold
// elements i.. and i + R/2..; all others are 16 consecutive elements.
template <bool ADJ>
__device__ __forceinline__ void unit_chunks(int u, int rot, int &c0, int &c1) {
    if (!ADJ && 16 * u < rot) {
        c0 = 8 * u;
        c1 = 8 * u + rot / 2;
    } else {
        c0 = 16 * u;
        c1 = 16 * u + 8;
    }
}

// Rotates a unit in place.  row: the table's row of the position.
template <bool ADJ>
__device__ __forceinline__ void rotate_unit(float a[8], float b[8], int u, int rot, const float *row) {
    if (16 * u >= rot) return;
    const float4 *cp = reinterpret_cast<const float4 *>(row + 8 * u);
    const float4 *sp = reinterpret_cast<const float4 *>(row + rot / 2 + 8 * u);
    const float4 c0 = cp[0], c1 = cp[1], s0 = sp[0], s1 = sp[1];
    const float cs[8] = {c0.x, c0.y, c0.z, c0.w, c1.x, c1.y, c1.z, c1.w};
    const float sn[8] = {s0.x, s0.y, s0.z, s0.w, s1.x, s1.y, s1.z, s1.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
#pragma clang fp contract(off)   // each product and sum is rounded once, as the formula says
        float &x = ADJ ? (i < 4 ? a[2 * i] : b[2 * i - 8]) : a[i];
        float &y = ADJ ? (i < 4 ? a[2 * i + 1] : b[2 * i - 7]) : b[i];
        const float p = x * cs[i] - y * sn[i];
        const float q = y * cs[i] + x * sn[i];
        x = p;
        y = q;
    }
}

__device__ __forceinline__ bool finite(float f) {
    return (__builtin_bit_cast(uint32_t, f) & 0x7F800000u) != 0x7F800000u;
}

template <typename T, int D, bool ADJ>
__global__ void __launch_bounds__(kThreads) append_kernel(AppendArgs p) {
    constexpr int kUnits = D / 16;
    __shared__ float red[2][kThreads / 64];
    __shared__ int bad[kMaxPage];
    const KvView &c = p.c;
    const int tid = threadIdx.x;
    const int h = blockIdx.y, b = blockIdx.z;
    const Seq s = load_seq(c, b);
    const int P = 1 << c.log2_page;
    const int group = p.q_heads / c.kv_heads;
    const int first = s.first();                       // position of row 0 (below 0: rows without a place)
    // positions in [from, to) have a place in the page table and a row in the rotation's table
    const int from = max(first, 0);
    const int to = p.rot ? min(s.len, p.rope_positions) : s.len;
    if (from >= to) return;
    const int j0 = from >> c.log2_page, j1 = (to - 1) >> c.log2_page;
    for (int j = j0 + blockIdx.x; j <= j1; j += gridDim.x) {
        const int base = j << c.log2_page;
        const int lo = max(from, base), hi = min(to, base + P);
        const int count = hi - lo;
        const long long row = s.row0 + (lo - first);
        // queries of this page's tokens and this head's group
        if (p.q != nullptr) {
            for (int i = tid; i < count * group * kUnits; i += kThreads) {
                const int u = i % kUnits, g = (i / kUnits) % group, t = i / (kUnits * group);
                const int head = h * group + g;
                const uint16_t *src = p.q + (row + t) * p.q_stride + head * D;
                uint16_t *dst = p.q_out + ((row + t) * p.q_heads + head) * D;
                int c0, c1;
                unit_chunks<ADJ>(u, p.rot, c0, c1);
                float x[8], y[8];
                load8<T>(src + c0, x);
                load8<T>(src + c1, y);
                rotate_unit<ADJ>(x, y, u, p.rot, p.rope + (long long)(lo + t) * p.rot);
                *reinterpret_cast<uint4 *>(dst + c0) = pack8<T>(x);
                *reinterpret_cast<uint4 *>(dst + c1) = pack8<T>(y);
            }
        }
        const int id = c.page_table[(long long)b * c.table_width + j];
        if (id < 0 || id >= c.pages) continue;         // names no page: nothing is appended
        const uint16_t *krow = p.k + row * p.k_stride + h * D;
        const uint16_t *vrow = p.v + row * p.v_stride + h * D;
        for (int i = tid; i < count; i += kThreads) bad[i] = 0;
        __syncthreads();
        // largest finite magnitudes
        float ka = 0.0f, va = 0.0f;
        for (int i = tid; i < count * kUnits; i += kThreads) {
            const int u = i % kUnits, t = i / kUnits;
            int c0, c1;
            unit_chunks<ADJ>(u, p.rot, c0, c1);
            float x[8], y[8];
            load8<T>(krow + t * p.k_stride + c0, x);
            load8<T>(krow + t * p.k_stride + c1, y);
            rotate_unit<ADJ>(x, y, u, p.rot, p.rope + (long long)(lo + t) * p.rot);
            bool ok = true;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                ok = ok && finite(x[e]) && finite(y[e]);
                ka = fmaxf(ka, fmaxf(finite(x[e]) ? fabsf(x[e]) : 0.0f, finite(y[e]) ? fabsf(y[e]) : 0.0f));
            }
            load8<T>(vrow + t * p.v_stride + 16 * u, x);
            load8<T>(vrow + t * p.v_stride + 16 * u + 8, y);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                ok = ok && finite(x[e]) && finite(y[e]);
                va = fmaxf(va, fmaxf(finite(x[e]) ? fabsf(x[e]) : 0.0f, finite(y[e]) ? fabsf(y[e]) : 0.0f));
            }
            if (!ok) bad[t] = 1;
        }
        for (int m = 32; m > 0; m >>= 1) {
            ka = fmaxf(ka, __shfl_xor(ka, m));
            va = fmaxf(va, __shfl_xor(va, m));
        }
        if ((tid & 63) == 0) {
            red[0][tid >> 6] = ka;
            red[1][tid >> 6] = va;
        }
        __syncthreads();
        ka = va = 0.0f;
#pragma unroll
        for (int w = 0; w < kThreads / 64; ++w) {
            ka = fmaxf(ka, red[0][w]);
            va = fmaxf(va, red[1][w]);
        }
        const long long ph = (long long)id * c.kv_heads + h;
        const int held = lo - base;                    // slots that hold tokens from before
        const float ks0 = c.k_scales[ph], vs0 = c.v_scales[ph];
        float ks = scale_for(ka), vs = scale_for(va);
        if (held > 0) {
            ks = fmaxf(ks, ks0);
            vs = fmaxf(vs, vs0);
        }
        const float ki = 1.0f / ks, vi = 1.0f / vs;    // exact
        uint8_t *kslab = c.k + ph * P * D;
        uint8_t *vslab = c.v + ph * P * D;
        if (held > 0 && ks != ks0) {
            const float f = ks0 * ki;
            for (int i = tid; i < held * (D / 4); i += kThreads) {
                uint32_t *w = reinterpret_cast<uint32_t *>(kslab) + i;
                float x[4];
                from_e4m3x4(*w, x);
                *w = to_e4m3x4(x[0] * f, x[1] * f, x[2] * f, x[3] * f);
            }
        }
        for (int i = tid; i < count * kUnits; i += kThreads) {
            const int u = i % kUnits, t = i / kUnits;
            int c0, c1;
            unit_chunks<ADJ>(u, p.rot, c0, c1);
            float x[8], y[8];
            load8<T>(krow + t * p.k_stride + c0, x);
            load8<T>(krow + t * p.k_stride + c1, y);
            rotate_unit<ADJ>(x, y, u, p.rot, p.rope + (long long)(lo + t) * p.rot);
            uint32_t w[4] = {0x7F7F7F7Fu, 0x7F7F7F7Fu, 0x7F7F7F7Fu, 0x7F7F7F7Fu};
            if (!bad[t]) {
                w[0] = to_e4m3x4(x[0] * ki, x[1] * ki, x[2] * ki, x[3] * ki);
                w[1] = to_e4m3x4(x[4] * ki, x[5] * ki, x[6] * ki, x[7] * ki);
                w[2] = to_e4m3x4(y[0] * ki, y[1] * ki, y[2] * ki, y[3] * ki);
                w[3] = to_e4m3x4(y[4] * ki, y[5] * ki, y[6] * ki, y[7] * ki);
            }
            uint8_t *dst = kslab + (held + t) * D;
            *reinterpret_cast<uint2 *>(dst + c0) = make_uint2(w[0], w[1]);
            *reinterpret_cast<uint2 *>(dst + c1) = make_uint2(w[2], w[3]);
        }
        // values: a thread takes eight elements of four slots, one word of each of eight rows
        const bool moved = held > 0 && vs != vs0;
        const float f = vs0 * vi;
        const int s0 = (moved ? 0 : held) >> 2, s1 = (held + count + 3) >> 2;
        for (int i = tid; i < (s1 - s0) * (D / 8); i += kThreads) {
            const int u = i % (D / 8), sg = s0 + i / (D / 8);
            float x[4][8];
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                const int slot = 4 * sg + t;
                if (slot >= held && slot < held + count) load8<T>(vrow + (slot - held) * p.v_stride + 8 * u, x[t]);
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                uint32_t *w = reinterpret_cast<uint32_t *>(vslab + (8 * u + e) * P) + sg;
                const uint32_t was = (4 * sg >= held && 4 * sg + 4 <= held + count) ? 0u : *w;
                float o[4], n[4];
                from_e4m3x4(was, o);
#pragma unroll
                for (int t = 0; t < 4; ++t) {
                    const int slot = 4 * sg + t;
                    n[t] = slot < held ? (moved ? o[t] * f : o[t]) : slot < held + count ? (finite(x[t][e]) ? x[t][e] * vi : 0.0f) : 0.0f;
                }
                const uint32_t now = to_e4m3x4(n[0], n[1], n[2], n[3]);
                // slots behind the last token stay as they were
                const int live = held + count - 4 * sg;
                const uint32_t keep = live >= 4 ? 0u : 0xFFFFFFFFu << (8 * live);
                *w = (now & ~keep) | (was & keep);
            }
        }
        __syncthreads();                               // everyone has read the old scales
        if (tid == 0) {
            c.k_scales[ph] = ks;
            c.v_scales[ph] = vs;
        }
    }
}

template <typename T, int D>
hipError_t launch(const AppendArgs &p, bool adjacent, int touched, hipStream_t s) {
    const dim3 grid(touched, p.c.kv_heads, p.c.seqs);
    if (adjacent)
        append_kernel<T, D, true><<<grid, kThreads, 0, s>>>(p);
    else
        append_kernel<T, D, false><<<grid, kThreads, 0, s>>>(p);
    return hipGetLastError();
}

template <typename T>
hipError_t launch_dim(const AppendArgs &p, int D, bool adjacent, int touched, hipStream_t s) {
    switch (D) {
    case 64: return launch<T, 64>(p, adjacent, touched, s);
    case 128: return launch<T, 128>(p, adjacent, touched, s);
    case 256: return launch<T, 256>(p, adjacent, touched, s);
    }
    return hipErrorInvalidValue;
}

}  // namespace

bool kv_head_dim_supported(int head_dim) { return head_dim == 64 || head_dim == 128 || head_dim == 256; }

hipError_t launch_kv_append(const KvView &c, int head_dim, const uint16_t *q, long long q_stride,
                            const uint16_t *k, long long k_stride, const uint16_t *v,
                            long long v_stride, uint16_t *q_out, int q_heads, const float *rope,
                            int rope_positions, int rot, bool adjacent, bool bf16, int max_q,
                            hipStream_t s) {
    AppendArgs p{c, q, k, v, q_stride, k_stride, v_stride, q_out, rope, rope_positions, rot, q_heads};
    // pages that a sequence's rows can touch (the kernel steps on if there are more)
    const int most = max_q < 1 ? 1 : max_q > c.rows ? c.rows : max_q;
    const int touched = most == 1 ? 1 : ((most - 2) >> c.log2_page) + 2;
    return bf16 ? launch_dim<bhalf_t>(p, head_dim, adjacent, touched, s)
                : launch_dim<half_t>(p, head_dim, adjacent, touched, s);
}

}  // namespace awq
