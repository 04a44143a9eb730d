// awq_kv_append, awq_kv_append_at: rotates the new rows' queries and keys by their positions and
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
// One workgroup owns one (page, kv head), for the page's new tokens: nobody else
// writes that slab or its scales, so no atomics.  Bound: HBM for prompts, launch latency for single tokens.
//
// AT, not 0 (awq_kv_append_at): the rows' rotary positions are given, up to four of each row, and
// frequency f takes the one that the map names; places in the cache stay those of the
// sequence.  A position behind the table turns by NaN, so such a token comes out as one
// that is not finite.
#pragma once

#include <algorithm>
#include <limits>

#include "awq_internal.h"
#include "awq_kv.h"

namespace awq {

struct AppendArgs {
    KvView c;
    const uint16_t *q, *k, *v;
    long long q_stride, k_stride, v_stride;   // elements between rows
    uint16_t *q_out;
    const float *rope;                        // [positions][rot]: cos | sin
    int rope_positions, rot, q_heads;
    const int32_t *positions;                 // (AT) [rows][axes]
    int axes;
    AxisMap map;
};
hipError_t launch_append_in_turn(const AppendArgs &p, int head_dim, bool adjacent, bool bf16, int max_q, hipStream_t s);

namespace {

constexpr int kMaxPage = 256, kMaxRot = 256;
enum { kSections = 1, kInTurn = 2 };        // AT: how axes share the frequencies, mostly
constexpr int kMinExp = -64;

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

// Sixteen elements of a head row: those of unit u of the D / 16 units, as two chunks
// of eight, at elements c0 and c1.  The first and the second chunks of a row's units
// each lie side by side, so that a wave's loads and stores are of whole lines.
template <int D, bool ADJ>
__device__ __forceinline__ void unit_chunks(int u, int rot, int &c0, int &c1) {
    if (ADJ) {
        c0 = 8 * u;
        c1 = 8 * u + D / 2;
    } else if (16 * u < rot) {                         // pairs (i, i + rot / 2)
        c0 = 8 * u;
        c1 = 8 * u + rot / 2;
    } else {
        c0 = 8 * u + rot / 2;
        c1 = 8 * u + D / 2;
    }
}

// Queries of a prompt are read and written once, and are more than the caches hold:
// past them (8192 tokens of 32 heads: 58 -> 49 us; 16384 of 64: 161 -> 146 us).
typedef uint32_t words_t __attribute__((ext_vector_type(4)));
template <bool ONCE>
__device__ __forceinline__ uint4 load16(const uint16_t *p) {
    const words_t *w = reinterpret_cast<const words_t *>(p);
    const words_t v = ONCE ? __builtin_nontemporal_load(w) : *w;
    return make_uint4(v[0], v[1], v[2], v[3]);
}
template <bool ONCE>
__device__ __forceinline__ void store16(uint16_t *p, uint4 u) {
    words_t *w = reinterpret_cast<words_t *>(p);
    const words_t v = {u.x, u.y, u.z, u.w};
    if (ONCE)
        __builtin_nontemporal_store(v, w);
    else
        *w = v;
}

__device__ __forceinline__ bool finite(float f) {
    return (__builtin_bit_cast(uint32_t, f) & 0x7F800000u) != 0x7F800000u;
}

// Sums up one element: whether it is finite, and the largest finite magnitude.
__device__ __forceinline__ void take(float x, float &most, bool &ok) {
    const bool f = finite(x);
    ok = ok && f;
    most = fmaxf(most, f ? fabsf(x) : 0.0f);
}

// Cosines and sines of the frequencies f .. f + 3 from a row of the table: cosines, then sines.
__device__ __forceinline__ auto table_row(const float *row, int rot) {
    return [=](int f, float4 &c, float4 &s) {
        c = *reinterpret_cast<const float4 *>(row + f);
        s = *reinterpret_cast<const float4 *>(row + rot / 2 + f);
    };
}

// The same where each frequency takes the table's row of the position on its axis.  Sections of
// the frequencies leave four of them on one axis: then it is one load for the four, and at a border
// one for each.  With the axes in turn it is one for each axis that they are on (4 x 2048 tokens 58.4
// us; as at borders 64.5.  For sections 57.3 and 53.5, and both in one kernel cost 16384 tokens 10 us).
template <bool TURN>
__device__ __forceinline__ void given_turns(const AppendArgs &p, const uint8_t *axis, long long row, int f, float4 &c, float4 &s) {
    const float none = std::numeric_limits<float>::quiet_NaN();
    const int32_t *at = p.positions + row * p.axes;
    const uint32_t four = *reinterpret_cast<const uint32_t *>(axis + f);
    if constexpr (TURN) {
        int pos[4];                                    // (all on the way at once; behind the last axis the last again)
#pragma unroll
        for (int a = 0; a < 4; ++a) pos[a] = at[min(a, p.axes - 1)];
        float cs[4] = {}, ss[4] = {};
#pragma unroll
        for (int a = 0; a < 4; ++a) {
            bool on[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) on[e] = (four >> (8 * e) & 0xFF) == (uint32_t)a;
            if (on[0] | on[1] | on[2] | on[3]) {
                const bool in = (uint32_t)pos[a] < (uint32_t)p.rope_positions;
                const float *from = p.rope + (long long)(in ? pos[a] : 0) * p.rot + f;
                const float4 x = *reinterpret_cast<const float4 *>(from), y = *reinterpret_cast<const float4 *>(from + p.rot / 2);
                const float xs[4] = {x.x, x.y, x.z, x.w}, ys[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    cs[e] = on[e] ? (in ? xs[e] : none) : cs[e];
                    ss[e] = on[e] ? (in ? ys[e] : none) : ss[e];
                }
            }
        }
        c = make_float4(cs[0], cs[1], cs[2], cs[3]);
        s = make_float4(ss[0], ss[1], ss[2], ss[3]);
    } else if (four == (four & 0xFF) * 0x01010101u) {
        const int pos = at[four & 0xFF];
        const bool in = (uint32_t)pos < (uint32_t)p.rope_positions;
        const float *from = p.rope + (long long)(in ? pos : 0) * p.rot + f;
        c = *reinterpret_cast<const float4 *>(from);
        s = *reinterpret_cast<const float4 *>(from + p.rot / 2);
        if (!in) c = s = make_float4(none, none, none, none);
    } else {
        float cs[4], ss[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int pos = at[four >> (8 * e) & 0xFF];
            const bool in = (uint32_t)pos < (uint32_t)p.rope_positions;
            const float *from = p.rope + (long long)(in ? pos : 0) * p.rot + f + e;
            cs[e] = in ? from[0] : none;
            ss[e] = in ? from[p.rot / 2] : none;
        }
        c = make_float4(cs[0], cs[1], cs[2], cs[3]);
        s = make_float4(ss[0], ss[1], ss[2], ss[3]);
    }
}

// A unit's elements x[0..7] of its first chunk and x[8..15] of the second, turned by
// turns(f, c, s): the cosines and sines of the frequencies f .. f + 3.
template <bool ADJ, typename F>
__device__ __forceinline__ void turn_unit(float x[16], int c0, int c1, int rot, F turns) {
    const auto turn = [](float &a, float &b, float c, float s) {
#pragma clang fp contract(off)   // each product and sum is rounded once, as the formula says
        const float p = a * c - b * s;
        const float q = b * c + a * s;
        a = p;
        b = q;
    };
    if (ADJ) {                                         // pairs (2 i, 2 i + 1): four in a chunk
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const int at = k ? c1 : c0;
            if (at >= rot) continue;
            float4 c, s;
            turns(at / 2, c, s);
            turn(x[8 * k], x[8 * k + 1], c.x, s.x);
            turn(x[8 * k + 2], x[8 * k + 3], c.y, s.y);
            turn(x[8 * k + 4], x[8 * k + 5], c.z, s.z);
            turn(x[8 * k + 6], x[8 * k + 7], c.w, s.w);
        }
    } else if (c0 < rot / 2) {                         // pairs (i, i + rot / 2): a chunk and the other
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            float4 c, s;
            turns(c0 + 4 * k, c, s);
            turn(x[4 * k], x[4 * k + 8], c.x, s.x);
            turn(x[4 * k + 1], x[4 * k + 9], c.y, s.y);
            turn(x[4 * k + 2], x[4 * k + 10], c.z, s.z);
            turn(x[4 * k + 3], x[4 * k + 11], c.w, s.w);
        }
    }
}

// kThreads: 256 for prompts, 128 for a few tokens.  kKeys: units of keys that a thread
// can hold (and half as many tiles of values): 2, or 4 where pages of 128 tokens of
// 128 elements, or as much, need it.  There 16384 tokens of 64/8 heads go 146 -> 136 us with
// adjacent pairs and 140 -> 137 with the others, whose instance spills 17 to 21 registers, 4 x
// 2048 of 32/8 heads 56 -> 50 and 51 -> 50; 8 x 300 tokens 22.8 -> 22.3 and 20.8 -> 22.2.  (With 4
// for pages of 64 the registers cost 45.6 -> 49 us.)  Workgroups 0 .. pages - 1 of a
// (sequence, kv head) take its pages, the others its queries: those are two thirds
// of a prompt's bytes at four query heads to a kv head, and with them in the pages'
// workgroups the last round of these was long.
template <typename T, int D, bool ADJ, int kThreads, int kKeys, int AT>
__global__ void __launch_bounds__(kThreads, 3) append_kernel(AppendArgs p, int pages) {     // 0: flat
    constexpr int U = D / 16;                          // units of a head row
    constexpr int kValues = kKeys / 2;                 // tiles of values, 4 slots by 8 elements, a thread holds
    __shared__ float red[2][kThreads / 64];
    __shared__ int bad[kMaxPage];
    __shared__ __align__(4) uint8_t axis[AT ? kMaxRot / 2 : 4];     // of a frequency
    __shared__ __align__(16) uint32_t turned[8 * kValues * kThreads + D];    // value codes [D][words + 1], four slots to a word
    const KvView &c = p.c;
    constexpr int kTokens = 8 * kThreads / D;          // of a workgroup of queries
    const int tid = threadIdx.x;
    const int h = blockIdx.y;
    // positions in [from, to) have a place in the page table and a row in the rotation's table
    // (first, that of row 0, may be below 0: rows without a place)
    const auto from_of = [](const Seq &s) { return max(s.first(), 0); };
    const auto to_of = [&](const Seq &s) { return p.rot && AT == 0 ? min(s.len, p.rope_positions) : s.len; };
    int b = blockIdx.z, piece = blockIdx.x, blocks = gridDim.x - pages;
    if (pages == 0) {
        const auto pages_of = [&](const Seq &s) {
            return from_of(s) < to_of(s) ? ((to_of(s) - 1) >> c.log2_page) - (from_of(s) >> c.log2_page) + 1 : 0;
        };
        const int2 at = seq_of_piece(c, blockIdx.x, [&](const Seq &s) {
            return pages_of(s) + (p.q && from_of(s) < to_of(s) ? (to_of(s) - from_of(s) + kTokens - 1) / kTokens : 0);
        });
        if (at.x >= c.seqs) return;
        b = at.x;
        piece = at.y;
        pages = pages_of(load_seq(c, b));
        blocks = 1 << 20;
    }
    const Seq s = load_seq(c, b);
    const int P = 1 << c.log2_page;
    const int group = p.q_heads / c.kv_heads;
    const int first = s.first(), from = from_of(s), to = to_of(s);
    if (from >= to) return;
    if constexpr (AT != 0) {                                // (read behind a barrier of both kinds of work)
        if (tid < p.rot / 2) axis[tid] = p.map.at(tid);
    }
    if (piece >= pages) {
        if (p.q == nullptr) return;
        // queries: kTokens tokens at a time, with their rows of the table in LDS; a wave's units lie
        // side by side, and each thread has kAhead of them on the way
        constexpr int kAhead = 4;
        constexpr bool kOnce = kThreads == 256;
        float *rows = reinterpret_cast<float *>(turned);
        const int width = group * U;
        for (int pos = from + (piece - pages) * kTokens; pos < to; pos += blocks * kTokens) {
            const int items = min(kTokens, to - pos) * width;
            const long long row = s.row0 + (pos - first);
            uint4 r[kAhead][2];
            auto load = [&](int i0) {
#pragma unroll
                for (int n = 0; n < kAhead; ++n) {
                    const int i = i0 + tid + n * kThreads;
                    if (i < items) {
                        const int t = i / width, g = i % width / U;
                        int c0, c1;
                        unit_chunks<D, ADJ>(i % U, p.rot, c0, c1);
                        const uint16_t *src = p.q + (row + t) * p.q_stride + (h * group + g) * D;
                        r[n][0] = load16<kOnce>(src + c0);
                        r[n][1] = load16<kOnce>(src + c1);
                    }
                }
            };
            load(0);
            __syncthreads();                           // the rows of the step before are done with
            if constexpr (AT != 0) {
                const int quads = p.rot / 8;           // of frequencies
                for (int i = tid; i < items / width * quads; i += kThreads) {
                    const int t = i / quads, f = i % quads * 4;
                    float4 c, s;
                    given_turns<AT == kInTurn>(p, axis, row + t, f, c, s);
                    *reinterpret_cast<float4 *>(rows + t * p.rot + f) = c;
                    *reinterpret_cast<float4 *>(rows + t * p.rot + p.rot / 2 + f) = s;
                }
            } else if (p.rot) {
                const float4 *from_row = reinterpret_cast<const float4 *>(p.rope + (long long)pos * p.rot);
                for (int i = tid; i < items / width * p.rot / 4; i += kThreads) reinterpret_cast<float4 *>(rows)[i] = from_row[i];
            }
            __syncthreads();
            for (int i0 = 0; i0 < items; i0 += kAhead * kThreads) {
                if (i0 > 0) load(i0);
#pragma unroll
                for (int n = 0; n < kAhead; ++n) {
                    const int i = i0 + tid + n * kThreads;
                    if (i < items) {
                        const int t = i / width, g = i % width / U, u = i % U;
                        int c0, c1;
                        unit_chunks<D, ADJ>(u, p.rot, c0, c1);
                        float x[16];
                        unpack8<T>(r[n][0], x);
                        unpack8<T>(r[n][1], x + 8);
                        if (p.rot) turn_unit<ADJ>(x, c0, c1, p.rot, table_row(rows + t * p.rot, p.rot));
                        uint16_t *dst = p.q_out + ((row + t) * p.q_heads + h * group + g) * D;
                        store16<kOnce>(dst + c0, pack8<T>(x));
                        store16<kOnce>(dst + c1, pack8<T>(x + 8));
                    }
                }
            }
        }
        return;
    }
    const int j0 = from >> c.log2_page, j1 = (to - 1) >> c.log2_page;
    for (int j = j0 + piece; j <= j1; j += pages) {
        const int base = j << c.log2_page;
        const int lo = max(from, base), hi = min(to, base + P);
        const int count = hi - lo, held = lo - base;   // new tokens; slots that hold tokens from before
        const int items = count * U;
        const long long row = s.row0 + (lo - first);
        const int id = c.page_table[(long long)b * c.table_width + j];
        if (id < 0 || id >= c.pages) continue;         // names no page: nothing is appended
        const uint16_t *krow = p.k + row * p.k_stride + h * D;
        const uint16_t *vrow = p.v + row * p.v_stride + h * D;
        for (int i = tid; i < count; i += kThreads) bad[i] = 0;
        const long long ph = (long long)id * c.kv_heads + h;
        const float ks0 = c.k_scales[ph], vs0 = c.v_scales[ph];

        // values, in tiles of four slots by eight elements; the page's words that hold new slots
        const int w0 = held >> 2, w1 = (held + count + 3) >> 2, tiles = (w1 - w0) * (D / 8);
        // keys and values stay in registers between the passes, if they are few enough
        const bool once = items <= kKeys * kThreads && tiles <= kValues * kThreads;
        uint4 vr[kValues][4];
        auto load_values = [&](int i, uint4 (&r)[4]) {
            const int u = i % (D / 8), w = w0 + i / (D / 8);
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                const int slot = 4 * w + t - held;
                r[t] = slot >= 0 && slot < count ? *reinterpret_cast<const uint4 *>(vrow + slot * p.v_stride + 8 * u) : make_uint4(0, 0, 0, 0);
            }
        };
        if (once) {
#pragma unroll
            for (int n = 0; n < kValues; ++n)
                if (tid + n * kThreads < tiles) load_values(tid + n * kThreads, vr[n]);
        }
        auto load_keys = [&](int i, uint4 (&r)[2]) {
            int c0, c1;
            unit_chunks<D, ADJ>(i % U, p.rot, c0, c1);
            const uint16_t *src = krow + i / U * p.k_stride;
            r[0] = *reinterpret_cast<const uint4 *>(src + c0);
            r[1] = *reinterpret_cast<const uint4 *>(src + c1);
        };
        auto rotated = [&](int i, const uint4 (&r)[2], float (&x)[16]) {
            unpack8<T>(r[0], x);
            unpack8<T>(r[1], x + 8);
            int c0, c1;
            unit_chunks<D, ADJ>(i % U, p.rot, c0, c1);
            if constexpr (AT != 0)
                turn_unit<ADJ>(x, c0, c1, p.rot, [&](int f, float4 &c, float4 &s) { given_turns<AT == kInTurn>(p, axis, row + i / U, f, c, s); });
            else if (p.rot)
                turn_unit<ADJ>(x, c0, c1, p.rot, table_row(p.rope + (long long)(lo + i / U) * p.rot, p.rot));
        };
        uint4 kr[kKeys][2];
        if (once) {
#pragma unroll
            for (int n = 0; n < kKeys; ++n)
                if (tid + n * kThreads < items) load_keys(tid + n * kThreads, kr[n]);
        }
        __syncthreads();
        // largest finite magnitudes
        float ka = 0.0f, va = 0.0f;
        auto take_keys = [&](int i, const uint4 (&r)[2]) {
            float x[16];
            bool ok = true;
            rotated(i, r, x);
#pragma unroll
            for (int e = 0; e < 16; ++e) take(x[e], ka, ok);
            if (!ok) bad[i / U] = 1;
        };
        if (once) {
#pragma unroll
            for (int n = 0; n < kKeys; ++n)
                if (tid + n * kThreads < items) take_keys(tid + n * kThreads, kr[n]);
        } else {
            for (int i = tid; i < items; i += kThreads) {
                load_keys(i, kr[0]);
                take_keys(i, kr[0]);
            }
        }
        auto take_values = [&](int i, const uint4 (&r)[4]) {
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                bool ok = true;
                const uint32_t w[4] = {r[t].x, r[t].y, r[t].z, r[t].w};
#pragma unroll
                for (int e = 0; e < 8; ++e) take(to_float<T>((uint16_t)(w[e / 2] >> (16 * (e & 1)))), va, ok);
                if (!ok) bad[4 * (w0 + i / (D / 8)) + t - held] = 1;       // (a slot of none is 0, finite)
            }
        };
        if (once) {
#pragma unroll
            for (int n = 0; n < kValues; ++n)
                if (tid + n * kThreads < tiles) take_values(tid + n * kThreads, vr[n]);
        } else {
            for (int i = tid; i < tiles; i += kThreads) {
                load_values(i, vr[0]);
                take_values(i, vr[0]);
            }
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
        float ks = scale_for(ka), vs = scale_for(va);
        if (held > 0) {
            ks = fmaxf(ks, ks0);
            vs = fmaxf(vs, vs0);
        }
        if (tid == 0) {                                // (everyone has read the old ones)
            c.k_scales[ph] = ks;
            c.v_scales[ph] = vs;
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
        auto write_keys = [&](int i, const uint4 (&r)[2]) {
            float x[16];
            rotated(i, r, x);
            const int u = i % U, t = i / U;
            int c0, c1;
            unit_chunks<D, ADJ>(u, p.rot, c0, c1);
            uint32_t w[4] = {0x7F7F7F7Fu, 0x7F7F7F7Fu, 0x7F7F7F7Fu, 0x7F7F7F7Fu};
            if (!bad[t]) {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    w[e] = to_e4m3x4(x[4 * e] * ki, x[4 * e + 1] * ki, x[4 * e + 2] * ki, x[4 * e + 3] * ki);
            }
            uint8_t *dst = kslab + (held + t) * D;
            *reinterpret_cast<uint2 *>(dst + c0) = make_uint2(w[0], w[1]);
            *reinterpret_cast<uint2 *>(dst + c1) = make_uint2(w[2], w[3]);
        };
        if (once) {
#pragma unroll
            for (int n = 0; n < kKeys; ++n)
                if (tid + n * kThreads < items) write_keys(tid + n * kThreads, kr[n]);
        } else {
            for (int i = tid; i < items; i += kThreads) {
                load_keys(i, kr[0]);
                write_keys(i, kr[0]);
            }
        }
        // values: eight words of four slots each from a tile
        const bool moved = held > 0 && vs != vs0;
        const float f = vs0 * vi;
        auto words = [&](int i, const uint4 (&r)[4], auto put) {
            const int u = i % (D / 8), w = w0 + i / (D / 8);
            const int live = held + count - 4 * w;     // slots behind the last token stay as they were
            const bool all = 4 * w >= held && live >= 4;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const uint32_t was = all ? 0u : reinterpret_cast<const uint32_t *>(vslab + (8 * u + e) * P)[w];
                float o[4], n[4];
                from_e4m3x4(was, o);
#pragma unroll
                for (int t = 0; t < 4; ++t) {
                    const uint32_t v[4] = {r[t].x, r[t].y, r[t].z, r[t].w};
                    const float x = to_float<T>((uint16_t)(v[e / 2] >> (16 * (e & 1))));
                    n[t] = 4 * w + t < held ? (moved ? o[t] * f : o[t]) : finite(x) ? x * vi : 0.0f;
                }
                const uint32_t now = to_e4m3x4(n[0], n[1], n[2], n[3]);
                const uint32_t keep = live >= 4 ? 0u : 0xFFFFFFFFu << (8 * live);
                put(8 * u + e, w, (now & ~keep) | (was & keep));
            }
        };
        // words that hold old slots only
        if (moved) {
            for (int i = tid; i < w0 * D; i += kThreads) {
                uint32_t *w = reinterpret_cast<uint32_t *>(vslab + (i / w0) * P) + i % w0;
                float x[4];
                from_e4m3x4(*w, x);
                *w = to_e4m3x4(x[0] * f, x[1] * f, x[2] * f, x[3] * f);
            }
        }
        if (once && count >= 16) {
            // by way of LDS, so that sixteen slots of an element go out as one store
            const int pitch = w1 - w0 + 1;
#pragma unroll
            for (int n = 0; n < kValues; ++n)
                if (tid + n * kThreads < tiles)
                    words(tid + n * kThreads, vr[n], [&](int d, int w, uint32_t x) { turned[d * pitch + w - w0] = x; });
            __syncthreads();
            const int q0 = w0 >> 2, q1 = (w1 + 3) >> 2;
            for (int i = tid; i < D * (q1 - q0); i += kThreads) {
                const int d = i / (q1 - q0), q = q0 + i % (q1 - q0);
                uint32_t *to = reinterpret_cast<uint32_t *>(vslab + d * P) + 4 * q;
                const int at = d * pitch + 4 * q - w0;
                if (4 * q >= w0 && 4 * q + 4 <= w1) {
                    *reinterpret_cast<uint4 *>(to) = make_uint4(turned[at], turned[at + 1], turned[at + 2], turned[at + 3]);
                } else {
                    for (int e = 0; e < 4; ++e)
                        if (4 * q + e >= w0 && 4 * q + e < w1) to[e] = turned[at + e];
                }
            }
        } else {
            const auto put = [&](int d, int w, uint32_t x) { reinterpret_cast<uint32_t *>(vslab + d * P)[w] = x; };
            if (once) {
#pragma unroll
                for (int n = 0; n < kValues; ++n)
                    if (tid + n * kThreads < tiles) words(tid + n * kThreads, vr[n], put);
            } else {
                for (int i = tid; i < tiles; i += kThreads) {
                    load_values(i, vr[0]);
                    words(i, vr[0], put);
                }
            }
        }
        __syncthreads();                               // bad and the words in LDS are free again
    }
}

template <typename T, int D, int AT>
hipError_t launch(const AppendArgs &p, bool adjacent, bool few, int most, int touched, hipStream_t s) {
    const int threads = few ? 128 : 256, tokens = 8 * threads / D;       // of a workgroup of queries
    dim3 grid(touched + (p.q ? (most + tokens - 1) / tokens : 0), p.c.kv_heads, p.c.seqs);
    // Prompts among single tokens: as many workgroups as there can be work for, which look for
    // theirs (one of 2048 rows and 255 of one: 163 -> 68 us)
    if ((long long)grid.x * grid.y * grid.z >= 4096 && rows_differ(p.c.seqs, p.c.rows, most)) {
        const int some = std::min(p.c.seqs, p.c.rows);
        grid = dim3((p.c.rows >> p.c.log2_page) + 2 * some + (p.q ? p.c.rows / tokens + some : 0), p.c.kv_heads);
        touched = 0;
    }
    const int elements = D << p.c.log2_page;
    if (few && adjacent)
        append_kernel<T, D, true, 128, 2, AT><<<grid, threads, 0, s>>>(p, touched);
    else if (few)
        append_kernel<T, D, false, 128, 2, AT><<<grid, threads, 0, s>>>(p, touched);
    else if (elements > 8192 && elements <= 16384 && adjacent)
        append_kernel<T, D, true, 256, 4, AT><<<grid, threads, 0, s>>>(p, touched);
    else if (elements > 8192 && elements <= 16384)
        append_kernel<T, D, false, 256, 4, AT><<<grid, threads, 0, s>>>(p, touched);
    else if (adjacent)
        append_kernel<T, D, true, 256, 2, AT><<<grid, threads, 0, s>>>(p, touched);
    else
        append_kernel<T, D, false, 256, 2, AT><<<grid, threads, 0, s>>>(p, touched);
    return hipGetLastError();
}

template <typename T, int AT>
hipError_t launch_dim(const AppendArgs &p, int D, bool adjacent, bool few, int most, int touched, hipStream_t s) {
    switch (D) {
    case 64: return launch<T, 64, AT>(p, adjacent, few, most, touched, s);
    case 128: return launch<T, 128, AT>(p, adjacent, few, most, touched, s);
    case 256: return launch<T, 256, AT>(p, adjacent, few, most, touched, s);
    }
    return hipErrorInvalidValue;
}

template <int AT>
hipError_t launch_append(const AppendArgs &p, int head_dim, bool adjacent, bool bf16, int max_q, hipStream_t s) {
    // pages that a sequence's rows can touch (the kernel steps on if there are more)
    const int most = max_q < 1 ? 1 : max_q > p.c.rows ? p.c.rows : max_q;
    const int touched = most == 1 ? 1 : ((most - 2) >> p.c.log2_page) + 2;
    const bool few = (long long)most * head_dim <= 2 * 128 * 16;
    return bf16 ? launch_dim<bhalf_t, AT>(p, head_dim, adjacent, few, most, touched, s)
                : launch_dim<half_t, AT>(p, head_dim, adjacent, few, most, touched, s);
}

}  // namespace
}  // namespace awq
