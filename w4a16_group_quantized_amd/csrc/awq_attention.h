// Shared by the attention kernels (awq_attention*.hip): arguments, the tiles of
// keys that rows see, and queries as matrix operands.
#pragma once

#include "awq_kv.h"

namespace awq {

constexpr int kTile = 64;                  // keys of a tile
constexpr float kEmpty = -0x1.fffffep127f; // running maximum of a row that has seen no key
// From here on a maximum is taken off the scores before anything is added: its steps are
// half an exponent's and more, and a sum with it would lose the rest.
constexpr float kFar = 0x1p23f;
constexpr float kNone = -0x1p14f;           // logarithm of a scale where there is none: below that of any
constexpr int kWidest = 1 << 30;           // a window of this many tokens sees all: no position is past it
constexpr float kLog2e = 1.44269504088896340736f;

struct AttnArgs {
    KvView c;
    const uint16_t *q;
    long long q_stride;
    uint16_t *out;
    float *part;             // partial results, or null with one chunk
    int q_heads, group;
    float scale;             // scale * log2(e)
    int window, sinks;
    int most, target;        // most chunks of a row tile in this kernel; workgroups that all chunks are dealt to
    int splits;              // chunks that a row has room for in the workspace
    int few;                 // rows (times query heads of a kv head) of a sequence from which the prompt kernel takes it
};

// The 64-key tiles that rows at positions lo .. hi see: tiles [0, a) that hold
// the first tokens and [b, e) that hold the window.
struct Tiles {
    int a, b, e;
    __device__ __forceinline__ int count() const { return a + e - b; }
    __device__ __forceinline__ int at(int i) const { return i < a ? i : b + i - a; }
};
__device__ __forceinline__ Tiles visible_tiles(const AttnArgs &p, int lo, int hi, int len) {
    Tiles t;
    const int end = min(hi + 1, len);
    t.e = end > 0 ? (end + kTile - 1) / kTile : 0;
    t.b = p.window > 0 ? min(max(lo - p.window + 1, 0) / kTile, t.e) : 0;
    t.a = p.window > 0 ? min((min(p.sinks, end > 0 ? end : 0) + kTile - 1) / kTile, t.b) : 0;
    return t;
}

// The sequence with the rank-th most tokens, among up to 64 of them (equal ones in
// their order); with more the order is as it comes.  All 64 lanes have to ask.
__device__ __forceinline__ int seq_of_rank(const KvView &c, int rank) {
    if (c.seqs == 1 || c.seqs > 64) return rank;
    const int lane = threadIdx.x & 63;
    const int len = lane < c.seqs ? c.kv_lens[lane] : 0;
    int above = 0;
    for (int i = 0; i < c.seqs; ++i) {
        const int other = __builtin_amdgcn_readlane(len, i);
        above += other > len || (other == len && i < lane);
    }
    return (int)__builtin_ctzll(__ballot(lane < c.seqs && above == rank));
}

// The scale that a row's outputs count in, and the largest so far in terms of the running
// maximum, as logarithms: quotients of scales may leave fp32.  A weight times its page's scale
// is what it adds to an output, so the largest such product (need) says how high the unit has
// to be, which a page of large values and no weight to speak of does not.  Down it goes where
// the maximum rises to a key of smaller values, whose product is then what counts, and with the
// pages' scales (most), so that weights are normal halves whatever these are; but not further
// than 2^60 from the largest: outputs, below 2^45 of their unit, stay far from fp32's end.  (A
// page of zeros has 2^-64, and values of bf16 reach 2^127.)
struct OutUnit {
    static constexpr float kDrop = 6.0f, kMostFall = 60.0f;
    float at = kNone, peak = kNone;
    // whether a tile of the largest product 2^need and the largest scale 2^most calls for another
    __device__ __forceinline__ bool moves(float need, float most) const { return need > at || (most < at - kDrop && most > kNone); }
    // goes along where the maximum rises by -down; returns what the outputs are to be multiplied by
    __device__ __forceinline__ float move(float need, float most, float down) {
        peak = fmaxf(peak, at) + down;
        const bool by_need = need > at || (down < 0.0f && need < at - kDrop);
        const float next = fmaxf(by_need ? fminf(most, need + kDrop) : moves(need, most) ? most : at, peak - kMostFall);
        const float turn = __builtin_amdgcn_exp2f(down + (at - next));
        at = next;
        return turn;
    }
};
// From here on a tile's weights, times a page's scale to the unit, are too small to sum up the
// weights from.
constexpr float kLeastToUnit = -60.0f;

template <typename T>
__device__ __forceinline__ half8_t as_row_half(const uint16_t *p, float f) {
    float x[8];
    load8<T>(p, x);
    half8_t h;
#pragma unroll
    for (int i = 0; i < 8; ++i) h[i] = (half_t)(x[i] * f);
    return h;
}

// The lane's value and that of its partner in the other half of the wave, the
// lower half's first.  (The elements go through variables of their own: a bit
// cast straight from an element of the result takes element 0.)
__device__ __forceinline__ float2 halves(float x) {
    const uint32_t u = __builtin_bit_cast(uint32_t, x);
    const auto r = __builtin_amdgcn_permlane32_swap(u, u, false, false);
    const uint32_t a = r[0], b = r[1];
    return make_float2(__builtin_bit_cast(float, a), __builtin_bit_cast(float, b));
}
__device__ __forceinline__ float half_max(float x) {
    const float2 v = halves(x);
    return fmaxf(v.x, v.y);
}
__device__ __forceinline__ float half_sum(float x) {
    const float2 v = halves(x);
    return v.x + v.y;
}
// Matrix results before inline assembly reads them, and what it wrote before products read
// it.  The compiler puts the wait states that a vector instruction needs behind a matrix one
// (12 behind a 32x32x16), and a matrix one behind a vector one (2), around its own
// instructions only.
__device__ __forceinline__ void settle(float16_t &acc) { asm volatile("s_nop 15" : "+v"(acc)); }
__device__ __forceinline__ void settle(float16_t &a, float16_t &b) { asm volatile("s_nop 15" : "+v"(a), "+v"(b)); }
__device__ __forceinline__ void settle(uint32_t (&w)[8]) {
    asm volatile("s_nop 1" : "+v"(w[0]), "+v"(w[1]), "+v"(w[2]), "+v"(w[3]), "+v"(w[4]), "+v"(w[5]), "+v"(w[6]), "+v"(w[7]));
}

// The largest of three (NaN only if all are), without the instructions that the
// compiler puts before fmaxf to quiet NaNs.  Not of matrix results as they come: settle() first.
__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("v_max3_f32 %0, %1, %2, %3" : "=v"(r) : "v"(a), "v"(b), "v"(c));
    return r;
}
// The same over the four lanes that share lane % 16.
__device__ __forceinline__ float2 quarters(float x) {
    const uint32_t u = __builtin_bit_cast(uint32_t, x);
    const auto r = __builtin_amdgcn_permlane16_swap(u, u, false, false);
    const uint32_t a = r[0], b = r[1];
    return make_float2(__builtin_bit_cast(float, a), __builtin_bit_cast(float, b));
}
__device__ __forceinline__ float group_max(float x) {
    const float2 v = quarters(x);
    return half_max(fmaxf(v.x, v.y));
}
__device__ __forceinline__ float group_sum(float x) {
    const float2 v = quarters(x);
    return half_sum(v.x + v.y);
}

// Two weights as halves, and what their roundings leave, as halves again: together they are
// off by 2^-22 of a weight (or 2^-25, where the weight is below 2^-3 and the remainder a
// subnormal), so that a product with both is one with fp32 weights.  One conversion and two
// multiply-adds, which take a half as it lies.  (Remainders before products: settle().)
__device__ __forceinline__ void lead_and_rest(float a, float b, uint32_t &lead, uint32_t &rest) {
    const half2_t h = {(half_t)a, (half_t)b};
    lead = __builtin_bit_cast(uint32_t, h);
    asm("v_fma_mixlo_f16 %0, %1, -1.0, %2 op_sel_hi:[1,0,0]" : "=v"(rest) : "v"(lead), "v"(a));
    asm("v_fma_mixhi_f16 %0, %1, -1.0, %2 op_sel:[1,0,0] op_sel_hi:[1,0,0]" : "+v"(rest) : "v"(lead), "v"(b));
}
__device__ __forceinline__ half8_t halves8(const uint32_t w[4]) {
    return __builtin_bit_cast(half8_t, make_uint4(w[0], w[1], w[2], w[3]));
}

// Four masks of four bytes each: the first `live` of sixteen bytes.
__device__ __forceinline__ void live_bytes(int live, uint32_t keep[4]) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const int n = live - 4 * e;
        keep[e] = n >= 4 ? 0xFFFFFFFFu : n <= 0 ? 0u : (1u << (8 * n)) - 1u;
    }
}

// A partial result of a chunk of keys, in the workspace: D outputs (over the sum), the
// maximum, the sum and (of chunk 0) the number of chunks.
template <int D>
constexpr int kPart = D + 4;

// Rows by rows of 32 to a wave, for prompts (awq_attention_prefill.hip).
// row_tiles: of each sequence, or with `flat` of all of them, one after the other.
int prefill_row_tiles(int seqs, int rows, int kv_heads, int group, int head_dim, int max_q, int few, bool flat);
int prefill_splits(int seqs, int kv_heads, int row_tiles, bool flat, long long key_tiles);
hipError_t launch_attention_prefill(const AttnArgs &p, int head_dim, bool bf16, int row_tiles, bool flat, hipStream_t s);

}  // namespace awq
