// Shared by the kernels of the 8-bit paged key/value cache (awq_kv_append,
// awq_attention): the views that reach them, types, and e4m3 conversions.
#pragma once

#include "awq_device.h"

namespace awq {

// The cache and batch of include/awq.h, as kernel arguments.  log2_page: the
// page size is a power of two.
struct KvView {
    uint8_t *k;            // e4m3 [pages][kv_heads][page][dim]
    uint8_t *v;            // e4m3 [pages][kv_heads][dim][page]
    float *k_scales;       // [pages][kv_heads]
    float *v_scales;
    const int32_t *page_table;
    const int32_t *kv_lens;
    const int32_t *q_starts;
    int pages, log2_page, kv_heads;
    int seqs, table_width, rows;
};

// What a sequence has in a call: rows [row0, row0 + n) at positions
// len - n + t.  Everything is clamped to the arrays that the host checked, so
// no content of the device arrays leads out of them.
struct Seq {
    int row0, n, len;
    __device__ __forceinline__ int first() const { return len - n; }
};
__device__ __forceinline__ Seq load_seq(const KvView &c, int b) {
    Seq s;
    const int a = min(max(c.q_starts[b], 0), c.rows);
    const int e = min(max(c.q_starts[b + 1], 0), c.rows);
    s.row0 = a;
    s.n = max(e - a, 0);
    s.len = min(max(c.kv_lens[b], 0), c.table_width << c.log2_page);   // at most 2^30
    return s;
}

// The n-th of the pieces of work that the sequences have, one sequence after the other:
// its sequence (or seqs, if there are fewer) and its number there.  All lanes of a wave
// have to ask, for the same n.
template <typename F>
__device__ __forceinline__ int2 seq_of_piece(const KvView &c, int n, F pieces) {
    const int lane = threadIdx.x & 63;
    for (int b = 0; b < c.seqs; b += 64) {
        const int own = b + lane < c.seqs ? pieces(load_seq(c, b + lane)) : 0;
        int upto = own;
#pragma unroll
        for (int k = 1; k < 64; k <<= 1) {
            const int other = __shfl_up(upto, k);
            upto += lane >= k ? other : 0;
        }
        const int all = __builtin_amdgcn_readlane(upto, 63);
        if (n < all) {
            const int at = (int)__builtin_ctzll(__ballot(upto > n));
            return make_int2(b + at, n - (__builtin_amdgcn_readlane(upto, at) - __builtin_amdgcn_readlane(own, at)));
        }
        n -= all;
    }
    return make_int2(c.seqs, 0);
}
// A call whose sequences have, but for the longest, less than half its rows on average
// (prompts among single tokens): grids for the longest would be mostly empty.
inline bool rows_differ(int seqs, int rows, int max_q) {
    return seqs > 1 && 2ll * (rows - max_q) < (long long)(seqs - 1) * max_q;
}

// Activation types: fp16 (T = half_t) and bf16 (T = bhalf_t), as 16-bit patterns.
struct bhalf_t {};
template <typename T>
__device__ __forceinline__ float to_float(uint16_t u);
template <>
__device__ __forceinline__ float to_float<half_t>(uint16_t u) {
    return (float)as_half(u);
}
template <>
__device__ __forceinline__ float to_float<bhalf_t>(uint16_t u) {
    return __builtin_bit_cast(float, (uint32_t)u << 16);
}
template <typename T>
__device__ __forceinline__ uint16_t from_float(float f);
template <>
__device__ __forceinline__ uint16_t from_float<half_t>(float f) {
    return as_u16((half_t)f);
}
template <>
__device__ __forceinline__ uint16_t from_float<bhalf_t>(float f) {
    return __builtin_bit_cast(uint16_t, (__bf16)f);
}

template <typename T>
__device__ __forceinline__ void unpack8(uint4 u, float f[8]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = to_float<T>((uint16_t)w[i]);
        f[2 * i + 1] = to_float<T>((uint16_t)(w[i] >> 16));
    }
}
template <typename T>
__device__ __forceinline__ void load8(const uint16_t *p, float f[8]) {
    unpack8<T>(*reinterpret_cast<const uint4 *>(p), f);
}
template <typename T>
__device__ __forceinline__ uint4 pack8(const float f[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        w[i] = (uint32_t)from_float<T>(f[2 * i]) | ((uint32_t)from_float<T>(f[2 * i + 1]) << 16);
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// e4m3 codes (1-4-3, bias 7, largest 448, 0x7F NaN): four floats of magnitude
// at most 448 to a word, nearest, ties to even; and a word back.
__device__ __forceinline__ uint32_t to_e4m3x4(float a, float b, float c, float d) {
    int w = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
    w = __builtin_amdgcn_cvt_pk_fp8_f32(c, d, w, true);
    return (uint32_t)w;
}
__device__ __forceinline__ void from_e4m3x4(uint32_t w, float f[4]) {
    f[0] = __builtin_amdgcn_cvt_f32_fp8((int)w, 0);
    f[1] = __builtin_amdgcn_cvt_f32_fp8((int)w, 1);
    f[2] = __builtin_amdgcn_cvt_f32_fp8((int)w, 2);
    f[3] = __builtin_amdgcn_cvt_f32_fp8((int)w, 3);
}
// Eight codes (two words) to eight halves, exactly (e4m3 is a subset of fp16),
// one instruction for two.
__device__ __forceinline__ half8_t e4m3x8_to_half(uint32_t lo, uint32_t hi) {
    const half2_t a = __builtin_bit_cast(half2_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8((int)lo, 1.0f, false));
    const half2_t b = __builtin_bit_cast(half2_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8((int)lo, 1.0f, true));
    const half2_t c = __builtin_bit_cast(half2_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8((int)hi, 1.0f, false));
    const half2_t d = __builtin_bit_cast(half2_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8((int)hi, 1.0f, true));
    return half8_t{a.x, a.y, b.x, b.y, c.x, c.y, d.x, d.y};
}

// 2^e as a float, e in [-126, 127].
__device__ __forceinline__ float pow2(int e) {
    return __builtin_bit_cast(float, (uint32_t)(e + 127) << 23);
}

}  // namespace awq
