// awq_kv_keep: compaction.  Of a sequence's rows, its last tokens, the kept ones move together,
// in place: token first + i becomes the token that was first + kept[i].
//
//   scale   of a page that tokens come to: the largest of the scales of the pages that its
//           tokens (those that come, and those before them that stay) were in
//   codes   c as it is where the scales are alike, else e4m3_rne(c * (old / new)): scales that are
//           powers of two only shift the exponent, exact but for codes that become subnormal
//
// kept ascends, so a token never moves up: what is read for a place lies there or behind it.
// One workgroup owns a (sequence, kv head) and takes the pages from the first, each in pieces
// that are read, then (after a barrier) written: a piece's places are behind all that was written
// before, and in front of all that is read later.  Nobody else writes these slabs or scales: no
// atomics, and the same bits each time.  Bound: latency; a page after the other.
#include "awq_internal.h"
#include "awq_kv.h"

namespace awq {
namespace {

constexpr int kThreads = 256, kMaxPage = 256, kAtOnce = 4;

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
__global__ void __launch_bounds__(kThreads) keep_kernel(KeepArgs p) {
    constexpr int U = D / 16;                  // 16-byte pieces of a key
    __shared__ int m_s, id_s[kMaxPage], slot_s[kMaxPage];
    __shared__ float fk_s[kMaxPage], fv_s[kMaxPage], red[2][kThreads / 64];
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
    for (int i = tid; i < most; i += kThreads) {
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
            for (int i = tid; i < held * (D / 4); i += kThreads) {
                uint32_t *w = reinterpret_cast<uint32_t *>(kslab) + i;
                *w = rescaled(*w, f);
            }
        }
        const int w0 = held >> 2, w1 = (held + count + 3) >> 2, words = w1 - w0;
        if (w0 > 0 && va != vs0) {
            const float f = vs0 / va;
            for (int i = tid; i < w0 * D; i += kThreads) {
                uint32_t *w = reinterpret_cast<uint32_t *>(vslab + (i / w0) * P) + i % w0;
                *w = rescaled(*w, f);
            }
        }
        // keys that come, token after token
        for (int x0 = 0; x0 < count * U; x0 += kAtOnce * kThreads) {
            uint4 r[kAtOnce];
#pragma unroll
            for (int n = 0; n < kAtOnce; ++n) {
                const int x = x0 + n * kThreads + tid, t = held + x / U;
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
                const int x = x0 + n * kThreads + tid;
                if (x < count * U) *reinterpret_cast<uint4 *>(kslab + (held + x / U) * D + 16 * (x % U)) = r[n];
            }
        }
        // values, element after element: four slots to a word
        for (int x0 = 0; x0 < words * D; x0 += kAtOnce * kThreads) {
            uint32_t r[kAtOnce];
#pragma unroll
            for (int n = 0; n < kAtOnce; ++n) {
                const int x = x0 + n * kThreads + tid, d = x / words, w = w0 + x % words;
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
                const int x = x0 + n * kThreads + tid;
                if (x < words * D) reinterpret_cast<uint32_t *>(vslab + (x / words) * P)[w0 + x % words] = r[n];
            }
        }
        __syncthreads();                       // what the page's tokens came from is read no more
    }
}

}  // namespace

hipError_t launch_kv_keep(const KvView &c, int head_dim, const int32_t *kept, int width, const int32_t *counts, int32_t *lens_out, hipStream_t s) {
    const KeepArgs p{c, kept, counts, lens_out, width};
    const dim3 grid(c.kv_heads, c.seqs);
    switch (head_dim) {
    case 64: keep_kernel<64><<<grid, kThreads, 0, s>>>(p); break;
    case 128: keep_kernel<128><<<grid, kThreads, 0, s>>>(p); break;
    case 256: keep_kernel<256><<<grid, kThreads, 0, s>>>(p); break;
    default: return hipErrorInvalidValue;
    }
    return hipGetLastError();
}

}  // namespace awq
