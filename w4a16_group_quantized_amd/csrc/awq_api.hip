// C ABI of libawq (declared in include/awq.h): argument validation on the
// host, then one launch on the caller's stream.  Validation runs before any
// HIP call, so a rejected call touches neither the device nor the stream.
#include "../../include/awq.h"

#include <hip/hip_runtime.h>

#include <math.h>
#include <stdlib.h>

#include "awq_internal.h"
#include "awq_kv.h"

namespace {

constexpr long long kMaxElems = (1LL << 31) - 1;
constexpr int kMaxSplits = 16;
constexpr long long kMaxTokens = 1LL << 30;   // of one sequence in the paged cache

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

awq_status check_layer(const awq_layer *w) {
    if (w == nullptr || w->qweight == nullptr || w->scales == nullptr)
        return AWQ_ERROR_INVALID_VALUE;
    const long long K = w->K, N = w->N, G = w->group_size;
    if (K <= 0 || N <= 0 || G <= 0) return AWQ_ERROR_INVALID_VALUE;
    if (w->layout != AWQ_LAYOUT_CANONICAL && w->layout != AWQ_LAYOUT_INTERLEAVED &&
        w->layout != AWQ_LAYOUT_BLOCKED)
        return AWQ_ERROR_INVALID_VALUE;
    if (K % 8 || N % 8 || G % 8 || K % G) return AWQ_ERROR_SHAPE;
    if (w->layout == AWQ_LAYOUT_BLOCKED && N % 128) return AWQ_ERROR_SHAPE;
    if (K * N > kMaxElems) return AWQ_ERROR_SHAPE;  // the dequantized weight's element count
    if (!aligned16(w->qweight) || !aligned16(w->scales) ||
        (w->qzeros != nullptr && !aligned16(w->qzeros)))
        return AWQ_ERROR_ALIGNMENT;
    return AWQ_SUCCESS;
}

awq_status check_io(const uint16_t *x, const uint16_t *y, const awq_layer *w, int32_t M) {
    if (M < 0) return AWQ_ERROR_INVALID_VALUE;
    if (M == 0) return AWQ_SUCCESS;
    if (x == nullptr || y == nullptr) return AWQ_ERROR_INVALID_VALUE;
    if ((long long)M * w->K > kMaxElems || (long long)M * w->N > kMaxElems) return AWQ_ERROR_SHAPE;
    if (!aligned16(x) || !aligned16(y)) return AWQ_ERROR_ALIGNMENT;
    return AWQ_SUCCESS;
}

hipStream_t as_stream(void *s) { return reinterpret_cast<hipStream_t>(s); }

// AWQ_SYNC set to anything but "" or "0" in the environment (read once, at the
// first call): every call that launched work waits for its stream and reports
// a fault of its own kernels as AWQ_ERROR_HIP, instead of leaving it to the
// caller's next synchronization.  A stream that is being captured into a graph
// is not waited for (a capture cannot synchronize).  For debugging only: the
// wait serializes the caller with the GPU.
bool sync_mode() {
    static const bool on = [] {
        const char *v = getenv("AWQ_SYNC");
        return v != nullptr && v[0] != '\0' && !(v[0] == '0' && v[1] == '\0');
    }();
    return on;
}

// The status of a call whose launches returned e on `stream`.
awq_status done(void *stream, hipError_t e) {
    if (e != hipSuccess) return AWQ_ERROR_HIP;
    if (!sync_mode()) return AWQ_SUCCESS;
    hipStreamCaptureStatus capture = hipStreamCaptureStatusNone;
    if (hipStreamIsCapturing(as_stream(stream), &capture) != hipSuccess) return AWQ_ERROR_HIP;
    if (capture != hipStreamCaptureStatusNone) return AWQ_SUCCESS;
    if (hipStreamSynchronize(as_stream(stream)) != hipSuccess) return AWQ_ERROR_HIP;
    return hipGetLastError() == hipSuccess ? AWQ_SUCCESS : AWQ_ERROR_HIP;
}

// The launchers take the layout as AWQ_LAYOUT_* (checked by check_layer).
int layout_of(const awq_layer *w) { return w->layout; }

// Calibration X [M][K] and fp16 weight W [K][N] of the scale search.
awq_status check_calibration(const uint16_t *x, int32_t M, const uint16_t *w, int32_t K, int32_t N,
                             int32_t G) {
    if (x == nullptr || w == nullptr || M <= 0 || K <= 0 || N <= 0 || G <= 0)
        return AWQ_ERROR_INVALID_VALUE;
    if (K % 8 || N % 8 || G % 8 || K % G) return AWQ_ERROR_SHAPE;
    if ((long long)M * K > kMaxElems || (long long)K * N > kMaxElems || (long long)M * N > kMaxElems)
        return AWQ_ERROR_SHAPE;
    if (!aligned16(x) || !aligned16(w)) return AWQ_ERROR_ALIGNMENT;
    return AWQ_SUCCESS;
}

// The paged cache and the batch of the attention calls.
awq_status check_kv(const awq_kv_cache *c, const awq_kv_batch *b) {
    if (c == nullptr || b == nullptr) return AWQ_ERROR_INVALID_VALUE;
    if (c->k == nullptr || c->v == nullptr || c->k_scales == nullptr || c->v_scales == nullptr ||
        (b->seqs > 0 && (b->page_table == nullptr || b->kv_lens == nullptr || b->q_starts == nullptr)))
        return AWQ_ERROR_INVALID_VALUE;
    if (c->pages <= 0 || c->page_size <= 0 || c->kv_heads <= 0 || c->head_dim <= 0 || b->seqs < 0 ||
        b->rows < 0 || b->table_width <= 0 || b->max_q < 0 || b->max_kv < 0)
        return AWQ_ERROR_INVALID_VALUE;
    if (c->page_size & (c->page_size - 1) || c->page_size < 16 || c->page_size > 256)
        return AWQ_ERROR_SHAPE;
    // grid dimensions
    if (c->kv_heads > 65535 || b->seqs > 65535 || (long long)c->kv_heads * b->seqs >= 1 << 20)
        return AWQ_ERROR_SHAPE;
    if ((long long)c->pages * c->kv_heads > kMaxElems || (long long)b->seqs * b->table_width > kMaxElems)
        return AWQ_ERROR_SHAPE;
    if (!aligned16(c->k) || !aligned16(c->v) || !aligned16(c->k_scales) || !aligned16(c->v_scales) ||
        !aligned16(b->page_table) || !aligned16(b->kv_lens) || !aligned16(b->q_starts))
        return AWQ_ERROR_ALIGNMENT;
    if ((long long)b->table_width * c->page_size > kMaxTokens) return AWQ_ERROR_SHAPE;
    if (!awq::kv_head_dim_supported(c->head_dim)) return AWQ_ERROR_UNSUPPORTED;
    return AWQ_SUCCESS;
}

// Rows [rows][heads][dim] of 16-bit values, `stride` elements from row to row.
awq_status check_rows(const uint16_t *p, long long rows, int32_t stride, int32_t heads, int32_t dim) {
    if (p == nullptr || heads <= 0) return AWQ_ERROR_INVALID_VALUE;
    const long long width = (long long)heads * dim;
    if (stride < width || stride % 8 || rows * width > kMaxElems) return AWQ_ERROR_SHAPE;
    if (!aligned16(p)) return AWQ_ERROR_ALIGNMENT;
    return AWQ_SUCCESS;
}

awq::KvView kv_view(const awq_kv_cache *c, const awq_kv_batch *b) {
    int log2_page = 0;
    while ((1 << log2_page) < c->page_size) ++log2_page;
    return awq::KvView{c->k, c->v, c->k_scales, c->v_scales, b->page_table, b->kv_lens, b->q_starts,
                       c->pages, log2_page, c->kv_heads, b->seqs, b->table_width, b->rows};
}

bool known_type(int32_t t) { return t == AWQ_TYPE_FP16 || t == AWQ_TYPE_BF16; }

// The largest row and token counts of a sequence as they size a grid: within
// what the arrays can hold.
int grid_rows(const awq_kv_batch *b) { return b->max_q < 1 ? 1 : b->max_q < b->rows ? b->max_q : b->rows > 0 ? b->rows : 1; }
int grid_keys(const awq_kv_cache *c, const awq_kv_batch *b) {
    const long long cap = (long long)b->table_width * c->page_size;
    return b->max_kv < 1 ? 1 : b->max_kv < cap ? b->max_kv : (int)cap;
}

}  // namespace

extern "C" {

const char *awq_status_string(awq_status status) {
    switch (status) {
    case AWQ_SUCCESS: return "AWQ_SUCCESS";
    case AWQ_ERROR_INVALID_VALUE: return "AWQ_ERROR_INVALID_VALUE: null pointer or non-positive size";
    case AWQ_ERROR_SHAPE: return "AWQ_ERROR_SHAPE: K%8, N%8, G%8, K%G must be 0 (and N%128 in the blocked layout) and arrays below 2^31 elements";
    case AWQ_ERROR_ALIGNMENT: return "AWQ_ERROR_ALIGNMENT: tensor pointers must be 16-byte aligned";
    case AWQ_ERROR_UNSUPPORTED: return "AWQ_ERROR_UNSUPPORTED: outside this entry point (awq_gemv takes M <= 16; awq_gemv_gate_up also needs G % 128 == 0; awq_gemm_gate_up needs G % 64 == 0 and K % 256 == 0; awq_gemm_splitk needs slices of whole groups (or one group) and whole 128- or 256-k ring turns)";
    case AWQ_ERROR_WORKSPACE: return "AWQ_ERROR_WORKSPACE: null, unaligned or smaller than the *_workspace_bytes query";
    case AWQ_ERROR_HIP: return "AWQ_ERROR_HIP: the HIP runtime refused the launch";
    }
    return "AWQ_ERROR_UNKNOWN";
}

awq_status awq_pack(const uint8_t *codes, int32_t *qweight, int32_t K, int32_t N, void *stream) {
    if (codes == nullptr || qweight == nullptr || K <= 0 || N <= 0) return AWQ_ERROR_INVALID_VALUE;
    if (K % 8 || N % 8 || (long long)K * N > kMaxElems) return AWQ_ERROR_SHAPE;
    if (!aligned16(codes) || !aligned16(qweight)) return AWQ_ERROR_ALIGNMENT;
    return done(stream, awq::launch_pack(codes, qweight, K, N, as_stream(stream)));
}

awq_status awq_pack_zeros(const uint8_t *zeros, int32_t *qzeros, int32_t groups, int32_t N,
                          void *stream) {
    if (zeros == nullptr || qzeros == nullptr || groups <= 0 || N <= 0)
        return AWQ_ERROR_INVALID_VALUE;
    if (N % 8 || (long long)groups * N > kMaxElems) return AWQ_ERROR_SHAPE;
    if (!aligned16(zeros) || !aligned16(qzeros)) return AWQ_ERROR_ALIGNMENT;
    return done(stream, awq::launch_pack_zeros(zeros, qzeros, groups, N, as_stream(stream)));
}

awq_status awq_repack(const int32_t *src, int32_t *dst, int32_t K, int32_t N, int32_t from,
                      int32_t to, void *stream) {
    if (src == nullptr || dst == nullptr || K <= 0 || N <= 0) return AWQ_ERROR_INVALID_VALUE;
    const auto known = [](int32_t l) {
        return l == AWQ_LAYOUT_CANONICAL || l == AWQ_LAYOUT_INTERLEAVED || l == AWQ_LAYOUT_BLOCKED;
    };
    if (!known(from) || !known(to)) return AWQ_ERROR_INVALID_VALUE;
    // In place only where no word moves: the blocked layout moves words.
    if (src == dst && (from == AWQ_LAYOUT_BLOCKED) != (to == AWQ_LAYOUT_BLOCKED))
        return AWQ_ERROR_INVALID_VALUE;
    if (K % 8 || N % 8 || (long long)K * N > kMaxElems) return AWQ_ERROR_SHAPE;
    if ((from == AWQ_LAYOUT_BLOCKED || to == AWQ_LAYOUT_BLOCKED) && N % 128) return AWQ_ERROR_SHAPE;
    if (!aligned16(src) || !aligned16(dst)) return AWQ_ERROR_ALIGNMENT;
    const long long words = (long long)(K / 8) * N;
    if (from == to) {
        if (src == dst) return AWQ_SUCCESS;
        return done(stream, hipMemcpyAsync(dst, src, (size_t)words * 4, hipMemcpyDeviceToDevice,
                                       as_stream(stream)));
    }
    return done(stream, awq::launch_repack(src, dst, K, N, from, to, as_stream(stream)));
}

awq_status awq_dequant(const awq_layer *layer, uint16_t *w_out, void *stream) {
    awq_status st = check_layer(layer);
    if (st != AWQ_SUCCESS) return st;
    if (w_out == nullptr) return AWQ_ERROR_INVALID_VALUE;
    if (!aligned16(w_out)) return AWQ_ERROR_ALIGNMENT;
    return done(stream, awq::launch_dequant(layer->qweight, layer->scales, layer->qzeros, w_out,
                                        layer->K, layer->N, layer->group_size, layout_of(layer), as_stream(stream)));
}

size_t awq_gemv_workspace_bytes(int32_t M, int32_t K, int32_t N) {
    (void)M;
    (void)K;
    (void)N;
    return 0;   // the K split is reduced inside each workgroup (LDS)
}

awq_status awq_gemv(const uint16_t *x, const awq_layer *layer, uint16_t *y, int32_t M,
                    void *workspace, size_t workspace_bytes, void *stream) {
    awq_status st = check_layer(layer);
    if (st != AWQ_SUCCESS) return st;
    st = check_io(x, y, layer, M);
    if (st != AWQ_SUCCESS || M == 0) return st;
    if (M > 16) return AWQ_ERROR_UNSUPPORTED;
    if (workspace != nullptr && !aligned16(workspace)) return AWQ_ERROR_WORKSPACE;
    if (workspace_bytes < awq_gemv_workspace_bytes(M, layer->K, layer->N)) return AWQ_ERROR_WORKSPACE;
    return done(stream, awq::launch_gemv(x, layer->qweight, layer->scales, layer->qzeros, y, M,
                                     layer->K, layer->N, layer->group_size, layout_of(layer), as_stream(stream)));
}

awq_status awq_gemm(const uint16_t *x, const awq_layer *layer, uint16_t *y, int32_t M,
                    void *stream) {
    awq_status st = check_layer(layer);
    if (st != AWQ_SUCCESS) return st;
    st = check_io(x, y, layer, M);
    if (st != AWQ_SUCCESS || M == 0) return st;
    return done(stream, awq::launch_gemm(x, layer->qweight, layer->scales, layer->qzeros, y, M,
                                     layer->K, layer->N, layer->group_size, layout_of(layer), as_stream(stream)));
}

awq_status awq_quantize(const uint16_t *w, int32_t K, int32_t N, int32_t group_size,
                        int32_t symmetric, int32_t *qweight, uint16_t *scales, int32_t *qzeros,
                        void *stream) {
    if (w == nullptr || qweight == nullptr || scales == nullptr || (!symmetric && qzeros == nullptr))
        return AWQ_ERROR_INVALID_VALUE;
    if (K <= 0 || N <= 0 || group_size <= 0) return AWQ_ERROR_INVALID_VALUE;
    if (K % 8 || N % 8 || group_size % 8 || K % group_size || (long long)K * N > kMaxElems)
        return AWQ_ERROR_SHAPE;
    if (!aligned16(w) || !aligned16(qweight) || !aligned16(scales) ||
        (!symmetric && !aligned16(qzeros)))
        return AWQ_ERROR_ALIGNMENT;
    return done(stream, awq::launch_quantize(w, qweight, scales, qzeros, K, N, group_size,
                                         symmetric != 0, as_stream(stream)));
}

awq_status awq_gemv_gate_up(const uint16_t *x, const awq_layer *layer, uint16_t *h, int32_t M,
                            void *stream) {
    awq_status st = check_layer(layer);
    if (st != AWQ_SUCCESS) return st;
    if (layer->N % 16) return AWQ_ERROR_SHAPE;
    st = check_io(x, h, layer, M);
    if (st != AWQ_SUCCESS || M == 0) return st;
    if (!awq::gemv_gate_up_supported(M, layer->K, layer->N, layer->group_size))
        return AWQ_ERROR_UNSUPPORTED;
    return done(stream, awq::launch_gemv_gate_up(x, layer->qweight, layer->scales, layer->qzeros, h, M,
                                             layer->K, layer->N, layer->group_size,
                                             layout_of(layer), as_stream(stream)));
}

awq_status awq_gemm_gate_up(const uint16_t *x, const awq_layer *layer, uint16_t *h, int32_t M,
                            void *stream) {
    awq_status st = check_layer(layer);
    if (st != AWQ_SUCCESS) return st;
    if (layer->N % 16) return AWQ_ERROR_SHAPE;
    st = check_io(x, h, layer, M);
    if (st != AWQ_SUCCESS || M == 0) return st;
    if (!awq::gemm_gate_up_supported(layer->K, layer->N, layer->group_size))
        return AWQ_ERROR_UNSUPPORTED;
    return done(stream, awq::launch_gemm_gate_up(x, layer->qweight, layer->scales, layer->qzeros, h, M,
                                             layer->K, layer->N, layer->group_size,
                                             layout_of(layer), as_stream(stream)));
}

size_t awq_gemm_splitk_workspace_bytes(int32_t M, int32_t N, int32_t splits) {
    if (M <= 0 || N <= 0 || splits < 1 || splits > kMaxSplits) return 0;
    return awq::gemm_splitk_workspace(M, N, splits);
}

awq_status awq_gemm_splitk(const uint16_t *x, const awq_layer *layer, uint16_t *y, int32_t M,
                           int32_t splits, void *workspace, size_t workspace_bytes, void *stream) {
    awq_status st = check_layer(layer);
    if (st != AWQ_SUCCESS) return st;
    if (splits < 1 || splits > kMaxSplits) return AWQ_ERROR_INVALID_VALUE;
    st = check_io(x, y, layer, M);
    if (st != AWQ_SUCCESS || M == 0) return st;
    if (splits == 1)
        return done(stream, awq::launch_gemm(x, layer->qweight, layer->scales, layer->qzeros, y, M,
                                         layer->K, layer->N, layer->group_size, layout_of(layer), as_stream(stream)));
    if (!awq::gemm_splitk_supported(layer->K, layer->group_size, splits)) return AWQ_ERROR_UNSUPPORTED;
    if ((long long)splits * M * layer->N > kMaxElems) return AWQ_ERROR_SHAPE;
    if (workspace == nullptr || !aligned16(workspace) ||
        workspace_bytes < awq::gemm_splitk_workspace(M, layer->N, splits))
        return AWQ_ERROR_WORKSPACE;
    return done(stream, awq::launch_gemm_splitk(x, layer->qweight, layer->scales, layer->qzeros, y, M,
                                            layer->K, layer->N, layer->group_size, splits, workspace,
                                            layout_of(layer), as_stream(stream)));
}

awq_status awq_gemm_splitk_static(const uint16_t *x, const awq_layer *layer, uint16_t *y,
                                  int32_t M, int32_t splits, void *stream) {
    static_assert(awq::kStaticScratchBytes == AWQ_GEMM_SPLITK_STATIC_SCRATCH_BYTES,
                  "the header states the scratch size");
    awq_status st = check_layer(layer);
    if (st != AWQ_SUCCESS) return st;
    if (splits < 1 || splits > kMaxSplits) return AWQ_ERROR_INVALID_VALUE;
    st = check_io(x, y, layer, M);
    if (st != AWQ_SUCCESS || M == 0) return st;
    if (splits == 1)
        return done(stream, awq::launch_gemm(x, layer->qweight, layer->scales, layer->qzeros, y, M,
                                         layer->K, layer->N, layer->group_size, layout_of(layer), as_stream(stream)));
    if (!awq::gemm_splitk_supported(layer->K, layer->group_size, splits)) return AWQ_ERROR_UNSUPPORTED;
    if (awq::gemm_splitk_workspace(M, layer->N, splits) > awq::kStaticScratchBytes)
        return AWQ_ERROR_WORKSPACE;
    return done(stream, awq::launch_gemm_splitk_static(x, layer->qweight, layer->scales, layer->qzeros,
                                                   y, M, layer->K, layer->N, layer->group_size,
                                                   splits, layout_of(layer), as_stream(stream)));
}

size_t awq_channel_stats_workspace_bytes(int32_t M, int32_t K, int32_t N, int32_t group_size) {
    if (M <= 0 || K <= 0 || N <= 0 || group_size <= 0 || K % group_size) return 0;
    return awq::channel_stats_workspace(M, K, N, group_size);
}

size_t awq_scale_search_workspace_bytes(int32_t M, int32_t K, int32_t N, int32_t group_size) {
    if (M <= 0 || K <= 0 || N <= 0 || group_size <= 0 || K % group_size) return 0;
    return awq::scale_search_workspace(M, K, N, group_size);
}

awq_status awq_channel_stats(const uint16_t *x, int32_t M, const uint16_t *w, int32_t K, int32_t N,
                             int32_t group_size, float *xbar, float *wbar, void *workspace,
                             size_t workspace_bytes, void *stream) {
    awq_status st = check_calibration(x, M, w, K, N, group_size);
    if (st != AWQ_SUCCESS) return st;
    if (xbar == nullptr || wbar == nullptr) return AWQ_ERROR_INVALID_VALUE;
    if (workspace == nullptr || !aligned16(workspace) ||
        workspace_bytes < awq::channel_stats_workspace(M, K, N, group_size))
        return AWQ_ERROR_WORKSPACE;
    return done(stream, awq::launch_channel_stats(x, M, w, K, N, group_size, xbar, wbar, workspace,
                                              as_stream(stream)));
}

awq_status awq_scale_search(const uint16_t *x, int32_t M, const uint16_t *w, int32_t K, int32_t N,
                            int32_t group_size, int32_t symmetric, const float *alphas,
                            int32_t n_alpha, double *losses, int32_t *best, float *best_scales,
                            void *workspace, size_t workspace_bytes, void *stream) {
    awq_status st = check_calibration(x, M, w, K, N, group_size);
    if (st != AWQ_SUCCESS) return st;
    if (alphas == nullptr || losses == nullptr || best == nullptr || n_alpha < 1 ||
        n_alpha > awq::kScaleSearchMaxAlphas)
        return AWQ_ERROR_INVALID_VALUE;
    for (int i = 0; i < n_alpha; ++i)
        if (!(alphas[i] >= 0.0f && alphas[i] <= 1.0f)) return AWQ_ERROR_INVALID_VALUE;   // also NaN
    if (workspace == nullptr || !aligned16(workspace) ||
        workspace_bytes < awq::scale_search_workspace(M, K, N, group_size))
        return AWQ_ERROR_WORKSPACE;
    return done(stream, awq::launch_scale_search(x, M, w, K, N, group_size, symmetric != 0, alphas,
                                             n_alpha, losses, best, best_scales, workspace,
                                             as_stream(stream)));
}

// What both forms of awq_kv_append check; `work`: whether there is any.
static awq_status check_append(const uint16_t *q, int32_t q_stride, const uint16_t *k, int32_t k_stride,
                               const uint16_t *v, int32_t v_stride, const uint16_t *q_out, int32_t q_heads,
                               int32_t type, const float *rope, int32_t rope_positions, int32_t rot_dim,
                               const awq_kv_cache *cache, const awq_kv_batch *batch, bool *work) {
    *work = false;
    awq_status st = check_kv(cache, batch);
    if (st != AWQ_SUCCESS) return st;
    if (!known_type(type) || rot_dim < 0 || q_heads <= 0) return AWQ_ERROR_INVALID_VALUE;
    if (q_heads % cache->kv_heads || rot_dim % 16 || rot_dim > cache->head_dim) return AWQ_ERROR_SHAPE;
    if (rot_dim > 0) {
        if (rope == nullptr || rope_positions <= 0) return AWQ_ERROR_INVALID_VALUE;
        if (!aligned16(rope)) return AWQ_ERROR_ALIGNMENT;
    }
    if (batch->seqs == 0 || batch->rows == 0) return AWQ_SUCCESS;
    st = check_rows(k, batch->rows, k_stride, cache->kv_heads, cache->head_dim);
    if (st == AWQ_SUCCESS) st = check_rows(v, batch->rows, v_stride, cache->kv_heads, cache->head_dim);
    if (st == AWQ_SUCCESS && (q == nullptr) != (q_out == nullptr)) st = AWQ_ERROR_INVALID_VALUE;
    if (st == AWQ_SUCCESS && q != nullptr)
        st = check_rows(q, batch->rows, q_stride, q_heads, cache->head_dim);
    if (st == AWQ_SUCCESS && q_out != nullptr && !aligned16(q_out)) st = AWQ_ERROR_ALIGNMENT;
    *work = st == AWQ_SUCCESS;
    return st;
}

awq_status awq_kv_append(const uint16_t *q, int32_t q_stride, const uint16_t *k, int32_t k_stride,
                         const uint16_t *v, int32_t v_stride, uint16_t *q_out, int32_t q_heads,
                         int32_t type, const float *rope, int32_t rope_positions, int32_t rot_dim,
                         int32_t interleaved, const awq_kv_cache *cache, const awq_kv_batch *batch,
                         void *stream) {
    bool work;
    const awq_status st = check_append(q, q_stride, k, k_stride, v, v_stride, q_out, q_heads, type, rope,
                                       rope_positions, rot_dim, cache, batch, &work);
    if (!work) return st;
    return done(stream, awq::launch_kv_append(kv_view(cache, batch), cache->head_dim, q, q_stride, k,
                                              k_stride, v, v_stride, q_out, q_heads, rope,
                                              rope_positions, rot_dim, interleaved != 0,
                                              type == AWQ_TYPE_BF16, grid_rows(batch), as_stream(stream)));
}

awq_status awq_kv_append_at(const uint16_t *q, int32_t q_stride, const uint16_t *k, int32_t k_stride,
                            const uint16_t *v, int32_t v_stride, uint16_t *q_out, int32_t q_heads,
                            int32_t type, const float *rope, int32_t rope_positions, int32_t rot_dim,
                            int32_t interleaved, const int32_t *positions, int32_t axes,
                            const uint8_t *axis_of, const awq_kv_cache *cache, const awq_kv_batch *batch,
                            void *stream) {
    bool work;
    const awq_status st = check_append(q, q_stride, k, k_stride, v, v_stride, q_out, q_heads, type, rope,
                                       rope_positions, rot_dim, cache, batch, &work);
    if (st != AWQ_SUCCESS) return st;
    if (axes < 1 || axes > AWQ_MAX_AXES) return AWQ_ERROR_INVALID_VALUE;
    awq::AxisMap map{};
    for (int f = 0; f < rot_dim / 2; ++f) {
        const int axis = axis_of == nullptr ? 0 : axis_of[f];
        if (axis >= axes) return AWQ_ERROR_INVALID_VALUE;
        map.set(f, axis);
    }
    if (!work) return st;
    if (positions == nullptr) return AWQ_ERROR_INVALID_VALUE;
    if ((long long)batch->rows * axes > kMaxElems) return AWQ_ERROR_SHAPE;
    if (!aligned16(positions)) return AWQ_ERROR_ALIGNMENT;
    return done(stream, awq::launch_kv_append_at(kv_view(cache, batch), cache->head_dim, q, q_stride, k,
                                                 k_stride, v, v_stride, q_out, q_heads, rope,
                                                 rope_positions, rot_dim, interleaved != 0, positions, axes, map,
                                                 type == AWQ_TYPE_BF16, grid_rows(batch), as_stream(stream)));
}

static size_t attention_workspace(int32_t q_heads, int32_t window, int32_t sinks, const awq_kv_cache *cache,
                                  const awq_kv_batch *batch, bool tree) {
    if (check_kv(cache, batch) != AWQ_SUCCESS || q_heads <= 0 || q_heads % cache->kv_heads || window < 0 ||
        sinks < 0 || batch->seqs == 0 || batch->rows == 0)
        return 0;
    return awq::attention_workspace(batch->seqs, batch->rows, q_heads, cache->kv_heads, cache->head_dim,
                                    grid_rows(batch), grid_keys(cache, batch), window, sinks, tree);
}

size_t awq_attention_workspace_bytes(int32_t q_heads, int32_t window, int32_t sinks,
                                     const awq_kv_cache *cache, const awq_kv_batch *batch) {
    return attention_workspace(q_heads, window, sinks, cache, batch, false);
}

// Both attentions; tree: whether the rows' bits are asked for.
static awq_status attention(const uint16_t *q, int32_t q_stride, uint16_t *out, int32_t q_heads, int32_t type,
                            float scale, int32_t window, int32_t sinks, bool tree, const uint32_t *mask,
                            int32_t mask_words, const awq_kv_cache *cache, const awq_kv_batch *batch,
                            void *workspace, size_t workspace_bytes, void *stream) {
    awq_status st = check_kv(cache, batch);
    if (st != AWQ_SUCCESS) return st;
    if (!known_type(type) || !isfinite(scale) || window < 0 || sinks < 0 || q_heads <= 0)
        return AWQ_ERROR_INVALID_VALUE;
    if (tree && mask_words <= 0) return AWQ_ERROR_INVALID_VALUE;
    if (q_heads % cache->kv_heads) return AWQ_ERROR_SHAPE;
    if (batch->seqs == 0 || batch->rows == 0) return AWQ_SUCCESS;
    st = check_rows(q, batch->rows, q_stride, q_heads, cache->head_dim);
    if (st == AWQ_SUCCESS && (out == nullptr || (tree && mask == nullptr))) st = AWQ_ERROR_INVALID_VALUE;
    if (st == AWQ_SUCCESS && tree && (long long)batch->rows * mask_words > kMaxElems) st = AWQ_ERROR_SHAPE;
    if (st == AWQ_SUCCESS && (!aligned16(out) || (tree && !aligned16(mask)))) st = AWQ_ERROR_ALIGNMENT;
    if (st != AWQ_SUCCESS) return st;
    const size_t need = attention_workspace(q_heads, window, sinks, cache, batch, tree);
    if (need > 0 && (workspace == nullptr || !aligned16(workspace) || workspace_bytes < need))
        return AWQ_ERROR_WORKSPACE;
    return done(stream, awq::launch_attention(kv_view(cache, batch), cache->head_dim, q, q_stride, out,
                                              q_heads, type == AWQ_TYPE_BF16, scale, window, sinks,
                                              grid_rows(batch), grid_keys(cache, batch), mask, mask_words,
                                              workspace, as_stream(stream)));
}

awq_status awq_attention(const uint16_t *q, int32_t q_stride, uint16_t *out, int32_t q_heads,
                         int32_t type, float scale, int32_t window, int32_t sinks,
                         const awq_kv_cache *cache, const awq_kv_batch *batch, void *workspace,
                         size_t workspace_bytes, void *stream) {
    return attention(q, q_stride, out, q_heads, type, scale, window, sinks, false, nullptr, 0, cache, batch,
                     workspace, workspace_bytes, stream);
}

awq_status awq_tree_rows(const int32_t *parents, uint32_t *mask, int32_t mask_words, int32_t *positions,
                         const awq_kv_batch *batch, void *stream) {
    if (batch == nullptr || batch->seqs < 0 || batch->rows < 0 || batch->max_q < 0 || mask_words <= 0 ||
        (batch->seqs > 0 && (batch->kv_lens == nullptr || batch->q_starts == nullptr)))
        return AWQ_ERROR_INVALID_VALUE;
    if (batch->seqs > 65535 || (long long)batch->rows * mask_words > kMaxElems) return AWQ_ERROR_SHAPE;
    if (!aligned16(batch->kv_lens) || !aligned16(batch->q_starts)) return AWQ_ERROR_ALIGNMENT;
    if (batch->seqs == 0 || batch->rows == 0) return AWQ_SUCCESS;
    if (parents == nullptr || mask == nullptr) return AWQ_ERROR_INVALID_VALUE;
    if (!aligned16(parents) || !aligned16(mask) || !aligned16(positions)) return AWQ_ERROR_ALIGNMENT;
    awq::KvView c{};
    c.kv_lens = batch->kv_lens;
    c.q_starts = batch->q_starts;
    c.seqs = batch->seqs;
    c.rows = batch->rows;
    return done(stream, awq::launch_tree_rows(parents, c, grid_rows(batch), mask, mask_words, positions, as_stream(stream)));
}

size_t awq_tree_attention_workspace_bytes(int32_t q_heads, int32_t window, int32_t sinks,
                                          const awq_kv_cache *cache, const awq_kv_batch *batch) {
    return attention_workspace(q_heads, window, sinks, cache, batch, true);
}

awq_status awq_tree_attention(const uint16_t *q, int32_t q_stride, uint16_t *out, int32_t q_heads,
                              int32_t type, float scale, int32_t window, int32_t sinks,
                              const uint32_t *mask, int32_t mask_words, const awq_kv_cache *cache,
                              const awq_kv_batch *batch, void *workspace, size_t workspace_bytes,
                              void *stream) {
    return attention(q, q_stride, out, q_heads, type, scale, window, sinks, true, mask, mask_words, cache,
                     batch, workspace, workspace_bytes, stream);
}

awq_status awq_kv_keep(const int32_t *kept, int32_t kept_width, const int32_t *counts, int32_t *lens_out,
                       const awq_kv_cache *cache, const awq_kv_batch *batch, void *stream) {
    const awq_status st = check_kv(cache, batch);
    if (st != AWQ_SUCCESS) return st;
    if (kept_width <= 0) return AWQ_ERROR_INVALID_VALUE;
    if ((long long)batch->seqs * kept_width > kMaxElems) return AWQ_ERROR_SHAPE;
    if (batch->seqs == 0) return AWQ_SUCCESS;
    if (kept == nullptr || counts == nullptr || lens_out == nullptr || lens_out == batch->kv_lens)
        return AWQ_ERROR_INVALID_VALUE;
    if (!aligned16(kept) || !aligned16(counts) || !aligned16(lens_out)) return AWQ_ERROR_ALIGNMENT;
    return done(stream, awq::launch_kv_keep(kv_view(cache, batch), cache->head_dim, kept, kept_width, counts,
                                            lens_out, as_stream(stream)));
}

size_t awq_kv_fork_workspace_bytes(int32_t new_seqs, const awq_kv_cache *cache, const awq_kv_batch *batch) {
    if (check_kv(cache, batch) != AWQ_SUCCESS || new_seqs <= 0 || new_seqs > 65535 ||
        (long long)new_seqs * batch->table_width > kMaxElems)
        return 0;
    return awq::kv_fork_workspace(new_seqs, batch->table_width, cache->pages);
}

awq_status awq_kv_fork(const int32_t *from, const int32_t *grow, int32_t new_seqs, const uint8_t *held,
                       const awq_kv_cache *cache, const awq_kv_batch *batch, int32_t *table_out,
                       int32_t *lens_out, int32_t *copies, int32_t *missing, void *workspace,
                       size_t workspace_bytes, void *stream) {
    const awq_status st = check_kv(cache, batch);
    if (st != AWQ_SUCCESS) return st;
    if (new_seqs < 0) return AWQ_ERROR_INVALID_VALUE;
    if (new_seqs > 65535 || (long long)new_seqs * batch->table_width > kMaxElems) return AWQ_ERROR_SHAPE;
    if (new_seqs == 0) return AWQ_SUCCESS;
    if (from == nullptr || grow == nullptr || table_out == nullptr || lens_out == nullptr || copies == nullptr ||
        missing == nullptr || table_out == batch->page_table || lens_out == batch->kv_lens)
        return AWQ_ERROR_INVALID_VALUE;
    if (!aligned16(from) || !aligned16(grow) || !aligned16(held) || !aligned16(table_out) || !aligned16(lens_out) ||
        !aligned16(copies) || !aligned16(missing))
        return AWQ_ERROR_ALIGNMENT;
    const size_t need = awq::kv_fork_workspace(new_seqs, batch->table_width, cache->pages);
    if (need > 0 && (workspace == nullptr || !aligned16(workspace) || workspace_bytes < need))
        return AWQ_ERROR_WORKSPACE;
    return done(stream, awq::launch_kv_fork(from, grow, new_seqs, held, kv_view(cache, batch), table_out, lens_out,
                                            copies, missing, workspace, as_stream(stream)));
}

awq_status awq_kv_copy(const int32_t *pairs, int32_t n, const awq_kv_cache *from, const awq_kv_cache *to, void *stream) {
    awq_kv_batch none{};
    none.table_width = 1;
    awq_status st = check_kv(from, &none);
    if (st == AWQ_SUCCESS) st = check_kv(to, &none);
    if (st != AWQ_SUCCESS) return st;
    if (n < 0) return AWQ_ERROR_INVALID_VALUE;
    if (from->page_size != to->page_size || from->kv_heads != to->kv_heads || from->head_dim != to->head_dim || n > 1 << 22)
        return AWQ_ERROR_SHAPE;
    if (n == 0) return AWQ_SUCCESS;
    if (pairs == nullptr) return AWQ_ERROR_INVALID_VALUE;
    if (!aligned16(pairs)) return AWQ_ERROR_ALIGNMENT;
    return done(stream, awq::launch_kv_copy(pairs, n, kv_view(from, &none), kv_view(to, &none), from->head_dim, as_stream(stream)));
}

}  // extern "C"
