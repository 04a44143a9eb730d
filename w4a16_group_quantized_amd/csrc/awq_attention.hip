// awq_attention and awq_tree_attention: which kernel takes a call, how its keys are cut into
// chunks, and the kernel that joins these.  awq_attention_split.h has the formula and the
// kernel of few rows, awq_attention_prefill.hip and awq_tree_attention_prefill.hip those of many.
#include <algorithm>

#include "awq_attention.h"
#include "awq_internal.h"

namespace awq {
namespace {

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
constexpr int kUncutTiles = 12, kManyGroups = 192, kLongTiles = 256, kMaxSplits = 256;
constexpr int kJoinGroups = 8192;          // workgroups that join chunks
constexpr size_t kMixedRoom = 1u << 28;    // bytes of partial results for single tokens among prompts

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

// The same where a row has few chunks: D / 4 lanes to a row and head, all of its chunks on the way
// at once, no LDS, and the same bits (the sums in combine_kernel's order).  1024 rows of 32 heads
// of 128 in up to three chunks: 34 -> 12 us.
constexpr int kFewChunks = 8;
template <typename T, int D>
__global__ void __launch_bounds__(256) combine_few_kernel(AttnArgs p) {
#pragma clang fp contract(off)   // (weights are rounded before they are summed up)
    constexpr int kLanes = D / 4, kParts = 256 / kLanes < kFewChunks ? 256 / kLanes : kFewChunks;
    const KvView &c = p.c;
    const int row0 = min(max(c.q_starts[0], 0), c.rows), row1 = min(max(c.q_starts[c.seqs], 0), c.rows);
    const int i = row0 * p.q_heads + (int)(blockIdx.x * (256 / kLanes) + threadIdx.x / kLanes), lane = threadIdx.x % kLanes;
    if (i >= row1 * p.q_heads) return;
    const float *src = p.part + (long long)i * p.splits * kPart<D>;
    const int n = min((int)src[D + 2], p.splits);
    if (n <= 1) return;                        // the one chunk has written its outputs
    float own[kFewChunks], l[kFewChunks];
    float4_t v[kFewChunks];
#pragma unroll
    for (int k = 0; k < kFewChunks; ++k) {     // (behind the last the last again)
        const float *from = src + min(k, n - 1) * kPart<D>;
        own[k] = from[D];
        l[k] = from[D + 1];
        v[k] = *reinterpret_cast<const float4_t *>(from + 4 * lane);
    }
    float mx = kEmpty;
#pragma unroll
    for (int k = 0; k < kFewChunks; ++k) mx = fmaxf(mx, own[k]);
#pragma unroll
    for (int k = 0; k < kFewChunks; ++k) l[k] = k < n ? l[k] * __builtin_amdgcn_exp2f(own[k] - mx) : 0.0f;
    const float sum = ((l[0] + l[4]) + (l[2] + l[6])) + ((l[1] + l[5]) + (l[3] + l[7]));
    const float inv = sum > 0.0f || !(sum == sum) ? 1.0f / sum : 0.0f;
    float4_t part[kParts];
#pragma unroll
    for (int k = 0; k < kParts; ++k) part[k] = float4_t{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int k = 0; k < kFewChunks; ++k) {
        const float w = l[k] * inv;
        if (k < n) {
#pragma unroll
            for (int e = 0; e < 4; ++e) part[k % kParts][e] = __builtin_fmaf(w, v[k][e], part[k % kParts][e]);
        }
    }
    float4_t o = part[0];
#pragma unroll
    for (int k = 1; k < kParts; ++k) o += part[k];
    if (kParts < 256 / kLanes) o += float4_t{0.0f, 0.0f, 0.0f, 0.0f};      // (of -0 this makes 0, as there)
    uint2 y;
    y.x = (uint32_t)from_float<T>(o[0]) | ((uint32_t)from_float<T>(o[1]) << 16);
    y.y = (uint32_t)from_float<T>(o[2]) | ((uint32_t)from_float<T>(o[3]) << 16);
    *reinterpret_cast<uint2 *>(p.out + (long long)i * D + 4 * lane) = y;
}

// The same for drafted trees in more chunks, up to 64: a wave to a row and head, a chunk's maximum and
// sum to a lane, then D / 4 lanes to a chunk.  No LDS and no barriers: 256 rows of 32 heads of 64 in nine
// chunks 13.1 -> 5.8 us, 48 of 64 heads of 128 in up to 23 10.4 -> 8.5.
// Bound: HBM and L2 (4 TB/s there), or latency.
constexpr int kWaveChunks = 64;
template <typename T, int D>
__global__ void __launch_bounds__(256) combine_wave_kernel(AttnArgs p) {
    constexpr int kLanes = D / 4, kAtOnce = 64 / kLanes, kAhead = 8;
    const KvView &c = p.c;
    const int row0 = min(max(c.q_starts[0], 0), c.rows), row1 = min(max(c.q_starts[c.seqs], 0), c.rows);
    const int lane = threadIdx.x & 63, i = row0 * p.q_heads + (int)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    if (i >= row1 * p.q_heads) return;
    const float *src = p.part + (long long)i * p.splits * kPart<D>;
    const int n = __builtin_amdgcn_readfirstlane(min((int)src[D + 2], p.splits));
    if (n <= 1) return;                        // the one chunk has written its outputs
    const float *mine = src + min(lane, n - 1) * kPart<D> + D;
    const float own = mine[0], some = mine[1];
    float mx = own;                            // (of the lanes behind the last chunk the last again)
    for (int k = 32; k > 0; k >>= 1) mx = fmaxf(mx, __shfl_xor(mx, k));
    const float l = lane < n ? some * __builtin_amdgcn_exp2f(own - mx) : 0.0f;
    float sum = l;
    for (int k = 32; k > 0; k >>= 1) sum += __shfl_xor(sum, k);
    const float weight = l * (sum > 0.0f || !(sum == sum) ? 1.0f / sum : 0.0f);
    const int at = lane / kLanes, col = 4 * (lane % kLanes);
    float4_t o = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int k0 = 0; k0 < n; k0 += kAhead * kAtOnce) {
        float4_t v[kAhead];
#pragma unroll
        for (int u = 0; u < kAhead; ++u)
            v[u] = *reinterpret_cast<const float4_t *>(src + min(k0 + u * kAtOnce + at, n - 1) * kPart<D> + col);
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            const int k = k0 + u * kAtOnce + at;
            const float w = __shfl(weight, min(k, 63));
            if (k < n) o += w * v[u];
        }
    }
#pragma unroll
    for (int k = kLanes; k < 64; k <<= 1)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[e] += __shfl_xor(o[e], k);
    if (at == 0) {
        uint2 y;
        y.x = (uint32_t)from_float<T>(o[0]) | ((uint32_t)from_float<T>(o[1]) << 16);
        y.y = (uint32_t)from_float<T>(o[2]) | ((uint32_t)from_float<T>(o[3]) << 16);
        *reinterpret_cast<uint2 *>(p.out + (long long)i * D + col) = y;
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
//
// Drafted trees have a kernel of their own for many rows, which takes over earlier (sequences x kv heads,
// rows times heads of a kv head, keys, us of the split / tree kernel): 16 x 8, 56 rows, 8000 108 / 89; 80, 4000 78 / 76; 160, 2000
// 73 / 73; 1 x 8, 96, 8000 33 / 28; heads of 64, 112, 8000 24 / 22; 320, 2000 38 / 26.  And where
// its row tiles fill the GPU without a cut: 64 x 8, 240 rows, 100 88 / 55; 16 x 8, 500 46 / 30; 1000 64 / 46; 160,
// 1000 45 / 44; but 8 x 8, 256 rows, 1000 37 / 51.  Heads of 256 as prompts, and those of 64 with eight sequences and
// more (16 x 8, 96 rows, 8000 78 / 90).
int prompt_rows(int seqs, int kv_heads, long long tiles, int head_dim, bool tree, long long most) {
    static const int rows[3][2][5] = {{{80, 80, 80, 144, 512}, {96, 128, 768, 768, 768}},
                                      {{72, 72, 72, 120, 288}, {64, 96, 256, 384, 768}},
                                      {{24, 24, 24, 72, 96}, {24, 24, 40, 72, 288}}};
    static const int tree_rows[2][2][5] = {{{80, 80, 80, 96, 256}, {96, 128, 768, 768, 768}},
                                           {{60, 72, 72, 80, 288}, {48, 80, 256, 384, 768}}};
    const long long pairs = (long long)seqs * kv_heads, all = pairs * tiles;
    const int width = head_dim > 128 ? 2 : head_dim > 64 ? 1 : 0;
    const int at = all >= 12000 ? 0 : all >= 3000 ? 1 : all >= 1500 ? 2 : all >= 400 ? 3 : 4;
    int from = (tree && width < 2 ? tree_rows : rows)[width][seqs >= kXcds][at];
    if (tree && width == 1 && tiles < kTreeCutTiles && pairs * ((most + 127) / 128) >= kTreeFullTiles) from = std::min(from, 200);
    return (int)std::max<long long>(from, (width == 2 ? 320 : 640) / pairs);
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
    TreePlan tree;           // of a tree's rows in the prompt kernel
    int row_tiles, splits, target;
    int room() const { return std::max(splits, prompt_splits); }
};
Plan plan(int seqs, int rows, int kv_heads, int group, int head_dim, int max_q, int max_kv, int window, int sinks, bool tree) {
    Plan pl;
    long long keys = max_kv;
    if (window > 0) keys = std::min(keys, (long long)window + max_q + std::min(sinks, max_kv) + 2 * kTile);
    const long long tiles = (keys + kTile - 1) / kTile;
    pl.few = prompt_rows(seqs, kv_heads, tiles, head_dim, tree, (long long)max_q * group);
    pl.prompt = (long long)max_q * group >= pl.few;
    pl.mixed = pl.prompt && rows_differ(seqs, rows, max_q);
    pl.row_tiles = pl.target = 0;
    pl.splits = pl.prompt_splits = 1;
    pl.tree = {};
    pl.wide = false;
    if (pl.prompt) {
        pl.prompt_tiles = prefill_row_tiles(seqs, rows, kv_heads, group, head_dim, max_q, pl.few, pl.mixed);
        pl.prompt_splits = prefill_splits(seqs, kv_heads, pl.prompt_tiles, pl.mixed, tiles);
        if (tree) {
            pl.tree = tree_plan(seqs, rows, kv_heads, group, head_dim, max_q, pl.mixed, pl.few, tiles);
            pl.prompt_splits = pl.tree.room;
        }
        if (!pl.mixed) return pl;
    }
    // (the kernel steps on where the grid is cut)
    const int units = (seqs + kXcds - 1) / kXcds * kXcds;
    const long long some = pl.mixed ? std::min((rows - max_q) / (seqs - 1) + 1, (pl.few - 1) / group + 1) : max_q;
    pl.row_tiles = (int)std::min<long long>((some * group + kSplitRows - 1) / kSplitRows,
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
    pl.splits = (int)std::max<long long>(1, std::min<long long>({want, (tiles + kSplitLeastChunk - 1) / kSplitLeastChunk, kMaxSplits}));
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

template <typename T, int D>
void combine_dim(const AttnArgs &p, hipStream_t s) {
    const long long items = (long long)p.c.rows * p.q_heads;
    if (p.splits <= kFewChunks)
        combine_few_kernel<T, D><<<(int)((items + 1024 / D - 1) / (1024 / D)), 256, 0, s>>>(p);
    else if (p.tree != nullptr && p.splits <= kWaveChunks)
        combine_wave_kernel<T, D><<<(int)((items + 3) / 4), 256, 0, s>>>(p);
    else
        combine_kernel<T, D><<<(int)std::min<long long>(items, kJoinGroups), 256, 0, s>>>(p);
}
template <typename T>
hipError_t combine(const AttnArgs &p, int D, hipStream_t s) {
    switch (D) {
    case 64: combine_dim<T, 64>(p, s); break;
    case 128: combine_dim<T, 128>(p, s); break;
    case 256: combine_dim<T, 256>(p, s); break;
    default: return hipErrorInvalidValue;
    }
    return hipGetLastError();
}

hipError_t launch(AttnArgs p, int D, const Plan &pl, bool bf16, hipStream_t s) {
    hipError_t e = hipSuccess;
    const bool tree = p.tree != nullptr;
    if (pl.prompt) {
        p.few = pl.mixed ? pl.few : 0;
        p.most = tree ? pl.tree.shares : pl.prompt_splits;
        e = tree ? launch_tree_attention_prefill(p, D, bf16, pl.tree.waves, s) : launch_attention_prefill(p, D, bf16, pl.prompt_tiles, pl.mixed, s);
        if (e != hipSuccess) return e;
    }
    if (!pl.prompt || pl.mixed) {
        p.few = pl.mixed ? pl.few : 0x7FFFFFFF;
        p.most = pl.splits;
        e = (tree ? launch_tree_attention_split : launch_attention_split)(p, D, bf16, pl.wide, pl.row_tiles, s);
    }
    if (e != hipSuccess || p.part == nullptr) return e;
    return bf16 ? combine<bhalf_t>(p, D, s) : combine<half_t>(p, D, s);
}

}  // namespace

size_t attention_workspace(int seqs, int rows, int q_heads, int kv_heads, int head_dim, int max_q,
                           int max_kv, int window, int sinks, bool tree) {
    const Plan pl = plan(seqs, rows, kv_heads, q_heads / kv_heads, head_dim, max_q, max_kv, window, sinks, tree);
    if (pl.room() == 1) return 0;
    return (size_t)rows * q_heads * pl.room() * (head_dim + 4) * sizeof(float);
}

hipError_t launch_attention(const KvView &c, int head_dim, const uint16_t *q, long long q_stride,
                            uint16_t *out, int q_heads, bool bf16, float scale, int window, int sinks,
                            int max_q, int max_kv, const uint32_t *tree, int tree_words, void *workspace, hipStream_t s) {
    const Plan pl = plan(c.seqs, c.rows, c.kv_heads, q_heads / c.kv_heads, head_dim, max_q, max_kv, window, sinks, tree != nullptr);
    AttnArgs p{c, q, q_stride, out, pl.room() > 1 ? (float *)workspace : nullptr, q_heads,
               q_heads / c.kv_heads, scale * kLog2e, std::min(window, kWidest), sinks, 1, pl.target, pl.room(), 0,
               tree, tree_words};
    return launch(p, head_dim, pl, bf16, s);
}

}  // namespace awq
