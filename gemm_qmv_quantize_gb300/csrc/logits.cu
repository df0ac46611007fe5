// logits.cu -- penalties for repeated tokens, biases and grammar masks on logits, one
// row a request. For token v of row m, with n = how often v is in the history from
// prompt_len on:
//   x = in the history at all ? (x > 0 ? x / repetition : x repetition) : x
//   x = x - (frequency n + presence [n > 0]) + (v's biases);  y = mask bit ? x : -inf
//
// A CTA owns a tile of a row's tokens, keeps their counts in shared memory and reads the
// whole history, which the row's other CTAs find in L2, counting what is in its tile; then
// its logits, loaded before that, pass through registers once. Counts are whole numbers:
// the order of the atomics does not matter. Bound by the logits' bytes, and by the latencies
// of history, logits and biases one after the other, which a wave of CTAs has. (Clusters
// that read the history once and count in each other's shared memory were slower at every
// size measured: 14 to 23 us against 11 for 8 rows with 16000 tokens of history, 51 to 54
// against 33 for 96 rows with 3000.)
#include <algorithm>

#include "decode_ops.h"
#include "qmv.h"
#include "qmv_device.cuh"

namespace qmv {
namespace {

__device__ uint32_t g_logits_error;

constexpr int kThreads = 512;
constexpr int kAhead = 3;             // float4 of logits and int4 of history that a thread loads
constexpr int kHistoryAhead = 1;      // before it waits for anything
constexpr int kMinTile = 2048, kMaxTile = 16384;
constexpr int kSms = 152, kCtasPerSm = 3;
constexpr uint32_t kSeen = 1u << 31;  // the bit above a token's count: it is in the prompt

struct RowTerms {
    float repetition, frequency, presence;
    const uint32_t *mask;   // of this row, or null
};

__device__ __forceinline__ bool allowed(const uint32_t *mask, int v)
{
    return !mask || (__ldg(mask + (v >> 5)) >> (v & 31)) & 1u;
}

// The logit x of a token whose count is not zero.
__device__ __forceinline__ float penalized(const RowTerms &t, float x, uint32_t count)
{
    x = x > 0.0f ? x / t.repetition : x * t.repetition;
    const uint32_t n = count & ~kSeen;
    return n ? x - (t.frequency * static_cast<float>(n) + t.presence) : x;
}

// Grid (tiles, M). Shared memory: tile + 4 counts, those of the row's 16-byte groups of
// logits on 16-byte boundaries.
__global__ void __launch_bounds__(kThreads, 3) logits_kernel(const __grid_constant__ LogitsArgs g, int tile)
{
    extern __shared__ __align__(16) uint32_t counts[];
    const int m = blockIdx.y, tid = threadIdx.x, v0 = static_cast<int>(blockIdx.x) * tile, n = min(tile, g.V - v0);
    grid_launch_dependents();
    grid_dependency_wait();
    const float *in = g.logits + static_cast<int64_t>(m) * g.V + v0;
    float *out = g.y + static_cast<int64_t>(m) * g.V + v0;
    const bool vec = ((reinterpret_cast<uintptr_t>(in) ^ reinterpret_cast<uintptr_t>(out)) & 15u) == 0;
    // tokens before the first 16-byte boundary, then groups of 4, then the rest
    const int head = vec ? min(n, static_cast<int>((16u - (reinterpret_cast<uintptr_t>(in) & 15u)) & 15u) / 4) : n;
    const int groups = (n - head) / 4;
    uint32_t *count = counts + ((4 - head) & 3);   // of token v0
    float4 ahead[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i)
        if (tid + i * kThreads < groups) ahead[i] = __ldcs(reinterpret_cast<const float4 *>(in + head) + tid + i * kThreads);
    const int32_t *tokens = g.tokens + static_cast<int64_t>(m) * g.max_history;
    const int all_fours = (reinterpret_cast<uintptr_t>(tokens) & 15u) == 0 ? g.max_history / 4 : 0;
    int4 early[kHistoryAhead];
#pragma unroll
    for (int i = 0; i < kHistoryAhead; ++i)
        if (tid + i * kThreads < all_fours) early[i] = __ldg(reinterpret_cast<const int4 *>(tokens) + tid + i * kThreads);
    RowTerms t;
    const int32_t *bias_tokens = g.bias_tokens + static_cast<int64_t>(m) * g.max_bias;
    const int bias_token = tid < g.max_bias ? __ldg(bias_tokens + tid) : -1;
    int total = g.total_len ? g.total_len[m] : 0;
    const int prompt = g.prompt_len ? g.prompt_len[m] : 0;
    const int mr = g.mask ? (g.mask_row ? g.mask_row[m] : m) : -1;
    t.repetition = g.repetition ? g.repetition[m] : 1.0f;
    t.frequency = g.frequency ? g.frequency[m] : 0.0f;
    t.presence = g.presence ? g.presence[m] : 0.0f;
    for (int i = tid; i < tile / 4 + 1; i += kThreads) reinterpret_cast<uint4 *>(counts)[i] = make_uint4(0, 0, 0, 0);
    if (total > g.max_history) {
        if (tid == 0) atomicOr(&g_logits_error, kErrIndex);
        total = g.max_history;
    }
    if (mr >= g.n_masks && g.mask && tid == 0) atomicOr(&g_logits_error, kErrIndex);
    t.mask = mr >= 0 && mr < g.n_masks ? g.mask + static_cast<int64_t>(mr) * ((g.V + 31) / 32) : nullptr;
    __syncthreads();
    auto tally = [&](int i, int v) {
        if (v >= g.V) atomicOr(&g_logits_error, kErrIndex);
        if (v < v0 || v >= v0 + n) return;
        if (i >= prompt) {
            atomicAdd(count + (v - v0), 1u);
        } else {
            atomicOr(count + (v - v0), kSeen);
        }
    };
    auto tally4 = [&](int i, int4 v) {
        tally(4 * i, v.x);
        tally(4 * i + 1, v.y);
        tally(4 * i + 2, v.z);
        tally(4 * i + 3, v.w);
    };
    const int fours = min(all_fours, total / 4);
#pragma unroll
    for (int i = 0; i < kHistoryAhead; ++i)
        if (tid + i * kThreads < fours) tally4(tid + i * kThreads, early[i]);
#pragma unroll 4
    for (int i = tid + kHistoryAhead * kThreads; i < fours; i += kThreads) tally4(i, __ldg(reinterpret_cast<const int4 *>(tokens) + i));
#pragma unroll 4
    for (int i = 4 * fours + tid; i < total; i += kThreads) tally(i, __ldg(tokens + i));
    __syncthreads();
    auto one = [&](int i) {
        float x = in[i];
        if (count[i]) x = penalized(t, x, count[i]);
        out[i] = allowed(t.mask, v0 + i) ? x : -INFINITY;
    };
    for (int i = tid; i < head; i += kThreads) one(i);
    for (int i = head + 4 * groups + tid; i < n; i += kThreads) one(i);
    auto four = [&](int group, float4 x) {
        const int i = head + 4 * group, v = v0 + i;
        const uint4 c = *reinterpret_cast<const uint4 *>(count + i);
        if (c.x | c.y | c.z | c.w) {
            const uint32_t cs[4] = {c.x, c.y, c.z, c.w};
            float e[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (cs[j]) e[j] = penalized(t, e[j], cs[j]);
            x = make_float4(e[0], e[1], e[2], e[3]);
        }
        if (t.mask) {
            const uint32_t lo = __ldg(t.mask + (v >> 5)), hi = (v & 31) > 28 ? __ldg(t.mask + (v >> 5) + 1) : 0u;
            const uint32_t bits = __funnelshift_r(lo, hi, v & 31);
            x.x = bits & 1u ? x.x : -INFINITY;
            x.y = bits & 2u ? x.y : -INFINITY;
            x.z = bits & 4u ? x.z : -INFINITY;
            x.w = bits & 8u ? x.w : -INFINITY;
        }
        __stcs(reinterpret_cast<float4 *>(out + head) + group, x);
    };
#pragma unroll
    for (int i = 0; i < kAhead; ++i)
        if (tid + i * kThreads < groups) four(tid + i * kThreads, ahead[i]);
#pragma unroll 2
    for (int i = tid + kAhead * kThreads; i < groups; i += kThreads) four(i, __ldcs(reinterpret_cast<const float4 *>(in + head) + i));
    if (g.max_bias == 0) return;
    // Biases, onto what this CTA has just written: the first entry of a token adds all of
    // that token's, in their order. Each entry looks at all others, which is cheap for the
    // hundred or so of a request (8 rows of 151936: 12 us with 300 entries, 5 without any) and
    // grows with the square of the list: 52 us with 1000, 790 with 4096. (Inside the pass above, each thread that met a token with
    // a bias searching the list, 8 rows with 100 biases took 13.5 us for 10.7; each such token
    // finished by the thread that marks it first, before the pass, 11.8.)
    __syncthreads();
    const float *bias_values = g.bias_values + static_cast<int64_t>(m) * g.max_bias;
    for (int j = tid; j < g.max_bias; j += kThreads) {
        const int v = j < kThreads ? bias_token : __ldg(bias_tokens + j);
        if (v >= g.V && blockIdx.x == 0) atomicOr(&g_logits_error, kErrIndex);
        if (v < v0 || v >= v0 + n || !allowed(t.mask, v)) continue;
        bool again = false;
#pragma unroll 8
        for (int k = 0; k < j; ++k) again |= __ldg(bias_tokens + k) == v;
        if (again) continue;
        float x = out[v - v0] + __ldg(bias_values + j);
#pragma unroll 8
        for (int k = j + 1; k < g.max_bias; ++k)
            if (__ldg(bias_tokens + k) == v) x += __ldg(bias_values + k);
        out[v - v0] = x;
    }
}

// The largest tile up to 16384 that leaves a wave of CTAs, three an SM (96 rows of 151936:
// 33 us, 36 with 8192, 44 with 4096); 4096 for fewer rows, and 2048 where that leaves SMs
// without a CTA (1 row of 151936 with 2000 tokens of history: 4.9 us for 5.5).
int tile_of(int M, int V)
{
    auto ctas = [&](int tile) { return static_cast<int64_t>(M) * ((V + tile - 1) / tile); };
    int tile = ctas(2 * kMinTile) < kSms ? kMinTile : 2 * kMinTile;
    while (tile > kMinTile && tile < kMaxTile && ctas(2 * tile) >= kCtasPerSm * kSms) tile *= 2;
    return tile;
}

}  // namespace

cudaError_t launch_logits(const LogitsArgs &g, cudaStream_t s)
{
    route_hit(kRouteLogits);
    const int tile = tile_of(g.M, g.V);
    const size_t smem = static_cast<size_t>(tile + 4) * 4;
    cudaError_t e = ensure_smem_attr(reinterpret_cast<const void *>(logits_kernel), static_cast<int>(smem));
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute attr[1];
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3(kThreads);
    cfg.gridDim = dim3(static_cast<unsigned>((g.V + tile - 1) / tile), static_cast<unsigned>(g.M));
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = set_launch_overlap_attr(attr);
    return cudaLaunchKernelEx(&cfg, logits_kernel, g, tile);
}

cudaError_t read_error_word_logits(uint32_t *out, bool clear)
{
    cudaError_t e = cudaMemcpyFromSymbol(out, g_logits_error, sizeof(uint32_t));
    if (e != cudaSuccess || !clear) return e;
    const uint32_t zero = 0;
    return cudaMemcpyToSymbol(g_logits_error, &zero, sizeof(uint32_t));
}

}  // namespace qmv
