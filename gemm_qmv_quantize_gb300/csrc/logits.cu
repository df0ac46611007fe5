// logits.cu -- penalties for repeated tokens, biases and grammar masks on logits, one
// row a request. For token v of row m, with n = how often v is in the history from
// prompt_len on:
//   x = in the history at all ? (x > 0 ? x / repetition : x repetition) : x
//   x = x - (frequency n + presence [n > 0]) + (v's biases);  y = mask bit ? x : -inf
//
// A cluster of CTAs shares a row's tokens (or a part of them): each CTA keeps the counts of
// its own tokens in shared memory and reads a share of the history, counting a token in
// whichever CTA of the cluster owns it, so that the history is read once a cluster. Counts
// are whole numbers: their order does not matter. The logits, loaded before the history is
// counted, pass through registers once; bound by their bytes.
#include <algorithm>

#include "decode_ops.h"
#include "qmv.h"
#include "qmv_device.cuh"

namespace qmv {
namespace {

__device__ uint32_t g_logits_error;

constexpr int kThreads = 512;
constexpr int kAhead = 6;             // float4 of logits a thread loads before the history is counted
constexpr int kMaxCluster = 8;
constexpr int kMaxOwned = 48 * 1024;  // tokens of a CTA at most: 192 KB of counts
constexpr int kSms = 152;
constexpr uint32_t kSeen = 1u << 31;  // the bit above a token's count: it is in the prompt

__device__ __forceinline__ uint32_t cluster_rank()
{
    uint32_t r;
    asm("mov.u32 %0, %cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync()
{
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// The shared-memory word at the same place in the cluster's CTA `rank`.
__device__ __forceinline__ uint32_t peer_addr(const uint32_t *local, int rank)
{
    uint32_t remote;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(remote) : "r"(smem_addr(local)), "r"(rank));
    return remote;
}
__device__ __forceinline__ void count_answered(uint32_t addr)
{
    asm volatile("red.relaxed.cluster.shared::cluster.add.u32 [%0], 1;" ::"r"(addr) : "memory");
}
__device__ __forceinline__ void mark_seen(uint32_t addr)
{
    asm volatile("red.relaxed.cluster.shared::cluster.or.b32 [%0], %1;" ::"r"(addr), "r"(kSeen) : "memory");
}

struct RowTerms {
    float repetition, frequency, presence;
    const uint32_t *mask;   // of this row, or null
};

__device__ __forceinline__ bool allowed(const RowTerms &t, int v)
{
    return !t.mask || (__ldg(t.mask + (v >> 5)) >> (v & 31)) & 1u;
}

__device__ __forceinline__ float penalized(const RowTerms &t, float x, uint32_t count)
{
    if (count) {
        x = x > 0.0f ? x / t.repetition : x * t.repetition;
        const uint32_t n = count & ~kSeen;
        if (n) x -= t.frequency * static_cast<float>(n) + t.presence;
    }
    return x;
}

// owned: tokens a CTA, a multiple of 4; grid (parts * cluster, M), a cluster a part of the
// row. kVec: the row's logits and outputs may be moved 16 bytes at a time from their first
// aligned token on.
template <bool kVec>
__global__ void __launch_bounds__(kThreads, 2) logits_kernel(const __grid_constant__ LogitsArgs g, int owned, int cluster)
{
    extern __shared__ __align__(16) uint32_t count[];
    const int m = blockIdx.y, tid = threadIdx.x;
    const int rank = cluster > 1 ? static_cast<int>(cluster_rank()) : 0;
    const int part0 = static_cast<int>(blockIdx.x) / cluster * cluster * owned;   // the cluster's first token
    const int v0 = min(part0 + rank * owned, g.V), n = min(owned, g.V - v0);
    grid_launch_dependents();
    grid_dependency_wait();
    const float *in = g.logits + static_cast<int64_t>(m) * g.V + v0;
    float *out = g.y + static_cast<int64_t>(m) * g.V + v0;
    // tokens before the first 16-byte boundary, then groups of 4, then the rest
    const int head = kVec ? min(n, static_cast<int>((16u - (reinterpret_cast<uintptr_t>(in) & 15u)) & 15u) / 4) : n;
    const int groups = kVec ? (n - head) / 4 : 0;
    float4 ahead[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i)
        if (tid + i * kThreads < groups) ahead[i] = reinterpret_cast<const float4 *>(in + head)[tid + i * kThreads];
    for (int i = tid; i < owned / 4; i += kThreads) reinterpret_cast<uint4 *>(count)[i] = make_uint4(0, 0, 0, 0);
    int total = g.total_len ? g.total_len[m] : 0;
    if (total > g.max_history) {
        if (tid == 0) atomicOr(&g_logits_error, kErrIndex);
        total = g.max_history;
    }
    const int prompt = total > 0 ? g.prompt_len[m] : 0;
    RowTerms t;
    t.repetition = g.repetition ? g.repetition[m] : 1.0f;
    t.frequency = g.frequency ? g.frequency[m] : 0.0f;
    t.presence = g.presence ? g.presence[m] : 0.0f;
    const int mr = g.mask ? (g.mask_row ? g.mask_row[m] : m) : -1;
    if (mr >= g.n_masks && g.mask && tid == 0) atomicOr(&g_logits_error, kErrIndex);
    t.mask = mr >= 0 && mr < g.n_masks ? g.mask + static_cast<int64_t>(mr) * ((g.V + 31) / 32) : nullptr;
    if (cluster > 1) {
        cluster_sync();   // every CTA's counts are zero
    } else {
        __syncthreads();
    }
    const int32_t *tokens = g.tokens + static_cast<int64_t>(m) * g.max_history;
    const int span = cluster * owned;
#pragma unroll 4
    for (int i = rank * kThreads + tid; i < total; i += cluster * kThreads) {
        const int v = tokens[i], at = v - part0;
        if (v >= g.V) {
            atomicOr(&g_logits_error, kErrIndex);
        } else if (v >= 0 && at >= 0 && at < span) {
            const int owner = at / owned;
            const uint32_t addr = peer_addr(count + (at - owner * owned), owner);
            if (i >= prompt) {
                count_answered(addr);
            } else {
                mark_seen(addr);
            }
        }
    }
    if (cluster > 1) {
        cluster_sync();   // all of the history is counted, and no CTA counts in another any more
    } else {
        __syncthreads();
    }
    auto one = [&](int i) {
        const float x = penalized(t, in[i], count[i]);
        out[i] = allowed(t, v0 + i) ? x : -INFINITY;
    };
    for (int i = tid; i < head; i += kThreads) one(i);
    for (int i = head + 4 * groups + tid; i < n; i += kThreads) one(i);
    auto four = [&](int group, float4 x) {
        const int i = head + 4 * group, v = v0 + i;
        float e[4] = {x.x, x.y, x.z, x.w};
        uint32_t bits = 0xfu;
        if (t.mask) {
            const uint32_t lo = __ldg(t.mask + (v >> 5)), hi = (v & 31) > 28 ? __ldg(t.mask + (v >> 5) + 1) : 0u;
            bits = __funnelshift_r(lo, hi, v & 31);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            e[j] = penalized(t, e[j], count[i + j]);
            if (!((bits >> j) & 1u)) e[j] = -INFINITY;
        }
        reinterpret_cast<float4 *>(out + head)[group] = make_float4(e[0], e[1], e[2], e[3]);
    };
#pragma unroll
    for (int i = 0; i < kAhead; ++i)
        if (tid + i * kThreads < groups) four(tid + i * kThreads, ahead[i]);
    for (int i = tid + kAhead * kThreads; i < groups; i += kThreads) four(i, reinterpret_cast<const float4 *>(in + head)[i]);
    if (g.max_bias == 0) return;
    // Biases, onto what this CTA has just written: the first entry of a token adds all of
    // that token's, in their order.
    __syncthreads();
    const int32_t *bt = g.bias_tokens + static_cast<int64_t>(m) * g.max_bias;
    const float *bv = g.bias_values + static_cast<int64_t>(m) * g.max_bias;
    for (int j = tid; j < g.max_bias; j += kThreads) {
        const int v = bt[j];
        if (v < v0 || v >= v0 + n || !allowed(t, v)) continue;
        bool first = true;
        for (int k = 0; k < j && first; ++k) first = bt[k] != v;
        if (!first) continue;
        float x = out[v - v0] + bv[j];
        for (int k = j + 1; k < g.max_bias; ++k)
            if (bt[k] == v) x += bv[k];
        out[v - v0] = x;
    }
}

}  // namespace

cudaError_t launch_logits(const LogitsArgs &g, cudaStream_t s)
{
    route_hit(kRouteLogits);
    // Up to 8 CTAs a cluster, of 2048 tokens at least; more clusters a row (each reads the
    // history) where the rows leave SMs idle, or a CTA's counts would not fit.
    int cluster = kMaxCluster;
    while (cluster > 1 && g.V < 2048 * cluster) cluster /= 2;
    const int fill = std::max(1, std::min(2 * kSms / (cluster * g.M), g.V / (2048 * cluster)));
    const int fit = (g.V + kMaxOwned * cluster - 1) / (kMaxOwned * cluster);
    const int parts = std::max(fill, fit);
    const int owned = ((g.V + parts * cluster - 1) / (parts * cluster) + 3) & ~3;
    const bool vec = ((reinterpret_cast<uintptr_t>(g.logits) ^ reinterpret_cast<uintptr_t>(g.y)) & 15u) == 0;
    auto kern = vec ? logits_kernel<true> : logits_kernel<false>;
    cudaError_t e = ensure_smem_attr(reinterpret_cast<const void *>(kern), owned * 4);
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute attr[2];
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3(kThreads);
    cfg.gridDim = dim3(static_cast<unsigned>(parts * cluster), static_cast<unsigned>(g.M));
    cfg.dynamicSmemBytes = static_cast<size_t>(owned) * 4;
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = set_launch_overlap_attr(attr);
    if (cluster > 1) {
        attr[cfg.numAttrs].id = cudaLaunchAttributeClusterDimension;
        attr[cfg.numAttrs].val.clusterDim.x = static_cast<unsigned>(cluster);
        attr[cfg.numAttrs].val.clusterDim.y = 1;
        attr[cfg.numAttrs].val.clusterDim.z = 1;
        ++cfg.numAttrs;
    }
    return cudaLaunchKernelEx(&cfg, kern, g, owned, cluster);
}

cudaError_t read_error_word_logits(uint32_t *out, bool clear)
{
    cudaError_t e = cudaMemcpyFromSymbol(out, g_logits_error, sizeof(uint32_t));
    if (e != cudaSuccess || !clear) return e;
    const uint32_t zero = 0;
    return cudaMemcpyToSymbol(g_logits_error, &zero, sizeof(uint32_t));
}

}  // namespace qmv
