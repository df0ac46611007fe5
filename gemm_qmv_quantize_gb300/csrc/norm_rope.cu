// norm_rope.cu -- RMS norms of a projection's q and k heads, rotary positions, and the append
// of k and v to a paged cache, held in 16 bits or as E4M3 codes with a scale for each block of
// 16 tokens and head. For a head x of D elements:
//   n = x / sqrt(mean(x^2) + eps) * w,   (a, b) -> (a c - b s, b c + a s)
// in fp32 from the projection's fp32 output, rounded once to q's and the cache's type. v is
// neither normed nor turned.
//
// Codes: a block's scale is the power of two s = 2^e with the least e >= -64 for which no
// finite new element of the block is above 448 s (448: E4M3's largest), but never below the
// scale that its earlier tokens have; when it grows these tokens' codes are multiplied by
// s_old / s and rounded again, which is exact unless they fall below 2^-6. A power of two
// costs no accuracy in a format with an exponent of its own, and makes x / s exact.
//
// A group of L lanes (8, 16 or 32: the power of two that holds D / 8) has a head of a token,
// a lane 8 of its elements: 4 pairs of the rotated part, or 8 elements beyond it. Bound by
// the bytes.
#include "decode_device.cuh"
#include "decode_ops.h"
#include "qmv.h"
#include "qmv_device.cuh"

namespace qmv {
namespace {

__device__ uint32_t g_norm_rope_error;

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

// The 8 elements e0 .. e0 + 3 and e1 .. e1 + 3 of a head that a lane has.
struct Unit {
    int e0, e1;
    bool live, turn;   // turn: (a[j], b[j]) or, interleaved, neighbours of a and of b are pairs
};

template <bool kInterleaved>
__device__ __forceinline__ Unit unit_of(int i, int D, int pairs, bool is_v)
{
    Unit u;
    u.live = i < D / 8;
    u.turn = !is_v && i < pairs / 4;
    u.e0 = u.turn && !kInterleaved ? 4 * i : 8 * i;
    u.e1 = u.turn && !kInterleaved ? pairs + 4 * i : 8 * i + 4;
    return u;
}

__device__ __forceinline__ void load8(float (&x)[8], const float *in, const Unit &u)
{
    const float4 p = __ldcs(reinterpret_cast<const float4 *>(in + u.e0)), q = __ldcs(reinterpret_cast<const float4 *>(in + u.e1));
    x[0] = p.x, x[1] = p.y, x[2] = p.z, x[3] = p.w, x[4] = q.x, x[5] = q.y, x[6] = q.z, x[7] = q.w;
}

// The norm, over the group of L lanes that has the head.
template <int L>
__device__ __forceinline__ void norm8(float (&x)[8], const float (&w)[8], int D, float eps)
{
    float sum = 0.0f;
#pragma unroll
    for (int j = 0; j < 8; ++j) sum = fmaf(x[j], x[j], sum);
#pragma unroll
    for (int o = L / 2; o > 0; o /= 2) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    const float r = 1.0f / sqrtf(sum / static_cast<float>(D) + eps);
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] = x[j] * r * w[j];
}

template <bool kInterleaved>
__device__ __forceinline__ void turn8(float (&x)[8], const float2 *cs, int i)
{
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int lo = kInterleaved ? 2 * j : j, hi = kInterleaved ? 2 * j + 1 : j + 4;
        const float2 t = cs[4 * i + j];
        const float a = x[lo], b = x[hi];
        x[lo] = a * t.x - b * t.y;
        x[hi] = b * t.x + a * t.y;
    }
}

// Angle `pair` of row m.
__device__ __forceinline__ float2 angle_of(const NormRopeArgs &g, int m, int pair)
{
    int pos = g.positions[static_cast<int64_t>(g.axis_of_pair[pair]) * g.M + m];
    if (pos < 0 || pos >= g.n_positions) {
        atomicOr(&g_norm_rope_error, kErrIndex);
        pos = pos < 0 ? 0 : g.n_positions - 1;
    }
    return reinterpret_cast<const float2 *>(g.table)[static_cast<int64_t>(pos) * (g.rot / 2) + pair];
}

template <typename T>
__device__ __forceinline__ void store8(void *base, int64_t head, int D, const Unit &u, const float (&x)[8])
{
    T *out = static_cast<T *>(base) + head * D;
    *reinterpret_cast<uint2 *>(out + u.e0) = make_uint2(pack2<T>(x[0], x[1]), pack2<T>(x[2], x[3]));
    *reinterpret_cast<uint2 *>(out + u.e1) = make_uint2(pack2<T>(x[4], x[5]), pack2<T>(x[6], x[7]));
}

// kThreads / L heads of row m, from head `first` on, of `heads` (q heads, then k, then v): q to
// g.q and, in a cache of 16 bits, k and v to their slot.
template <typename T, bool kInterleaved, int L>
__device__ __forceinline__ void row_heads(const NormRopeArgs &g, int m, int first, int heads, int64_t slot, float2 *cs)
{
    const int tid = threadIdx.x, pairs = g.rot / 2, i = tid % L, head = first + tid / L;
    const bool is_v = head >= g.Hq + g.Hkv;
    const Unit u = unit_of<kInterleaved>(i, g.D, pairs, is_v);
    const bool live = u.live && head < heads;
    float x[8] = {}, w[8] = {};
    if (live) load8(x, g.qkv + (static_cast<int64_t>(m) * (g.Hq + 2 * g.Hkv) + head) * g.D, u);
    const float *weight = is_v ? nullptr : head < g.Hq ? g.q_norm : g.k_norm;
    if (live && weight) {
#pragma unroll
        for (int j = 0; j < 8; ++j) w[j] = __ldg(weight + (j < 4 ? u.e0 + j : u.e1 + j - 4));
    }
    if (tid < pairs) cs[tid] = angle_of(g, m, tid);
    __syncthreads();
    if (g.q_norm || g.k_norm) {   // (all lanes take part)
        float y[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) y[j] = x[j];
        norm8<L>(y, w, g.D, g.eps);
        if (weight) {
#pragma unroll
            for (int j = 0; j < 8; ++j) x[j] = y[j];
        }
    }
    if (!live) return;
    if (u.turn) turn8<kInterleaved>(x, cs, i);
    if (head < g.Hq) {
        store8<T>(g.q, static_cast<int64_t>(m) * g.Hq + head, g.D, u, x);
    } else if (slot >= 0) {
        const int h = head - g.Hq - (is_v ? g.Hkv : 0);
        store8<T>(is_v ? g.v_cache : g.k_cache, slot * g.Hkv + h, g.D, u, x);
    }
}

__device__ __forceinline__ int64_t slot_of(const NormRopeArgs &g, int m)
{
    const int64_t slot = g.slots[m];
    if (slot < g.n_slots) return slot;
    if (threadIdx.x == 0) atomicOr(&g_norm_rope_error, kErrIndex);
    return -1;
}

// Grid (M, CTAs of kThreads / L heads).
template <typename T, bool kInterleaved, int L>
__global__ void __launch_bounds__(kThreads) norm_rope_kernel(const __grid_constant__ NormRopeArgs g)
{
    __shared__ float2 cs[kMaxRopePairs];
    grid_launch_dependents();
    grid_dependency_wait();
    const int m = blockIdx.x;
    row_heads<T, kInterleaved, L>(g, m, static_cast<int>(blockIdx.y) * (kThreads / L), g.Hq + 2 * g.Hkv, slot_of(g, m), cs);
}

// The least e >= -64 with largest <= 448 * 2^e, as the scale 2^e; `largest` the bits of a
// value that is finite and not negative. (448 = 1.75 * 2^8.)
__device__ __forceinline__ float scale_for(uint32_t largest)
{
    const int e = static_cast<int>(largest >> 23) - 127 - 8 + ((largest & 0x7fffffu) > 0x600000u ? 1 : 0);
    return __uint_as_float(static_cast<uint32_t>(max(e, -64) + 127) << 23);
}

// The codes of one head of k or of v: a warp a head. Row m is the first of a run of rows whose
// slots follow one another in one block; the warp takes the run's rows (n of them, at places
// `offset` .. of the block), so that it alone reads and writes the head's part of the block.
template <bool kInterleaved, int L>
__device__ __forceinline__ void block_head(const NormRopeArgs &g, int m, int n, int64_t slot, int task,
                                           const float2 (*cs)[kMaxRopePairs / 2], bool live_task)
{
    constexpr int kGroups = 32 / L, kTokens = kScaleTokens / kGroups;   // of a lane
    const int lane = threadIdx.x & 31, i = lane % L, group = lane / L, pairs = g.rot / 2, D = g.D;
    const bool is_v = task >= g.Hkv;
    const int h = is_v ? task - g.Hkv : task;
    const Unit u = unit_of<kInterleaved>(i, D, pairs, is_v);
    const int64_t row = static_cast<int64_t>(g.Hq + 2 * g.Hkv) * D;
    const float *in = g.qkv + static_cast<int64_t>(m) * row + static_cast<int64_t>(g.Hq + task) * D;
    float x[kTokens][8] = {}, w[8];
#pragma unroll
    for (int j = 0; j < kTokens; ++j)
        if (live_task && u.live && group + j * kGroups < n) load8(x[j], in + (group + j * kGroups) * row, u);
    const int64_t block = slot / kScaleTokens;
    const int offset = static_cast<int>(slot % kScaleTokens);
    float *scale_at = (is_v ? g.v_scale : g.k_scale) + block * g.Hkv + h;
    uint8_t *codes = static_cast<uint8_t *>(is_v ? g.v_cache : g.k_cache) + ((block * kScaleTokens) * g.Hkv + h) * D;
    const int64_t token = static_cast<int64_t>(g.Hkv) * D;   // bytes from a token to the next
    const float had = live_task && offset > 0 ? *scale_at : 0.0f;
    const bool norm = !is_v && g.k_norm;
    if (norm) {
#pragma unroll
        for (int j = 0; j < 8; ++j) w[j] = u.live ? __ldg(g.k_norm + (j < 4 ? u.e0 + j : u.e1 + j - 4)) : 0.0f;
    }
    __syncthreads();   // the angles
    if (!live_task) return;
    uint32_t largest = 0;
#pragma unroll
    for (int j = 0; j < kTokens; ++j) {
        if (j * kGroups >= n) break;
        if (norm) norm8<L>(x[j], w, D, g.eps);
        if (u.turn && group + j * kGroups < n) turn8<kInterleaved>(x[j], cs[group + j * kGroups], i);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const uint32_t bits = __float_as_uint(x[j][e]) & 0x7fffffffu;
            if (bits < 0x7f800000u) {
                largest = max(largest, bits);
            } else {
                x[j][e] = __uint_as_float(0x7fc00000u);   // there is no infinity among the codes
            }
        }
    }
    largest = __reduce_max_sync(0xffffffffu, largest);
    const float scale = fmaxf(scale_for(largest), had), inv = 1.0f / scale;
    if (had > 0.0f && scale > had) {   // earlier tokens follow: 16 codes a lane
        const float by = had * inv;
        for (int c = lane; c < offset * (D / 16); c += 32) {
            uint4 *at = reinterpret_cast<uint4 *>(codes + (c / (D / 16)) * token + (c % (D / 16)) * 16);
            uint4 v = *at;
            uint32_t words[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const uint32_t lo = e4m3x2_to_f16x2(words[k] & 0xffffu), hi = e4m3x2_to_f16x2(words[k] >> 16);
                const float2 a = __half22float2(*reinterpret_cast<const __half2 *>(&lo)), b = __half22float2(*reinterpret_cast<const __half2 *>(&hi));
                words[k] = e4m3x4(a.x * by, a.y * by, b.x * by, b.y * by);
            }
            *at = make_uint4(words[0], words[1], words[2], words[3]);
        }
    }
    if (lane == 0) *scale_at = scale;
    if (!u.live) return;
#pragma unroll
    for (int j = 0; j < kTokens; ++j) {
        const int t = group + j * kGroups;
        if (t >= n) break;
        uint8_t *out = codes + (offset + t) * token;
        *reinterpret_cast<uint32_t *>(out + u.e0) = e4m3x4(x[j][0] * inv, x[j][1] * inv, x[j][2] * inv, x[j][3] * inv);
        *reinterpret_cast<uint32_t *>(out + u.e1) = e4m3x4(x[j][4] * inv, x[j][5] * inv, x[j][6] * inv, x[j][7] * inv);
    }
}

// Grid (M, kv_ctas + CTAs of kThreads / L query heads). The first kv_ctas of a row have a warp
// for each k and v head; they go on only where the row starts a run.
template <typename T, bool kInterleaved, int L>
__global__ void __launch_bounds__(kThreads) rope_e4m3_kernel(const __grid_constant__ NormRopeArgs g, int kv_ctas)
{
    __shared__ float2 cs[kScaleTokens][kMaxRopePairs / 2];
    grid_launch_dependents();
    grid_dependency_wait();
    const int m = blockIdx.x, tid = threadIdx.x, pairs = g.rot / 2;
    if (static_cast<int>(blockIdx.y) >= kv_ctas) {
        row_heads<T, kInterleaved, L>(g, m, (static_cast<int>(blockIdx.y) - kv_ctas) * (kThreads / L), g.Hq, -1, &cs[0][0]);
        return;
    }
    const int64_t slot = blockIdx.y == 0 ? slot_of(g, m) : g.slots[m];
    if (slot < 0 || slot >= g.n_slots) return;
    if (slot % kScaleTokens != 0 && m > 0 && g.slots[m - 1] == slot - 1) return;   // an earlier row's run
    const int lane = tid & 31, most = kScaleTokens - static_cast<int>(slot % kScaleTokens);
    const bool goes_on = lane < most && lane < g.M - m && g.slots[m + lane] == slot + lane;
    const int n = __ffs(~__ballot_sync(0xffffffffu, goes_on)) - 1;   // at least 1, at most 16
    for (int a = tid; a < n * pairs; a += kThreads) cs[a / pairs][a % pairs] = angle_of(g, m + a / pairs, a % pairs);
    const int task = static_cast<int>(blockIdx.y) * kWarps + tid / 32;
    block_head<kInterleaved, L>(g, m, n, slot, task, cs, task < 2 * g.Hkv);
}

template <typename T, bool kInterleaved, int L>
cudaError_t launch_typed(const NormRopeArgs &g, cudaStream_t s)
{
    constexpr int kHeads = kThreads / L;
    const bool codes = g.k_scale != nullptr;
    const int kv_ctas = codes ? (2 * g.Hkv + kWarps - 1) / kWarps : 0, heads = codes ? g.Hq : g.Hq + 2 * g.Hkv;
    cudaLaunchAttribute attr[1];
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3(kThreads);
    cfg.gridDim = dim3(static_cast<unsigned>(g.M), static_cast<unsigned>(kv_ctas + (heads + kHeads - 1) / kHeads));
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = set_launch_overlap_attr(attr);
    if constexpr (L <= 16) {   // codes: heads of 128 at most
        if (codes) return cudaLaunchKernelEx(&cfg, rope_e4m3_kernel<T, kInterleaved, L>, g, kv_ctas);
    }
    return cudaLaunchKernelEx(&cfg, norm_rope_kernel<T, kInterleaved, L>, g);
}

template <typename T, bool kInterleaved>
cudaError_t launch_lanes(const NormRopeArgs &g, cudaStream_t s)
{
    if (g.D <= 64) return launch_typed<T, kInterleaved, 8>(g, s);
    if (g.D <= 128) return launch_typed<T, kInterleaved, 16>(g, s);
    return launch_typed<T, kInterleaved, 32>(g, s);
}

}  // namespace

cudaError_t launch_norm_rope(const NormRopeArgs &g, cudaStream_t s)
{
    route_hit(g.k_scale ? kRouteRopeE4m3 : kRouteNormRope);
    if (g.interleaved) return g.type == QMV_F16 ? launch_lanes<__half, true>(g, s) : launch_lanes<__nv_bfloat16, true>(g, s);
    return g.type == QMV_F16 ? launch_lanes<__half, false>(g, s) : launch_lanes<__nv_bfloat16, false>(g, s);
}

cudaError_t read_error_word_norm_rope(uint32_t *out, bool clear)
{
    cudaError_t e = cudaMemcpyFromSymbol(out, g_norm_rope_error, sizeof(uint32_t));
    if (e != cudaSuccess || !clear) return e;
    const uint32_t zero = 0;
    return cudaMemcpyToSymbol(g_norm_rope_error, &zero, sizeof(uint32_t));
}

}  // namespace qmv
