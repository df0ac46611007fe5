// rope_append.cu -- rotary positions on a projection's q and k, and the append of k and
// v to a paged cache. A pair (a, b) of a head turns by its position's angle:
//   (a, b) -> (a c - b s, b c + a s),  (c, s) = table[position on the pair's axis][pair]
// computed in fp32 from the projection's fp32 output and rounded once, to the 16-bit type
// of q and the cache.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "decode_device.cuh"
#include "decode_ops.h"
#include "qmv.h"
#include "qmv_device.cuh"

namespace qmv {
namespace {

__device__ uint32_t g_rope_error;

constexpr int kThreads = 256;

// A CTA takes 256 units of 8 elements of one token's heads, a thread a unit: 4 pairs of the
// rotated part, or 8 elements that are copied. The token's angles go to shared memory once
// for the CTA, while the units' elements are on their way. Bound by the bytes: 4001 tokens of
// 40 + 8 + 8 heads of 128 take 33 us, 5.3 TB/s (each thread loading its angles from the
// table: 53 us; four units a thread: 40).
template <typename T, bool kInterleaved>
__global__ void __launch_bounds__(kThreads) rope_append_kernel(const __grid_constant__ RopeArgs g)
{
    __shared__ float2 cs[kMaxRopePairs];
    const int m = blockIdx.x, pairs = g.rot / 2, tid = threadIdx.x;
    const int heads = g.Hq + 2 * g.Hkv, per_head = g.D / 8, u = blockIdx.y * kThreads + tid;
    grid_launch_dependents();
    grid_dependency_wait();
    const int head = u / per_head, i = u - head * per_head;
    const bool live = head < heads, turn = head < g.Hq + g.Hkv && i < pairs / 4;
    // this unit's elements e0 .. e0 + 3 and e1 .. e1 + 3 of its head
    const int e0 = turn && !kInterleaved ? 4 * i : 8 * i, e1 = turn && !kInterleaved ? pairs + 4 * i : 8 * i + 4;
    const float *in = g.qkv + (static_cast<int64_t>(m) * heads + head) * g.D;
    float4 p{}, q{};
    if (live) {
        p = __ldcs(reinterpret_cast<const float4 *>(in + e0));
        q = __ldcs(reinterpret_cast<const float4 *>(in + e1));
    }
    int64_t slot = g.slots[m];
    if (tid < pairs) {
        int pos = g.positions[static_cast<int64_t>(g.axis_of_pair[tid]) * g.M + m];
        if (pos < 0 || pos >= g.n_positions) {
            atomicOr(&g_rope_error, kErrIndex);
            pos = pos < 0 ? 0 : g.n_positions - 1;
        }
        cs[tid] = reinterpret_cast<const float2 *>(g.table)[static_cast<int64_t>(pos) * pairs + tid];
    }
    if (slot >= g.n_slots) {
        if (tid == 0) atomicOr(&g_rope_error, kErrIndex);
        slot = -1;
    }
    __syncthreads();
    if (!live) return;
    float a[4] = {p.x, p.y, p.z, p.w}, b[4] = {q.x, q.y, q.z, q.w};
    if (turn) {
        if (kInterleaved) {   // pair j = (elements 2 j, 2 j + 1): a holds pairs 4 i, 4 i + 1
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const float2 t = cs[4 * i + j], v = cs[4 * i + 2 + j];
                const float x = a[2 * j], y = a[2 * j + 1], z = b[2 * j], w = b[2 * j + 1];
                a[2 * j] = x * t.x - y * t.y;
                a[2 * j + 1] = y * t.x + x * t.y;
                b[2 * j] = z * v.x - w * v.y;
                b[2 * j + 1] = w * v.x + z * v.y;
            }
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float2 t = cs[4 * i + j];
                const float x = a[j], y = b[j];
                a[j] = x * t.x - y * t.y;
                b[j] = y * t.x + x * t.y;
            }
        }
    }
    T *out;
    if (head < g.Hq) {
        out = static_cast<T *>(g.q) + (static_cast<int64_t>(m) * g.Hq + head) * g.D;
    } else {
        if (slot < 0) return;
        const bool is_k = head < g.Hq + g.Hkv;
        out = static_cast<T *>(is_k ? g.k_cache : g.v_cache) + (slot * g.Hkv + head - g.Hq - (is_k ? 0 : g.Hkv)) * g.D;
    }
    *reinterpret_cast<uint2 *>(out + e0) = make_uint2(pack2<T>(a[0], a[1]), pack2<T>(a[2], a[3]));
    *reinterpret_cast<uint2 *>(out + e1) = make_uint2(pack2<T>(b[0], b[1]), pack2<T>(b[2], b[3]));
}

template <typename T, bool kInterleaved>
cudaError_t launch_typed(const RopeArgs &g, cudaStream_t s)
{
    const int total = (g.Hq + 2 * g.Hkv) * (g.D / 8);
    cudaLaunchAttribute attr[1];
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3(kThreads);
    cfg.gridDim = dim3(static_cast<unsigned>(g.M), static_cast<unsigned>((total + kThreads - 1) / kThreads));
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = set_launch_overlap_attr(attr);
    return cudaLaunchKernelEx(&cfg, rope_append_kernel<T, kInterleaved>, g);
}

}  // namespace

cudaError_t launch_rope(const RopeArgs &g, cudaStream_t s)
{
    route_hit(kRouteRopeAppend);
    if (g.interleaved) return g.type == QMV_F16 ? launch_typed<__half, true>(g, s) : launch_typed<__nv_bfloat16, true>(g, s);
    return g.type == QMV_F16 ? launch_typed<__half, false>(g, s) : launch_typed<__nv_bfloat16, false>(g, s);
}

cudaError_t read_error_word_rope(uint32_t *out, bool clear)
{
    cudaError_t e = cudaMemcpyFromSymbol(out, g_rope_error, sizeof(uint32_t));
    if (e != cudaSuccess || !clear) return e;
    const uint32_t zero = 0;
    return cudaMemcpyToSymbol(g_rope_error, &zero, sizeof(uint32_t));
}

}  // namespace qmv
