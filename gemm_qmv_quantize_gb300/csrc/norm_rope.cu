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
// the bytes and by what a lane executes for them: 4001 tokens of 40 + 8 + 8 heads of 128 take 30 us in 16
// bits (5.8 TB/s) and 40 us as codes (4.1).
#include <algorithm>

#include "decode_device.cuh"
#include "decode_ops.h"
#include "qmv.h"
#include "qmv_device.cuh"
#include "rows.h"

namespace qmv {
namespace {

__device__ uint32_t g_norm_rope_error;

constexpr int kThreads = 256;
constexpr int kTwoRows = 256;   // rows from which a CTA takes two: 512 of 56 heads 5.7 us for 6.1
// Rows a CTA, rounded down, from which CTAs that fill the SMs go through them, in 16 bits: with 56 heads from 1038 rows on, with
// 10 from 3648. 4001 rows of 56 heads (23 each) 29.8 us for 35.6 by CTAs of two rows, 1000 (5, or 6 for most) 10.3 for
// 10.4; at the border 1037 rows by CTAs of two 10.2 us, 1038 streamed 10.6, 1200 11.6. 1000 of 10 heads (1) 4.7 for 3.5, 8000 (13) 17.9
// for 17.6; at the border 8.4 and 9.1. (With codes, q in such a launch of its own 41 us for 40 with 4005 rows.)
constexpr int kStreamRows = 6;
// CTAs of so many threads, all on the SMs at once; a CTA's rows that are on their way and the one it works on. (4 or 3 for 2
// stages 31.6 and 29.9 us for 29.7; 256 threads 32.7, 64 30.1.)
constexpr int kStreamThreads = 128, kStreamCtas = kSms * 8, kStages = 2;
using Ring = float4[kStages][2][kStreamThreads];

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

// The norm, over the group of L lanes that has the head, where `norm`; w is 1 where not. (All lanes
// take part: the groups of a warp may have heads of both kinds.)
template <int L>
__device__ __forceinline__ void norm8(float (&x)[8], const float (&w)[8], bool norm, const NormRopeArgs &g)
{
    float sum = 0.0f;
#pragma unroll
    for (int j = 0; j < 8; ++j) sum = fmaf(x[j], x[j], sum);
#pragma unroll
    for (int o = L / 2; o > 0; o /= 2) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    const float r = norm ? rsqrtf(fmaf(sum, g.one_over_d, g.eps)) : 1.0f;
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] = x[j] * r * w[j];
}

// A unit's four angles, (cos, sin) each.
struct Angles {
    float4 a, b;
};

__device__ __forceinline__ int position_inside(const NormRopeArgs &g, int pos)
{
    if (pos < 0 || pos >= g.n_positions) {
        atomicOr(&g_norm_rope_error, kErrIndex);
        pos = pos < 0 ? 0 : g.n_positions - 1;
    }
    return pos;
}

__device__ __forceinline__ int position_of(const NormRopeArgs &g, int m, int axis) { return position_inside(g, g.positions[static_cast<int64_t>(axis) * g.M + m]); }

// Of a position and pairs 4 i .. 4 i + 3.
__device__ __forceinline__ Angles angles_at(const NormRopeArgs &g, int pos, int i)
{
    const float4 *at = reinterpret_cast<const float4 *>(g.table) + (static_cast<int64_t>(pos) * (g.rot / 2) + 4 * i) / 2;
    return Angles{__ldg(at), __ldg(at + 1)};
}

// Of row m and pairs 4 i .. 4 i + 3. Lanes with the same i of all of a CTA's heads read the same ones: L1
// serves all but the first. (Through shared memory, with a barrier, 4001 rows took 39 us for 35, and with codes
// 53 for 40.)
__device__ __forceinline__ Angles angles_of(const NormRopeArgs &g, int m, int i)
{
    const int pairs = g.rot / 2;
    Angles t;
    const uint32_t axes = reinterpret_cast<const uint32_t *>(g.axis_of_pair)[i], axis = axes & 0xffu;   // of the four pairs
    if (axes == axis * 0x01010101u) {
        t = angles_at(g, position_of(g, m, static_cast<int>(axis)), i);
    } else {
        float2 c[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
            c[j] = __ldg(reinterpret_cast<const float2 *>(g.table) + static_cast<int64_t>(position_of(g, m, static_cast<int>(axes >> (8 * j) & 0xffu))) * pairs + 4 * i + j);
        t.a = make_float4(c[0].x, c[0].y, c[1].x, c[1].y), t.b = make_float4(c[2].x, c[2].y, c[3].x, c[3].y);
    }
    return t;
}

template <bool kInterleaved>
__device__ __forceinline__ void turn8(float (&x)[8], const Angles &t)
{
    const float2 angles[4] = {make_float2(t.a.x, t.a.y), make_float2(t.a.z, t.a.w), make_float2(t.b.x, t.b.y), make_float2(t.b.z, t.b.w)};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int lo = kInterleaved ? 2 * j : j, hi = kInterleaved ? 2 * j + 1 : j + 4;
        const float a = x[lo], b = x[hi];
        x[lo] = a * angles[j].x - b * angles[j].y;
        x[hi] = b * angles[j].x + a * angles[j].y;
    }
}

template <typename T>
__device__ __forceinline__ void store8(void *base, int64_t head, int D, const Unit &u, const float (&x)[8])
{
    T *out = static_cast<T *>(base) + head * D;
    *reinterpret_cast<uint2 *>(out + u.e0) = make_uint2(pack2<T>(x[0], x[1]), pack2<T>(x[2], x[3]));
    *reinterpret_cast<uint2 *>(out + u.e1) = make_uint2(pack2<T>(x[4], x[5]), pack2<T>(x[6], x[7]));
}

__device__ __forceinline__ void load_weight(float (&w)[8], const float *weight, const Unit &u)
{
    const float4 p = __ldg(reinterpret_cast<const float4 *>(weight + u.e0)), q = __ldg(reinterpret_cast<const float4 *>(weight + u.e1));
    w[0] = p.x, w[1] = p.y, w[2] = p.z, w[3] = p.w, w[4] = q.x, w[5] = q.y, w[6] = q.z, w[7] = q.w;
}

// A slot, or -1 for one that lies outside.
__device__ __forceinline__ int64_t slot_inside(const NormRopeArgs &g, int64_t slot)
{
    if (slot < g.n_slots) return slot;
    atomicOr(&g_norm_rope_error, kErrIndex);
    return -1;
}

template <typename T>
__device__ __forceinline__ void put_head(const NormRopeArgs &g, int m, int head, bool is_v, int64_t slot, const Unit &u, const float (&x)[8])
{
    if (head < g.Hq) {
        store8<T>(g.q, static_cast<int64_t>(m) * g.Hq + head, g.D, u, x);
    } else if (slot >= 0) {
        store8<T>(is_v ? g.v_cache : g.k_cache, slot * g.Hkv + head - g.Hq - (is_v ? g.Hkv : 0), g.D, u, x);
    }
}

// kThreads / L heads of rows m .. m + R - 1, from head `first` on, of `heads` (q heads, then k,
// then v): q to g.q and, in a cache of 16 bits, k and v to their slots.
template <typename T, bool kInterleaved, int L, int R>
__device__ __forceinline__ void row_heads(const NormRopeArgs &g, int m, int first, int heads)
{
    const int tid = threadIdx.x, pairs = g.rot / 2, i = tid % L, head = first + tid / L, rows = min(R, g.M - m);
    const bool is_v = head >= g.Hq + g.Hkv;
    const Unit u = unit_of<kInterleaved>(i, g.D, pairs, is_v);
    const bool live = u.live && head < heads;
    const float *in = g.qkv + (static_cast<int64_t>(m) * (g.Hq + 2 * g.Hkv) + head) * g.D;
    float x[R][8] = {}, w[8] = {1.0f, 1.0f, 1.0f, 1.0f, 1.0f, 1.0f, 1.0f, 1.0f};
#pragma unroll
    for (int r = 0; r < R; ++r)
        if (live && r < rows) load8(x[r], in + static_cast<int64_t>(r) * (g.Hq + 2 * g.Hkv) * g.D, u);
    const float *weight = is_v ? nullptr : head < g.Hq ? g.q_norm : g.k_norm;
    if (live && weight) load_weight(w, weight, u);
    Angles t[R];
#pragma unroll
    for (int r = 0; r < R; ++r)
        if (live && u.turn && r < rows) t[r] = angles_of(g, m + r, i);
#pragma unroll
    for (int r = 0; r < R; ++r) {
        if (g.q_norm || g.k_norm) norm8<L>(x[r], w, weight != nullptr, g);
        if (!live || r >= rows) continue;
        if (u.turn) turn8<kInterleaved>(x[r], t[r]);
        put_head<T>(g, m + r, head, is_v, head < g.Hq ? 0 : slot_inside(g, g.slots[m + r]), u, x[r]);
    }
}

// The same of a CTA's rows in turn, kStreamThreads / L heads: each lane copies its own pieces of the next rows to shared memory, and
// has the row's angles on their way, while it works on a row.
template <typename T, bool kInterleaved, int L>
__device__ __forceinline__ void stream_heads(const NormRopeArgs &g, RowsInTurn at, int first, Ring &ring)
{
    const int tid = threadIdx.x, pairs = g.rot / 2, i = tid % L, head = first + tid / L;
    const bool is_v = head >= g.Hq + g.Hkv;
    const Unit u = unit_of<kInterleaved>(i, g.D, pairs, is_v);
    const bool live = u.live && head < g.Hq + 2 * g.Hkv, turn = live && u.turn, normed = g.q_norm || g.k_norm;
    const float *weight = is_v ? nullptr : head < g.Hq ? g.q_norm : g.k_norm;
    float w[8] = {1.0f, 1.0f, 1.0f, 1.0f, 1.0f, 1.0f, 1.0f, 1.0f};
    if (live && weight) load_weight(w, weight, u);
    const int64_t row = static_cast<int64_t>(g.Hq + 2 * g.Hkv) * g.D;
    const float *in = g.qkv + static_cast<int64_t>(head) * g.D;
    auto copy = [&](int n, int stage) {
        if (live && at.ahead(n)) {
            cp_async_16(&ring[stage][0][tid], in + at.row(n) * row + u.e0);
            cp_async_16(&ring[stage][1][tid], in + at.row(n) * row + u.e1);
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
#pragma unroll
    for (int j = 0; j < kStages - 1; ++j) copy(j, j);
    // of the four pairs; where they are of one axis, the position is there a row before the angles are asked for
    const uint32_t axes = turn ? reinterpret_cast<const uint32_t *>(g.axis_of_pair)[i] : 0, axis = axes & 0xffu;
    const bool one_axis = axes == axis * 0x01010101u, cached = live && head >= g.Hq;
    const int *positions = g.positions + static_cast<int64_t>(axis) * g.M;
    Angles next;
    if (turn) next = angles_of(g, at.row(0), i);
    int next_position = turn && at.ahead(1) ? positions[at.row(1)] : 0;
    int64_t next_slot = cached ? g.slots[at.row(0)] : 0;
    int stage = 0;
#pragma unroll 1
    for (; at.ahead(0); at.next()) {
        copy(kStages - 1, (stage + kStages - 1) % kStages);
        const Angles t = next;
        const int64_t slot = next_slot;
        const int position = next_position;
        if (at.ahead(1)) {
            if (turn) next = one_axis ? angles_at(g, position_inside(g, position), i) : angles_of(g, at.row(1), i);
            if (cached) next_slot = g.slots[at.row(1)];
            if (turn && at.ahead(2)) next_position = positions[at.row(2)];
        }
        asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 1) : "memory");
        float x[8] = {};
        if (live) {
            const float4 p = ring[stage][0][tid], q = ring[stage][1][tid];
            x[0] = p.x, x[1] = p.y, x[2] = p.z, x[3] = p.w, x[4] = q.x, x[5] = q.y, x[6] = q.z, x[7] = q.w;
        }
        stage = (stage + 1) % kStages;
        if (normed) norm8<L>(x, w, weight != nullptr, g);
        if (turn) turn8<kInterleaved>(x, t);
        if (live) put_head<T>(g, at.row(0), head, is_v, cached ? slot_inside(g, slot) : 0, u, x);
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
}

// Grid (rows / R, CTAs of kThreads / L heads).
template <typename T, bool kInterleaved, int L, int R>
__global__ void __launch_bounds__(kThreads) norm_rope_kernel(const __grid_constant__ NormRopeArgs g)
{
    grid_launch_dependents();
    grid_dependency_wait();
    row_heads<T, kInterleaved, L, R>(g, static_cast<int>(blockIdx.x) * R, static_cast<int>(blockIdx.y) * (kThreads / L), g.Hq + 2 * g.Hkv);
}

// Grid (CTAs that the rows go to in turn, CTAs of kStreamThreads / L heads).
template <typename T, bool kInterleaved, int L>
__global__ void __launch_bounds__(kStreamThreads, kStreamCtas / kSms) norm_rope_stream_kernel(const __grid_constant__ NormRopeArgs g)
{
    __shared__ Ring ring;
    grid_launch_dependents();
    grid_dependency_wait();
    stream_heads<T, kInterleaved, L>(g, RowsInTurn{blockIdx.x, static_cast<int>(gridDim.x), g.M - static_cast<int>(blockIdx.x)}, static_cast<int>(blockIdx.y) * (kStreamThreads / L), ring);
}

// The least e >= -64 with largest <= 448 * 2^e, as the scale 2^e; `largest` the bits of a
// value that is finite and not negative. (448 = 1.75 * 2^8.)
__device__ __forceinline__ float scale_for(uint32_t largest)
{
    const int e = static_cast<int>(largest >> 23) - 127 - 8 + ((largest & 0x7fffffu) > 0x600000u ? 1 : 0);
    return __uint_as_float(static_cast<uint32_t>(max(e, -64) + 127) << 23);
}

// The codes of one head of k (task < Hkv) or of v, of the runs that start in rows 16 `window`
// .. + 15: a run is rows whose slots follow one another in one block, so this CTA alone reads and
// writes the head's part of the block. A run that starts at the window's last row ends 15 rows
// later: the CTA looks at 31 rows, a group of L lanes a row or two.
template <bool kInterleaved, int L>
__device__ __forceinline__ void window_head(const NormRopeArgs &g, int window, int task, uint32_t *run_largest)
{
    constexpr int kGroups = kThreads / L, kEach = 2 * kScaleTokens / kGroups;   // groups of lanes, rows of a group: 2 or 1
    const int tid = threadIdx.x, lane = tid & 31, i = tid % L, group = tid / L, pairs = g.rot / 2, D = g.D;
    const int m0 = window * kScaleTokens;
    const bool is_v = task >= g.Hkv;
    const Unit u = unit_of<kInterleaved>(i, D, pairs, is_v);
    const int64_t row = static_cast<int64_t>(g.Hq + 2 * g.Hkv) * D;
    const float *in = g.qkv + static_cast<int64_t>(m0) * row + static_cast<int64_t>(g.Hq + task) * D;
    // which rows, in every warp: lane j looks at row m0 + j
    const bool there = row_ahead(m0, lane, g.M);
    const int64_t slot = there && lane < 2 * kScaleTokens - 1 ? g.slots[m0 + lane] : -1;
    const int64_t before = there && m0 + lane > 0 ? g.slots[m0 + lane - 1] : -1;
    const bool valid = slot >= 0 && slot < g.n_slots;
    if (slot >= g.n_slots && lane < kScaleTokens && tid < 32 && task == 0) atomicOr(&g_norm_rope_error, kErrIndex);
    const uint32_t starts = __ballot_sync(0xffffffffu, valid && (before != slot - 1 || slot % kScaleTokens == 0));
    const uint32_t up_to = starts & (0xffffffffu >> (31 - lane));
    const int start = up_to && valid ? 31 - __clz(up_to) : -1;   // the row (of 32) that this row's run starts at
    const int run = start < kScaleTokens ? start : -1;            // a later window's run is not this CTA's
    const uint32_t mine = __ballot_sync(0xffffffffu, run >= 0);
    float x[kEach][8] = {}, w[8], had[kEach];
    int my_run[kEach];
    int64_t my_slot[kEach];
#pragma unroll
    for (int k = 0; k < kEach; ++k) {
        const int j = group + k * kGroups;
        my_run[k] = __shfl_sync(0xffffffffu, run, j);
        my_slot[k] = __shfl_sync(0xffffffffu, slot, j);
        if (my_run[k] >= 0 && u.live) load8(x[k], in + j * row, u);
    }
    float *scales = is_v ? g.v_scale : g.k_scale;
    const int h = is_v ? task - g.Hkv : task;
    const bool norm = !is_v && g.k_norm;
#pragma unroll
    for (int j = 0; j < 8; ++j) w[j] = 1.0f;
    if (norm && u.live) load_weight(w, g.k_norm, u);
#pragma unroll
    for (int k = 0; k < kEach; ++k) {   // the scale of tokens that are there before the run
        const int j = group + k * kGroups;
        const int64_t first = my_slot[k] - (j - my_run[k]);
        had[k] = my_run[k] >= 0 && first % kScaleTokens > 0 ? scales[first / kScaleTokens * g.Hkv + h] : 0.0f;
    }
    Angles t[kEach];
#pragma unroll
    for (int k = 0; k < kEach; ++k)
        if (u.turn && my_run[k] >= 0) t[k] = angles_of(g, m0 + group + k * kGroups, i);
    if (tid < kScaleTokens) run_largest[tid] = 0;
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kEach; ++k) {
        if (!(mine >> (tid / 32 * (32 / L) + k * kGroups) & ((1u << (32 / L)) - 1))) continue;   // no rows for this warp's groups
        if (norm) norm8<L>(x[k], w, true, g);
        if (u.turn && my_run[k] >= 0) turn8<kInterleaved>(x[k], t[k]);
        uint32_t largest = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const uint32_t bits = __float_as_uint(x[k][e]) & 0x7fffffffu;
            if (bits < 0x7f800000u) {
                largest = max(largest, bits);
            } else {
                x[k][e] = __uint_as_float(0x7fc00000u);   // there is no infinity among the codes
            }
        }
#pragma unroll
        for (int o = L / 2; o > 0; o /= 2) largest = max(largest, __shfl_xor_sync(0xffffffffu, largest, o));
        if (i == 0 && my_run[k] >= 0) atomicMax(run_largest + my_run[k], largest);
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kEach; ++k) {
        const int j = group + k * kGroups;
        if (my_run[k] < 0) continue;
        if (!(had[k] >= 0.0f && had[k] < INFINITY)) had[k] = NAN;   // no scale: what it is of becomes NaN
        const float scale = fmaxf(scale_for(run_largest[my_run[k]]), had[k]), inv = 1.0f / scale;
        uint8_t *codes = static_cast<uint8_t *>(is_v ? g.v_cache : g.k_cache);
        const int64_t token = static_cast<int64_t>(g.Hkv) * D;   // bytes from a token to the next
        if (j == my_run[k]) {   // the run's first row: its group sees to the scale and the earlier tokens
            const int64_t block = my_slot[k] / kScaleTokens;
            const int offset = static_cast<int>(my_slot[k] % kScaleTokens), pieces = D / 16;
            if (offset > 0 && scale != had[k]) {   // 16 codes a lane
                const float by = had[k] * inv;
                for (int c = i; c < offset * pieces; c += L) {
                    uint4 *at = reinterpret_cast<uint4 *>(codes + (block * kScaleTokens + c / pieces) * token + h * D + c % pieces * 16);
                    const uint4 v = *at;
                    uint32_t words[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                    for (int n = 0; n < 4; ++n) {
                        const uint32_t lo = e4m3x2_to_f16x2(words[n] & 0xffffu), hi = e4m3x2_to_f16x2(words[n] >> 16);
                        const float2 a = __half22float2(*reinterpret_cast<const __half2 *>(&lo)), b = __half22float2(*reinterpret_cast<const __half2 *>(&hi));
                        words[n] = e4m3x4(a.x * by, a.y * by, b.x * by, b.y * by);
                    }
                    *at = make_uint4(words[0], words[1], words[2], words[3]);
                }
            }
            if (i == 0) scales[block * g.Hkv + h] = scale;
        }
        if (!u.live) continue;
        uint8_t *out = codes + my_slot[k] * token + h * D;
        *reinterpret_cast<uint32_t *>(out + u.e0) = e4m3x4(x[k][0] * inv, x[k][1] * inv, x[k][2] * inv, x[k][3] * inv);
        *reinterpret_cast<uint32_t *>(out + u.e1) = e4m3x4(x[k][4] * inv, x[k][5] * inv, x[k][6] * inv, x[k][7] * inv);
    }
}

// Grid: windows * 2 Hkv CTAs of a window's head, then rows / R * q_ctas of kThreads / L query heads.
template <typename T, bool kInterleaved, int L, int R>
__global__ void __launch_bounds__(kThreads) rope_e4m3_kernel(const __grid_constant__ NormRopeArgs g, int windows, int q_ctas)
{
    __shared__ uint32_t run_largest[kScaleTokens];
    grid_launch_dependents();
    grid_dependency_wait();
    const int kv = windows * 2 * g.Hkv, c = static_cast<int>(blockIdx.x);
    if (c < kv) {
        window_head<kInterleaved, L>(g, c / (2 * g.Hkv), c % (2 * g.Hkv), run_largest);
    } else {
        row_heads<T, kInterleaved, L, R>(g, (c - kv) / q_ctas * R, (c - kv) % q_ctas * (kThreads / L), g.Hq);
    }
}

template <typename T, bool kInterleaved, int L>
cudaError_t launch_typed(const NormRopeArgs &g, cudaStream_t s)
{
    constexpr int kHeads = kThreads / L, kStreamHeads = kStreamThreads / L;
    const int rows = g.M >= kTwoRows ? 2 : 1, row_ctas = groups_of(g.M, rows);
    cudaLaunchAttribute attr[1];
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3(kThreads);
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = set_launch_overlap_attr(attr);
    if constexpr (L <= 16) {   // codes: heads of 128 at most
        if (g.k_scale) {
            const int windows = groups_of(g.M, kScaleTokens), q_ctas = (g.Hq + kHeads - 1) / kHeads;
            const int64_t grid = static_cast<int64_t>(windows) * 2 * g.Hkv + static_cast<int64_t>(row_ctas) * q_ctas;
            if (grid > 0x7fffffff) return cudaErrorInvalidValue;
            cfg.gridDim = dim3(static_cast<unsigned>(grid));
            return rows == 2 ? cudaLaunchKernelEx(&cfg, rope_e4m3_kernel<T, kInterleaved, L, 2>, g, windows, q_ctas)
                             : cudaLaunchKernelEx(&cfg, rope_e4m3_kernel<T, kInterleaved, L, 1>, g, windows, q_ctas);
        }
    }
    const int heads = g.Hq + 2 * g.Hkv, stream_head_ctas = (heads + kStreamHeads - 1) / kStreamHeads;
    const int at_once = std::max(1, kStreamCtas / stream_head_ctas);   // rows
    if (g.M / at_once >= kStreamRows) {
        cfg.blockDim = dim3(kStreamThreads);
        cfg.gridDim = dim3(static_cast<unsigned>(at_once), static_cast<unsigned>(stream_head_ctas));
        return cudaLaunchKernelEx(&cfg, norm_rope_stream_kernel<T, kInterleaved, L>, g);
    }
    cfg.gridDim = dim3(static_cast<unsigned>(row_ctas), static_cast<unsigned>((heads + kHeads - 1) / kHeads));
    return rows == 2 ? cudaLaunchKernelEx(&cfg, norm_rope_kernel<T, kInterleaved, L, 2>, g)
                     : cudaLaunchKernelEx(&cfg, norm_rope_kernel<T, kInterleaved, L, 1>, g);
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
