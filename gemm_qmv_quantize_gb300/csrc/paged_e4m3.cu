// paged_e4m3.cu -- attention of T tokens of each of B requests over a paged cache of E4M3
// codes with a scale for each block of 16 tokens and head:
//   o = sum_j p_j sv_j V_j,  p = softmax_j(scale sk_j q . K_j)
//
// A warp takes blocks of 16 keys of one key head against up to 8 NT query rows (the T tokens
// and G query heads that read the key head), on m16n8k16 products with the keys as the 16
// rows of A and the query rows as the 8 columns of B:
//   S^T = K Q^T (16 keys x 8 rows a product),   O^T += V^T P^T (16 dimensions x 8 rows).
// So a product's rows are full however few query rows there are, and a block has one scale.
// Which key or dimension a row or column of a product stands for is free: it is chosen so
// that every lane's operands are whole 16-byte pieces of the cache's rows, which the lane
// copies to shared memory and reads back itself; nothing is shared between lanes, and codes
// become binary16, exactly, on their way into the product. P^T is S^T transposed in registers.
//
// Numerics: q is held in binary16 (bfloat16 rows are scaled by a power of two that brings
// their largest element to 2^14 or more: elements 2^-28 of it and less lose bits); S, the softmax's
// statistics, and O are fp32. A column's running maxima are two: m of z = c sk S for the
// denominator l = sum 2^(z - m), and m' of z + log2 sv for the numerator, whose terms
// 2^(z + log2 sv - m') are rounded to binary16, the product's operand: with a maximum of its
// own the largest term is near 1, whatever the scales of the blocks. Both follow the true
// maxima with a slack of 2^8, so that O is rescaled rarely.
#include <algorithm>
#include <cmath>

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "decode_device.cuh"
#include "decode_ops.h"
#include "qmv.h"
#include "qmv_device.cuh"

namespace qmv {
namespace {

__device__ uint32_t g_paged_error;

constexpr int kBlock = kScaleTokens;    // keys a step of a warp
constexpr int kWarps = 8, kThreads = 32 * kWarps;
constexpr int64_t kWorkspaceBytes = 2 * 152 * 4352 * 4;   // two parts for each of the most runs, whatever the sizes
constexpr int kBatch = 32;              // blocks whose page and scales a warp looks up at a time, a lane a block
constexpr float kSlack = 8.0f;
constexpr float kLowest = -3.402823466e38f;   // a maximum of no scores: the difference to it is never NaN
constexpr float kLog2e = 1.4426950408889634f;

template <int D>
struct Ring {   // a stage: 16-byte pieces, [piece][lane]
    static constexpr int kKPieces = 2 * D / 64;
    static constexpr int kBytes = 32 * kBlock * D / 16;   // keys and values of a block: 2 * 16 * D
};

// Stages of a warp's ring, and CTAs an SM, by the registers that NT row tiles of O take.
template <int D, int NT>
struct Shape {
    static constexpr int kCtas = NT * D <= 256 ? 2 : 1;
    static constexpr int kStages = (128 / D) * (kCtas == 2 ? 3 : 6);
};

__device__ __forceinline__ void cp_async_16_zfill(uint32_t dst, const void *src, bool there)
{
    asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(there ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_async_8_zfill(uint32_t dst, const void *src, bool there)
{
    asm volatile("cp.async.ca.shared.global.L2::128B [%0], [%1], 8, %2;" ::"r"(dst), "l"(src), "r"(there ? 8 : 0) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

__device__ __forceinline__ uint4 lds128(uint32_t at)
{
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at) : "memory");
    return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t at)
{
    uint2 v;
    asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(at) : "memory");
    return v;
}

// The 8 x 8 matrix of 16-bit elements that a warp holds (lane l: row l / 4, columns 2 (l % 4)
// and the next), transposed.
__device__ __forceinline__ uint32_t transpose8x8(uint32_t v)
{
    uint32_t r;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}

__device__ __forceinline__ float exp2_fast(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ uint32_t half2_bits(float a, float b)
{
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
}

// A warp's part of the result for 8 NT rows: column 2 t + c of tile n (t = lane % 4) is a row.
template <int D, int NT>
struct Part {
    float o[NT][D / 16][4];        // O^T: [0], [1] dimension d of columns 0 and 1; [2], [3] of d + 1
    float l[NT][2], m[NT][2], mv[NT][2];
};

// Where a request's keys lie.
struct Place {
    const uint8_t *k, *v;          // of the key head
    const float *ks, *vs;
    const int32_t *table;
    int64_t token, pages;          // bytes from a token to the next; pages of the cache
    int page_shift, Hkv;
    int len, first_seen;           // keys; the first token sees first_seen of them, each further one more
};

// The page and the log2 scales of a block, a lane a block.
struct Found {
    int64_t block;                 // of 16 tokens, in the cache; -1: outside
    float ks, vs;
};

__device__ __forceinline__ Found find(const Place &p, int block, bool any)
{
    Found f{-1, 0.0f, 0.0f};
    if (!any) return f;
    const int per_page = p.page_shift - 4;
    const int page = __ldg(p.table + (block >> per_page));
    if (page < 0 || page >= p.pages) {
        atomicOr(&g_paged_error, kErrIndex);
        return f;
    }
    f.block = (static_cast<int64_t>(page) << per_page) + (block & ((1 << per_page) - 1));
    f.ks = __ldg(p.ks + f.block * p.Hkv);
    f.vs = __ldg(p.vs + f.block * p.Hkv);
    return f;
}

template <int D>
__device__ __forceinline__ void copy_block(const Place &p, int64_t block, uint32_t stage, int lane)
{
    const int gid = lane / 4, t = lane % 4;
    const bool there = block >= 0;
    const int64_t first = (there ? block : 0) * kBlock * p.token;
#pragma unroll
    for (int i = 0; i < Ring<D>::kKPieces; ++i) {   // piece i: key gid + 8 (i % 2), 16 of dimensions 64 (i / 2) ..
        const uint8_t *src = p.k + first + (gid + 8 * (i % 2)) * p.token + 64 * (i / 2) + 16 * t;
        cp_async_16_zfill(stage + (i * 32 + lane) * 16, src, there);
    }
    const uint32_t values = stage + Ring<D>::kKPieces * 512;
#pragma unroll
    for (int i = 0; i < 4; ++i) {                   // piece i: key 2 t + i % 2 + 8 (i / 2), D / 8 dimensions from gid D / 8 on
        const uint8_t *src = p.v + first + (2 * t + i % 2 + 8 * (i / 2)) * p.token + gid * (D / 8);
        if constexpr (D == 128) {
            cp_async_16_zfill(values + (i * 32 + lane) * 16, src, there);
        } else {
            cp_async_8_zfill(values + (i * 32 + lane) * 8, src, there);
        }
    }
}

__device__ __forceinline__ bool has_nan(uint32_t codes)
{
    return ((codes & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;
}

// Values that are NaN, in a block that not every row sees whole: 0 x NaN is NaN, so in the
// product they are cleared, and only the rows that see their keys get the NaN, here.
template <int D, int NT>
__device__ __forceinline__ void add_nan(Part<D, NT> &r, uint32_t (&v)[4][D / 32], const int (&seen)[NT][2], int key0, int lane)
{
    for (int t = 0; t < 4; ++t) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int key = key0 + 2 * t + i % 2 + 8 * (i / 2);
#pragma unroll
            for (int w = 0; w < D / 32; ++w) {
                const uint32_t word = __shfl_sync(0xffffffffu, v[i][w], (lane & ~3) + t);
#pragma unroll
                for (int b = 0; b < 4; ++b) {
                    if ((word >> (8 * b) & 0x7fu) != 0x7fu) continue;
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        if (key < seen[n][0]) r.o[n][2 * w + b / 2][2 * (b % 2)] = NAN;
                        if (key < seen[n][1]) r.o[n][2 * w + b / 2][2 * (b % 2) + 1] = NAN;
                    }
                }
            }
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
#pragma unroll
        for (int w = 0; w < D / 32; ++w) {
            const uint32_t nan = ((v[i][w] & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;   // a byte's top bit: it is NaN
            v[i][w] &= ~((nan >> 7) * 0xffu);
        }
    }
}

// One block of 16 keys into the warp's part. q: columns' rows as the B operand of S^T.
template <int D, int NT, typename Q>
__device__ __forceinline__ void add_block(Part<D, NT> &r, const Q &q, const float (&c)[NT][2],
                                          const int (&seen)[NT][2], uint32_t stage, int lane, int key0, int len, float ks,
                                          float lv, bool masked)
{
    const int gid = lane / 4, t = lane % 4;
    float s[NT][4];
#pragma unroll
    for (int n = 0; n < NT; ++n) s[n][0] = s[n][1] = s[n][2] = s[n][3] = 0.0f;
#pragma unroll
    for (int i = 0; i < D / 64; ++i) {
        const uint4 lo = lds128(stage + (2 * i * 32 + lane) * 16), hi = lds128(stage + ((2 * i + 1) * 32 + lane) * 16);
        const uint32_t low[4] = {lo.x, lo.y, lo.z, lo.w}, high[4] = {hi.x, hi.y, hi.z, hi.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint32_t a0 = e4m3x2_to_f16x2(low[j] & 0xffffu), a2 = e4m3x2_to_f16x2(low[j] >> 16);
            const uint32_t a1 = e4m3x2_to_f16x2(high[j] & 0xffffu), a3 = e4m3x2_to_f16x2(high[j] >> 16);
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                const uint2 b = q.at(n, 4 * i + j);
                mma_16816(s[n], a0, a1, a2, a3, b.x, b.y);
            }
        }
    }
    bool grow = false;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            s[n][e] *= c[n][e & 1] * ks;
            if (masked && key0 + gid + (e >> 1) * 8 >= seen[n][e & 1]) s[n][e] = -INFINITY;
            grow |= s[n][e] > r.m[n][e & 1] + kSlack || s[n][e] + lv > r.mv[n][e & 1] + kSlack;
        }
    }
    if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
        for (int n = 0; n < NT; ++n) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float top = fmaxf(s[n][e], s[n][e + 2]);
#pragma unroll
                for (int o = 4; o < 32; o *= 2) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
                const float m = fmaxf(r.m[n][e], top), mv = fmaxf(r.mv[n][e], top + lv);
                r.l[n][e] *= exp2_fast(r.m[n][e] - m);
                const float by = exp2_fast(r.mv[n][e] - mv);
                r.m[n][e] = m;
                r.mv[n][e] = mv;
#pragma unroll
                for (int j = 0; j < D / 16; ++j) {
                    r.o[n][j][e] *= by;
                    r.o[n][j][e + 2] *= by;
                }
            }
        }
    }
    uint32_t p[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        float w[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            r.l[n][e & 1] += exp2_fast(s[n][e] - r.m[n][e & 1]);
            w[e] = exp2_fast(s[n][e] + lv - r.mv[n][e & 1]);
        }
        p[n][0] = transpose8x8(half2_bits(w[0], w[1]));
        p[n][1] = transpose8x8(half2_bits(w[2], w[3]));
    }
    const uint32_t values = stage + Ring<D>::kKPieces * 512;
    uint32_t v[4][D / 32];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (D == 128) {
            const uint4 x = lds128(values + (i * 32 + lane) * 16);
            v[i][0] = x.x, v[i][1] = x.y, v[i][2] = x.z, v[i][3] = x.w;
        } else {
            const uint2 x = lds64(values + (i * 32 + lane) * 8);
            v[i][0] = x.x, v[i][1] = x.y;
        }
        if (masked && key0 + 2 * t + i % 2 + 8 * (i / 2) >= len) {   // behind the last token: whatever lies there
#pragma unroll
            for (int w = 0; w < D / 32; ++w) v[i][w] = 0;
        }
    }
    if (masked) {
        bool nan = false;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
#pragma unroll
            for (int w = 0; w < D / 32; ++w) nan |= has_nan(v[i][w]);
        }
        if (__any_sync(0xffffffffu, nan)) add_nan<D, NT>(r, v, seen, key0, lane);
    }
#pragma unroll
    for (int w = 0; w < D / 32; ++w) {
        // dimensions gid D / 8 + 4 w + 0, 1 (tile 2 w) and + 2, 3 (tile 2 w + 1), two keys a register
        const uint32_t lo01 = __byte_perm(v[0][w], v[1][w], 0x5140), lo23 = __byte_perm(v[0][w], v[1][w], 0x7362);
        const uint32_t hi01 = __byte_perm(v[2][w], v[3][w], 0x5140), hi23 = __byte_perm(v[2][w], v[3][w], 0x7362);
        const uint32_t a0 = e4m3x2_to_f16x2(lo01 & 0xffffu), a1 = e4m3x2_to_f16x2(lo01 >> 16);
        const uint32_t a2 = e4m3x2_to_f16x2(hi01 & 0xffffu), a3 = e4m3x2_to_f16x2(hi01 >> 16);
        const uint32_t b0 = e4m3x2_to_f16x2(lo23 & 0xffffu), b1 = e4m3x2_to_f16x2(lo23 >> 16);
        const uint32_t b2 = e4m3x2_to_f16x2(hi23 & 0xffffu), b3 = e4m3x2_to_f16x2(hi23 >> 16);
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            mma_16816(r.o[n][2 * w], a0, a1, a2, a3, p[n][0], p[n][1]);
            mma_16816(r.o[n][2 * w + 1], b0, b1, b2, b3, p[n][0], p[n][1]);
        }
    }
}

// A warp's way through the blocks first, first + kWarps, ... (count of them): pages and scales
// are looked up a batch ahead, copies run kStages - 1 blocks ahead.
template <int D, int NT>
struct Walk {
    static constexpr int kStages = Shape<D, NT>::kStages;
    const Place &p;
    uint32_t ring;
    int lane, first, count, issued = 0;
    Found ahead, next{};
    float ks32 = 0.0f, lv32 = 0.0f;   // of the batch that is being added, a lane a block

    __device__ __forceinline__ Found batch(int n) const   // blocks 32 n .. of the warp's
    {
        const int i = n * kBatch + lane;
        return find(p, first + i * kWarps, i < count);
    }
    __device__ __forceinline__ Walk(const Place &place, uint32_t ring_at, int lane_, int first_, int count_)
        : p(place), ring(ring_at), lane(lane_), first(first_), count(count_)
    {
        ahead = batch(0);
        if (count > kBatch) next = batch(1);
#pragma unroll
        for (int i = 0; i < kStages - 1; ++i) issue();
    }
    __device__ __forceinline__ void issue()
    {
        if (issued < count) {
            if (issued % kBatch == 0 && issued > 0) {
                ahead = next;
                if ((issued / kBatch + 1) * kBatch < count) next = batch(issued / kBatch + 1);
            }
            const int64_t block = __shfl_sync(0xffffffffu, ahead.block, issued % kBatch);
            copy_block<D>(p, block, ring + (issued % kStages) * Ring<D>::kBytes, lane);
        }
        ++issued;
        cp_async_commit();
    }
    template <typename Q>
    __device__ __forceinline__ void add(Part<D, NT> &r, const Q &q, const float (&c)[NT][2], const int (&seen)[NT][2])
    {
        for (int j = 0; j < count; ++j) {
            cp_async_wait<kStages - 2>();
            if (j % kBatch == 0) {   // copies are less than a batch ahead
                ks32 = ahead.ks;
                lv32 = log2f(ahead.vs);
            }
            issue();
            const float ks = __shfl_sync(0xffffffffu, ks32, j % kBatch), lv = __shfl_sync(0xffffffffu, lv32, j % kBatch);
            const int key0 = (first + j * kWarps) * kBlock;
            add_block<D, NT>(r, q, c, seen, ring + (j % kStages) * Ring<D>::kBytes, lane, key0, p.len, ks, lv,
                             key0 + kBlock > p.first_seen);
        }
        cp_async_wait<0>();
    }
};

template <int D, int NT>
__device__ __forceinline__ void merge(Part<D, NT> &r, const float *other, int lane)
{
    int at = 0;
    auto get = [&]() { return other[32 * at++ + lane]; };
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        float mine[2], theirs[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const float l = get(), m1 = get(), mv1 = get();
            const float m = fmaxf(r.m[n][e], m1), mv = fmaxf(r.mv[n][e], mv1);
            r.l[n][e] = r.l[n][e] * exp2_fast(r.m[n][e] - m) + l * exp2_fast(m1 - m);
            mine[e] = exp2_fast(r.mv[n][e] - mv);
            theirs[e] = exp2_fast(mv1 - mv);
            r.m[n][e] = m;
            r.mv[n][e] = mv;
        }
#pragma unroll
        for (int j = 0; j < D / 16; ++j) {
#pragma unroll
            for (int e = 0; e < 4; ++e) r.o[n][j][e] = r.o[n][j][e] * mine[e & 1] + get() * theirs[e & 1];
        }
    }
}

template <int D, int NT>
__device__ __forceinline__ void put(const Part<D, NT> &r, float *to, int lane)
{
    int at = 0;
    auto set = [&](float v) { to[32 * at++ + lane] = v; };
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            set(r.l[n][e]);
            set(r.m[n][e]);
            set(r.mv[n][e]);
        }
#pragma unroll
        for (int j = 0; j < D / 16; ++j) {
#pragma unroll
            for (int e = 0; e < 4; ++e) set(r.o[n][j][e]);
        }
    }
}

template <int D, int NT>
constexpr int part_floats() { return 32 * NT * (6 + D / 4); }

// The work is cut into units, a block of an item each, an item being a request, a key head and a group of
// 8 NT query rows, in that order. A CTA takes a run of units; a run's piece of an item that
// is not all of it leaves a part in the workspace.
struct Cut {
    int b, item;          // item of the request: key head * groups + group
    int64_t at;           // units before it in its item (blocks)
    int64_t left;         // units of the run
    int64_t from, units;  // where the run starts; all units
};

// Where run c of `ctas` starts: shares of equal length, the first ones longer by one.
__device__ __forceinline__ int64_t start_of(int64_t units, int c, int ctas)
{
    return units / ctas * c + min(static_cast<int64_t>(c), units % ctas);
}

__device__ __forceinline__ int blocks_of(const PagedArgs &g, int b)
{
    return (static_cast<int>(min(static_cast<int64_t>(max(g.lens[b], 0)), g.max_len)) + kBlock - 1) / kBlock;
}

// Sum over a CTA's threads before this one, and of all.
__device__ __forceinline__ int64_t scan_before(int64_t v, int64_t *sums, int64_t &all)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x / 32, warps = blockDim.x / 32;
    int64_t upto = v;
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
        const int64_t x = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += x;
    }
    __syncthreads();
    if (lane == 31) sums[warp] = upto;
    __syncthreads();
    int64_t before = upto - v;
    all = 0;
    for (int i = 0; i < warps; ++i) {
        if (i < warp) before += sums[i];
        all += sums[i];
    }
    return before;
}

// The c-th run. items: of a request.
__device__ __forceinline__ Cut cut_of(const PagedArgs &g, int c, int ctas, int items, int64_t *sums, Cut *shared)
{
    const int tid = threadIdx.x, step = static_cast<int>(blockDim.x);
    int64_t total = 0, all, mine = 0, before = 0;
    for (int b0 = 0; b0 < g.B; b0 += step) {
        mine = b0 + tid < g.B ? blocks_of(g, b0 + tid) : 0;
        before = scan_before(mine, sums, all);
        total += all;
    }
    const int64_t units = total * items, from = start_of(units, c, ctas), to = start_of(units, c + 1, ctas);
    if (tid == 0) *shared = Cut{0, 0, 0, 0, from, units};
    if (g.B > step) total = 0;
    for (int b0 = 0; b0 < g.B; b0 += step) {
        int64_t base = 0;
        if (g.B > step) {
            mine = b0 + tid < g.B ? blocks_of(g, b0 + tid) : 0;
            before = scan_before(mine, sums, all);
            base = total;
            total += all;
        } else {
            __syncthreads();
        }
        const int64_t start = (base + before) * items;
        if (start <= from && from < start + mine * items && from < to)
            *shared = Cut{b0 + tid, static_cast<int>((from - start) / mine), (from - start) % mine, to - from, from, units};
    }
    __syncthreads();
    return *shared;
}

template <int D, int NT>
struct Staged {                                // in shared memory, behind the rings
    uint2 q[NT][D / 16][32];                   // B operands of S^T
    float back[8 * NT];                        // what q's rows were divided by
    int64_t sums[kWarps];
    Cut cut;
};

template <int NT, int D>
struct QRegs {
    uint2 v[NT][D / 16];
    __device__ __forceinline__ uint2 at(int n, int k) const { return v[n][k]; }
};
struct QShared {
    uint32_t base;   // of this lane
    int ks;
    __device__ __forceinline__ uint2 at(int n, int k) const { return lds64(base + (n * ks + k) * 256); }
};

// Row tile n of the item's q, as B operands: lane (gid, t) has row gid.
template <int D, int NT>
__device__ __forceinline__ void stage_q(const PagedArgs &g, Staged<D, NT> &s, int n, const uint16_t *q, bool live, int lane)
{
    const int gid = lane / 4, t = lane % 4;
    uint32_t words[D / 8];
#pragma unroll
    for (int i = 0; i < D / 64; ++i) {
#pragma unroll
        for (int w = 0; w < 2; ++w) {
            uint4 x = make_uint4(0, 0, 0, 0);
            if (live) x = *(reinterpret_cast<const uint4 *>(q + 64 * i + 16 * t) + w);
            words[8 * i + 4 * w] = x.x, words[8 * i + 4 * w + 1] = x.y, words[8 * i + 4 * w + 2] = x.z, words[8 * i + 4 * w + 3] = x.w;
        }
    }
    float back = 1.0f;
    if (g.type == QMV_BF16) {
        uint32_t largest = 0;   // of the finite elements, as the upper half of an fp32's bits
#pragma unroll
        for (int w = 0; w < D / 8; ++w) {
            const uint32_t lo = words[w] & 0x7fffu, hi = words[w] >> 16 & 0x7fffu;
            largest = max(largest, max(lo < 0x7f80u ? lo : 0u, hi < 0x7f80u ? hi : 0u));
        }
        largest = max(largest, __shfl_xor_sync(0xffffffffu, largest, 1));
        largest = max(largest, __shfl_xor_sync(0xffffffffu, largest, 2));
        const int e = largest ? min(max(14 - (static_cast<int>(largest >> 7) - 127), -126), 126) : 0;
        const float by = __uint_as_float(static_cast<uint32_t>(e + 127) << 23);
        back = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
#pragma unroll
        for (int w = 0; w < D / 8; ++w)
            words[w] = half2_bits(__uint_as_float(words[w] << 16) * by, __uint_as_float(words[w] & 0xffff0000u) * by);
    }
#pragma unroll
    for (int k = 0; k < D / 16; ++k) s.q[n][k][lane] = make_uint2(words[2 * k], words[2 * k + 1]);
    if (t == 0) s.back[8 * n + gid] = back;
}

// A part in the workspace: 8 NT rows of D floats, then of (l, m, m', 0).
template <int D, int NT>
constexpr int slot_floats() { return 8 * NT * (D + 4); }

// direct: CTA i has item i % items of request i / items, whole. Otherwise: the i-th run.
template <int D, int NT>
__global__ void __launch_bounds__(kThreads, Shape<D, NT>::kCtas) paged_kernel(const __grid_constant__ PagedArgs g, int groups, bool direct)
{
    extern __shared__ __align__(128) uint8_t smem[];
    constexpr int kRings = kWarps * Shape<D, NT>::kStages * Ring<D>::kBytes;
    Staged<D, NT> &staged = *reinterpret_cast<Staged<D, NT> *>(smem + kRings);
    const int lane = threadIdx.x & 31, warp = threadIdx.x / 32, gid = lane / 4, t = lane % 4;
    const int G = g.Hq / g.Hkv, rows = g.T * G, items = g.Hkv * groups;
    grid_launch_dependents();
    grid_dependency_wait();
    Cut cut;
    if (direct) {
        cut.b = static_cast<int>(blockIdx.x) / items;
        cut.item = static_cast<int>(blockIdx.x) % items;
        cut.at = 0;
        cut.left = 1;
    } else {
        cut = cut_of(g, static_cast<int>(blockIdx.x), static_cast<int>(gridDim.x), items, staged.sums, &staged.cut);
        // rows of requests without keys are no units
        for (int b = static_cast<int>(blockIdx.x); b < g.B; b += static_cast<int>(gridDim.x)) {
            if (g.lens[b] > g.max_len && threadIdx.x == 0) atomicOr(&g_paged_error, kErrIndex);
            if (blocks_of(g, b) > 0) continue;
            uint4 *out = reinterpret_cast<uint4 *>(static_cast<uint16_t *>(g.out) + static_cast<int64_t>(b) * g.T * g.Hq * D);
            for (int64_t i = threadIdx.x; i < static_cast<int64_t>(g.T) * g.Hq * D / 8; i += kThreads) out[i] = make_uint4(0, 0, 0, 0);
        }
    }
    bool first_piece = true;
    while (cut.left > 0) {
        const int b = cut.b, h = cut.item / groups, row0 = cut.item % groups * 8 * NT;
        if (direct && g.lens[b] > g.max_len && threadIdx.x == 0) atomicOr(&g_paged_error, kErrIndex);
        const int len = static_cast<int>(min(static_cast<int64_t>(max(g.lens[b], 0)), g.max_len));
        const int blocks = (len + kBlock - 1) / kBlock;
        const int block0 = static_cast<int>(cut.at);
        const int block1 = direct ? blocks : static_cast<int>(min(static_cast<int64_t>(blocks), cut.at + cut.left));
        Place p;
        p.token = static_cast<int64_t>(g.Hkv) * D;
        p.k = static_cast<const uint8_t *>(g.k) + h * D;
        p.v = static_cast<const uint8_t *>(g.v) + h * D;
        p.ks = g.ks + h;
        p.vs = g.vs + h;
        p.table = g.table + static_cast<int64_t>(b) * g.table_pages;
        p.pages = g.n_pages;
        p.page_shift = 31 - __clz(g.page);
        p.Hkv = g.Hkv;
        p.len = len;
        p.first_seen = len - g.T + 1;
        const int first = block0 + warp;
        Walk<D, NT> walk(p, smem_addr(smem) + warp * Shape<D, NT>::kStages * Ring<D>::kBytes, lane, first,
                         first < block1 ? (block1 - first + kWarps - 1) / kWarps : 0);
        auto row_at = [&](int r) { return ((static_cast<int64_t>(b) * g.T + r / G) * g.Hq + static_cast<int64_t>(h) * G + r % G) * D; };
        for (int n = warp; n < NT; n += kWarps) {
            const int row = row0 + 8 * n + gid;
            stage_q<D, NT>(g, staged, n, static_cast<const uint16_t *>(g.q) + (row < rows ? row_at(row) : 0), row < rows, lane);
        }
        __syncthreads();
        float c[NT][2];
        int seen[NT][2];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int r = row0 + 8 * n + 2 * t + e;
                c[n][e] = g.scale * kLog2e * staged.back[8 * n + 2 * t + e];
                seen[n][e] = r < rows ? p.first_seen + r / G : 0;
            }
        }
        Part<D, NT> part;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
#pragma unroll
            for (int e = 0; e < 2; ++e) part.l[n][e] = 0.0f, part.m[n][e] = part.mv[n][e] = kLowest;
#pragma unroll
            for (int j = 0; j < D / 16; ++j) part.o[n][j][0] = part.o[n][j][1] = part.o[n][j][2] = part.o[n][j][3] = 0.0f;
        }
        if constexpr (NT == 1) {
            QRegs<NT, D> q;
#pragma unroll
            for (int k = 0; k < D / 16; ++k) q.v[0][k] = staged.q[0][k][lane];
            walk.add(part, q, c, seen);
        } else {
            walk.add(part, QShared{smem_addr(&staged.q[0][0][lane]), D / 16}, c, seen);
        }
        // the warps' parts, half of them into the other half at a time, over the rings
        float *parts = reinterpret_cast<float *>(smem);
#pragma unroll
        for (int half = kWarps / 2; half > 0; half /= 2) {
            __syncthreads();
            if (warp >= half && warp < 2 * half) put(part, parts + (warp - half) * part_floats<D, NT>(), lane);
            __syncthreads();
            if (warp < half) merge(part, parts + warp * part_floats<D, NT>(), lane);
        }
        const bool whole = block0 == 0 && block1 == blocks;
        if (warp == 0) {
            float *slot = static_cast<float *>(g.workspace) + (2 * static_cast<int64_t>(blockIdx.x) + (first_piece ? 0 : 1)) * slot_floats<D, NT>();
#pragma unroll
            for (int n = 0; n < NT; ++n) {
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float l = part.l[n][e];
#pragma unroll
                    for (int o = 4; o < 32; o *= 2) l += __shfl_xor_sync(0xffffffffu, l, o);
                    const int row = row0 + 8 * n + 2 * t + e;
                    if (row >= rows) continue;
                    if (!whole) {
                        float4 *to = reinterpret_cast<float4 *>(slot + (8 * n + 2 * t + e) * D + gid * (D / 8));
#pragma unroll
                        for (int j = 0; j < D / 32; ++j)
                            to[j] = make_float4(part.o[n][2 * j][e], part.o[n][2 * j][e + 2], part.o[n][2 * j + 1][e], part.o[n][2 * j + 1][e + 2]);
                        if (gid == 0)
                            reinterpret_cast<float4 *>(slot + 8 * NT * D)[8 * n + 2 * t + e] = make_float4(l, part.m[n][e], part.mv[n][e], 0.0f);
                        continue;
                    }
                    const float by = exp2f(part.mv[n][e] - part.m[n][e]) / l;
                    const bool none = seen[n][e] <= 0;
                    uint16_t *out = static_cast<uint16_t *>(g.out) + row_at(row) + gid * (D / 8);
                    uint32_t words[D / 16];
#pragma unroll
                    for (int j = 0; j < D / 16; ++j) {
                        const float a = none ? 0.0f : part.o[n][j][e] * by, z = none ? 0.0f : part.o[n][j][e + 2] * by;
                        words[j] = g.type == QMV_F16 ? pack2<__half>(a, z) : pack2<__nv_bfloat16>(a, z);
                    }
#pragma unroll
                    for (int j = 0; j < D / 64; ++j)
                        reinterpret_cast<uint4 *>(out)[j] = make_uint4(words[4 * j], words[4 * j + 1], words[4 * j + 2], words[4 * j + 3]);
                }
            }
        }
        if (direct) return;
        first_piece = false;
        cut.left -= block1 - block0;
        cut.at = 0;
        if (++cut.item == items) {
            cut.item = 0;
            do {
                ++cut.b;
            } while (cut.left > 0 && cut.b < g.B && blocks_of(g, cut.b) == 0);
        }
        if (cut.left > 0) __syncthreads();   // the parts have been read
    }
}

// The rows of items of which more than one run has a part. Grid (runs - 1, rows): CTA (i, r) has
// row r of the item that the cut between runs i and i + 1 goes through, unless an earlier cut
// goes through it too.
template <int D, int NT>
__global__ void __launch_bounds__(128) paged_join_kernel(const __grid_constant__ PagedArgs g, int groups, int ctas)
{
    constexpr int kWarpsJoin = 4, kD4 = D / 4;
    __shared__ int64_t sums[kWarpsJoin];
    __shared__ Cut found;
    __shared__ float4 sum_o[kWarpsJoin][kD4];
    __shared__ float sum_l[kWarpsJoin], sum_m[kWarpsJoin], sum_mv[kWarpsJoin];
    const int lane = threadIdx.x & 31, warp = threadIdx.x / 32, c = static_cast<int>(blockIdx.x) + 1, r = blockIdx.y;
    const int G = g.Hq / g.Hkv, rows = g.T * G, items = g.Hkv * groups;
    grid_launch_dependents();
    grid_dependency_wait();   // in every CTA: this launch ends after the one before it
    const Cut cut = cut_of(g, c, ctas, items, sums, &found);
    if (cut.left == 0 || cut.at == 0) return;
    const int row = cut.item % groups * 8 * NT + r, h = cut.item / groups;
    const int64_t item0 = cut.from - cut.at, item1 = item0 + blocks_of(g, cut.b), last = start_of(cut.units, c - 1, ctas);
    if (row >= rows || last > item0) return;
    // piece 0: of run c - 1, its first if it starts with the item; piece i: the first of run c - 1 + i
    float l = 0.0f, m = kLowest, mv = kLowest;
    float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    auto take = [&](float l1, float m1, float mv1, float4 x) {
        const float mn = fmaxf(m, m1), mvn = fmaxf(mv, mv1), a = exp2_fast(mv - mvn), z = exp2_fast(mv1 - mvn);
        l = l * exp2_fast(m - mn) + l1 * exp2_fast(m1 - mn);
        o = make_float4(o.x * a + x.x * z, o.y * a + x.y * z, o.z * a + x.z * z, o.w * a + x.w * z);
        m = mn;
        mv = mvn;
    };
#pragma unroll 4
    for (int i = warp; c - 1 + i < ctas; i += kWarpsJoin) {
        const int run = c - 1 + i;
        if (i > 0 && start_of(cut.units, run, ctas) >= item1) break;
        if (i > 0 && start_of(cut.units, run + 1, ctas) == start_of(cut.units, run, ctas)) continue;   // an empty run
        const float *slot = static_cast<const float *>(g.workspace) + (2 * static_cast<int64_t>(run) + (i == 0 && last < item0 ? 1 : 0)) * slot_floats<D, NT>();
        const float4 st = reinterpret_cast<const float4 *>(slot + 8 * NT * D)[r];
        const float4 x = lane < kD4 ? reinterpret_cast<const float4 *>(slot + r * D)[lane] : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        take(st.x, st.y, st.z, x);
    }
    if (lane < kD4) sum_o[warp][lane] = o;
    if (lane == 0) sum_l[warp] = l, sum_m[warp] = m, sum_mv[warp] = mv;
    __syncthreads();
    if (warp > 0 || lane >= kD4) return;
#pragma unroll
    for (int w = 1; w < kWarpsJoin; ++w) take(sum_l[w], sum_m[w], sum_mv[w], sum_o[w][lane]);
    const int seen = static_cast<int>(min(static_cast<int64_t>(g.lens[cut.b]), g.max_len)) - g.T + 1 + row / G;
    const float by = seen <= 0 ? 0.0f : exp2f(mv - m) / l;
    if (seen <= 0) o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    o = make_float4(o.x * by, o.y * by, o.z * by, o.w * by);
    uint16_t *out = static_cast<uint16_t *>(g.out) + ((static_cast<int64_t>(cut.b) * g.T + row / G) * g.Hq + static_cast<int64_t>(h) * G + row % G) * D;
    reinterpret_cast<uint2 *>(out)[lane] = g.type == QMV_F16 ? make_uint2(pack2<__half>(o.x, o.y), pack2<__half>(o.z, o.w))
                                                             : make_uint2(pack2<__nv_bfloat16>(o.x, o.y), pack2<__nv_bfloat16>(o.z, o.w));
}

constexpr int kSms = 152;
constexpr int kDirectBlocks = 64;   // of a request, up to which an item is one CTA's

template <int D, int NT>
cudaError_t launch_typed(const PagedArgs &g, int groups, cudaStream_t s)
{
    using S = Shape<D, NT>;
    const int64_t items = static_cast<int64_t>(g.Hkv) * groups, blocks = (g.max_len + kBlock - 1) / kBlock;
    constexpr int kSmem = kWarps * S::kStages * Ring<D>::kBytes + static_cast<int>(sizeof(Staged<D, NT>));
    static_assert(kWarps / 2 * part_floats<D, NT>() * 4 <= kWarps * S::kStages * Ring<D>::kBytes, "the parts fit the rings");
    static_assert(2 * kSms * S::kCtas * slot_floats<D, NT>() * 4 <= kWorkspaceBytes, "the workspace has every run's parts");
    const bool direct = blocks <= kDirectBlocks && items * g.B <= 0x7fffffff;
    const int64_t most = kSms * S::kCtas;
    const int ctas = static_cast<int>(direct ? items * g.B : std::max<int64_t>(1, std::min(most, items * g.B * blocks / kWarps)));
    cudaError_t e = ensure_smem_attr(reinterpret_cast<const void *>(paged_kernel<D, NT>), kSmem);
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute attr[1];
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3(kThreads);
    cfg.gridDim = dim3(static_cast<unsigned>(ctas));
    cfg.dynamicSmemBytes = kSmem;
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = set_launch_overlap_attr(attr);
    e = cudaLaunchKernelEx(&cfg, paged_kernel<D, NT>, g, groups, direct);
    if (e != cudaSuccess || direct || ctas == 1) return e;
    // the join starts while the runs still go on, and waits for their end on the device
    cudaLaunchConfig_t join = {};
    join.blockDim = dim3(128);
    join.gridDim = dim3(static_cast<unsigned>(ctas - 1), static_cast<unsigned>(std::min(8 * NT, g.T * (g.Hq / g.Hkv))));
    join.stream = s;
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    join.attrs = attr;
    join.numAttrs = 1;
    return cudaLaunchKernelEx(&join, paged_join_kernel<D, NT>, g, groups, ctas);
}

// Groups of up to 8 NT rows, all of nearly the same number.
template <int D>
cudaError_t launch_rows(const PagedArgs &g, cudaStream_t s)
{
    constexpr int kMost = D == 64 ? 48 : 32;
    const int rows = g.T * (g.Hq / g.Hkv);
    const int groups = (rows + kMost - 1) / kMost, each = (rows + groups - 1) / groups;
    if (each <= 8) return launch_typed<D, 1>(g, groups, s);
    if (each <= 16) return launch_typed<D, 2>(g, (rows + 15) / 16, s);
    if (each <= 32) return launch_typed<D, 4>(g, (rows + 31) / 32, s);
    if constexpr (D == 64) return launch_typed<D, 6>(g, (rows + 47) / 48, s);
    return cudaErrorInvalidValue;
}

}  // namespace

int64_t paged_workspace_bytes() { return kWorkspaceBytes; }

cudaError_t launch_paged_e4m3(const PagedArgs &g, cudaStream_t s)
{
    route_hit(kRoutePagedE4m3);
    return g.D == 64 ? launch_rows<64>(g, s) : launch_rows<128>(g, s);
}

cudaError_t read_error_word_paged(uint32_t *out, bool clear)
{
    cudaError_t e = cudaMemcpyFromSymbol(out, g_paged_error, sizeof(uint32_t));
    if (e != cudaSuccess || !clear) return e;
    const uint32_t zero = 0;
    return cudaMemcpyToSymbol(g_paged_error, &zero, sizeof(uint32_t));
}

}  // namespace qmv
