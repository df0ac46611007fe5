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
// that every lane's operands are whole 16-byte pieces of the cache's rows, and codes become
// binary16, exactly, on their way from shared memory into the product. P^T is S^T transposed in registers.
//
// Numerics: q is held in binary16 (bfloat16 rows are scaled by a power of two that brings
// their largest element to 2^14 or more: elements 2^-28 of it and less lose bits); S, the
// softmax's statistics and O are fp32. The running maximum of a column is that of z + log2 sv, z = c sk S:
// the terms 2^(z + log2 sv - m) of the numerator are then of one size where they are largest, whatever the
// scales of the blocks. Each goes into the products as two binary16, itself rounded and what that left: 2^-22 of
// it, or 2^-32 of the row's largest, is lost. (Rounded once, outputs differed from a plain form's in fp32 by 2.5e-4 for 6e-6 now, and
// were 2.6e-4 off for 2.1e-4, binary16's own rounding. With 5 rows a key head of 128 that costs nothing that shows, where the products' instructions
// bound a call up to a tenth: 40 rows of heads of 64 30 us for 28.6, 64 requests of 16384 keys and 16 rows of 64 143 for 129.)
// The denominator's are 2^(z - m), in fp32, whose range holds them. m is the true maximum less 7, and follows it
// with a slack of 2^8, so that O is rescaled rarely: the largest terms are 2^7 .. 2^15, binary16's range ends at 2^16.
//
// Bound by the cache's bytes: 64 requests of up to 16384 tokens, 40 query heads over 8 key heads of
// 128, take 164 to 166 us, by the GPU, 6.6 TB/s. What it took to get there, us: a CTA an item 482; equal runs of blocks over
// all SMs 223; key heads of the same blocks side by side, and copies of whole rows (half rows
// were as many requests to L2 again, which bound it), 174; scores of the next block beside this
// one's softmax, starting on an item counted as blocks 165. The smaller the call, the more of it
// is starting and joining: 12 us or so (8 where clusters have the items), a chain of lengths, pages, scales, codes and parts that wait for
// one another. Of the cycles between a warp's instructions in a cluster 27 % are at barriers, 18 fixed latencies, 16 reads of memory and 7 the
// fetching of instructions; in a join 37 % reads.
#include <algorithm>
#include <cmath>

#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "decode_device.cuh"
#include "decode_ops.h"
#include "qmv.h"
#include "qmv_device.cuh"

namespace cg = cooperative_groups;

namespace qmv {
namespace {

__device__ uint32_t g_paged_error;

constexpr int kBlock = kScaleTokens;    // keys a step of a warp
constexpr int kMostWarps = 8;           // of a CTA, a key head each
constexpr int64_t kFewBytes = 11ll << 20, kMostBytes = 22ll << 20;   // of the workspace's slots, with 8 rows and 16
constexpr int kStartUnits = 8;          // what starting on an item costs, in blocks of a warp's
constexpr int kLeastBlocks = 2;         // of a run, where there are few
// Blocks a CTA up to which a cluster has an item: one launch for two. 560 keys of one request 8.5 us for
// 11.1, 12 requests of 1000 keys 12.3 for 16.8; one of 2000 keys, the most there is for one, 12.6 for 12.3.
constexpr int kClusterBlocks = 8;
// Blocks after which a warp leaves its part in the workspace and begins a new one, which the first is added to in fp32: the products truncate their
// sums to fp32, and with values of one sign a sum over n blocks is 5e-8 n too small (152 requests of 65536 keys 4e-4, of 1048576 6.7e-3;
// now 3e-5). A launch whose runs may have so many of one item has the code for it: 24 requests of up to 131072 keys take 511 us for 506,
// 64 of 2000 with that bound 45 for 44 (16 rows of 64: 48 for 46). In all launches it would be 169 us for 165.5 with 64 requests of up to 16384
// keys, and 33 for 30 with 40 rows of heads of 64.
constexpr int kFold = 512;
constexpr int kBatch = 32;              // blocks whose page and scales a warp looks up at a time, a lane a block
constexpr float kLift = 7.0f, kSlack = 15.0f;   // log2 of the largest term when m is set, and at most
constexpr float kLowest = -3.402823466e38f;   // a maximum of no scores: the difference to it is never NaN
// log2 of a scale of 0; smaller ones are taken for 0. A row's denominator is up to 2^(15 + 81) for each of 2^30 keys, where all scales are as
// small: that fits fp32.
constexpr float kLeastLog = -81.0f;
constexpr float kLog2e = 1.4426950408889634f;

template <int D>
struct Ring {
    static constexpr int kBytes = 32 * kBlock * D / 16;   // keys and values of a block: 2 * 16 * D
};

// Warps an SM, and stages of a warp's ring, by the shared memory that is left beside q's operands:
// 8 warps with six stages. (16 with three end at the same time where there is much, 166 us for 165, but have twice
// the parts: 75 us for 54 with one request of 131072 tokens. A block of 64 dimensions is half the bytes.)
template <int D, int NT>
struct Shape {
    static constexpr int kWarpsSm = D == 128 ? 8 : 16;
    static constexpr int kQueries = NT == 1 ? 0 : NT * D * 16;   // bytes a warp
    static constexpr int kFit = (216 * 1024 / kWarpsSm - kQueries) / (32 * D), kStages = kFit < 3 ? 3 : kFit > 6 ? 6 : kFit;
    static constexpr int kOwn = kStages * 32 * D + kQueries;     // a warp's shared memory
    static constexpr int kMostWarpsOfRuns = kSms * kWarpsSm;
};

__device__ __forceinline__ void cp_async_16_zfill(uint32_t dst, const void *src, bool there)
{
    asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(there ? 16 : 0) : "memory");
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

// Four E4M3 codes as two pairs of binary16, exactly, the lowest byte first.
__device__ __forceinline__ void decode4(uint32_t codes, uint32_t &lo, uint32_t &hi)
{
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(codes));
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
    float l[NT][2], m[NT][2];
    uint32_t nan;                  // of a lane, not 0: there are NaN values that some rows do not see
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
    const int page = p.table[block >> per_page];
    if (page < 0 || page >= p.pages) {
        atomicOr(&g_paged_error, kErrIndex);
        return f;
    }
    f.block = (static_cast<int64_t>(page) << per_page) + (block & ((1 << per_page) - 1));
    f.ks = p.ks[f.block * p.Hkv];   // (no read-only loads: an append that this launch overlapped with may have written them)
    f.vs = p.vs[f.block * p.Hkv];
    return f;
}

// A block to a stage: 16 rows of keys, then 16 of values, D bytes each. Whole rows by
// neighbouring lanes; 16-byte piece c of row r lies at piece c ^ (r % 8) of it (D = 128) or c ^ (r / 2 % 4)
// (D = 64), so that the lanes that read together, below, meet all banks.
template <int D>
__device__ __forceinline__ uint32_t piece_at(int row, int c)
{
    return static_cast<uint32_t>(row * D + ((D == 128 ? c ^ (row & 7) : c ^ (row >> 1 & 3)) * 16));
}
template <int D>
__device__ __forceinline__ void copy_block(const Place &p, int64_t block, uint32_t stage, int lane)
{
    constexpr int kPieces = D / 16, kRows = 32 / kPieces;   // pieces of a row, rows at a time
    const bool there = block >= 0;
    const int64_t at = (there ? block : 0) * kBlock * p.token + lane / kPieces * p.token + lane % kPieces * 16;
#pragma unroll
    for (int i = 0; i < 16 / kRows; ++i) {
        const uint32_t to = stage + piece_at<D>(lane / kPieces + i * kRows, lane % kPieces);
        cp_async_16_zfill(to, p.k + at + i * kRows * p.token, there);
        cp_async_16_zfill(to + 16 * D, p.v + at + i * kRows * p.token, there);
    }
}

// The top bit of each byte that is a NaN code.
__device__ __forceinline__ uint32_t nan_bytes(uint32_t codes) { return ((codes & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u; }

// S^T of a block of 16 keys. q: columns' rows as the B operand.
template <int D, int NT, typename Q>
__device__ __forceinline__ void scores(float (&s)[NT][4], const Q &q, uint32_t stage, int lane)
{
    float odd[NT][4] = {};   // two chains of products
#pragma unroll
    for (int n = 0; n < NT; ++n) s[n][0] = s[n][1] = s[n][2] = s[n][3] = 0.0f;
#pragma unroll
    for (int i = 0; i < D / 64; ++i) {
        // keys gid and gid + 8, 16 dimensions from 16 (D / 64 t + i) on
        const uint4 lo = lds128(stage + piece_at<D>(lane / 4, D / 64 * (lane % 4) + i)), hi = lds128(stage + piece_at<D>(lane / 4 + 8, D / 64 * (lane % 4) + i));
        const uint32_t low[4] = {lo.x, lo.y, lo.z, lo.w}, high[4] = {hi.x, hi.y, hi.z, hi.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            uint32_t a0, a1, a2, a3;
            decode4(low[j], a0, a2);
            decode4(high[j], a1, a3);
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                const uint2 b = q.at(n, 4 * i + j);
                mma_16816(j & 1 ? odd[n] : s[n], a0, a1, a2, a3, b.x, b.y);
            }
        }
    }
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
        for (int e = 0; e < 4; ++e) s[n][e] += odd[n][e];
    }
}

// What S is multiplied by: never 0, which a score of -inf (a key that is not seen) would turn into
// NaN; the least normal number makes 0 of any finite one.
__device__ __forceinline__ float factor(float c, float ks) { return fmaxf(c * ks, 1.17549435e-38f); }

// The block's share of the sums, from its S^T. lv: log2 of its values' scale.
template <int D, int NT>
__device__ __forceinline__ void add_block(Part<D, NT> &r, float (&s)[NT][4], const float (&c)[NT][2], const int (&seen)[NT][2],
                                          uint32_t stage, int lane, int key0, int len, int first_seen, float ks, float lv)
{
    const int gid = lane / 4, t = lane % 4;
    const bool zero = lv <= kLeastLog, masked = key0 + kBlock > first_seen || zero;   // some rows do not see all of it, or its values are 0
    uint32_t v[4][D / 32];
#pragma unroll
    for (int i = 0; i < 4; ++i) {   // value of key 2 t + i % 2 + 8 (i / 2), dimensions gid D / 8 on
        const int row = 2 * t + i % 2 + 8 * (i / 2);
        if constexpr (D == 128) {
            const uint4 x = lds128(stage + 16 * D + piece_at<D>(row, gid));
            v[i][0] = x.x, v[i][1] = x.y, v[i][2] = x.z, v[i][3] = x.w;
        } else {
            const uint2 x = lds64(stage + 16 * D + piece_at<D>(row, gid / 2) + gid % 2 * 8);
            v[i][0] = x.x, v[i][1] = x.y;
        }
    }
    if (masked) {
#pragma unroll
        for (int n = 0; n < NT; ++n) {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (key0 + gid + (e >> 1) * 8 >= seen[n][e & 1]) s[n][e] = -INFINITY;   // (c is positive)
        }
        // Values behind the last token are cleared, whatever lies there; of a scale of 0, all but NaN, which
        // stays NaN. Of keys that not every row sees, NaN is cleared (0 x NaN is NaN), and the rows that see it
        // get it when they are written.
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int key = key0 + 2 * t + i % 2 + 8 * (i / 2);
            const uint32_t there = key < len ? ~0u : 0u, some = key >= first_seen ? ~0u : 0u;
#pragma unroll
            for (int w = 0; w < D / 32; ++w) {
                const uint32_t nan = nan_bytes(v[i][w]) & there, bytes = (nan >> 7) * 0xffu;
                v[i][w] &= (zero ? bytes : there) & ~(bytes & some);
                r.nan |= nan & some;
            }
        }
    }
    // u = z + log2 sv - m of the numerator's terms; the denominator's are u - log2 sv
    float u[NT][4];
    bool grow = false;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        const float ck[2] = {factor(c[n][0], ks), factor(c[n][1], ks)}, off[2] = {lv - r.m[n][0], lv - r.m[n][1]};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            u[n][e] = fmaf(s[n][e], ck[e & 1], off[e & 1]);
            grow |= u[n][e] > kSlack;
        }
    }
    if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
        for (int n = 0; n < NT; ++n) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const float ck = factor(c[n][e], ks);
                float top = fmaxf(s[n][e], s[n][e + 2]);
#pragma unroll
                for (int o = 4; o < 32; o *= 2) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
                const float m = fmaxf(r.m[n][e], fmaf(top, ck, lv) - kLift), by = exp2_fast(r.m[n][e] - m);
                r.m[n][e] = m;
                r.l[n][e] *= by;
                u[n][e] = fmaf(s[n][e], ck, lv - m);
                u[n][e + 2] = fmaf(s[n][e + 2], ck, lv - m);
#pragma unroll
                for (int j = 0; j < D / 16; ++j) {
                    r.o[n][j][e] *= by;
                    r.o[n][j][e + 2] *= by;
                }
            }
        }
    }
    uint32_t p[NT][2], rest[NT][2];   // the terms, and what their rounding left
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
        for (int e = 0; e < 4; ++e) r.l[n][e & 1] += exp2_fast(u[n][e] - lv);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const float a = exp2_fast(u[n][2 * i]), b = exp2_fast(u[n][2 * i + 1]);
            const __half2 h = __floats2half2_rn(a, b);
            p[n][i] = transpose8x8(*reinterpret_cast<const uint32_t *>(&h));
            rest[n][i] = transpose8x8(half2_bits(a - __low2float(h), b - __high2float(h)));
        }
    }
#pragma unroll
    for (int w = 0; w < D / 32; ++w) {
        // dimensions gid D / 8 + 4 w + 0, 1 (tile 2 w) and + 2, 3 (tile 2 w + 1), two keys a register
        const uint32_t lo01 = __byte_perm(v[0][w], v[1][w], 0x5140), lo23 = __byte_perm(v[0][w], v[1][w], 0x7362);
        const uint32_t hi01 = __byte_perm(v[2][w], v[3][w], 0x5140), hi23 = __byte_perm(v[2][w], v[3][w], 0x7362);
        uint32_t a0, a1, a2, a3, b0, b1, b2, b3;
        decode4(lo01, a0, a1);
        decode4(hi01, a2, a3);
        decode4(lo23, b0, b1);
        decode4(hi23, b2, b3);
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            mma_16816(r.o[n][2 * w], a0, a1, a2, a3, p[n][0], p[n][1]);
            mma_16816(r.o[n][2 * w + 1], b0, b1, b2, b3, p[n][0], p[n][1]);
            mma_16816(r.o[n][2 * w], a0, a1, a2, a3, rest[n][0], rest[n][1]);
            mma_16816(r.o[n][2 * w + 1], b0, b1, b2, b3, rest[n][0], rest[n][1]);
        }
    }
}

// A warp's way through `count` blocks from `first` on: pages and scales are looked up a batch
// ahead, copies run kStages - 1 blocks ahead.
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
        return find(p, first + i, i < count);
    }
    __device__ __forceinline__ Walk(const Place &place, uint32_t ring_at, int lane_, int first_, int count_)
        : p(place), ring(ring_at), lane(lane_), first(first_), count(count_)
    {
        ahead = batch(0);
        if (count > kBatch) next = batch(1);
    }
    __device__ __forceinline__ void issue(uint32_t stage)
    {
        if (issued < count) {
            if (issued % kBatch == 0 && issued > 0) {
                ahead = next;
                if ((issued / kBatch + 1) * kBatch < count) next = batch(issued / kBatch + 1);
            }
            copy_block<D>(p, __shfl_sync(0xffffffffu, ahead.block, issued % kBatch), stage, lane);
        }
        ++issued;
        cp_async_commit();
    }
    // Block j's softmax and values beside block j + 1's scores, whose instructions do not wait for
    // one another. (One loop, so that its code is there once.)
    template <typename Q>
    __device__ __forceinline__ void add(Part<D, NT> &r, const Q &q, const float (&c)[NT][2], const int (&seen)[NT][2])
    {
        constexpr uint32_t kBytes = Ring<D>::kBytes, kEnd = kStages * kBytes;
        uint32_t to = 0, now = 0;   // stages of the block that is copied next, and of block j
        float s[NT][4];
#pragma unroll 1
        for (int j = 1 - kStages; j < count; ++j) {
            const uint32_t then = now + kBytes == kEnd || j < 0 ? 0 : now + kBytes;
            if (j >= -1) cp_async_wait<kStages - 3>();
            __syncwarp();   // all lanes' copies have landed, and all have read the stage that is copied to next
            if (j >= 0 && j % kBatch == 0) {   // copies are less than a batch ahead
                ks32 = ahead.ks;
                lv32 = fmaxf(log2f(ahead.vs), kLeastLog);
            }
            issue(ring + to);
            to = to + kBytes == kEnd ? 0 : to + kBytes;
            float next_s[NT][4] = {};
            if (j >= -1 && j + 1 < count) scores<D, NT>(next_s, q, ring + then, lane);
            if (j >= 0) {
                const float ks = __shfl_sync(0xffffffffu, ks32, j % kBatch), lv = __shfl_sync(0xffffffffu, lv32, j % kBatch);
                add_block<D, NT>(r, s, c, seen, ring + now, lane, (first + j) * kBlock, p.len, p.first_seen, ks, lv);
                now = then;
            }
#pragma unroll
            for (int n = 0; n < NT; ++n) {
#pragma unroll
                for (int e = 0; e < 4; ++e) s[n][e] = next_s[n][e];
            }
        }
        cp_async_wait<0>();
    }
};

// A part outside registers: 8 NT rows of D floats of O, then l, m and whether there are NaN
// values that not every row sees.
template <int D, int NT>
constexpr int slot_floats() { return 8 * NT * (D + 4); }

// A block is gone through once for each pair of a key head and a group of 8 NT of its query rows, by a
// warp each. The work is cut into units: a block of an item, an item being a request and up to 8 of its
// pairs, in that order. A CTA takes a run of units, its warps a pair each, so that the rows
// of a block, which lie side by side for all heads, are read together (reads alone: 7.0 TB/s;
// one head at a time by all warps of a CTA 6.2). All runs are of equal length, whatever the requests'
// lengths; so that a run with more items does not end later, an item counts kStartUnits more,
// before its blocks. What a run has of an item that is not all of it is a part (an empty one, where
// it has none of the blocks), which paged_join_kernel joins with the others'.
struct Cut {
    int b, item;          // item of the request
    int64_t at;           // units before it in its item
    int64_t left;         // units of the run
    int64_t from, units;  // where the run starts; all units
};

// a / b of numbers that are not negative: most fit 32 bits, where it takes a tenth of the time.
__device__ __forceinline__ int64_t quotient(int64_t a, int64_t b)
{
    return (a | b) >> 32 ? a / b : static_cast<int64_t>(static_cast<uint32_t>(a) / static_cast<uint32_t>(b));
}

__device__ __forceinline__ int len_of(const PagedArgs &g, int b) { return static_cast<int>(min(static_cast<int64_t>(max(g.lens[b], 0)), g.max_len)); }

// Units of an item of a request.
__device__ __forceinline__ int units_of(const PagedArgs &g, int b)
{
    const int len = len_of(g, b);
    return len > 0 ? (len + kBlock - 1) / kBlock + kStartUnits : 0;
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
    if (lane == 31) sums[warp] = upto;
    __syncthreads();
    int64_t before = upto - v;
    all = 0;
    for (int i = 0; i < warps; ++i) {
        if (i < warp) before += sums[i];
        all += sums[i];
    }
    __syncthreads();
    return before;
}

// The c-th run. items: of a request. starts: where not null, gets the units (of one item) before
// each request, and of all.
__device__ __forceinline__ Cut cut_of(const PagedArgs &g, int c, int ctas, int items, int64_t *sums, Cut *shared, int64_t *starts)
{
    const int tid = threadIdx.x, step = static_cast<int>(blockDim.x);
    int64_t total = 0, all, mine = 0, before = 0;
    for (int b0 = 0; b0 < g.B; b0 += step) {
        mine = b0 + tid < g.B ? units_of(g, b0 + tid) : 0;
        before = scan_before(mine, sums, all);
        if (starts && b0 + tid < g.B) starts[b0 + tid] = total + before;
        total += all;
    }
    if (starts && tid == 0) starts[g.B] = total;
    const int64_t units = total * items, q = quotient(units, ctas), rest = units - q * ctas;
    const int64_t from = q * c + min(static_cast<int64_t>(c), rest), to = from + q + (c < rest ? 1 : 0);
    if (tid == 0 && from == to) *shared = Cut{0, 0, 0, 0, from, units};   // an empty run; else one thread finds its start
    if (g.B > step) total = 0;
    for (int b0 = 0; b0 < g.B; b0 += step) {
        int64_t base = 0;
        if (g.B > step) {
            mine = b0 + tid < g.B ? units_of(g, b0 + tid) : 0;
            before = scan_before(mine, sums, all);
            base = total;
            total += all;
        }
        const int64_t start = (base + before) * items;
        if (start <= from && from < start + mine * items && from < to) {
            const int64_t item = quotient(from - start, mine);
            *shared = Cut{b0 + tid, static_cast<int>(item), from - start - item * mine, to - from, from, units};
        }
    }
    __syncthreads();
    return *shared;
}

// q's operands of a warp: in registers, or, where they are too many, in its shared memory
// behind the ring, each lane its own.
template <int D, int NT>
struct Queries {
    uint32_t base;   // of this lane
    __device__ __forceinline__ uint2 at(int n, int k) const { return lds64(base + (n * (D / 16) + k) * 256); }
    __device__ __forceinline__ void set(int n, int k, uint2 v) { asm volatile("st.shared.v2.u32 [%0], {%1,%2};" ::"r"(base + (n * (D / 16) + k) * 256), "r"(v.x), "r"(v.y) : "memory"); }
};
template <int D>
struct Queries<D, 1> {
    uint32_t base;
    uint2 v[D / 16];
    __device__ __forceinline__ uint2 at(int, int k) const { return v[k]; }
    __device__ __forceinline__ void set(int, int k, uint2 x) { v[k] = x; }
};

// Row tile n of the item's q, as B operands: lane (gid, t) has row gid, D / 4 elements from t D / 4 on.
template <int D>
__device__ __forceinline__ void fetch_q(uint32_t (&words)[D / 8], const uint16_t *q, bool live, int t)
{
#pragma unroll
    for (int i = 0; i < D / 64; ++i) {
#pragma unroll
        for (int w = 0; w < 2; ++w) {
            uint4 x = make_uint4(0, 0, 0, 0);
            if (live) x = *(reinterpret_cast<const uint4 *>(q + D / 4 * t + 16 * i) + w);
            words[8 * i + 4 * w] = x.x, words[8 * i + 4 * w + 1] = x.y, words[8 * i + 4 * w + 2] = x.z, words[8 * i + 4 * w + 3] = x.w;
        }
    }
}

// As binary16. Returns what the row was divided by.
template <int D, int NT>
__device__ __forceinline__ float set_q(Queries<D, NT> &s, int n, uint32_t (&words)[D / 8], int type)
{
    float back = 1.0f;
    if (type == QMV_BF16) {
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
    for (int k = 0; k < D / 16; ++k) s.set(n, k, make_uint2(words[2 * k], words[2 * k + 1]));
    return back;
}

// Four outputs of a row whose request has NaN among the values of keys that earlier rows do not
// see: NaN where the row sees one.
__device__ __noinline__ float4 with_nan(const PagedArgs &g, int b, int h, int len, int token, int d, int D, float4 o)
{
    const int per_page = 31 - __clz(g.page);
    for (int key = max(0, len - g.T + 1); key < len - g.T + 1 + token; ++key) {
        const int page = g.table[static_cast<int64_t>(b) * g.table_pages + (key >> per_page)];
        if (page < 0 || page >= g.n_pages) continue;
        const int64_t place = (static_cast<int64_t>(page) << per_page) + (key & (g.page - 1));
        const uint32_t nan = nan_bytes(*reinterpret_cast<const uint32_t *>(static_cast<const uint8_t *>(g.v) + (place * g.Hkv + h) * D + d));
        o = make_float4(nan & 0x80u ? NAN : o.x, nan & 0x8000u ? NAN : o.y, nan & 0x800000u ? NAN : o.z, nan & 0x80000000u ? NAN : o.w);
    }
    return o;
}

template <int D, int NT>
__device__ __forceinline__ void put(const Part<D, NT> &r, float *slot, int lane)
{
    const int gid = lane / 4, t = lane % 4;
    const bool nan = __any_sync(0xffffffffu, r.nan != 0);
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            float l = r.l[n][e];
#pragma unroll
            for (int o = 4; o < 32; o *= 2) l += __shfl_xor_sync(0xffffffffu, l, o);
            float *row = slot + (8 * n + 2 * t + e) * (D + 4);
#pragma unroll
            for (int j = 0; j < D / 32; ++j)
                reinterpret_cast<float4 *>(row + gid * (D / 8))[j] = make_float4(r.o[n][2 * j][e], r.o[n][2 * j][e + 2], r.o[n][2 * j + 1][e], r.o[n][2 * j + 1][e + 2]);
            if (gid == 0) *reinterpret_cast<float4 *>(row + D) = make_float4(l, r.m[n][e], nan ? 1.0f : 0.0f, 0.0f);
        }
    }
}

// Adds a part that `put` has left in a slot, by the same warp.
template <int D, int NT>
__device__ __forceinline__ void add_put(Part<D, NT> &r, const float *slot, int lane)
{
    const int gid = lane / 4, t = lane % 4;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const float *row = slot + (8 * n + 2 * t + e) * (D + 4);
            const float4 st = *reinterpret_cast<const float4 *>(row + D);
            const float m = fmaxf(r.m[n][e], st.y), by = exp2_fast(r.m[n][e] - m), weight = exp2_fast(st.y - m);
            r.m[n][e] = m;
            r.l[n][e] = r.l[n][e] * by + (gid == 0 ? st.x * weight : 0.0f);
            if (st.z != 0.0f) r.nan = 1;
#pragma unroll
            for (int j = 0; j < D / 32; ++j) {
                const float4 x = reinterpret_cast<const float4 *>(row + gid * (D / 8))[j];
                r.o[n][2 * j][e] = r.o[n][2 * j][e] * by + x.x * weight;
                r.o[n][2 * j][e + 2] = r.o[n][2 * j][e + 2] * by + x.y * weight;
                r.o[n][2 * j + 1][e] = r.o[n][2 * j + 1][e] * by + x.z * weight;
                r.o[n][2 * j + 1][e + 2] = r.o[n][2 * j + 1][e + 2] * by + x.w * weight;
            }
        }
    }
}

// Adds those of an item's parts that are in the slot, and leaves all in it, if more follow.
template <int D, int NT>
__device__ __forceinline__ void fold(Part<D, NT> &r, float *slot, int lane, bool before, bool after)
{
    if (before) add_put<D, NT>(r, slot, lane);
    __syncwarp();   // all have read the slot
    if (after) put<D, NT>(r, slot, lane);
    __syncwarp();
}
template <int D, int NT>
__device__ __noinline__ Part<D, NT> fold_called(Part<D, NT> r, float *slot, int lane, bool before, bool after)
{
    fold<D, NT>(r, slot, lane, before, after);
    return r;
}

// Four outputs of row `row` of a key head, from their sums over V and the denominator l.
__device__ __forceinline__ void write_row(const PagedArgs &g, int b, int h, int len, int row, int G, int d, int D, float l, bool nan, float4 o)
{
    const bool none = len - g.T + 1 + row / G <= 0;
    const float by = 1.0f / l;
    float4 y = none ? make_float4(0.0f, 0.0f, 0.0f, 0.0f) : make_float4(o.x * by, o.y * by, o.z * by, o.w * by);
    if (nan && !none) y = with_nan(g, b, h, len, row / G, d, D, y);
    const int64_t at = (static_cast<int64_t>(b) * g.T + row / G) * g.Hq + static_cast<int64_t>(h) * G + row % G;
    *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(g.out) + at * D + d) =
        g.type == QMV_F16 ? make_uint2(pack2<__half>(y.x, y.y), pack2<__half>(y.z, y.w)) : make_uint2(pack2<__nv_bfloat16>(y.x, y.y), pack2<__nv_bfloat16>(y.z, y.w));
}

// The workspace: two slots for each warp of a run, [run][first or last][warp]; then the units
// before each request, and of all.
template <int D, int NT>
__device__ __forceinline__ float *slot_of(const PagedArgs &g, int run, bool first, int warps, int warp)
{
    return static_cast<float *>(g.workspace) + ((2 * static_cast<int64_t>(run) + (first ? 0 : 1)) * warps + warp) * slot_floats<D, NT>();
}
template <int D, int NT>
__device__ __forceinline__ int64_t *starts_of(const PagedArgs &g)
{
    return reinterpret_cast<int64_t *>(static_cast<float *>(g.workspace) + 2ll * Shape<D, NT>::kMostWarpsOfRuns * slot_floats<D, NT>());
}

// A warp's part of an item: `count` blocks from block `at` on of request b, against 8 NT rows of
// key head h from row0 on.
template <int D, int NT>
__device__ __forceinline__ void add_item(Part<D, NT> &part, const PagedArgs &g, Queries<D, NT> &q, uint32_t ring, int b, int h, int row0,
                                 int len, int at, int count, int lane)
{
    const int gid = lane / 4, t = lane % 4, G = g.Hq / g.Hkv, rows = g.T * G;
    int seen[NT][2];
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
    auto row_at = [&](int r) { return ((static_cast<int64_t>(b) * g.T + r / G) * g.Hq + static_cast<int64_t>(h) * G + r % G) * D; };
    uint32_t words[D / 8];   // the first row tile's, on their way while the pages are looked up
    fetch_q<D>(words, static_cast<const uint16_t *>(g.q) + (row0 + gid < rows ? row_at(row0 + gid) : 0), row0 + gid < rows, t);
    Walk<D, NT> walk(p, ring, lane, at, count);
    float c[NT][2];
    part.nan = 0;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        const float back = set_q<D, NT>(q, n, words, g.type);
        const int next = row0 + 8 * (n + 1) + gid;
        if (n + 1 < NT) fetch_q<D>(words, static_cast<const uint16_t *>(g.q) + (next < rows ? row_at(next) : 0), next < rows, t);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int r = row0 + 8 * n + 2 * t + e;
            c[n][e] = g.scale * kLog2e * __shfl_sync(0xffffffffu, back, (2 * t + e) * 4);
            seen[n][e] = r < rows ? p.first_seen + r / G : 0;
            part.l[n][e] = 0.0f;
            part.m[n][e] = kLowest;
        }
#pragma unroll
        for (int j = 0; j < D / 16; ++j) part.o[n][j][0] = part.o[n][j][1] = part.o[n][j][2] = part.o[n][j][3] = 0.0f;
    }
    walk.add(part, q, c, seen);
}

// A run a CTA. row_groups: groups of 8 NT query rows. kLong: of an item, a run can have more than kFold blocks.
template <int D, int NT, bool kLong>
__global__ void __launch_bounds__(32 * kMostWarps, Shape<D, NT>::kWarpsSm / kMostWarps) paged_kernel(const __grid_constant__ PagedArgs g, int row_groups)
{
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ int64_t sums[kMostWarps];
    __shared__ Cut shared_cut;
    const int lane = threadIdx.x & 31, warp = threadIdx.x / 32, warps = blockDim.x / 32, gid = lane / 4, t = lane % 4;
    const int G = g.Hq / g.Hkv, rows = g.T * G, pairs = g.Hkv * row_groups, items = (pairs + warps - 1) / warps;
    const uint32_t my_ring = smem_addr(smem) + warp * Shape<D, NT>::kOwn;
    grid_launch_dependents();
    grid_dependency_wait();
    Cut cut = cut_of(g, static_cast<int>(blockIdx.x), static_cast<int>(gridDim.x), items, sums, &shared_cut,
                     blockIdx.x == 0 ? starts_of<D, NT>(g) : nullptr);
    // rows of requests without keys are no units
    for (int i = static_cast<int>(blockIdx.x); i < g.B; i += static_cast<int>(gridDim.x)) {
        if (g.lens[i] > g.max_len && threadIdx.x == 0) atomicOr(&g_paged_error, kErrIndex);
        if (len_of(g, i) > 0) continue;
        uint4 *out = reinterpret_cast<uint4 *>(static_cast<uint16_t *>(g.out) + static_cast<int64_t>(i) * g.T * g.Hq * D);
        for (int64_t j = threadIdx.x; j < static_cast<int64_t>(g.T) * g.Hq * D / 8; j += blockDim.x) out[j] = make_uint4(0, 0, 0, 0);
    }
    Part<D, NT> part{};
    Queries<D, NT> q;
    q.base = my_ring + Shape<D, NT>::kStages * Ring<D>::kBytes + lane * 8;
    for (bool first = true; cut.left > 0; first = false) {
        const int b = cut.b, pair = cut.item * warps + warp, h = pair / row_groups, row0 = pair % row_groups * 8 * NT;
        const int len = len_of(g, b), units = units_of(g, b), taken = static_cast<int>(min(units - cut.at, cut.left));
        const int at = max(static_cast<int>(cut.at) - kStartUnits, 0), count = max(static_cast<int>(cut.at) + taken - kStartUnits, 0) - at;
        if (pair < pairs) {
            float *slot = slot_of<D, NT>(g, static_cast<int>(blockIdx.x), first, warps, warp);
            if constexpr (kLong) {
#pragma unroll 1
                for (int done = 0;;) {
                    const int n = min(count - done, kFold);
                    add_item<D, NT>(part, g, q, my_ring, b, h, row0, len, at + done, n, lane);
                    // Heads of 64 have 128 registers a thread, of which the loop is left more where this is called: 64 requests of
                    // 2000 keys, 16 rows, 48 us for 53. (With 128, and 5 rows, 24 requests of up to 131072 keys 532 called, 517 not.)
                    if constexpr (D == 64) {
                        if (count > kFold) part = fold_called<D, NT>(part, slot, lane, done > 0, done + n < count);
                    } else {
                        fold<D, NT>(part, slot, lane, done > 0, done + n < count);
                    }
                    if ((done += n) == count) break;
                }
            } else {
                add_item<D, NT>(part, g, q, my_ring, b, h, row0, len, at, count, lane);
            }
            // the output, or a part
            const bool whole = taken == units, nan = __any_sync(0xffffffffu, part.nan != 0);
#pragma unroll
            for (int n = 0; n < NT; ++n) {
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float l = part.l[n][e];
#pragma unroll
                    for (int o = 4; o < 32; o *= 2) l += __shfl_xor_sync(0xffffffffu, l, o);
                    const int r = 8 * n + 2 * t + e;
                    if (row0 + r >= rows) continue;
#pragma unroll
                    for (int j = 0; j < D / 32; ++j) {
                        const float4 y = make_float4(part.o[n][2 * j][e], part.o[n][2 * j][e + 2], part.o[n][2 * j + 1][e], part.o[n][2 * j + 1][e + 2]);
                        if (whole) {
                            write_row(g, b, h, len, row0 + r, G, gid * (D / 8) + 4 * j, D, l, nan, y);
                        } else {
                            reinterpret_cast<float4 *>(slot + r * (D + 4) + gid * (D / 8))[j] = y;
                        }
                    }
                    if (!whole && gid == 0) *reinterpret_cast<float4 *>(slot + r * (D + 4) + D) = make_float4(l, part.m[n][e], nan ? 1.0f : 0.0f, 0.0f);
                }
            }
        }
        cut.left -= taken;
        cut.at = 0;
        if (++cut.item == items && cut.left > 0) {
            cut.item = 0;
            do {
                ++cut.b;
            } while (units_of(g, cut.b) == 0);   // ends: there are units left
        }
    }
}

// The rows of which runs have parts. A CTA has blockDim / 32 / share rows of all B * pairs * n of them
// (n: rows of a group), `share` warps a row, each every share-th part.
template <int D, int NT>
__global__ void __launch_bounds__(1024) paged_join_kernel(const __grid_constant__ PagedArgs g, int row_groups, int warps, int ctas, int share, int n)
{
    constexpr int kD4 = D / 4;
    __shared__ float4 sum_o[32][kD4];
    __shared__ float4 sum_l[32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x / 32, mine = warp % share;
    const uint32_t pairs = static_cast<uint32_t>(g.Hkv * row_groups), task = blockIdx.x * (blockDim.x / 32 / share) + warp / share;
    const uint32_t of_row = task / static_cast<uint32_t>(n), b = of_row / pairs, pair = of_row - b * pairs;
    const int r = static_cast<int>(task - of_row * n), row = static_cast<int>(pair) % row_groups * 8 * NT + r;
    const int item = static_cast<int>(pair) / warps, items = (static_cast<int>(pairs) + warps - 1) / warps;
    grid_launch_dependents();
    grid_dependency_wait();   // in every CTA: this launch ends after the one before it
    const bool live = b < static_cast<uint32_t>(g.B) && row < g.T * (g.Hq / g.Hkv);
    int parts = 0;
    const float *part0 = nullptr;   // this row's part of the item's first run; the further ones are `stride` apart
    int64_t stride = 0, skip = 0;   // skip: from the slots for a run's first piece to those for its last
    if (live) {
        const int64_t *starts = starts_of<D, NT>(g);
        const int64_t before = starts[b], blocks = starts[b + 1] - before, units = starts[g.B] * items;
        const int64_t item0 = before * items + blocks * item, q = quotient(units, ctas), long_ones = units - q * ctas;
        // of runs of q + 1 units, long_ones of them, and then of q: that of a unit, and where it starts
        auto run_of = [&](int64_t unit, int64_t &start) {
            const bool l = unit < long_ones * (q + 1);
            const int64_t rest = l ? unit : unit - long_ones * (q + 1), each = l ? q + 1 : q, run = quotient(rest, each);
            start = unit - (rest - run * each);
            return static_cast<int>(run + (l ? 0 : long_ones));
        };
        if (blocks > 0) {
            int64_t start, end;
            const int run0 = run_of(item0, start);
            parts = run_of(item0 + blocks - 1, end) - run0 + 1;
            skip = static_cast<int64_t>(warps) * slot_floats<D, NT>();
            stride = 2 * skip;
            part0 = slot_of<D, NT>(g, run0, true, warps, static_cast<int>(pair) % warps) + r * (D + 4);
            if (start == item0) skip = 0;   // the run starts with the item
        }
    }
    float l = 0.0f, m = kLowest, nan = 0.0f;
    float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    // 32 parts at a time: their statistics a lane a part, then their weights to all lanes
    for (int i0 = mine; parts > 1 && i0 < parts; i0 += 32 * share) {
        const int i = i0 + lane * share, count = min(32, (parts - i0 + share - 1) / share);
        float4 st = make_float4(0.0f, kLowest, 0.0f, 0.0f);
        if (i < parts) st = *reinterpret_cast<const float4 *>(part0 + i * stride + (i > 0 ? 0 : skip) + D);
        float top = fmaxf(m, st.y);
#pragma unroll
        for (int x = 16; x > 0; x /= 2) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
        const float by = exp2_fast(m - top), weight = exp2_fast(st.y - top);
        l = l * by + st.x * weight;   // of this lane's parts; by is 1 but for more than 32
        o = make_float4(o.x * by, o.y * by, o.z * by, o.w * by);
        m = top;
        nan = fmaxf(nan, st.z);
        const float *x_at = part0 + i0 * stride + 4 * (lane % kD4);
        int64_t skipped = i0 > 0 ? 0 : skip;
#pragma unroll 4
        for (int k = 0; k < count; ++k) {
            const float4 x = *reinterpret_cast<const float4 *>(x_at + skipped);
            const float w = __shfl_sync(0xffffffffu, weight, k);
            x_at += share * stride;
            skipped = 0;
            o = make_float4(o.x + x.x * w, o.y + x.y * w, o.z + x.z * w, o.w + x.w * w);
        }
    }
#pragma unroll
    for (int x = 16; x > 0; x /= 2) {
        l += __shfl_xor_sync(0xffffffffu, l, x);
        nan = fmaxf(nan, __shfl_xor_sync(0xffffffffu, nan, x));
    }
    if (share > 1) {
        if (lane < kD4) sum_o[warp][lane] = o;
        if (lane == 0) sum_l[warp] = make_float4(l, m, nan, 0.0f);
        __syncthreads();
        if (mine > 0) return;
        for (int w = 1; w < share; ++w) m = fmaxf(m, sum_l[warp + w].y);
        l = 0.0f;
        o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 1
        for (int w = 0; w < share; ++w) {
            const float4 st = sum_l[warp + w], x = sum_o[warp + w][lane % kD4];
            const float by = exp2_fast(st.y - m);
            l += st.x * by;
            nan = fmaxf(nan, st.z);
            o = make_float4(o.x + x.x * by, o.y + x.y * by, o.z + x.z * by, o.w + x.w * by);
        }
    }
    if (parts > 1 && lane < kD4)
        write_row(g, static_cast<int>(b), static_cast<int>(pair) / row_groups, static_cast<int>(min(static_cast<int64_t>(g.lens[b]), g.max_len)), row,
                  g.Hq / g.Hkv, 4 * lane, D, l, nan != 0.0f, o);
}

// Few and short requests: a cluster an item, its CTAs equal shares of the item's blocks, joined in their
// shared memory. One launch, and no search for where a run begins.
template <int D, int NT>
__global__ void __launch_bounds__(32 * kMostWarps) paged_cluster_kernel(const __grid_constant__ PagedArgs g, int row_groups)
{
    extern __shared__ __align__(128) uint8_t smem[];
    cg::cluster_group cluster = cg::this_cluster();
    const int R = static_cast<int>(cluster.num_blocks()), rank = static_cast<int>(cluster.block_rank());
    const int lane = threadIdx.x & 31, warp = threadIdx.x / 32, warps = blockDim.x / 32;
    const int G = g.Hq / g.Hkv, rows = g.T * G, pairs = g.Hkv * row_groups, items = (pairs + warps - 1) / warps;
    const int of = static_cast<int>(blockIdx.x) / R, b = of / items, pair = of % items * warps + warp;
    const int h = pair / row_groups, row0 = pair % row_groups * 8 * NT;
    uint8_t *own = smem + warp * Shape<D, NT>::kOwn;
    grid_launch_dependents();
    grid_dependency_wait();
    if (g.lens[b] > g.max_len && rank == 0 && threadIdx.x == 0) atomicOr(&g_paged_error, kErrIndex);
    const int len = len_of(g, b), blocks = (len + kBlock - 1) / kBlock;
    const int at = blocks * rank / R, count = blocks * (rank + 1) / R - at;
    float *slot = reinterpret_cast<float *>(own);   // over the ring
    if (pair < pairs) {
        Part<D, NT> part{};
        Queries<D, NT> q;
        q.base = smem_addr(own) + Shape<D, NT>::kStages * Ring<D>::kBytes + lane * 8;
        add_item<D, NT>(part, g, q, smem_addr(own), b, h, row0, len, at, count, lane);
        __syncwarp();
        put<D, NT>(part, slot, lane);
    }
    cluster.sync();
    constexpr int kD4 = D / 4;
    // a row a warp: rows rank, rank + R, .. of the warp's pair
    for (int r = rank; pair < pairs && r < 8 * NT && row0 + r < rows; r += R) {
        const float *row = slot + r * (D + 4);
        const float4 st = lane < R ? *reinterpret_cast<const float4 *>(cluster.map_shared_rank(const_cast<float *>(row) + D, lane)) : make_float4(0.0f, kLowest, 0.0f, 0.0f);
        float top = st.y;
#pragma unroll
        for (int x = 16; x > 0; x /= 2) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
        const float weight = exp2_fast(st.y - top);
        float l = st.x * weight, nan = st.z;
#pragma unroll
        for (int x = 16; x > 0; x /= 2) {
            l += __shfl_xor_sync(0xffffffffu, l, x);
            nan = fmaxf(nan, __shfl_xor_sync(0xffffffffu, nan, x));
        }
        float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 8
        for (int k = 0; k < R; ++k) {
            const float4 x = reinterpret_cast<const float4 *>(cluster.map_shared_rank(const_cast<float *>(row), k))[lane % kD4];
            const float w = __shfl_sync(0xffffffffu, weight, k);
            o = make_float4(o.x + x.x * w, o.y + x.y * w, o.z + x.z * w, o.w + x.w * w);
        }
        if (lane < kD4) write_row(g, b, h, len, row0 + r, G, 4 * lane, D, l, nan != 0.0f, o);
    }
    cluster.sync();   // nobody leaves while others read its memory
}

// CTAs of a cluster for each of `items` of up to `blocks` blocks, or 0. (16 to a cluster only for four items: more
// such clusters wait for one another's places, 9.7 us for 15.6 with 8 requests.)
int cluster_for(int64_t items, int64_t blocks)
{
    const int R = items <= 4 ? 16 : 8;
    return items * R <= 128 && blocks <= kClusterBlocks * R ? R : 0;
}

template <int D, int NT>
cudaError_t launch_typed(const PagedArgs &g, int row_groups, cudaStream_t s)
{
    using S = Shape<D, NT>;
    static_assert(S::kWarpsSm * S::kOwn <= 224 * 1024, "the warps' memory fits an SM");
    static_assert(2ll * S::kMostWarpsOfRuns * slot_floats<D, NT>() * 4 <= (NT == 1 ? kFewBytes : kMostBytes), "the workspace has every run's parts");
    const int64_t pairs = static_cast<int64_t>(g.Hkv) * row_groups, items = (pairs + kMostWarps - 1) / kMostWarps;
    const int warps = static_cast<int>((pairs + items - 1) / items);
    const int64_t blocks = (g.max_len + kBlock - 1) / kBlock;
    const int ctas = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(kSms * (S::kWarpsSm / warps), items * g.B * blocks / kLeastBlocks)));
    const int smem = warps * S::kOwn;
    cudaLaunchAttribute attr[2];
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3(static_cast<unsigned>(32 * warps));
    cfg.dynamicSmemBytes = static_cast<size_t>(smem);
    cfg.stream = s;
    cfg.attrs = attr;
    const int R = cluster_for(items * g.B, blocks);
    if (R > 0) {
        cudaError_t e = ensure_smem_attr(reinterpret_cast<const void *>(paged_cluster_kernel<D, NT>), smem);
        if (e == cudaSuccess && R > 8) e = cudaFuncSetAttribute(paged_cluster_kernel<D, NT>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
        if (e != cudaSuccess) return e;
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = static_cast<unsigned>(R);
        attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
        cfg.gridDim = dim3(static_cast<unsigned>(items * g.B * R));
        cfg.numAttrs = 1 + set_launch_overlap_attr(attr + 1);
        return cudaLaunchKernelEx(&cfg, paged_cluster_kernel<D, NT>, g, row_groups);
    }
    const auto kernel = std::min<int64_t>(blocks, items * g.B * (blocks + kStartUnits) / ctas + 1) > kFold ? paged_kernel<D, NT, true> : paged_kernel<D, NT, false>;
    cudaError_t e = ensure_smem_attr(reinterpret_cast<const void *>(kernel), smem);
    if (e != cudaSuccess) return e;
    cfg.gridDim = dim3(static_cast<unsigned>(ctas));
    cfg.numAttrs = set_launch_overlap_attr(attr);
    e = cudaLaunchKernelEx(&cfg, kernel, g, row_groups);
    if (e != cudaSuccess || ctas == 1) return e;
    // the join starts while the runs still go on, and waits for their end on the device
    const int rows = std::min(8 * NT, g.T * (g.Hq / g.Hkv));
    const int64_t tasks = g.B * pairs * rows;
    int share = 1;   // two parts a warp or more, by the mean, and as many warps as the SMs take at once
    while (share < 32 && 4 * share * g.B * items <= ctas && 2 * share * tasks <= 16 * kSms) share *= 2;
    const int join_warps = std::max(share, 8);
    cudaLaunchConfig_t join = {};
    join.blockDim = dim3(static_cast<unsigned>(32 * join_warps));
    join.gridDim = dim3(static_cast<unsigned>((tasks * share + join_warps - 1) / join_warps));
    join.stream = s;
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    join.attrs = attr;
    join.numAttrs = 1;
    return cudaLaunchKernelEx(&join, paged_join_kernel<D, NT>, g, row_groups, warps, ctas, share, rows);
}

// Groups of 8 rows, or of up to 16: where there are more, further warps take them beside each other, and
// find the keys in L2. (With terms of one binary16: 25 rows of 8 requests in one group of 32 43 us for 26; of 64 requests of up to 8191
// tokens, bound by the products' instructions, 236 for 225 (228 now). 40 rows of 64 dimensions in one of 48 56 for 33 (30 now).)
template <int D>
cudaError_t launch_rows(const PagedArgs &g, cudaStream_t s)
{
    const int rows = g.T * (g.Hq / g.Hkv);
    return rows <= 8 ? launch_typed<D, 1>(g, 1, s) : launch_typed<D, 2>(g, (rows + 15) / 16, s);
}

}  // namespace

// By the query rows of a key head alone: as many parts as the SMs hold warps, of 8 rows or of more.
int64_t paged_workspace_bytes(int B, int rows)
{
    return (rows <= 8 ? kFewBytes : kMostBytes) + 8 * (static_cast<int64_t>(B) + 1);
}

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
