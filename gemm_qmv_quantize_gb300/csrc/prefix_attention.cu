// prefix_attention.cu -- attention of a batch whose requests share a long prefix: query
// rows see the prefix's keys and their request's own, both in a paged cache:
//   o = softmax(scale [q Kp^T, q Ko^T]) [Vp; Vo]
//
// The rows of all requests that read one key head meet the same prefix keys, so they are
// the rows of one matrix product: B T G rows (G = query heads a key head) x 128 keys a
// step on the 5th-generation tensor cores, the prefix read once for up to 256 of them.
// A request's own keys are the same product with its T G rows. Both are "jobs" of one
// kernel: a key head, up to 256 consecutive rows i = (b T + t) G + g, and a range of
// 128-key tiles; a row's jobs leave partial results that a second kernel joins.
//
// A job (one CTA; TMEM columns: S0, S1, O0, O1 of 128 each):
//   S = Q K^T into tensor memory (fp32); 128 threads, a row each, take the running
//   maximum m, write P = 2^(c S - m) in 16 bits over S, and P V adds onto O in tensor
//   memory (fp32). Two such streams run against each other, so that one's products fill
//   the tensor cores while the other's exponentials run: the two 128-row halves of the
//   rows, each over every tile, or, for up to 128 rows, the even and the odd tiles of the
//   same rows. m follows the true maximum with a slack of 2^8: O is rescaled only when a
//   row's maximum has grown by more, which is rare, and P stays far below the 16-bit
//   types' range. Statistics and sums are fp32; P is rounded to the inputs' type, the
//   operand that the product takes.
#include <algorithm>
#include <cmath>
#include <type_traits>

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "decode_ops.h"
#include "qmv.h"
#include "qmv_device.cuh"
#include "umma_device.cuh"

namespace qmv {
namespace {

__device__ uint32_t g_attention_error;

constexpr int kTile = 128;              // keys a tile = rows a stream = TMEM lanes
constexpr int kMmaWarp = 8, kLoadWarpV = 10;
constexpr int kThreads = 32 * 11;       // two streams of 4 warps, the product warp, the loading warps of K and of V
constexpr int kTmemCols = 512;
constexpr int kMaxSlots = 8;
constexpr int kSmemBytes = 232448 - 2048;   // dynamic shared memory: a CTA's limit but the barriers and statistics
constexpr int kSms = 152;
constexpr float kSlack = 8.0f;          // log2 of the growth of a row's maximum that rescales O

// Splits of the work, by sizes alone.
struct AttnPlan {
    int pair_groups, lone;              // row groups of the prefix: of 256 rows, and one of up to 128
    int pair_splits, lone_splits;       // ranges of prefix tiles for each
    int own_groups, own_splits, own_tiles;   // row groups of a request, ranges of own_tiles own tiles
    int64_t prefix_jobs, own_jobs;
    int slots;                          // partial results a row: own_splits, then the prefix's
};

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// The prefix's jobs fill the SMs once: a pair group's tile costs two products where a
// lone group's costs one, so ranges are cut to the same cost, of two tiles at least (a
// tile a stream). Own keys: a range a request where the requests and key heads fill the
// SMs, else as many as fill them, of 256 keys at least.
AttnPlan plan_attention(int B, int T, int Hq, int Hkv, int64_t prefix_len, int64_t max_own)
{
    AttnPlan p{};
    const int64_t G = Hq / Hkv, rows = static_cast<int64_t>(B) * T * G, tiles = ceil_div(prefix_len, kTile);
    if (tiles > 0 && rows > 0) {
        const int64_t row_tiles = ceil_div(rows, kTile);
        p.pair_groups = static_cast<int>(row_tiles / 2);
        p.lone = static_cast<int>(row_tiles % 2);
        const int64_t cost = Hkv * row_tiles * tiles;   // in products of 128 x 128
        const int64_t budget = std::max<int64_t>(2, ceil_div(cost, kSms));
        auto splits = [&](int64_t per_tile) {
            return static_cast<int>(std::min<int64_t>({std::max<int64_t>(1, (per_tile * tiles + budget / 2) / budget), tiles, 256}));
        };
        p.pair_splits = p.pair_groups ? splits(2) : 0;
        p.lone_splits = p.lone ? splits(1) : 0;
        p.prefix_jobs = Hkv * (static_cast<int64_t>(p.pair_groups) * p.pair_splits + p.lone_splits);
    }
    const int64_t own_tiles = ceil_div(max_own, kTile);
    if (own_tiles > 0 && rows > 0) {
        p.own_groups = static_cast<int>(ceil_div(T * G, 2 * kTile));
        const int64_t jobs = static_cast<int64_t>(B) * Hkv * p.own_groups;
        const int64_t want = std::max<int64_t>(1, std::min<int64_t>({kSms / jobs, ceil_div(own_tiles, 2), 256}));
        p.own_tiles = static_cast<int>(ceil_div(own_tiles, want));
        p.own_splits = static_cast<int>(ceil_div(own_tiles, p.own_tiles));
        p.own_jobs = jobs * p.own_splits;
    }
    p.slots = p.own_splits + std::max(p.pair_splits, p.lone_splits);
    return p;
}

struct AttnParams {
    CUtensorMap k, v;    // {D, page, Hkv, pages}: boxes of 64 d x min(page, 128) keys
    AttnArgs g;
    AttnPlan plan;
    float *part;         // [slots][B T Hq][D], each divided by its sum
    float *lse;          // [slots][B T Hq], log2 of the sum of exponentials; -inf: no key
};

__device__ __forceinline__ float exp2_fast(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

template <typename T>
__device__ __forceinline__ uint32_t pack2(float a, float b)
{
    if constexpr (std::is_same_v<T, __half>) {
        const __half2 h = __floats2half2_rn(a, b);
        return *reinterpret_cast<const uint32_t *>(&h);
    } else {
        const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
        return *reinterpret_cast<const uint32_t *>(&h);
    }
}

// The order in which tiles go through the ring of slots, K0 K1 V0 K2 V1 K3 ...: a tile's
// K is needed one step before its V.
__device__ __forceinline__ int ring_pos(bool v, int j) { return v ? 2 * j + 2 : (j == 0 ? 0 : 2 * j - 1); }

template <typename T, int kD>
__global__ void __launch_bounds__(kThreads, 1) attention_kernel(const __grid_constant__ AttnParams p)
{
    constexpr bool kBf16 = std::is_same_v<T, __nv_bfloat16>;
    constexpr float kLift = kBf16 ? 0.0f : 6.0f;   // P = 2^(c S - m + kLift): small probabilities stay
                                                   // in binary16's normal range, the largest below 2^14
    constexpr int kChunks = kD / 64;               // 64-wide (128-byte) blocks of a row
    constexpr uint32_t kBlock = kTile * 128;       // bytes of one block of a tile
    constexpr uint32_t kSlotBytes = kChunks * kBlock;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    __shared__ __align__(8) uint64_t full[kMaxSlots], freed[kMaxSlots], s_full[2], p_full[2], o_done[2], drained;
    __shared__ uint32_t tmem_slot, abort_flag;
    __shared__ float merge_m[kTile], merge_l[kTile];
    uint8_t *smem = smem_raw;
    volatile uint32_t *abort_word = &abort_flag;
    const AttnArgs &g = p.g;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int G = g.Hq / g.Hkv;

    grid_dependency_wait();

    // ---- the job: key head h, rows i0 .. i0 + nrows - 1, keys [key0, key1), result slot
    int64_t id = blockIdx.x, i0, key0, key1;
    int h, nrows, slot, own_b = -1;
    const int64_t rows_all = static_cast<int64_t>(g.B) * g.T * G;
    if (id < p.plan.prefix_jobs) {
        const int64_t tiles = (g.prefix_len + kTile - 1) / kTile, pair_jobs = static_cast<int64_t>(g.Hkv) * p.plan.pair_groups * p.plan.pair_splits;
        int splits, group, split;
        if (id < pair_jobs) {
            splits = p.plan.pair_splits;
            split = static_cast<int>(id % splits);
            group = static_cast<int>(id / splits % p.plan.pair_groups);
            h = static_cast<int>(id / splits / p.plan.pair_groups);
        } else {
            splits = p.plan.lone_splits;
            split = static_cast<int>((id - pair_jobs) % splits);
            group = p.plan.pair_groups;
            h = static_cast<int>((id - pair_jobs) / splits);
        }
        i0 = static_cast<int64_t>(group) * 2 * kTile;
        nrows = static_cast<int>(min(rows_all - i0, static_cast<int64_t>(2 * kTile)));
        key0 = tiles * split / splits * kTile;
        key1 = min(tiles * (split + 1) / splits * kTile, g.prefix_len);
        slot = p.plan.own_splits + split;
    } else {
        id -= p.plan.prefix_jobs;
        const int split = static_cast<int>(id % p.plan.own_splits);
        id /= p.plan.own_splits;
        const int group = static_cast<int>(id % p.plan.own_groups);
        id /= p.plan.own_groups;
        h = static_cast<int>(id % g.Hkv);
        own_b = static_cast<int>(id / g.Hkv);
        const int per = g.T * G;
        i0 = static_cast<int64_t>(own_b) * per + group * 2 * kTile;
        nrows = min(per - group * 2 * kTile, 2 * kTile);
        int64_t len = g.own_len[own_b];
        if (len > g.max_own) {
            if (tid == 0) atomicOr(&g_attention_error, kErrIndex);
            len = g.max_own;
        }
        key0 = static_cast<int64_t>(split) * p.plan.own_tiles * kTile;
        key1 = min(key0 + static_cast<int64_t>(p.plan.own_tiles) * kTile, len);
        slot = split;
    }
    const int64_t out_row0 = static_cast<int64_t>(slot) * g.B * g.T * g.Hq;
    // row i of key head h is query head h G + i % G of token i / G
    auto q_row = [&](int64_t i) { return i / G * g.Hq + h * G + i % G; };
    if (key1 <= key0) {   // no key: nothing of these rows in this slot
        for (int r = tid; r < nrows; r += kThreads) p.lse[out_row0 + q_row(i0 + r)] = -INFINITY;
        grid_launch_dependents();
        return;
    }
    const bool pair = nrows > kTile;
    const int ntiles = static_cast<int>((key1 - key0 + kTile - 1) / kTile);
    // stream s takes tiles first, first + step, ...
    auto steps_of = [&](int s) { return pair ? ntiles : (ntiles - s + 1) / 2; };
    const int last_keys = static_cast<int>(key1 - key0 - static_cast<int64_t>(ntiles - 1) * kTile);   // keys of the last tile
    const uint32_t q_bytes = (pair ? 2u : 1u) * kSlotBytes;
    uint8_t *ring = smem + q_bytes;
    const int nslots = min(kMaxSlots, static_cast<int>((kSmemBytes - q_bytes) / kSlotBytes));
    auto fail = [&]() { note_wait_timeout(&g_attention_error, abort_word); };
    auto wait_all = [&](uint64_t *bar, uint32_t parity) {
        return __all_sync(0xffffffffu, mbar_wait_bounded(bar, parity) ? 1 : 0) != 0;
    };

    if (tid == 0) {
        for (int i = 0; i < nslots; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&freed[i], 1);
        }
        for (int s = 0; s < 2; ++s) {
            mbar_init(&s_full[s], 1);
            mbar_init(&p_full[s], 4);
            mbar_init(&o_done[s], 1);
        }
        mbar_init(&drained, 1);
        abort_flag = 0u;
        fence_barrier_init();
    }
    if (warp == kMmaWarp) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(&tmem_slot)),
                     "r"(kTmemCols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    // Q into the K-major swizzled layout, rows past the job's as zeros
    {
        const int q_rows = pair ? 2 * kTile : kTile;
        for (int u = tid; u < q_rows * (kD / 8); u += kThreads) {
            const int r = u / (kD / 8), c = u % (kD / 8);
            uint4 v = make_uint4(0, 0, 0, 0);
            if (r < nrows) v = *(reinterpret_cast<const uint4 *>(static_cast<const T *>(g.q) + q_row(i0 + r) * kD) + c);
            uint8_t *dst = smem + (r / kTile) * kSlotBytes + (c / 8) * kBlock + (r % kTile) * 128 + 16 * ((c % 8) ^ (r % 8));
            *reinterpret_cast<uint4 *>(dst) = v;
        }
        fence_proxy_async_shared();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_slot;
    grid_launch_dependents();

    if (warp < 8) {
        // ------------------------------------------------ softmax of stream s: a row a thread
        const int s = warp >> 2, r = tid & (kTile - 1), steps = steps_of(s);
        const int rel = pair ? s * kTile + r : r;               // row within the job
        const bool live = rel < nrows;
        const bool warp_live = (pair ? s * kTile : 0) + (r & ~31) < nrows;   // any row of this warp
        const uint32_t lanes = static_cast<uint32_t>(32 * (warp & 3)) << 16;
        const uint32_t s_col = tmem + lanes + static_cast<uint32_t>(s * kTile);
        const uint32_t o_col = tmem + lanes + 256u + static_cast<uint32_t>(s * kTile);
        // keys of this row: all of the prefix's, or its request's up to its own token
        int64_t limit = key1;
        if (own_b >= 0 && live) {
            const int t = static_cast<int>((i0 + rel) / G % g.T);
            limit = min(key1, min(static_cast<int64_t>(g.own_len[own_b]), g.max_own) - g.T + 1 + t);
        }
        const int64_t least = own_b >= 0 ? min(key1, min(static_cast<int64_t>(g.own_len[own_b]), g.max_own) - g.T + 1) : key1;
        const float c = g.scale * 1.4426950408889634f;
        float m = -INFINITY, l = 0.0f;
        bool ok = true;
        for (int i = 0; i < steps; ++i) {
            const int64_t k0 = key0 + static_cast<int64_t>(pair ? i : 2 * i + s) * kTile;
            if (*abort_word || !wait_all(&s_full[s], static_cast<uint32_t>(i) & 1u)) {
                fail();
                ok = false;
                break;
            }
            if (warp_live) {
                tc_fence_after();
                float v[kTile];
#pragma unroll
                for (int j = 0; j < kTile; j += 32) tmem_ld32_async(s_col + j, v + j);
#pragma unroll
                for (int j = 0; j < kTile; j += 32) tmem_wait_ld32(v + j);
                if (least - k0 < kTile) {
                    const int n = static_cast<int>(max(static_cast<int64_t>(0), min(limit - k0, static_cast<int64_t>(kTile))));
#pragma unroll
                    for (int j = 0; j < kTile; ++j)
                        if (j >= n) v[j] = -INFINITY;
                }
                float top[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) top[j] = v[j];
#pragma unroll
                for (int j = 4; j < kTile; ++j) top[j & 3] = fmaxf(top[j & 3], v[j]);
                const float best = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])) * c;
                const bool grow = best > m + kSlack;   // (m = -inf: the row's first keys)
                if (__any_sync(0xffffffffu, grow)) {
                    const float next = grow ? best : m;
                    const float fix = grow ? exp2_fast(m - next) : 1.0f;
                    l *= fix;
                    m = next;
                    // the sums so far are complete: S of this step was issued after P V of the last
                    if (i > 0) {
#pragma unroll
                        for (int j = 0; j < kD; j += 16) {
                            float o[16];
                            tmem_ld16(o_col + j, o);
                            uint32_t w[16];
#pragma unroll
                            for (int x = 0; x < 16; ++x) w[x] = __float_as_uint(o[x] * fix);
                            tmem_st16(o_col + j, w);
                        }
                    }
                }
                const float shift = (m == -INFINITY ? 0.0f : m) - kLift;
                float sum[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                for (int q = 0; q < kTile; q += 32) {
                    uint32_t w[16];
#pragma unroll
                    for (int j = 0; j < 16; ++j) {
                        const float a = exp2_fast(fmaf(v[q + 2 * j], c, -shift));
                        const float b = exp2_fast(fmaf(v[q + 2 * j + 1], c, -shift));
                        sum[j & 3] += a + b;
                        w[j] = pack2<T>(a, b);
                    }
                    tmem_st16(s_col + q / 2, w);
                }
                l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
                tmem_wait_st();
                tc_fence_before();
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&p_full[s]);
        }
        // (up to 128 rows: stream 1 hands its part over in the memory that stream 0's products read)
        if (ok && ((steps > 0 && !wait_all(&o_done[s], 0u)) || (!pair && s == 1 && !wait_all(&o_done[0], 0u)))) {
            fail();
            ok = false;
        }
        tc_fence_after();
        // ---- results
        float *acc_smem = reinterpret_cast<float *>(smem);   // Q and the ring are idle now: [d][128 rows]
        if (!pair) {   // the two streams hold the same rows: stream 1 hands its part over
            if (s == 1) {
                merge_m[r] = m;
                merge_l[r] = l;
                if (steps > 0 && warp_live && ok) {
#pragma unroll
                    for (int j = 0; j < kD; j += 32) {
                        float o[32];
                        tmem_ld32_async(o_col + j, o);
                        tmem_wait_ld32(o);
#pragma unroll
                        for (int x = 0; x < 32; ++x) acc_smem[(j + x) * kTile + r] = o[x];
                    }
                }
            }
            asm volatile("bar.sync 1, 256;" ::: "memory");
        }
        if (ok && warp_live && !(s == 1 && !pair) && !*abort_word) {
            float w0 = 1.0f, w1 = 0.0f;
            const bool both = !pair && steps_of(1) > 0;
            if (both) {
                const float m1 = merge_m[r], top = fmaxf(m, m1);
                w0 = m == -INFINITY ? 0.0f : exp2_fast(m - top);
                w1 = m1 == -INFINITY ? 0.0f : exp2_fast(m1 - top);
                l = l * w0 + merge_l[r] * w1;
                m = top;
            }
            const float inv = 1.0f / l;
            const int64_t row = live ? out_row0 + q_row(i0 + rel) : 0;
            if (live) p.lse[row] = l == 0.0f ? -INFINITY : m - kLift + log2f(l);
#pragma unroll
            for (int j = 0; j < kD; j += 32) {
                float o[32];
                tmem_ld32_async(o_col + j, o);
                tmem_wait_ld32(o);
                if (both) {
#pragma unroll
                    for (int x = 0; x < 32; ++x) o[x] = o[x] * w0 + acc_smem[(j + x) * kTile + r] * w1;
                }
                if (live && l != 0.0f) {
#pragma unroll
                    for (int x = 0; x < 32; x += 4)
                        *reinterpret_cast<float4 *>(p.part + row * kD + j + x) =
                            make_float4(o[x] * inv, o[x + 1] * inv, o[x + 2] * inv, o[x + 3] * inv);
                }
            }
        }
        tc_fence_before();
    } else if (warp == kMmaWarp) {
        // ------------------------------------------------ products (lane 0 issues; the warp clears tails)
        const uint32_t idesc_s = idesc_16bit_f32(kTile, kTile, kBf16, false);
        const uint32_t idesc_o = idesc_16bit_f32(kTile, kD, kBf16, true);
        const uint32_t q_addr = smem_addr(smem), ring_addr = smem_addr(ring);
        const int n0 = steps_of(0);
        auto tile_of = [&](int s, int i) { return pair ? i : 2 * i + s; };
        // S of stream s, step i; its K slot is free after the last stream that reads it
        auto issue_s = [&](int s, int i) {
            const int j = tile_of(s, i), pos = ring_pos(false, j), at = pos % nslots;
            if (*abort_word || !wait_all(&full[at], static_cast<uint32_t>(pos / nslots) & 1u)) return false;
            if (lane == 0) {
                tc_fence_after();
                const uint32_t qa = q_addr + (pair ? static_cast<uint32_t>(s) * kSlotBytes : 0u);
                const uint32_t ka = ring_addr + static_cast<uint32_t>(at) * kSlotBytes;
#pragma unroll
                for (int k = 0; k < kD / 16; ++k) {
                    const uint32_t off = static_cast<uint32_t>(k / 4) * kBlock + 32u * (k % 4);
                    umma_f16_ss(tmem + static_cast<uint32_t>(s * kTile), smem_desc_sw128(qa + off), smem_desc_sw128(ka + off),
                                idesc_s, k > 0 ? 1u : 0u);
                }
                umma_commit(&s_full[s]);
                if (!pair || s == 1) umma_commit(&freed[at]);
            }
            __syncwarp();
            return true;
        };
        bool ok = true;
        for (int s = 0; s < 2 && ok; ++s)
            if (steps_of(s) > 0) ok = issue_s(s, 0);
        for (int i = 0; i < n0 && ok; ++i) {
            for (int s = 0; s < 2 && ok; ++s) {
                if (i >= steps_of(s)) break;
                const int j = tile_of(s, i), pos = ring_pos(true, j), at = pos % nslots;
                if (*abort_word || !wait_all(&full[at], static_cast<uint32_t>(pos / nslots) & 1u)) {
                    ok = false;
                    break;
                }
                if (j == ntiles - 1 && last_keys < kTile && (!pair || s == 0)) {
                    // what lies past the last key may be anything, NaN too: zeros, since 0 x NaN is NaN
                    for (int u = lane; u < (kTile - last_keys) * 8 * kChunks; u += 32) {
                        const int row = last_keys + u / (8 * kChunks), x = u % (8 * kChunks);
                        *reinterpret_cast<uint4 *>(ring + at * kSlotBytes + (x / 8) * kBlock + row * 128 + 16 * (x % 8)) =
                            make_uint4(0, 0, 0, 0);
                    }
                    fence_proxy_async_shared();
                    __syncwarp();
                }
                if (*abort_word || !wait_all(&p_full[s], static_cast<uint32_t>(i) & 1u)) {
                    ok = false;
                    break;
                }
                if (lane == 0) {
                    tc_fence_after();
                    const uint32_t va = ring_addr + static_cast<uint32_t>(at) * kSlotBytes;
#pragma unroll
                    for (int k = 0; k < kTile / 16; ++k)
                        umma_f16_ta(tmem + 256u + static_cast<uint32_t>(s * kTile), tmem + static_cast<uint32_t>(s * kTile) + 8u * k,
                                    smem_desc_sw128_mn(va + 2048u * k, kBlock), idesc_o, (i > 0 || k > 0) ? 1u : 0u);
                    if (!pair || s == 1) umma_commit(&freed[at]);
                    if (i + 1 == steps_of(s)) umma_commit(&o_done[s]);
                }
                __syncwarp();
                if (i + 1 < steps_of(s)) ok = issue_s(s, i + 1);
            }
        }
        if (!ok) fail();
        // every product has completed before tensor memory is released: a normal end is
        // seen by the streams' waits on o_done; after a failure this thread waits itself
        if (!ok && lane == 0) {
            umma_commit(&drained);
            (void)mbar_wait_bounded(&drained, 0u);
        }
        __syncwarp();
    } else {
        // ------------------------------------------------ K (warp 9) or V (warp 10): a lane a page of a tile
        const bool is_v = warp == kLoadWarpV;
        const CUtensorMap *map = is_v ? &p.v : &p.k;
        const int box = min(g.page, kTile), shift = __ffs(g.page) - 1;
        const int32_t *table = own_b < 0 ? g.prefix_table : g.own_table + static_cast<int64_t>(own_b) * g.own_pages;
        // the page of this lane's keys of tile j, outside the cache (read as zeros) where it is no page
        auto page_of = [&](int j) {
            const int64_t k = key0 + static_cast<int64_t>(j) * kTile + lane * box;
            if (j >= ntiles || lane * box >= kTile || k >= key1) return -1;
            const int pg = table[k >> shift];
            if (pg >= 0 && pg < g.n_pages) return pg;
            atomicOr(&g_attention_error, kErrIndex);
            return static_cast<int>(g.n_pages);
        };
        int pg = page_of(0), last = -1;
        for (int j = 0; j < ntiles && !*abort_word; ++j) {
            const int pos = ring_pos(is_v, j), at = pos % nslots;
            if (pos >= nslots && !wait_all(&freed[at], static_cast<uint32_t>(pos / nslots - 1) & 1u)) {
                fail();
                break;
            }
            const int boxes = __popc(__ballot_sync(0xffffffffu, pg >= 0));
            if (lane == 0) mbar_arrive_expect_tx(&full[at], static_cast<uint32_t>(boxes) * box * 128u * kChunks);
            __syncwarp();
            if (pg >= 0) {
                const int64_t k = key0 + static_cast<int64_t>(j) * kTile + lane * box;
                uint8_t *dst = ring + at * kSlotBytes + lane * box * 128;
                for (int c = 0; c < kChunks; ++c)
                    tma_load_4d(dst + c * kBlock, map, 64 * c, static_cast<int>(k & (g.page - 1)), h, pg, &full[at]);
            }
            last = j;
            pg = page_of(j + 1);
        }
        // every copy has landed before the CTA can exit: the slots of the last positions are
        // not used again (after a failure an earlier one may have been, by the other loading
        // warp; the wait is bounded)
        for (int j = max(0, last - nslots); j <= last; ++j) {
            const int pos = ring_pos(is_v, j);
            if (last + 1 < ntiles || pos > ring_pos(true, ntiles - 1) - nslots)
                (void)mbar_wait_bounded(&full[pos % nslots], static_cast<uint32_t>(pos / nslots) & 1u);
        }
        __syncwarp();
    }
    tc_fence_before();
    __syncthreads();
    if (warp == kMmaWarp) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols) : "memory");
    }
}

// Joins a row's partial results, one warp a row: weights 2^(lse - max) over their sum.
template <typename T, int kD>
__global__ void __launch_bounds__(256) attention_join_kernel(const __grid_constant__ AttnParams p)
{
    const AttnArgs &g = p.g;
    const int lane = threadIdx.x & 31;
    const int64_t rows = static_cast<int64_t>(g.B) * g.T * g.Hq, row = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
    grid_launch_dependents();
    grid_dependency_wait();
    if (row >= rows) return;
    // this row's prefix slots: those of its row group
    const int G = g.Hq / g.Hkv;
    const int64_t i = row / g.Hq * G + row % G;
    const bool in_pair = i < static_cast<int64_t>(p.plan.pair_groups) * 2 * kTile;
    const int slots = p.plan.own_splits + (in_pair ? p.plan.pair_splits : p.plan.lone_splits);
    float top = -INFINITY;
    for (int k = lane; k < slots; k += 32) top = fmaxf(top, p.lse[k * rows + row]);
    for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    constexpr int kPer = kD / 32;
    float acc[kPer], sum = 0.0f;
#pragma unroll
    for (int x = 0; x < kPer; ++x) acc[x] = 0.0f;
    for (int k = 0; k < slots; ++k) {
        const float lse = p.lse[k * rows + row];
        if (lse == -INFINITY) continue;
        const float w = exp2_fast(lse - top);
        sum += w;
        const float *o = p.part + (k * rows + row) * kD + lane * kPer;
#pragma unroll
        for (int x = 0; x < kPer; ++x) acc[x] = fmaf(w, o[x], acc[x]);
    }
    const float inv = sum > 0.0f || isnan(sum) ? 1.0f / sum : 0.0f;   // no key at all: zeros
    uint32_t *out = reinterpret_cast<uint32_t *>(static_cast<T *>(g.out) + row * kD + lane * kPer);
#pragma unroll
    for (int x = 0; x < kPer; x += 2) out[x / 2] = pack2<T>(acc[x] * inv, acc[x + 1] * inv);
}

cudaError_t encode_cache_map(CUtensorMap *map, const void *cache, const AttnArgs &g)
{
    const uint64_t dims[4] = {static_cast<uint64_t>(g.D), static_cast<uint64_t>(g.page), static_cast<uint64_t>(g.Hkv),
                              static_cast<uint64_t>(g.n_pages)};
    const uint64_t head = static_cast<uint64_t>(g.D) * 2;
    const uint64_t strides[3] = {head * g.Hkv, head, head * g.Hkv * g.page};
    const uint32_t box[4] = {64, static_cast<uint32_t>(std::min(g.page, kTile)), 1, 1};
    return encode_map_nd(map, g.type == QMV_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4,
                         cache, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B);
}

template <typename T, int kD>
cudaError_t launch_typed(const AttnParams &p, cudaStream_t s)
{
    const AttnArgs &g = p.g;
    cudaLaunchAttribute attr[1];
    cudaLaunchConfig_t cfg = {};
    cfg.stream = s;
    cfg.attrs = attr;
    const int64_t jobs = p.plan.prefix_jobs + p.plan.own_jobs;
    if (jobs > 0) {
        auto kern = attention_kernel<T, kD>;
        cudaError_t e = ensure_smem_attr(reinterpret_cast<const void *>(kern), kSmemBytes);
        if (e != cudaSuccess) return e;
        cfg.blockDim = dim3(kThreads);
        cfg.gridDim = dim3(static_cast<unsigned>(jobs));
        cfg.dynamicSmemBytes = kSmemBytes;
        cfg.numAttrs = set_launch_overlap_attr(attr);
        if ((e = cudaLaunchKernelEx(&cfg, kern, p)) != cudaSuccess) return e;
    }
    const int64_t rows = static_cast<int64_t>(g.B) * g.T * g.Hq;
    cfg.blockDim = dim3(256);
    cfg.gridDim = dim3(static_cast<unsigned>((rows + 7) / 8));
    cfg.dynamicSmemBytes = 0;
    if (jobs > 0) {   // starts as the last jobs run, and waits for all of them
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        cfg.numAttrs = 1;
    } else {
        cfg.numAttrs = set_launch_overlap_attr(attr);
    }
    return cudaLaunchKernelEx(&cfg, attention_join_kernel<T, kD>, p);
}

int64_t part_bytes(const AttnPlan &plan, int B, int T, int Hq, int D)
{
    return static_cast<int64_t>(plan.slots) * B * T * Hq * D * 4;
}

}  // namespace

int64_t attn_workspace_bytes(int B, int T, int Hq, int Hkv, int D, int64_t prefix_len, int64_t max_own)
{
    const AttnPlan plan = plan_attention(B, T, Hq, Hkv, prefix_len, max_own);
    return part_bytes(plan, B, T, Hq, D) + static_cast<int64_t>(plan.slots) * B * T * Hq * 4;
}

cudaError_t launch_attention(const DeviceInfo &, const AttnArgs &g, cudaStream_t s)
{
    route_hit(kRoutePrefixAttention);
    AttnParams p{};
    p.g = g;
    p.plan = plan_attention(g.B, g.T, g.Hq, g.Hkv, g.prefix_len, g.max_own);
    if (p.plan.prefix_jobs + p.plan.own_jobs > 0x7fffffffLL) return cudaErrorInvalidValue;
    p.part = static_cast<float *>(g.workspace);
    p.lse = reinterpret_cast<float *>(static_cast<uint8_t *>(g.workspace) + part_bytes(p.plan, g.B, g.T, g.Hq, g.D));
    if (g.n_pages > 0) {
        cudaError_t e = encode_cache_map(&p.k, g.k_cache, g);
        if (e == cudaSuccess) e = encode_cache_map(&p.v, g.v_cache, g);
        if (e != cudaSuccess) return e;
    }
    if (g.D == 64)
        return g.type == QMV_F16 ? launch_typed<__half, 64>(p, s) : launch_typed<__nv_bfloat16, 64>(p, s);
    return g.type == QMV_F16 ? launch_typed<__half, 128>(p, s) : launch_typed<__nv_bfloat16, 128>(p, s);
}

cudaError_t read_error_word_attention(uint32_t *out, bool clear)
{
    cudaError_t e = cudaMemcpyFromSymbol(out, g_attention_error, sizeof(uint32_t));
    if (e != cudaSuccess || !clear) return e;
    const uint32_t zero = 0;
    return cudaMemcpyToSymbol(g_attention_error, &zero, sizeof(uint32_t));
}

}  // namespace qmv
