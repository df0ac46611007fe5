// prefix_attention.cu -- attention of a batch whose requests share a long prefix: query
// rows see the prefix's keys and their request's own, both in a paged cache:
//   o = softmax(scale [q Kp^T, q Ko^T]) [Vp; Vo]
//
// The rows of all requests that read one key head meet the same prefix keys, so they are
// the rows of one matrix product: B T G rows (G = query heads a key head) x 128 keys a
// step on the 5th-generation tensor cores, the prefix read once for up to 256 of them. A
// "job" is a key head, up to 256 consecutive rows i = (b T + t) G + g, and a share of the
// 128-key tiles. A request's own keys against more than 64 rows are jobs of the same kernel;
// for up to 64 rows, and for a prefix that at most 16 rows see, few_rows_kernel further down
// has products of 16 rows. What a row's jobs leave is joined by a last kernel.
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
//
// 51 requests of 5 query heads a key head (255 rows) behind 65536 keys take 70 us, 984
// TFLOP/s; 25 of them (125 rows, bound by the keys' bytes) 56 us, 4.8 TB/s. A stream's
// products, softmax and P V follow one another, about 3000 cycles a tile; its exponentials
// and the handing over, not the tensor cores (56 % busy), bound the first.
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
constexpr int kMmaWarp = 8;             // and 9: a thread each issues a stream's products
constexpr int kLoadWarp = 10;            // and 11: each loads half of every tile
constexpr int kThreads = 32 * 12;       // two streams of 4 warps, the product warps, the loading warps
// Registers a thread: the softmax warpgroups hold a row of S each; 256 x 224 + 128 x 56 of
// the 384 x 168 that the launch has.
constexpr int kRegsSoftmax = 224, kRegsOther = 56;
constexpr int kTmemCols = 512;
constexpr int kMaxSlots = 8;
constexpr int kSmemBytes = 224 * 1024;   // dynamic shared memory: a CTA's 227 KB but the barriers and statistics
constexpr int kSms = 152;
constexpr int kFewRows = 64;            // rows of a request and key head up to which its own keys have a kernel of their own
constexpr float kSlack = 8.0f;          // log2 of the growth of a row's maximum that rescales O

// Splits of the work, by sizes alone.
struct AttnPlan {
    int pair_groups, lone;              // row groups of the prefix: of 256 rows, and one of up to 128
    int pair_splits, lone_splits;       // ranges of prefix tiles for each
    int own_groups, own_splits, own_tiles;   // row groups of a request, ranges of own_tiles own tiles
    int few_row_tiles, few_keys;        // requests of few rows, by the kernel for those: 16-row tiles, keys a range
    int64_t few_jobs;
    int few_prefix_keys;                // the same for the prefix, where all rows together are 16 at most
    int64_t few_prefix_jobs;
    int64_t prefix_jobs, own_jobs;
    int prefix_ctas, own_ctas;          // CTAs that take the ones, and the others, in turn
    int slots;                          // partial results a row: own_splits, then the prefix's
};

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Keys of each of `splits` ranges, whole blocks of 64, within 31 bits.
int range_of(int64_t keys, int64_t splits)
{
    return static_cast<int>(std::min<int64_t>(ceil_div(ceil_div(keys, splits), 64) * 64, 0x7fffffc0));
}

// Costs, in thousands of cycles as measured: a tile 3 for a pair of streams, 2 where the
// streams take every other tile; a job 8 beside its tiles. The SMs are divided
// between the prefix and the own keys by their shares of the cost (own lengths are on the
// device: 0.6 of the bound is taken), so that no CTA starts on the one after the other; the
// prefix is then cut into a range a CTA, of equal cost and two tiles at least, and own keys
// into ranges that leave each CTA several, of two tiles at least.
AttnPlan plan_attention(int B, int T, int Hq, int Hkv, int64_t prefix_len, int64_t max_own)
{
    AttnPlan p{};
    const int64_t G = Hq / Hkv, rows = static_cast<int64_t>(B) * T * G, tiles = ceil_div(prefix_len, kTile);
    const int64_t own_tiles = ceil_div(max_own, kTile);
    int64_t own_cost = 0, prefix_cost = 0;
    if (own_tiles > 0 && rows > 0 && T * G <= kFewRows) {
        // ranges of 256 keys at least (four steps a warp), for four CTAs a place on the SMs
        p.few_row_tiles = static_cast<int>(ceil_div(T * G, 16));
        const int64_t jobs = static_cast<int64_t>(B) * Hkv * p.few_row_tiles;
        const int64_t splits = std::max<int64_t>(1, std::min<int64_t>({8 * kSms / jobs, ceil_div(max_own, 256), 256}));
        p.few_keys = range_of(max_own, splits);
        p.own_splits = static_cast<int>(ceil_div(max_own, p.few_keys));
        p.few_jobs = jobs * p.own_splits;
    } else if (own_tiles > 0 && rows > 0) {
        p.own_groups = static_cast<int>(ceil_div(T * G, 2 * kTile));
        const int64_t jobs = static_cast<int64_t>(B) * Hkv * p.own_groups;
        const int64_t most = std::max<int64_t>({2, jobs * own_tiles / (2 * kSms), ceil_div(own_tiles, 256)});
        const int64_t splits = ceil_div(own_tiles, most);
        p.own_tiles = static_cast<int>(ceil_div(own_tiles, splits));
        p.own_splits = static_cast<int>(ceil_div(own_tiles, p.own_tiles));
        p.own_jobs = jobs * p.own_splits;
        own_cost = 8 * p.own_jobs + jobs * own_tiles * 6 / 5;
    }
    if (tiles > 0 && rows > 0 && rows <= 16) {
        // (with 32 rows, the prefix read twice: 18 us for 16 with 4096 keys)
        const int64_t splits = std::max<int64_t>(1, std::min<int64_t>({2 * kSms / Hkv, ceil_div(prefix_len, 128), 256}));
        p.few_prefix_keys = range_of(prefix_len, splits);
        p.lone_splits = static_cast<int>(ceil_div(prefix_len, p.few_prefix_keys));
        p.few_prefix_jobs = static_cast<int64_t>(Hkv) * p.lone_splits;
    } else if (tiles > 0 && rows > 0) {
        const int64_t row_tiles = ceil_div(rows, kTile);
        p.pair_groups = static_cast<int>(row_tiles / 2);
        p.lone = static_cast<int>(row_tiles % 2);
        prefix_cost = Hkv * ((3 * p.pair_groups + 2 * p.lone) * tiles + 8 * (p.pair_groups + p.lone));
        int64_t ctas = own_cost == 0 ? kSms : std::min<int64_t>(std::max<int64_t>({1, kSms * prefix_cost / (prefix_cost + own_cost), kSms - p.own_jobs}), kSms - 1);
        const int64_t budget = std::max<int64_t>(4, ceil_div(prefix_cost, ctas));
        auto splits = [&](int64_t per_tile) {
            return static_cast<int>(std::min<int64_t>({std::max<int64_t>(1, (per_tile * tiles + budget / 2) / budget), tiles, 256}));
        };
        p.pair_splits = p.pair_groups ? splits(3) : 0;
        p.lone_splits = p.lone ? splits(2) : 0;
        p.prefix_jobs = Hkv * (static_cast<int64_t>(p.pair_groups) * p.pair_splits + p.lone_splits);
        // a CTA a range, unless whole row groups are several a CTA
        if (p.pair_splits > 1 || p.lone_splits > 1) ctas = std::max<int64_t>(ctas, p.prefix_jobs);
        p.prefix_ctas = static_cast<int>(std::min<int64_t>({ctas, p.prefix_jobs, own_cost == 0 ? kSms : kSms - 1}));
    }
    p.own_ctas = static_cast<int>(std::min<int64_t>(p.own_jobs, kSms - p.prefix_ctas));
    p.slots = p.own_splits + std::max(p.pair_splits, p.lone_splits);
    return p;
}

struct AttnParams {
    CUtensorMap k, v;    // {D, page, Hkv, pages}: boxes of 64 d x min(page, 128) keys
    AttnArgs g;
    AttnPlan plan;
    // Partial results, each divided by its sum: [slots][Hkv][blocks of 32 rows][D / 4][32][4], so
    // that the 32 threads of a warp, a row each, store whole lines; lse [slots][Hkv][rows], the
    // log2 of the sum of exponentials; -inf: no key (and no partial result).
    float *part, *lse;
    int row_blocks;
    bool chained;        // launched beside the own-key kernel: waits for that at its end
};

__device__ __forceinline__ float exp2_fast(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Two fp32 values side by side, one instruction for both.
__device__ __forceinline__ uint64_t pair_of(float a, float b)
{
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float2 both_of(uint64_t v)
{
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
    return r;
}
__device__ __forceinline__ uint64_t fma_pair(uint64_t a, uint64_t b, uint64_t c)
{
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t add_pair(uint64_t a, uint64_t b)
{
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ float max3(float a, float b, float c)
{
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
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

// The order in which a job's n tiles go through the ring of slots, K0 K1 V0 K2 V1 ... Vn-1:
// a tile's K is needed a step before its V.
__device__ __forceinline__ int k_pos(int j) { return j == 0 ? 0 : 2 * j - 1; }
__device__ __forceinline__ int v_pos(int j, int n) { return j == n - 1 ? 2 * n - 1 : 2 * j + 2; }

struct Job {
    int h, i0, nrows;       // key head; rows i0 .. i0 + nrows - 1
    int slot;               // of the partial results
    int own_b;              // request whose own keys these are, or -1: the prefix's
    int64_t key0;           // first key, a multiple of 128
    int step;               // tile t holds the keys key0 + 128 step t ...
    int keys, ntiles;       // number of keys, of tiles (0: no key)
    int own_end;            // own keys: the request's length - key0
};

// A bounded wait in few instructions (mbar_wait_bounded reads the clock too): a poll of a
// phase that is not complete returns after some microseconds, so the bound is about a second.
__device__ __forceinline__ bool wait_for(uint64_t *bar, uint32_t parity)
{
#pragma unroll 1
    for (int i = 0; i < 1 << 18; ++i)
        if (mbar_try_wait_sleep(bar, parity, 1000000u)) return true;
    return false;
}

// The length of job `id`'s request, where it has own keys.
__device__ __forceinline__ int own_length(const AttnParams &p, int id)
{
    if (id < p.plan.prefix_jobs || id >= p.plan.prefix_jobs + p.plan.own_jobs) return 0;
    const int b = (id - static_cast<int>(p.plan.prefix_jobs)) / (p.plan.own_splits * p.plan.own_groups * p.g.Hkv);
    return __ldg(p.g.own_len + b);
}

// Job `id`; len: own_length of it (loaded ahead). (What runs once a job has one place in
// the code and is not unrolled: a launch finds little of its code in the caches, since the keys pass
// through them, and fetches it at about a microsecond a miss.)
__device__ __forceinline__ Job job_of(const AttnParams &p, int id, int len)
{
    const AttnArgs &g = p.g;
    const int G = g.Hq / g.Hkv;
    Job j;
    if (id < p.plan.prefix_jobs) {
        const int tiles = static_cast<int>((g.prefix_len + kTile - 1) / kTile), rows = g.B * g.T * G;
        const int pair_jobs = g.Hkv * p.plan.pair_groups * p.plan.pair_splits;
        const bool lone = id >= pair_jobs;
        const int splits = lone ? p.plan.lone_splits : p.plan.pair_splits;
        int k = lone ? id - pair_jobs : id;
        const int split = k % splits;
        k /= splits;
        const int group = lone ? p.plan.pair_groups : k % p.plan.pair_groups;
        j.h = lone ? k : k / p.plan.pair_groups;
        j.i0 = group * 2 * kTile;
        j.nrows = min(rows - j.i0, 2 * kTile);
        // Every splits-th tile, not a run of them: all row groups of a key head then pass over
        // the prefix side by side and find one another's tiles in L2 (runs: 447 MB read from
        // memory for 268 MB of keys, 64 requests behind 65536).
        j.key0 = static_cast<int64_t>(split) * kTile;
        j.step = splits;
        j.ntiles = (tiles - split + splits - 1) / splits;
        j.keys = (j.ntiles - 1) * kTile +
                 static_cast<int>(min(static_cast<int64_t>(kTile), g.prefix_len - (j.key0 + static_cast<int64_t>(j.ntiles - 1) * splits * kTile)));
        j.slot = p.plan.own_splits + split;
        j.own_b = -1;
        j.own_end = 0;
    } else {
        int k = id - static_cast<int>(p.plan.prefix_jobs);
        const int split = k % p.plan.own_splits;
        k /= p.plan.own_splits;
        const int group = k % p.plan.own_groups;
        k /= p.plan.own_groups;
        j.h = k % g.Hkv;
        j.own_b = k / g.Hkv;
        const int per = g.T * G;
        j.i0 = j.own_b * per + group * 2 * kTile;
        j.nrows = min(per - group * 2 * kTile, 2 * kTile);
        const int64_t n = min(static_cast<int64_t>(len), g.max_own);
        j.key0 = static_cast<int64_t>(split) * p.plan.own_tiles * kTile;
        const int64_t key1 = min(j.key0 + static_cast<int64_t>(p.plan.own_tiles) * kTile, n);
        j.step = 1;
        j.keys = static_cast<int>(max(static_cast<int64_t>(0), key1 - j.key0));
        j.ntiles = (j.keys + kTile - 1) / kTile;
        j.slot = split;
        j.own_end = static_cast<int>(max(static_cast<int64_t>(0), n - j.key0));
    }
    return j;
}

// Piece u (16 bytes) of the Q of rows i0 ... of key head h: row i is query head h G + i % G
// of token i / G.
template <int kD>
__device__ __forceinline__ const uint4 *q_piece(const AttnArgs &g, int h, int i0, int u)
{
    const int G = g.Hq / g.Hkv, i = i0 + u / (kD / 8);
    const int64_t row = static_cast<int64_t>(i / G) * g.Hq + h * G + i % G;
    return static_cast<const uint4 *>(g.q) + row * (kD / 8) + u % (kD / 8);
}

// nrows of Q into the K-major swizzled layout, by 256 threads, their first pieces at hand.
// (Rows past these keep what is there: their S, P and O are never used.)
template <int kD>
__device__ __forceinline__ void store_q(uint8_t *smem, const AttnArgs &g, int h, int i0, int nrows, int tid, uint4 first)
{
    const int pieces = nrows * (kD / 8);
    auto place = [&](int u) {
        const int r = u / (kD / 8), x = u % (kD / 8);
        return smem + (r / kTile) * (kTile * kD * 2) + (x / 8) * (kTile * 128) + (r % kTile) * 128 + 16 * ((x % 8) ^ (r % 8));
    };
    if (tid < pieces) *reinterpret_cast<uint4 *>(place(tid)) = first;
#pragma unroll 1
    for (int u = tid + 256; u < pieces; u += 256) cp_async_16(place(u), q_piece<kD>(g, h, i0, u));
    cp_async_wait_all();
}

// kWide: the launch has jobs of more than 128 rows (two Q tiles, one slot less).
template <typename T, int kD, bool kWide>
__global__ void __launch_bounds__(kThreads, 1) attention_kernel(const __grid_constant__ AttnParams p)
{
    constexpr bool kBf16 = std::is_same_v<T, __nv_bfloat16>;
    constexpr float kLift = kBf16 ? 0.0f : 6.0f;   // P = 2^(c S - m + kLift): small probabilities stay
                                                   // in binary16's normal range, the largest below 2^14
    constexpr int kChunks = kD / 64;               // 64-wide (128-byte) blocks of a row
    constexpr uint32_t kBlock = kTile * 128;       // bytes of one block of a tile
    constexpr uint32_t kSlotBytes = kChunks * kBlock;
    constexpr uint32_t kQBytes = (kWide ? 2 : 1) * kSlotBytes;
    constexpr int kSlots = std::min(kMaxSlots, static_cast<int>((kSmemBytes - kQBytes) / kSlotBytes));
    extern __shared__ __align__(1024) uint8_t smem[];
    // full: a slot's copies have landed; freed: its readers are done (two arrivals: each
    // stream's, or two by the one stream that reads it); s_full / p_half / p_full: S, P for the
    // first 64 keys, all of P of a stream's step; q_full: a job's Q is in place; o_done: its products are complete; o_free: its
    // results have been read; merged: the streams' statistics of a job are there for one another;
    // turn: the other stream's products have been issued
    __shared__ __align__(8) uint64_t full[kSlots], freed[kSlots], s_full[2], p_half[2], p_full[2], q_full, o_done, o_free, merged, turn[2], drained[2];
    __shared__ uint32_t tmem_slot, abort_flag;
    __shared__ float merge_m[2][kTile], merge_l[2][kTile];
    volatile uint32_t *abort_word = &abort_flag;
    uint8_t *ring = smem + kQBytes;
    const AttnArgs &g = p.g;
    // (the product and loading warps are the CTA's first)
    const int tid = (threadIdx.x + 256) % kThreads, warp = tid >> 5, lane = tid & 31;
    const int G = g.Hq / g.Hkv, cta = static_cast<int>(blockIdx.x);
    // this CTA's jobs: id, id + stride, ... below `jobs`
    const bool on_prefix = cta < p.plan.prefix_ctas;
    const int jobs = static_cast<int>(p.plan.prefix_jobs + (on_prefix ? 0 : p.plan.own_jobs));
    const int stride = on_prefix ? p.plan.prefix_ctas : p.plan.own_ctas;
    auto fail = [&]() { note_wait_timeout(&g_attention_error, abort_word); };
    auto wait_all = [&](uint64_t *bar, uint32_t parity) {
        return __all_sync(0xffffffffu, wait_for(bar, parity) ? 1 : 0) != 0;
    };
    auto full_parity = [](int pos) { return static_cast<uint32_t>(pos / kSlots) & 1u; };
    // Ring position `pos` has landed. A wait is a parity test, right only if the phase
    // before is known to be over. Where a stream sees half of the tiles, the slot's copy
    // before may be the other stream's, and late: it is over once its readers have freed
    // the slot (and the use before that one was, when the loading warp came this far).
    auto landed = [&](int pos, bool pair) {
        const int at = pos % kSlots;
        if (!pair && pos >= kSlots && !wait_for(&freed[at], full_parity(pos) ^ 1u)) return false;
        return wait_for(&full[at], full_parity(pos));
    };

    if (tid == 0) {
        for (int i = 0; i < kSlots; ++i) {
            mbar_init(&full[i], 2);
            mbar_init(&freed[i], 2);
        }
        for (int s = 0; s < 2; ++s) {
            mbar_init(&s_full[s], 1);
            mbar_init(&p_half[s], 4);
            mbar_init(&p_full[s], 4);
        }
        mbar_init(&q_full, 8);
        mbar_init(&o_done, 2);
        mbar_init(&o_free, 8);
        mbar_init(&merged, 8);
        mbar_init(&turn[0], 1);
        mbar_init(&turn[1], 1);
        mbar_init(&drained[0], 1);
        mbar_init(&drained[1], 1);
        abort_flag = 0u;
        fence_barrier_init();
    }
    if (warp == kMmaWarp) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(&tmem_slot)),
                     "r"(kTmemCols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_slot;
    if (!p.chained) grid_dependency_wait();   // (chained: the own-key kernel began after the inputs were there)
    grid_launch_dependents();

    int id = on_prefix ? cta : static_cast<int>(p.plan.prefix_jobs) + cta - p.plan.prefix_ctas;
    int len = own_length(p, id);
    if (warp < 8) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoftmax));
        // ------------------------------------------------ softmax of stream s: a row a thread
        const int s = warp >> 2, r = tid & (kTile - 1);
        const uint32_t lanes = static_cast<uint32_t>(32 * (warp & 3)) << 16;
        const uint32_t s_col = tmem + lanes + static_cast<uint32_t>(s * kTile);
        const uint32_t o_col = tmem + lanes + 256u + static_cast<uint32_t>(s * kTile);
        const float c = g.scale * 1.4426950408889634f;
        // The first 256 16-byte pieces of a job's Q, all of a decode step's own-key job, are
        // loaded while the job before ends.
        auto has_q = [&](const Job &j) { return j.ntiles > 0 && tid < j.nrows * (kD / 8); };
        auto load_q = [&](const Job &j, uint4 first) {
            store_q<kD>(smem, g, j.h, j.i0, j.nrows, tid, first);
            fence_proxy_async_shared();
            __syncwarp();
            if (lane == 0) mbar_arrive(&q_full);
        };
        int pos0 = 0;            // ring positions before this job's
        uint32_t step = 0, done = 0, merges = 0;   // this stream's steps, the jobs with keys and those joined, so far
        bool ok = true, running = false;
        Job job{};
        // A turn: the steps of a job; the next job's Q, so that its first products run beside
        // this job's results; these.
        for (;;) {
            const bool pair = kWide && job.nrows > kTile;
            const int n = job.ntiles, steps = !running ? 0 : pair ? n : (n - s + 1) / 2;
            const int rel = pair ? s * kTile + r : r;   // row within the job
            const bool live = rel < job.nrows;
            const bool warp_live = (pair ? s * kTile : 0) + (r & ~31) < job.nrows;   // any row of this warp
            const int64_t out_row0 = (static_cast<int64_t>(job.slot) * g.Hkv + job.h) * p.row_blocks * 32 + job.i0;
            // keys of this row: all of the prefix's, or its request's up to its own token; and the fewest of any row
            const int limit = job.own_b < 0 ? job.keys : min(job.keys, job.own_end - g.T + 1 + (job.i0 + rel) / G % g.T);
            const int least = job.own_b < 0 ? job.keys : min(job.keys, job.own_end - g.T + 1);
            const uint32_t arrivals = pair ? 1u : 2u;
            float m = -INFINITY, l = 0.0f;
            for (int i = 0; i < steps; ++i, ++step) {
                const int t = pair ? i : 2 * i + s;
                if (*abort_word || !wait_all(&s_full[s], step & 1u)) {
                    fail();
                    ok = false;
                    break;
                }
                if ((warp & 3) == 0 && lane == 0) {   // S is complete, and P V of the last step
                    mbar_arrive_n(&freed[(pos0 + k_pos(t)) % kSlots], arrivals);
                    if (i > 0) mbar_arrive_n(&freed[(pos0 + v_pos(pair ? t - 1 : t - 2, n)) % kSlots], arrivals);
                }
                if (t == n - 1 && job.keys % kTile != 0) {
                    // what lies past the last key may be anything, NaN too: zeros, since 0 x NaN is NaN
                    // (each stream that reads the tile writes them before its own product)
                    const int pos = pos0 + v_pos(t, n), first = job.keys % kTile;
                    if (*abort_word || !__all_sync(0xffffffffu, landed(pos, pair) ? 1 : 0)) {
                        fail();
                        ok = false;
                        break;
                    }
                    for (int u = r; u < (kTile - first) * 8 * kChunks; u += kTile) {
                        const int row = first + u / (8 * kChunks), x = u % (8 * kChunks);
                        *reinterpret_cast<uint4 *>(ring + (pos % kSlots) * kSlotBytes + (x / 8) * kBlock + row * 128 + 16 * (x % 8)) =
                            make_uint4(0, 0, 0, 0);
                    }
                    fence_proxy_async_shared();
                }
                if (warp_live) {
                    tc_fence_after();
                    if (least - t * kTile < kTile) {   // the last tile, or the request's own tokens
                        const int x = limit - t * kTile;
#pragma unroll 1
                        for (int j = 0; j < kTile; j += 16) {
                            float o[16];
                            tmem_ld16(s_col + j, o);
                            uint32_t w[16];
#pragma unroll
                            for (int y = 0; y < 16; ++y) w[y] = __float_as_uint(j + y < x ? o[y] : -INFINITY);
                            tmem_st16(s_col + j, w);
                        }
                        tmem_wait_st();
                    }
                    float v[kTile];
#pragma unroll
                    for (int j = 0; j < kTile; j += 32) tmem_ld32_async(s_col + j, v + j);
#pragma unroll
                    for (int j = 0; j < kTile; j += 32) tmem_wait_ld32(v + j);
                    float top[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) top[j] = v[j];
#pragma unroll
                    for (int j = 4; j < kTile - 4; j += 8)
#pragma unroll
                        for (int x = 0; x < 4; ++x) top[x] = max3(top[x], v[j + 2 * x], v[j + 2 * x + 1]);
#pragma unroll
                    for (int j = kTile - 4; j < kTile; ++j) top[j & 3] = fmaxf(top[j & 3], v[j]);
                    const float best = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])) * c;
                    const bool grow = best > m + kSlack;   // (m = -inf: the row's first keys)
                    if (__any_sync(0xffffffffu, grow)) {
                        const float next = grow ? best : m;
                        const float fix = grow ? exp2_fast(m - next) : 1.0f;
                        l *= fix;
                        m = next;
                        // the sums so far are complete: S of this step was issued after P V of the last
                        if (i > 0) {
#pragma unroll 1
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
                    const float shift = kLift - (m == -INFINITY ? 0.0f : m);
                    const uint64_t shift2 = pair_of(shift, shift), c2 = pair_of(c, c);
                    uint64_t sum[2] = {0, 0};
#pragma unroll
                    for (int q = 0; q < kTile; q += 32) {
                        uint32_t w[16];
#pragma unroll
                        for (int j = 0; j < 16; ++j) {
                            const float2 x = both_of(fma_pair(pair_of(v[q + 2 * j], v[q + 2 * j + 1]), c2, shift2));
                            const float a = exp2_fast(x.x), b = exp2_fast(x.y);
                            sum[j & 1] = add_pair(sum[j & 1], pair_of(a, b));
                            w[j] = pack2<T>(a, b);
                        }
                        tmem_st16(s_col + q / 2, w);
                        if (q == kTile / 2 - 32) {   // the products with the first 64 keys may begin
                            tmem_wait_st();
                            tc_fence_before();
                            __syncwarp();
                            if (lane == 0) mbar_arrive(&p_half[s]);
                        }
                    }
                    const float2 sums = both_of(add_pair(sum[0], sum[1]));
                    l += sums.x + sums.y;
                    tmem_wait_st();
                    tc_fence_before();
                } else {
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&p_half[s]);
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&p_full[s]);
            }
            Job next{};
            uint4 first_q{};
            if (id < jobs) {   // (while this job's last products run)
                next = job_of(p, id, len);
                if (has_q(next)) first_q = __ldg(q_piece<kD>(g, next.h, next.i0, tid));
                if (next.own_b >= 0 && len > g.max_own && tid == 0) atomicOr(&g_attention_error, kErrIndex);
            }
            if (running) {
                if (ok && (*abort_word || !wait_all(&o_done, done & 1u))) {
                    fail();
                    ok = false;
                }
                if (!ok) break;
                ++done;
                if (steps > 0 && (warp & 3) == 0 && lane == 0)
                    mbar_arrive_n(&freed[(pos0 + v_pos(pair ? n - 1 : 2 * (steps - 1) + s, n)) % kSlots], arrivals);
                pos0 += 2 * n;
            }
            if (next.ntiles > 0) load_q(next, first_q);
            if (running) {
                // ---- results: O / l and the log2 of the sum. Up to 128 rows, both streams hold the
                // same rows: each joins both parts for half of D.
                tc_fence_after();
                float w0 = 1.0f, w1 = 0.0f;
                if (!pair) {
                    merge_m[s][r] = m;
                    merge_l[s][r] = l;
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&merged);
                    if (!wait_all(&merged, merges & 1u)) {
                        fail();
                        break;
                    }
                    ++merges;
                    const float m0 = merge_m[0][r], m1 = merge_m[1][r];
                    m = fmaxf(m0, m1);
                    w0 = m0 == -INFINITY ? 0.0f : exp2_fast(m0 - m);
                    w1 = m1 == -INFINITY ? 0.0f : exp2_fast(m1 - m);
                    l = merge_l[0][r] * w0 + merge_l[1][r] * w1;
                }
                if (warp_live) {
                    const bool both = !pair && n > 1;
                    const int d0 = pair ? 0 : s * (kD / 2), d1 = pair ? kD : d0 + kD / 2;
                    const float inv = 1.0f / l;
                    w0 *= inv;
                    w1 *= inv;
                    const int64_t row = out_row0 + rel;
                    float4 *dst = reinterpret_cast<float4 *>(p.part) + (row >> 5) * (8 * kD) + (row & 31);
                    const uint32_t col = pair ? o_col : tmem + lanes + 256u;
#pragma unroll 1
                    for (int j = d0; j < d1; j += 32) {
                        float o[32], o1[32];
                        tmem_ld32_async(col + j, o);
                        if (both) tmem_ld32_async(col + kTile + j, o1);
                        tmem_wait_ld32(o);
                        if (both) tmem_wait_ld32(o1);
#pragma unroll
                        for (int x = 0; x < 32; ++x) {
                            o[x] *= w0;
                            if (both) o[x] = fmaf(o1[x], w1, o[x]);
                        }
                        if (live && l != 0.0f) {
#pragma unroll
                            for (int x = 0; x < 8; ++x) dst[(j / 4 + x) * 32] = make_float4(o[4 * x], o[4 * x + 1], o[4 * x + 2], o[4 * x + 3]);
                        }
                    }
                    if (live && (pair || s == 0)) p.lse[row] = l == 0.0f ? -INFINITY : m - kLift + log2f(l);
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&o_free);   // O may be written again
            }
            if (id >= jobs) break;
            job = next;
            running = job.ntiles > 0;
            id += stride;
            len = own_length(p, id);
            if (!running) {   // no key: nothing of these rows in this slot
                float *lse = p.lse + (static_cast<int64_t>(job.slot) * g.Hkv + job.h) * p.row_blocks * 32 + job.i0;
                for (int x = tid; x < job.nrows; x += 256) lse[x] = -INFINITY;
            }
        }
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsOther));
    if (warp < kLoadWarp) {
        // ------------------------------------------------ products of stream s: one thread, in the
        // order S(0) PV(0) S(1) PV(1) ...; a thread a stream, since what one waits for must not
        // hold up the other's products
        const int s = warp - kMmaWarp;
        if (elect_one()) {
            constexpr uint32_t idesc_s = idesc_16bit_f32(kTile, kTile, kBf16, false);
            constexpr uint32_t idesc_o = idesc_16bit_f32(kTile, kD, kBf16, true);
            const uint64_t q_desc = smem_desc_sw128(smem_addr(smem)), k_desc = smem_desc_sw128(smem_addr(ring));
            const uint64_t v_desc = smem_desc_sw128_mn(smem_addr(ring), kBlock);
            const uint32_t s_tmem = tmem + static_cast<uint32_t>(s * kTile), o_tmem = s_tmem + 256u;
            int pos0 = 0;
            uint32_t done = 0, step = 0, turns = 0;
            bool ok = true;
            for (; id < jobs && ok; id += stride) {
                const Job job = job_of(p, id, len);
                len = own_length(p, id + stride);
                const int n = job.ntiles;
                if (n == 0) continue;
                const bool pair = kWide && job.nrows > kTile;
                const int steps = pair ? n : (n - s + 1) / 2;
                const uint64_t qd = q_desc + (pair && s == 1 ? kSlotBytes >> 4 : 0u);
                auto k_at = [&](int i) { return pos0 + k_pos(pair ? i : 2 * i + s); };
                ok = !*abort_word && wait_for(&q_full, done & 1u);
#pragma unroll 1
                for (int i = -1; i < steps && ok; ++i) {
                    ok = i + 1 >= steps || landed(k_at(i + 1), pair);
                    if (i >= 0 && ok) {
                        const int pos = pos0 + v_pos(pair ? i : 2 * i + s, n);
                        const uint64_t vd = v_desc + static_cast<uint32_t>(pos % kSlots) * (kSlotBytes >> 4);
                        ok = landed(pos, pair) && !*abort_word;
                        // the last job's results have been read before O is written again
                        if (ok && i == 0 && done > 0) ok = wait_for(&o_free, (done - 1) & 1u);
                        ok = ok && wait_for(&p_half[s], step & 1u);
                        if (!ok) break;
                        tc_fence_after();
                        auto issue_pv = [&](int k) {   // 16 keys: 2048 bytes of V, 8 columns of P
                            umma_f16_ta(o_tmem, s_tmem + 8u * k, vd + 128u * k, idesc_o, (i > 0 || k > 0) ? 1u : 0u);
                        };
#pragma unroll
                        for (int k = 0; k < kTile / 32; ++k) issue_pv(k);
                        // Two streams over the same tiles take turns: their products, mixed, would
                        // end together, and then their exponentials would run together.
                        if (pair) {
                            if (s == 1 || turns > 0) ok = wait_for(&turn[s], (turns + s - 1) & 1u);
                            ++turns;
                        }
                        ok = ok && wait_for(&p_full[s], step & 1u);
                        ++step;
                        if (!ok) break;
                        tc_fence_after();
#pragma unroll
                        for (int k = kTile / 32; k < kTile / 16; ++k) issue_pv(k);
                    }
                    if (i + 1 < steps && ok) {
                        const uint64_t kd = k_desc + static_cast<uint32_t>(k_at(i + 1) % kSlots) * (kSlotBytes >> 4);
                        tc_fence_after();
#pragma unroll
                        for (int k = 0; k < kD / 16; ++k) {
                            const uint32_t off = (static_cast<uint32_t>(k / 4) * kBlock + 32u * (k % 4)) >> 4;
                            umma_f16_ss(s_tmem, qd + off, kd + off, idesc_s, k > 0 ? 1u : 0u);
                        }
                        umma_commit(&s_full[s]);
                    }
                    if (i >= 0 && pair) mbar_arrive(&turn[1 - s]);
                }
                if (ok) umma_commit(&o_done);
                ++done;
                pos0 += 2 * n;
            }
            if (!ok) fail();
            // every product has completed before tensor memory is released
            umma_commit(&drained[s]);
            (void)wait_for(&drained[s], 0u);
        }
        __syncwarp();
    } else {
        // ------------------------------------------------ K and V: a thread of warp 10 loads the
        // first, one of warp 11 the second 64 elements of each row (64-wide heads: the even and
        // the odd pages). One thread for all took 500 cycles a slot to issue its copies, and a
        // whole warp, a lane a page, as long.
        if (elect_one()) {
            const int box = min(g.page, kTile), shift = __ffs(g.page) - 1, half = warp - kLoadWarp;
            constexpr int kStep = kChunks == 1 ? 2 : 1, kMost = kTile / 16 / kStep;   // this thread's pages of a tile:
            const int first = kChunks == 1 ? half : 0;                                // first, first + kStep, ...
            int pos = 0;
            bool ok = true;
            for (; id < jobs && ok; id += stride) {
                const Job job = job_of(p, id, len);
                len = own_length(p, id + stride);
                const int32_t *table = (job.own_b < 0 ? g.prefix_table : g.own_table + static_cast<int64_t>(job.own_b) * g.own_pages) + (job.key0 >> shift);
                const int in_page = static_cast<int>(job.key0 & (g.page - 1));   // (0 but for pages of 256)
#pragma unroll 1
                for (int q = 0; q < 2 * job.ntiles; ++q, ++pos) {   // K0 K1 V0 K2 V1 ...
                    const bool v = (q > 0 && q % 2 == 0) || q == 2 * job.ntiles - 1;
                    const int t = !v ? (q + 1) / 2 : q % 2 == 0 ? q / 2 - 1 : job.ntiles - 1;
                    const int at = pos % kSlots, pages = (min(kTile, job.keys - t * kTile) + box - 1) / box;
                    // the pages' numbers, all on their way at once
                    int page[kMost];
#pragma unroll
                    for (int x = 0; x < kMost; ++x)
                        if (first + kStep * x < pages) page[x] = __ldg(table + ((in_page + t * job.step * kTile + (first + kStep * x) * box) >> shift));
                    if (*abort_word || (pos >= kSlots && !wait_for(&freed[at], full_parity(pos) ^ 1u))) {
                        ok = false;
                        break;
                    }
                    mbar_arrive_expect_tx(&full[at], static_cast<uint32_t>(max((pages - first + kStep - 1) / kStep, 0)) * box * 128u);
                    uint8_t *dst = ring + at * kSlotBytes + (kChunks == 1 ? first * box * 128 : half * kBlock);
#pragma unroll
                    for (int x = 0; x < kMost; ++x) {
                        if (first + kStep * x >= pages) break;
                        if (page[x] < 0 || page[x] >= g.n_pages) {   // no page: read past the cache, zeros
                            atomicOr(&g_attention_error, kErrIndex);
                            page[x] = static_cast<int>(g.n_pages);
                        }
                        tma_load_4d(dst + kStep * x * box * 128, v ? &p.v : &p.k, kChunks == 1 ? 0 : 64 * half,
                                    (in_page + t * job.step * kTile) & (g.page - 1), job.h, page[x], &full[at]);
                    }
                }
                if (!ok) fail();
            }
            // Every copy lands before the CTA can exit: the products wait for each of them, unless
            // something gave up; then this thread waits (bounded) for those it last started.
            if (*abort_word) {
                for (int x = max(0, pos - kSlots); x < pos; ++x) (void)wait_for(&full[x % kSlots], full_parity(x));
            }
        }
        __syncwarp();
    }
    }
    if (p.chained) grid_dependency_wait();   // whoever waits for this launch waits for both
    tc_fence_before();
    __syncthreads();
    if (warp == kMmaWarp) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols) : "memory");
    }
}

// ---- few rows: a request's own keys against its rows (T G <= 64), and the prefix where all
// requests together have 16 at most
//
// A decode step's requests have a handful of rows each and no own key in common: bound by
// the bytes of K and V. A CTA takes 16 rows (m16n8k16 products) and a range of keys; its four
// warps take 16 keys in turn, each with a ring of asynchronous copies, statistics and output
// sums of its own, so that nothing waits for anything but memory, and are joined at the end.
// (As jobs of the kernel above, 128 rows a product and one range at a time an SM, 64
// requests of up to 1024 keys took 48 to 65 us; so 40.)
constexpr int kFewWarps = 4, kFewStages = 3;
template <int kD>
constexpr int few_smem() { return kFewWarps * kFewStages * 2 * 16 * kD * 2; }

__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], uint32_t addr)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void ldmatrix4_trans(uint32_t (&r)[4], uint32_t addr)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
template <typename T>
__device__ __forceinline__ void mma_16bit(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    if constexpr (std::is_same_v<T, __half>) {
        mma_16816(d, a[0], a[1], a[2], a[3], b0, b1);
    } else {
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    }
}

template <typename T, int kD>
__global__ void __launch_bounds__(32 * kFewWarps) few_rows_kernel(const __grid_constant__ AttnParams p)
{
    constexpr float kLift = std::is_same_v<T, __half> ? 6.0f : 0.0f;   // as above
    constexpr int kRowBytes = kD * 2, kTileBytes = 16 * kRowBytes, kPieces = kD / 8;
    extern __shared__ __align__(1024) uint8_t smem[];
    __shared__ float stat_m[kFewWarps][16], stat_l[kFewWarps][16];
    const AttnArgs &g = p.g;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, gid = lane >> 2, t = lane & 3;
    const int G = g.Hq / g.Hkv, per = g.T * G;
    grid_dependency_wait();
    grid_launch_dependents();
    // the job: 16 rows of key head h, a range of a request's own keys or of the prefix
    const bool on_prefix = blockIdx.x >= static_cast<unsigned>(p.plan.few_jobs);
    int id = static_cast<int>(blockIdx.x) - (on_prefix ? static_cast<int>(p.plan.few_jobs) : 0);
    const int tiles = on_prefix ? 1 : p.plan.few_row_tiles;
    const int splits = on_prefix ? p.plan.lone_splits : p.plan.own_splits, most = on_prefix ? p.plan.few_prefix_keys : p.plan.few_keys;
    const int rt = id % tiles;
    id /= tiles;
    const int split = id % splits;
    id /= splits;
    const int h = id % g.Hkv, b = id / g.Hkv;   // (b: 0 on the prefix)
    int64_t len = on_prefix ? g.prefix_len : g.own_len[b];
    if (!on_prefix && len > g.max_own) {
        if (tid == 0) atomicOr(&g_attention_error, kErrIndex);
        len = g.max_own;
    }
    const int rows = on_prefix ? g.B * per : per, i0 = b * per + rt * 16, nrows = min(16, rows - rt * 16);
    const int slot = (on_prefix ? p.plan.own_splits : 0) + split;
    const int64_t out_row0 = (static_cast<int64_t>(slot) * g.Hkv + h) * p.row_blocks * 32 + i0;
    const int64_t key0 = static_cast<int64_t>(split) * most;
    const int keys = static_cast<int>(max(static_cast<int64_t>(0), min(static_cast<int64_t>(most), len - key0)));
    if (keys == 0) {
        if (tid < nrows) p.lse[out_row0 + tid] = -INFINITY;
        return;
    }
    // ---- this warp's 16-key tiles warp, warp + 4, ...: page lookup and copies
    const int ntiles = (keys + 15) / 16, mine = (ntiles - warp + kFewWarps - 1) / kFewWarps;
    const int32_t *table = on_prefix ? g.prefix_table : g.own_table + static_cast<int64_t>(b) * g.own_pages;
    const int shift = __ffs(g.page) - 1;
    uint8_t *ring = smem + warp * kFewStages * 2 * kTileBytes;
    auto page_of = [&](int x) { return x < mine ? __ldg(table + ((key0 + (warp + kFewWarps * x) * 16) >> shift)) : 0; };
    auto load = [&](int x, int page) {
        if (x < mine) {
            const int k = (warp + kFewWarps * x) * 16;   // first key, from key0
            const bool there = page >= 0 && page < g.n_pages;   // (elsewhere: zeros)
            if (!there && lane == 0) atomicOr(&g_attention_error, kErrIndex);
            const int64_t at = ((static_cast<int64_t>(there ? page : 0) * g.page + ((key0 + k) & (g.page - 1))) * g.Hkv + h) * kD;
            const T *kc = static_cast<const T *>(g.k_cache) + at, *vc = static_cast<const T *>(g.v_cache) + at;
            uint8_t *dst = ring + (x % kFewStages) * 2 * kTileBytes;
#pragma unroll
            for (int i = 0; i < 16 * kPieces / 32; ++i) {
                const int key = (i * 32 + lane) / kPieces, c = (i * 32 + lane) % kPieces;
                const int64_t off = static_cast<int64_t>(key) * g.Hkv * kD + 8 * c;
                const int n = there && k + key < keys ? 16 : 0;   // past the last key: zeros, whatever is there
                const uint32_t to = smem_addr(dst) + key * kRowBytes + 16 * (c ^ (key & 7));
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(n ? kc + off : kc), "r"(n) : "memory");
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to + kTileBytes), "l"(n ? vc + off : vc), "r"(n) : "memory");
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    int ahead[kFewStages - 1];
#pragma unroll
    for (int x = 0; x < kFewStages - 1; ++x) ahead[x] = page_of(x);
    int page = page_of(kFewStages - 1);
#pragma unroll
    for (int x = 0; x < kFewStages - 1; ++x) load(x, ahead[x]);
    // ---- Q: row gid and gid + 8 of the tile, 16 of D a step
    uint32_t q[kD / 16][4];
    {
        const int ra = i0 + gid, rb = i0 + gid + 8;
        const bool has_a = gid < nrows, has_b = gid + 8 < nrows;
        const uint32_t *qa = reinterpret_cast<const uint32_t *>(static_cast<const T *>(g.q) + (static_cast<int64_t>(ra / G) * g.Hq + h * G + ra % G) * kD);
        const uint32_t *qb = reinterpret_cast<const uint32_t *>(static_cast<const T *>(g.q) + (static_cast<int64_t>(rb / G) * g.Hq + h * G + rb % G) * kD);
#pragma unroll
        for (int k = 0; k < kD / 16; ++k) {
            q[k][0] = has_a ? __ldg(qa + 8 * k + t) : 0u;
            q[k][1] = has_b ? __ldg(qb + 8 * k + t) : 0u;
            q[k][2] = has_a ? __ldg(qa + 8 * k + 4 + t) : 0u;
            q[k][3] = has_b ? __ldg(qb + 8 * k + 4 + t) : 0u;
        }
    }
    // keys, from key0, that rows gid and gid + 8 see: the prefix's, or their request's up to
    // their own token
    const int end = static_cast<int>(len - key0) - g.T + 1;
    const int limit[2] = {on_prefix ? keys : min(keys, end + (rt * 16 + gid) / G),
                          on_prefix ? keys : min(keys, end + (rt * 16 + gid + 8) / G)};
    const float c = g.scale * 1.4426950408889634f;
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f}, o[kD / 8][4];
#pragma unroll
    for (int d = 0; d < kD / 8; ++d)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[d][e] = 0.0f;
    for (int x = 0; x < mine; ++x) {
        asm volatile("cp.async.wait_group %0;" ::"n"(kFewStages - 2) : "memory");
        __syncwarp();   // every lane's copies of this tile have landed, and all have read the last one
        load(x + kFewStages - 1, page);
        page = page_of(x + kFewStages);
        const uint32_t kt = smem_addr(ring + (x % kFewStages) * 2 * kTileBytes), vt = kt + kTileBytes;
        float s[2][4] = {};
#pragma unroll
        for (int k = 0; k < kD / 16; ++k) {
            uint32_t f[4];   // keys 0 .. 7 and 8 .. 15, two halves of 16 of D each
            const int key = (lane & 7) + 8 * (lane >> 4), piece = 2 * k + ((lane >> 3) & 1);
            ldmatrix4(f, kt + key * kRowBytes + 16 * (piece ^ (key & 7)));
            mma_16bit<T>(s[0], q[k], f[0], f[1]);
            mma_16bit<T>(s[1], q[k], f[2], f[3]);
        }
        const int k0 = (warp + kFewWarps * x) * 16 + 2 * t;
        uint32_t pr[4];
#pragma unroll
        for (int r = 0; r < 2; ++r) {   // rows gid, gid + 8
            float e[4] = {s[0][2 * r], s[0][2 * r + 1], s[1][2 * r], s[1][2 * r + 1]};
#pragma unroll
            for (int y = 0; y < 4; ++y)
                if (k0 + (y & 1) + 8 * (y >> 1) >= limit[r]) e[y] = -INFINITY;
            float best = fmaxf(fmaxf(e[0], e[1]), fmaxf(e[2], e[3]));
            best = fmaxf(best, __shfl_xor_sync(0xffffffffu, best, 1));
            best = fmaxf(best, __shfl_xor_sync(0xffffffffu, best, 2)) * c;
            const bool grow = best > m[r] + kSlack;
            if (__any_sync(0xffffffffu, grow)) {
                const float next = grow ? best : m[r], fix = grow ? exp2_fast(m[r] - next) : 1.0f;
                m[r] = next;
                l[r] *= fix;
#pragma unroll
                for (int d = 0; d < kD / 8; ++d) {
                    o[d][2 * r] *= fix;
                    o[d][2 * r + 1] *= fix;
                }
            }
            const float shift = kLift - (m[r] == -INFINITY ? 0.0f : m[r]);
#pragma unroll
            for (int y = 0; y < 4; ++y) {
                e[y] = exp2_fast(fmaf(e[y], c, shift));
                l[r] += e[y];
            }
            pr[r] = pack2<T>(e[0], e[1]);       // keys 0 .. 7 of P
            pr[2 + r] = pack2<T>(e[2], e[3]);   // keys 8 .. 15
        }
#pragma unroll
        for (int d = 0; d < kD / 8; d += 2) {
            uint32_t f[4];   // 8 of D: keys 0 .. 7, 8 .. 15; the next 8: the same
            const int key = (lane & 7) + 8 * ((lane >> 3) & 1), piece = d + (lane >> 4);
            ldmatrix4_trans(f, vt + key * kRowBytes + 16 * (piece ^ (key & 7)));
            mma_16bit<T>(o[d], pr, f[0], f[1]);
            mma_16bit<T>(o[d + 1], pr, f[2], f[3]);
        }
    }
    // ---- the warps' parts joined
    asm volatile("cp.async.wait_all;" ::: "memory");
#pragma unroll
    for (int r = 0; r < 2; ++r) {
        l[r] += __shfl_xor_sync(0xffffffffu, l[r], 1);
        l[r] += __shfl_xor_sync(0xffffffffu, l[r], 2);
        if (t == 0) {
            stat_m[warp][gid + 8 * r] = m[r];
            stat_l[warp][gid + 8 * r] = l[r];
        }
    }
    __syncthreads();
    constexpr int kPitch = kD + 4;
    float *part = reinterpret_cast<float *>(ring);   // this warp's ring, [16][kD + 4]
#pragma unroll
    for (int r = 0; r < 2; ++r) {
        // A warp without a key for this row has the sum 0 beside m = -inf. A sum of NaN stands
        // beside -inf too where all its scores are NaN (no maximum is above -inf then): it goes on.
        float top = -INFINITY, sum = 0.0f;
#pragma unroll
        for (int w = 0; w < kFewWarps; ++w) top = fmaxf(top, stat_m[w][gid + 8 * r]);
#pragma unroll
        for (int w = 0; w < kFewWarps; ++w) {
            const float lw = stat_l[w][gid + 8 * r];
            sum += lw == 0.0f ? 0.0f : lw * exp2_fast(stat_m[w][gid + 8 * r] - top);
        }
        const float fix = l[r] == 0.0f ? 0.0f : exp2_fast(m[r] - top) / sum;
#pragma unroll
        for (int d = 0; d < kD / 8; ++d)
            *reinterpret_cast<float2 *>(part + (gid + 8 * r) * kPitch + 8 * d + 2 * t) = make_float2(o[d][2 * r] * fix, o[d][2 * r + 1] * fix);
        if (warp == 0 && t == 0 && gid + 8 * r < nrows) p.lse[out_row0 + gid + 8 * r] = sum == 0.0f ? -INFINITY : top - kLift + log2f(sum);
    }
    __syncthreads();
    constexpr int kRingFloats = kFewStages * 2 * kTileBytes / 4;
    static_assert(16 * kPitch <= kRingFloats, "a warp's part fits its ring");
    for (int e = tid; e < 16 * (kD / 4); e += 32 * kFewWarps) {
        const int r = e % 16, d4 = e / 16;
        if (r >= nrows) continue;
        const float *src = reinterpret_cast<const float *>(smem) + r * kPitch + 4 * d4;
        float4 v = *reinterpret_cast<const float4 *>(src);
#pragma unroll
        for (int w = 1; w < kFewWarps; ++w) {
            const float4 u = *reinterpret_cast<const float4 *>(src + w * kRingFloats);
            v.x += u.x;
            v.y += u.y;
            v.z += u.z;
            v.w += u.w;
        }
        const int64_t row = out_row0 + r;
        reinterpret_cast<float4 *>(p.part)[(row >> 5) * (8 * kD) + d4 * 32 + (row & 31)] = v;
    }
}

template <typename T>
__device__ __forceinline__ float2 widen2(uint32_t two)
{
    if constexpr (std::is_same_v<T, __half>) {
        return __half22float2(*reinterpret_cast<const __half2 *>(&two));
    } else {
        return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&two));
    }
}

// Columns d0 .. d0 + 7 of row i once more, where they did not come out finite. In the products
// above a key that the row does not see (a later token of its request) has P = 0, which an
// infinity or NaN among that key's values turns into NaN. If there is one, the row's own keys
// are gone through one by one, only those that it sees, beside the prefix's partial results:
// what is still not finite is the formula's. Bound by latency, 2 us a key, for such rows alone.
// (Looking through those values before each product
// instead cost 3 to 5 % of the calls with several tokens a request.)
template <typename T, int kD>
__device__ __forceinline__ void row_again(const AttnParams &p, int h, int i, int d0, int64_t per_slot, int slots, const float *lse,
                                          const float4 *part, float (&acc)[8], float &sum)
{
    const AttnArgs &g = p.g;
    const int G = g.Hq / g.Hkv, b = i / G / g.T, shift = __ffs(g.page) - 1;
    const int64_t own = min(static_cast<int64_t>(__ldg(g.own_len + b)), g.max_own), seen = own - g.T + 1 + i / G % g.T;
    // where an own key's row of the caches begins, or -1: its page is outside
    auto place = [&](int64_t key) -> int64_t {
        const int page = __ldg(g.own_table + static_cast<int64_t>(b) * g.own_pages + (key >> shift));
        return page < 0 || page >= g.n_pages ? -1 : ((static_cast<int64_t>(page) * g.page + (key & (g.page - 1))) * g.Hkv + h) * kD;
    };
    auto load_v = [&](int64_t at, float (&v)[8]) {
        const uint4 eight = __ldg(reinterpret_cast<const uint4 *>(static_cast<const T *>(g.v_cache) + at + d0));
        const uint32_t twos[4] = {eight.x, eight.y, eight.z, eight.w};
#pragma unroll
        for (int x = 0; x < 4; ++x) {
            const float2 e = widen2<T>(twos[x]);
            v[2 * x] = e.x;
            v[2 * x + 1] = e.y;
        }
    };
    bool hidden = false;
#pragma unroll 1
    for (int64_t key = max(static_cast<int64_t>(0), seen); key < own && !hidden; ++key) {
        const int64_t at = place(key);
        if (at < 0) continue;
        float v[8];
        load_v(at, v);
#pragma unroll
        for (int x = 0; x < 8; ++x) hidden |= !isfinite(v[x]);
    }
    if (!hidden) return;   // what is not finite is the formula's own
    const float c = g.scale * 1.4426950408889634f;
    const int64_t q_row = (static_cast<int64_t>(i / G) * g.Hq + h * G + i % G) * kD;
    float top = -INFINITY;
    sum = 0.0f;
#pragma unroll
    for (int x = 0; x < 8; ++x) acc[x] = 0.0f;
    // eight values v with the logarithm e of their weight
    auto add = [&](float e, const float *v) {
        if (e == -INFINITY) return;
        const float next = fmaxf(top, e), fix = top == -INFINITY ? 1.0f : exp2_fast(top - next), w = exp2_fast(e - next);
        top = next;
        sum = fmaf(sum, fix, w);
#pragma unroll
        for (int x = 0; x < 8; ++x) acc[x] = fmaf(w, v[x], acc[x] * fix);
    };
#pragma unroll 1
    for (int k = p.plan.own_splits; k < slots; ++k) {
        const float4 lo = part[k * per_slot * (kD / 4)], hi = part[k * per_slot * (kD / 4) + 32];
        const float v[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
        add(lse[k * per_slot], v);
    }
#pragma unroll 1
    for (int64_t key = 0; key < seen; ++key) {
        float s = 0.0f, v[8] = {};   // (what a page outside the cache reads as)
        const int64_t at = place(key);
        if (at >= 0) {
            const uint4 *k8 = reinterpret_cast<const uint4 *>(static_cast<const T *>(g.k_cache) + at);
            const uint4 *q8 = reinterpret_cast<const uint4 *>(static_cast<const T *>(g.q) + q_row);
            load_v(at, v);
#pragma unroll 4
            for (int d = 0; d < kD / 8; ++d) {
                const uint4 a = __ldg(q8 + d), e = __ldg(k8 + d);
                const uint32_t as[4] = {a.x, a.y, a.z, a.w}, es[4] = {e.x, e.y, e.z, e.w};
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    const float2 u = widen2<T>(as[x]), y = widen2<T>(es[x]);
                    s = fmaf(u.x, y.x, fmaf(u.y, y.y, s));
                }
            }
        }
        add(s * c, v);
    }
}

// Joins the partial results of 32 rows of a key head for 8 of D, a row a lane: weights
// 2^(lse - max) over their sum. Bound by latency: the four warps take every fourth slot, so
// that about all loads are under way at once, statistics and results alike, and are joined
// in shared memory. (A warp for all slots of 8 of D: 24 requests behind 8191 keys took 30 us in all, so 26.)
template <typename T, int kD>
__global__ void __launch_bounds__(128) attention_join_kernel(const __grid_constant__ AttnParams p)
{
    constexpr int kWarps = 4, kAhead = 6, kParts = kD / 8;
    __shared__ float tops[kWarps][32], sums[kWarps][32], accs[kWarps][8][32];
    const AttnArgs &g = p.g;
    const int lane = threadIdx.x & 31, warp = static_cast<int>(threadIdx.x >> 5), d0 = static_cast<int>(blockIdx.x) % kParts * 8;
    const int block = static_cast<int>(blockIdx.x) / kParts % p.row_blocks, h = static_cast<int>(blockIdx.x) / kParts / p.row_blocks;
    const int G = g.Hq / g.Hkv, i = block * 32 + lane;
    const bool live = i < g.B * g.T * G;
    // these rows' prefix slots: those of their row group
    const int slots = p.plan.own_splits + (block * 32 < p.plan.pair_groups * 2 * kTile ? p.plan.pair_splits : p.plan.lone_splits);
    const int64_t per_slot = static_cast<int64_t>(g.Hkv) * p.row_blocks * 32;
    const float *lse = p.lse + static_cast<int64_t>(h) * p.row_blocks * 32 + i;
    const float4 *part = reinterpret_cast<const float4 *>(p.part) + (static_cast<int64_t>(h) * p.row_blocks + block) * 8 * kD + d0 * 8 + lane;
    grid_launch_dependents();
    grid_dependency_wait();
    float acc[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f}, sum = 0.0f, top = -INFINITY;
    for (int k0 = warp; k0 < slots; k0 += kWarps * kAhead) {
        float e[kAhead];
        float4 v[kAhead][2];
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            const int k = k0 + u * kWarps;
            const bool in = k < slots && live;
            e[u] = in ? lse[k * per_slot] : -INFINITY;
#pragma unroll
            for (int x = 0; x < 2; ++x)   // (where lse is -inf nothing was written: looked at no further)
                v[u][x] = in ? part[k * per_slot * (kD / 4) + 32 * x] : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        }
        float best = top;
#pragma unroll
        for (int u = 0; u < kAhead; ++u) best = fmaxf(best, e[u]);
        const float fix = top == -INFINITY ? 0.0f : exp2_fast(top - best);
        top = best;
        sum *= fix;
#pragma unroll
        for (int x = 0; x < 8; ++x) acc[x] *= fix;
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            if (e[u] == -INFINITY) continue;
            const float w = exp2_fast(e[u] - top);
            sum += w;
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                acc[4 * x] = fmaf(w, v[u][x].x, acc[4 * x]);
                acc[4 * x + 1] = fmaf(w, v[u][x].y, acc[4 * x + 1]);
                acc[4 * x + 2] = fmaf(w, v[u][x].z, acc[4 * x + 2]);
                acc[4 * x + 3] = fmaf(w, v[u][x].w, acc[4 * x + 3]);
            }
        }
    }
    tops[warp][lane] = top;
    sums[warp][lane] = sum;
#pragma unroll
    for (int x = 0; x < 8; ++x) accs[warp][x][lane] = acc[x];
    __syncthreads();
    if (warp > 0 || !live) return;
#pragma unroll
    for (int w = 1; w < kWarps; ++w) top = fmaxf(top, tops[w][lane]);
    const float own = tops[0][lane], mine = own == -INFINITY ? 0.0f : exp2_fast(own - top);
    sum *= mine;
#pragma unroll
    for (int x = 0; x < 8; ++x) acc[x] *= mine;
#pragma unroll
    for (int w = 1; w < kWarps; ++w) {
        if (tops[w][lane] == -INFINITY && sums[w][lane] == 0.0f) continue;
        const float f = exp2_fast(tops[w][lane] - top);
        sum = fmaf(f, sums[w][lane], sum);
#pragma unroll
        for (int x = 0; x < 8; ++x) acc[x] = fmaf(f, accs[w][x][lane], acc[x]);
    }
    if (g.T > 1 && p.plan.own_splits > 0) {
        bool finite = true;
#pragma unroll
        for (int x = 0; x < 8; ++x) finite &= isfinite(acc[x]);
        if (!finite) row_again<T, kD>(p, h, i, d0, per_slot, slots, lse, part, acc, sum);
    }
    float inv = 1.0f / sum;   // (all scores -inf: 0 / 0, as the formula has it)
    if (sum == 0.0f && g.prefix_len == 0) {   // no key at all: zeros
        const int64_t own = g.max_own > 0 ? min(static_cast<int64_t>(g.own_len[i / G / g.T]), g.max_own) : 0;
        if (own - g.T + 1 + i / G % g.T <= 0) inv = 0.0f;
    }
    uint4 out;
    out.x = pack2<T>(acc[0] * inv, acc[1] * inv);
    out.y = pack2<T>(acc[2] * inv, acc[3] * inv);
    out.z = pack2<T>(acc[4] * inv, acc[5] * inv);
    out.w = pack2<T>(acc[6] * inv, acc[7] * inv);
    *reinterpret_cast<uint4 *>(static_cast<T *>(g.out) + (static_cast<int64_t>(i / G) * g.Hq + h * G + i % G) * kD + d0) = out;
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

template <typename T, int kD, bool kWide>
cudaError_t launch_typed(const AttnParams &p, cudaStream_t s)
{
    const AttnArgs &g = p.g;
    cudaLaunchAttribute attr[1];
    cudaLaunchConfig_t cfg = {};
    cfg.stream = s;
    cfg.attrs = attr;
    const int64_t jobs = p.plan.prefix_jobs + p.plan.own_jobs;
    auto beside_the_last = [&]() {   // starts as the last of the launch before run
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        cfg.numAttrs = 1;
    };
    cfg.numAttrs = set_launch_overlap_attr(attr);
    if (p.plan.few_jobs + p.plan.few_prefix_jobs > 0) {
        auto kern = few_rows_kernel<T, kD>;
        cudaError_t e = ensure_smem_attr(reinterpret_cast<const void *>(kern), few_smem<kD>());
        if (e != cudaSuccess) return e;
        cfg.blockDim = dim3(32 * kFewWarps);
        cfg.gridDim = dim3(static_cast<unsigned>(p.plan.few_jobs + p.plan.few_prefix_jobs));
        cfg.dynamicSmemBytes = few_smem<kD>();
        if ((e = cudaLaunchKernelEx(&cfg, kern, p)) != cudaSuccess) return e;
        beside_the_last();
    }
    if (jobs > 0) {
        auto kern = attention_kernel<T, kD, kWide>;
        cudaError_t e = ensure_smem_attr(reinterpret_cast<const void *>(kern), kSmemBytes);
        if (e != cudaSuccess) return e;
        cfg.blockDim = dim3(kThreads);
        cfg.gridDim = dim3(static_cast<unsigned>(p.plan.prefix_ctas + p.plan.own_ctas));
        cfg.dynamicSmemBytes = kSmemBytes;
        if ((e = cudaLaunchKernelEx(&cfg, kern, p)) != cudaSuccess) return e;
        beside_the_last();
    }
    cfg.blockDim = dim3(128);
    cfg.gridDim = dim3(static_cast<unsigned>(p.row_blocks * g.Hkv * (kD / 8)));
    cfg.dynamicSmemBytes = 0;
    return cudaLaunchKernelEx(&cfg, attention_join_kernel<T, kD>, p);
}

int64_t row_blocks_of(int B, int T, int Hq, int Hkv) { return ceil_div(static_cast<int64_t>(B) * T * (Hq / Hkv), 32); }

}  // namespace

// Bytes for any plan of at most these sizes: a caller keeps the workspace of its largest
// batch. (A plan's own need is not monotone, since fewer rows are split into more ranges.) In
// blocks of 32 rows of a key head, of which there are n: the prefix is cut into at most a
// range a tile, 256 ranges, and in all n + 8 blocks x 152 SMs (plan_attention gives a pair of
// streams, 8 blocks, 152 times its share of the cost, rounded); own keys into a range of 256
// keys at least, 256 ranges, and n + 8 x 152, or above 64 rows a request, of 8 blocks a job,
// n + 8 x 3/2 x 304.
int64_t attn_workspace_bytes(int B, int T, int Hq, int Hkv, int D, int64_t prefix_len, int64_t max_own)
{
    const int64_t n = Hkv * row_blocks_of(B, T, Hq, Hkv), most = 256;
    const int64_t prefix = std::min(n * std::min(ceil_div(prefix_len, kTile), most), n + 8 * kSms);
    const int64_t own = std::min(n * std::min(ceil_div(max_own, 2 * kTile), most),
                                 n + 8 * kSms * (static_cast<int64_t>(T) * (Hq / Hkv) > kFewRows ? 3 : 1));
    const int64_t planned = n * plan_attention(B, T, Hq, Hkv, prefix_len, max_own).slots;
    return std::max(prefix + own, planned) * 32 * (D + 1) * 4;
}

cudaError_t launch_attention(const AttnArgs &g, cudaStream_t s)
{
    route_hit(kRoutePrefixAttention);
    AttnParams p{};
    p.g = g;
    p.plan = plan_attention(g.B, g.T, g.Hq, g.Hkv, g.prefix_len, g.max_own);
    if (p.plan.prefix_jobs + p.plan.own_jobs > 0x7fffffffLL || p.plan.few_jobs + p.plan.few_prefix_jobs > 0x7fffffffLL) return cudaErrorInvalidValue;
    p.chained = p.plan.few_jobs + p.plan.few_prefix_jobs > 0;
    p.row_blocks = static_cast<int>(row_blocks_of(g.B, g.T, g.Hq, g.Hkv));
    p.part = static_cast<float *>(g.workspace);
    p.lse = p.part + p.plan.slots * static_cast<int64_t>(g.Hkv) * p.row_blocks * 32 * g.D;
    if (p.plan.prefix_jobs + p.plan.own_jobs > 0) {
        cudaError_t e = encode_cache_map(&p.k, g.k_cache, g);
        if (e == cudaSuccess) e = encode_cache_map(&p.v, g.v_cache, g);
        if (e != cudaSuccess) return e;
    }
    const bool wide = p.plan.pair_groups > 0 || (p.plan.own_jobs > 0 && static_cast<int64_t>(g.T) * (g.Hq / g.Hkv) > kTile);
    auto launch = [&](auto type) {
        using T = decltype(type);
        if (g.D == 64)
            return wide ? launch_typed<T, 64, true>(p, s) : launch_typed<T, 64, false>(p, s);
        return wide ? launch_typed<T, 128, true>(p, s) : launch_typed<T, 128, false>(p, s);
    };
    return g.type == QMV_F16 ? launch(__half()) : launch(__nv_bfloat16());
}

cudaError_t read_error_word_attention(uint32_t *out, bool clear)
{
    cudaError_t e = cudaMemcpyFromSymbol(out, g_attention_error, sizeof(uint32_t));
    if (e != cudaSuccess || !clear) return e;
    const uint32_t zero = 0;
    return cudaMemcpyToSymbol(g_attention_error, &zero, sizeof(uint32_t));
}

}  // namespace qmv
