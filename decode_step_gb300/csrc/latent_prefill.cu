// Attention of whole prompts over the latent cache, expanded form: every
// head's keys (w_uk[h] c, kr) and values w_uv[h] c are multiplied out once,
// then ordinary causal attention.  Per (row, token, head) that costs
// 2 (nope + 64 + v) flop where the absorbed form costs 2 (2 latent_dim + 64):
// 640 against 2176 at 128, 128 and 512, for 2 latent_dim (nope + v) more per
// (token, head).  Two kernels, the second a programmatic dependent of the
// first:
//
//  1. latent_expand_kernel: checks the streams, lays out their tokens in the
//     workspace (each stream from a 128-token boundary) and their query tiles,
//     and multiplies keys and values out: a tcgen05 GEMM whose token rows are
//     fetched through the block table.  37 us for 8891 tokens (16 heads, 512 ->
//     128 + 128: 1.0 PFLOP/s, 73 MB written), 9 us for 333, latency.
//  2. latent_prefill_kernel: attention of 256 rows of one head per CTA (two
//     128-row tiles that take turns on the tensor core: while one's weights
//     are computed, the other's products run).  S and O are in tensor memory;
//     the weights go back into S's columns (as f16) and are the A operand of
//     the second product.  Bound: the tensor core (640 flop a row, token and
//     head); 251 us for 8191 rows after 700 tokens, 1.60 PFLOP/s, 85% of the
//     measured rate of a large bf16 matrix product.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <atomic>
#include <cfloat>
#include <cmath>
#include <type_traits>

#include "latent_common.cuh"
#include "tcgen05.cuh"
#include "tts_common.cuh"
#include "tts_internal.h"

namespace tts {
namespace {

constexpr unsigned kFull = 0xFFFFFFFFu;
constexpr int kTile = 128;                 // tokens per tile, rows per query half
constexpr int kRows = 256;                 // query rows per work item
constexpr int kChunkBytes = kTile * 128;   // [128 rows][64 values] bf16, 128-byte swizzle
constexpr float kLog2e = 1.4426950408889634f;
// Running maximum before any token (log2 units): no finite score is below it, so
// that a row whose scores are all far below zero still has weights.
constexpr float kNoScore = -FLT_MAX;
constexpr float kSlack = 8.0f;             // scores may pass it by this much before it moves (log2 units)

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    const __nv_bfloat162 p = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&p);
}

// Values and softmax weights are f16: it holds them to 2^-11 where bf16 holds
// them to 2^-8, at the same rate.
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
    const __half2 p = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&p);
}
// Where f16 does not hold the values of a head's 128 tokens (of some token the
// largest is not in [2^-10, 65504]), each token's are kept divided by 2^e, e the
// exponent of its largest, and e is added to its scores (in log2 units): the
// weights are then w_t 2^e, held as precisely against the largest of them, and
// the sum of the weights w_t themselves is computed beside.  So a value is held to
// 2^-11 of itself or 2^-15 of its token's largest, and no finite one spreads to
// rows that do not see it.  e's limits keep the sum, relative to the largest
// w_t 2^e, between 2^-121 and 2^122 (2^24 tokens).
constexpr uint32_t kScaled = 0x100;
constexpr int kMinExp = -90, kMaxExp = 113;
__device__ __forceinline__ bool f16_holds(float largest) { return largest >= 0x1.0p-10f && largest <= 65504.0f; }
__device__ __forceinline__ int value_exp(float largest) {  // of a token's largest value
    return min(max(static_cast<int>(__float_as_uint(largest) >> 23) - 127, kMinExp), kMaxExp);
}

// kRows rows of one stream, what they see and where its keys and values are
struct __align__(16) QueryTile {
    int first, rows, ctx, tile0;  // of the stream: first row, rows, tokens, first token tile
    int q, unused[3];             // which of its tiles
};

struct PrefillArgs {
    const int32_t *table;
    int max_blocks, num_blocks;
    const int32_t *ctx_lens;
    const int32_t *row_start;
    int max_total, B, num_rows, Hq, L, nope, v;
    float scale_log2;
    int32_t *tile_start;   // [B] first token tile of each stream
    int32_t *num_qtiles;   // query tiles in all
    QueryTile *qtiles;     // [max_qtiles] those that see the most tokens first
    int max_qtiles;
    uint32_t *info;        // [Hq][max_tiles] bit i: block i of the tile is in the pool; kScaled: the head's values there are scaled
    int max_tiles;
    int8_t *exps;          // [Hq][max_tiles][128] the tokens' e, where scaled
    const __nv_bfloat16 *pool;
    __nv_bfloat16 *kr;     // [token tiles * 128][64]
    __nv_bfloat16 *out;
    int32_t *err;
    long long wait_limit;  // SM clock cycles per bounded wait of the attention
    int stall;             // test support: the first tile's keys expect 16 bytes that never come
};

// ------------------------------------------------------------------ expand

// K[t][h nope + d] = w_uk[h][d] . c_t (bf16) and V likewise (f16): a GEMM of
// 128-token x 256-feature units (128-feature ones for few tokens).  Persistent,
// one CTA per SM.  A unit reads 384 KB from L2 for 33 Mflop; 128 x 128 units
// were bound by those reads (10 TB/s of L2 to the SMs, 56 us at 8891 tokens x
// 4096 features x 512), and weights kept in shared memory left too short a ring
// (90 us).  (The weights are not multicast to pairs of CTAs: such copies are only
// for programs on one GPU, and replicas on several use this library too.)  The accumulator is double buffered: one unit's results
// leave (through shared memory, by TMA) while the next one's products run.
// Every CTA scans the streams by itself; CTA 0 writes the plan that the
// attention reads.  The first feature unit of a token tile also copies the
// tokens' rotated key parts and records which blocks are in the pool.
constexpr int kExpandThreads = 224;        // 4 epilogue warps, producer, MMA issuer, spare (tensor memory)
constexpr int kExpandSlots = 4;
constexpr int kExpandCtas = 152;
constexpr int kFeatures = 256, kWeightRows = 128;  // features per unit at most; weight rows per copy
constexpr int kSlotBytes = 3 * kChunkBytes;    // 128 token rows, 256 feature rows of 64 values
constexpr int kExpandSmem = kExpandSlots * kSlotBytes + 2 * kChunkBytes;

struct ExpandShared {
    uint64_t full[kExpandSlots], empty[kExpandSlots], acc_full[2], acc_empty[2], fin;
    uint32_t tmem;
    long long sums[kExpandThreads / 32];
    int tiles[kExpandThreads / 32], most[kExpandThreads / 32];
    int bucket[64];
    int limit;             // streams from here on exceed max_total
    int start_b, start_i;  // stream and tile of the first unit
};

// Rows and context of stream b; false: out of range.
__device__ __forceinline__ bool prefill_stream(const PrefillArgs &a, int b, int *n, int *ctx) {
    const int first = __ldcg(a.row_start + b), end = __ldcg(a.row_start + b + 1);
    *ctx = __ldcg(a.ctx_lens + b);
    *n = 0;
    if (first == end) return true;
    if (first < 0 || end < first || end > a.num_rows) return false;
    if (*ctx < end - first || *ctx > a.max_blocks * TTS_BLOCK_TOKENS) return false;
    *n = end - first;
    return true;
}
__device__ __forceinline__ int token_tiles(int ctx) { return (ctx + kTile - 1) / kTile; }

// Barrier of the four epilogue warps with an OR over their threads.
__device__ __forceinline__ bool epilogue_any(bool pred) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %1, 0;\n\t"
        "barrier.cta.red.or.pred q, 1, 128, p;\n\tselp.b32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"(static_cast<uint32_t>(pred))
        : "memory");
    return r != 0;
}

// Largest magnitude of 64 values, NaN if one of them is.
__device__ __forceinline__ float largest64(const uint32_t *x) {
    auto larger = [](float a, float b, float c) {
        float m;
        asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(m) : "f"(a), "f"(b), "f"(c));
        return m;
    };
    float m[4] = {};
#pragma unroll
    for (int i = 0; i < 64; i += 2)
        m[i / 2 % 4] = larger(m[i / 2 % 4], fabsf(__uint_as_float(x[i])), fabsf(__uint_as_float(x[i + 1])));
    return larger(larger(m[0], m[1], m[2]), m[3], m[3]);
}

// Whether a token's latent is finite (rare: asked when a product of it is not).
__device__ __noinline__ bool latent_finite(const PrefillArgs &a, int b, int t, int ctx) {
    if (t >= ctx) return true;
    const int id = a.table[static_cast<size_t>(b) * a.max_blocks + t / TTS_BLOCK_TOKENS];
    if (id < 0 || id >= a.num_blocks) return true;
    const uint4 *c = reinterpret_cast<const uint4 *>(
        a.pool + (static_cast<size_t>(id) * TTS_BLOCK_TOKENS + t % TTS_BLOCK_TOKENS) * (a.L + kLatentRope));
    bool finite = true;
    for (int i = 0; i < a.L / 8; ++i) {
        const uint4 x = c[i];
        for (const uint32_t w : {x.x, x.y, x.z, x.w})
            finite = finite && (w & 0x7F80u) != 0x7F80u && (w & 0x7F800000u) != 0x7F800000u;
    }
    return finite;
}

// Zeros in the rows of the refused streams (rare), by every thread of the grid:
// each warp of the CTA looks at 32 streams and finds the same ones.
__device__ __noinline__ void zero_refused(const PrefillArgs &a, int limit) {
    const int lane = threadIdx.x % 32;
    const size_t width = static_cast<size_t>(a.Hq) * a.v / 8;  // 16-byte pieces a row
    const size_t me = static_cast<size_t>(blockIdx.x) * blockDim.x + threadIdx.x, all = static_cast<size_t>(gridDim.x) * blockDim.x;
    for (int base = 0; base < a.B; base += 32) {
        bool bad = false;
        int n, ctx, r0 = 0, r1 = 0;
        if (base + lane < a.B) {
            const int b = base + lane;
            bad = !prefill_stream(a, b, &n, &ctx) || (n && b >= limit);
            r0 = max(0, a.row_start[b]);
            r1 = min(a.num_rows, a.row_start[b + 1]);
        }
        for (unsigned m = __ballot_sync(kFull, bad); m; m &= m - 1) {
            const int from = __shfl_sync(kFull, r0, __ffs(m) - 1), to = __shfl_sync(kFull, r1, __ffs(m) - 1);
            if (me == 0) flag_error(a.err, TTS_ERRBIT_CTX_LEN);
            if (from >= to) continue;
            for (size_t i = from * width + me; i < to * width; i += all) reinterpret_cast<uint4 *>(a.out)[i] = make_uint4(0, 0, 0, 0);
        }
    }
}

// Walks the units of a CTA (every feature tile of a token tile, then the next
// token tile); every warp keeps its own copy.
struct ExpandWalk {
    int left, f, t;               // units left; feature tile, token tile
    int feature_tiles;
    int b, i, n, limit;           // stream of the token tile, its tile in the stream, the stream's tiles
    int ctx;
    __device__ __forceinline__ void seek(const PrefillArgs &a) {          // b: the next stream that has tiles
        for (; b < limit; ++b) {
            int rows, c;
            const bool good = prefill_stream(a, b, &rows, &c);
            n = uniform(good && rows ? token_tiles(c) : 0);
            ctx = uniform(c);
            if (n) return;
        }
    }
    __device__ __forceinline__ void advance(const PrefillArgs &a) {
        --left;
        if (++f < feature_tiles) return;
        f = 0;
        ++t;
        if (++i == n) {
            i = 0;
            ++b;
            seek(a);
        }
    }
};

__global__ void __launch_bounds__(kExpandThreads, 1)
latent_expand_kernel(const __grid_constant__ CUtensorMap map_pool, const __grid_constant__ CUtensorMap map_uk,
                     const __grid_constant__ CUtensorMap map_uv, const __grid_constant__ CUtensorMap map_k,
                     const __grid_constant__ CUtensorMap map_v, const PrefillArgs a) {
    extern __shared__ __align__(1024) uint8_t raw[];
    __shared__ ExpandShared sh;
    const uint32_t ring = smem_addr(raw), stage = ring + kExpandSlots * kSlotBytes;
    const int warp = uniform(threadIdx.x / 32), lane = threadIdx.x % 32;
    const int chunks = a.L / 64;
    if (warp == 5 && lane == 0) {
        for (int i = 0; i < kExpandSlots; ++i) {
            mbar_init(smem_addr(&sh.full[i]), 1);
            mbar_init(smem_addr(&sh.empty[i]), 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_addr(&sh.acc_full[i]), 1);
            mbar_init(smem_addr(&sh.acc_empty[i]), 4);
        }
        mbar_init(smem_addr(&sh.fin), 1);
        sh.limit = a.B;
        fence_mbar_init();
    }
    if (warp == 4 && lane == 0) {
        prefetch_tensormap(&map_pool);
        prefetch_tensormap(&map_uk);
        prefetch_tensormap(&map_uv);
    }
    if (warp == 0 && lane == 0) {
        prefetch_tensormap(&map_k);
        prefetch_tensormap(&map_v);
    }
    pdl_wait_prerequisites();
    // (tensor memory only after the wait: the kernel before may be one that
    // still has to allocate its own)
    if (warp == 6) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_addr(&sh.tmem))
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    // ---- the streams' token tiles
    const int per = (a.B + kExpandThreads - 1) / kExpandThreads;
    const int b0 = min(a.B, static_cast<int>(threadIdx.x) * per), b1 = min(a.B, b0 + per);
    int n, ctx, limit = a.B;
    long long mine = 0;
    int t_mine = 0, most = 0;
    for (int b = b0; b < b1; ++b)
        if (prefill_stream(a, b, &n, &ctx) && n) {
            mine += ctx;
            t_mine += token_tiles(ctx);
            most = max(most, ctx);
        }
    long long incl = mine;
    int t_incl = t_mine;
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
        const long long x = __shfl_up_sync(kFull, incl, o);
        const int y = __shfl_up_sync(kFull, t_incl, o);
        if (lane >= o) {
            incl += x;
            t_incl += y;
        }
    }
    most = __reduce_max_sync(kFull, most);
    if (lane == 31) {
        sh.sums[warp] = incl;
        sh.tiles[warp] = t_incl;
        sh.most[warp] = most;
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    pdl_allow_dependents();
    long long at = incl - mine, total = 0;
#pragma unroll
    for (int w = 0; w < kExpandThreads / 32; ++w) {
        if (w < warp) at += sh.sums[w];
        total += sh.sums[w];
        most = max(most, sh.most[w]);
    }
    if (total > a.max_total) {  // rare: which streams fit, and their tiles
        for (int b = b0; b < b1 && at <= a.max_total; ++b)
            if (prefill_stream(a, b, &n, &ctx) && n) {
                at += ctx;
                if (at > a.max_total) atomicMin(&sh.limit, b);
            }
        __syncthreads();
        limit = sh.limit;
        t_mine = 0;
        for (int b = b0; b < min(b1, limit); ++b)
            if (prefill_stream(a, b, &n, &ctx) && n) t_mine += token_tiles(ctx);
        t_incl = t_mine;
#pragma unroll
        for (int o = 1; o < 32; o *= 2) {
            const int y = __shfl_up_sync(kFull, t_incl, o);
            if (lane >= o) t_incl += y;
        }
        if (lane == 31) sh.tiles[warp] = t_incl;
        __syncthreads();
    }
    int t_at = t_incl - t_mine, tiles = 0;
#pragma unroll
    for (int w = 0; w < kExpandThreads / 32; ++w) {
        if (w < warp) t_at += sh.tiles[w];
        tiles += sh.tiles[w];
    }
    // Units of 256 features, or of 128 where those still make one round of the
    // CTAs (one prompt of 333 rows, the whole call: 17.6 against 19.4 us; in
    // three rounds of 128 or two of 256, 16 prompts take 30.9 and 30.8)
    const int ctas = gridDim.x, me = blockIdx.x;
    auto tiles_of = [](int features, int each) { return (features + each - 1) / each; };
    auto units_of = [&](int each) { return tiles * (tiles_of(a.Hq * a.nope, each) + tiles_of(a.Hq * a.v, each)); };
    const int features = units_of(kFeatures / 2) <= ctas ? kFeatures / 2 : kFeatures;
    const int k_tiles = tiles_of(a.Hq * a.nope, features), feature_tiles = k_tiles + tiles_of(a.Hq * a.v, features);
    const int units = units_of(features);
    const int each = units / ctas;
    const int fewer = ctas - (units - each * ctas);  // the CTAs behind these take one more
    const int u0 = me * each + max(0, me - fewer), u1 = u0 + each + (me >= fewer);
    const int first_t = u0 / feature_tiles;
    bool refused = false;  // any of this thread's streams
    for (int b = b0; b < b1; ++b) {
        const bool good = prefill_stream(a, b, &n, &ctx);
        const int nt = good && n && b < limit ? token_tiles(ctx) : 0;
        if (first_t >= t_at && first_t < t_at + nt) {
            sh.start_b = b;
            sh.start_i = first_t - t_at;
        }
        if (blockIdx.x == 0) a.tile_start[b] = t_at;
        refused = refused || !good || (n && b >= limit);
        t_at += nt;
    }
    if (__syncthreads_or(refused)) zero_refused(a, limit);
    const uint32_t tmem = uniform(sh.tmem);
    ExpandWalk walk;
    walk.left = uniform(u1 - u0);
    walk.feature_tiles = feature_tiles;
    walk.f = uniform(u0 % feature_tiles);
    walk.t = uniform(first_t);
    walk.b = uniform(sh.start_b);
    walk.i = uniform(sh.start_i);
    walk.limit = uniform(limit);
    if (walk.left > 0) walk.seek(a);
    bool ok = true;

    if (warp == 4) {
        // ---- producer: the token tile's eight blocks and the weight chunk.  A
        // block outside the pool (or past the context) is read out of range,
        // which fills zeros.
        const uint32_t leader = elect_leader();
        uint32_t slot = 0, phase = 0, count = 0;
        int have = -1, ys[8] = {};
        for (; ok && walk.left > 0; walk.advance(a)) {
            if (walk.t != have) {
                const int block = walk.i * (kTile / TTS_BLOCK_TOKENS) + (lane & 7);
                int y = a.num_blocks * TTS_BLOCK_TOKENS;
                bool in_pool = false;
                if (block * TTS_BLOCK_TOKENS < walk.ctx) {
                    const int id = a.table[static_cast<size_t>(walk.b) * a.max_blocks + block];
                    in_pool = id >= 0 && id < a.num_blocks;
                    if (in_pool) y = id * TTS_BLOCK_TOKENS;
                    else if (walk.f == 0) flag_error(a.err, TTS_ERRBIT_BLOCK_ID);
                }
#pragma unroll
                for (int i = 0; i < 8; ++i) ys[i] = __shfl_sync(kFull, y, i);
            }
            have = walk.t;
            const bool is_k = walk.f < k_tiles;
            const int row = (is_k ? walk.f : walk.f - k_tiles) * features;
            for (int c = 0; c < chunks; ++c) {
                if (count >= kExpandSlots && !warp_wait(&sh.empty[slot], phase ^ 1)) {
                    ok = false;
                    break;
                }
                const uint32_t bar = smem_addr(&sh.full[slot]), to = ring + slot * kSlotBytes;
                mbar_expect_tx_by(leader, bar, kChunkBytes + features * 128);
                for (int i = 0; i < features; i += kWeightRows)
                    tma_load_2d_by(leader, to + kChunkBytes + i * 128, is_k ? &map_uk : &map_uv, c * 64, row + i, bar);
#pragma unroll
                for (int i = 0; i < 8; ++i) tma_load_2d_by(leader, to + i * 2048, &map_pool, c * 64, ys[i], bar);
                ++count;
                if (++slot == kExpandSlots) {
                    slot = 0;
                    phase ^= 1;
                }
            }
        }
        // every copy lands before the CTA ends
        for (uint32_t i = min(count, static_cast<uint32_t>(kExpandSlots)); i > 0; --i) {
            if (slot == 0) {
                slot = kExpandSlots;
                phase ^= 1;
            }
            --slot;
            warp_wait(&sh.full[slot], phase);
        }
    } else if (warp == 5) {
        // ---- MMA issuer; rows behind the context in its last block hold
        // anything and are cleared: their keys and values become zero
        const uint32_t leader = elect_leader();
        const uint32_t idesc = uniform(features == kFeatures ? mma_idesc(kTile, kFeatures) : mma_idesc(kTile, kFeatures / 2));
        uint32_t slot = 0, phase = 0, done = 0;
        for (; ok && walk.left > 0; walk.advance(a), ++done) {
            const uint32_t buf = done & 1;
            const int end = walk.ctx - walk.i * kTile;  // tokens of the context from this tile on
            const int stop = (end + TTS_BLOCK_TOKENS - 1) / TTS_BLOCK_TOKENS * TTS_BLOCK_TOKENS;
            for (int c = 0; c < chunks; ++c) {
                WarpWaits<2> w;
                w.set(0, &sh.full[slot], phase);
                w.none(1);
                if (c == 0 && done >= 2) w.set(1, &sh.acc_empty[buf], (done / 2 - 1) & 1);
                if (!w.wait()) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t sa = ring + slot * kSlotBytes, sb = sa + kChunkBytes;
                if (end < kTile && end < stop) {
                    for (int t = end + lane / 8; t < stop; t += 4)
                        asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(sa + t * 128 + lane % 8 * 16), "r"(0)
                                     : "memory");
                    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                    __syncwarp();
                }
#pragma unroll
                for (int kk = 0; kk < 4; ++kk)
                    mma_bf16_by(leader, tmem + buf * kFeatures, sw128_desc(sa + kk * 32), sw128_desc(sb + kk * 32),
                                idesc, (c | kk) != 0);
                mma_commit_by(leader, smem_addr(&sh.empty[slot]));
                if (++slot == kExpandSlots) {
                    slot = 0;
                    phase ^= 1;
                }
            }
            if (!ok) break;
            mma_commit_by(leader, smem_addr(&sh.acc_full[buf]));
        }
        mma_commit_by(leader, smem_addr(&sh.fin));
        if (!warp_wait(&sh.fin, 0)) ok = false;
    } else if (warp < 4) {
        // ---- rotated key parts, then the accumulators, 64 features at a time
        const int r = warp * 32 + lane;
        const uint32_t tl = tmem + (static_cast<uint32_t>(warp * 32) << 16);
        uint32_t done = 0, in_pool = 0, half = 0;
        int have = -1;
        for (; walk.left > 0; walk.advance(a), ++done) {
            if (warp == 0 && walk.f >= k_tiles && walk.t != have) {
                have = walk.t;
                const int block = walk.i * (kTile / TTS_BLOCK_TOKENS) + (lane & 7);
                const int id = block * TTS_BLOCK_TOKENS < walk.ctx ? a.table[static_cast<size_t>(walk.b) * a.max_blocks + block] : -1;
                in_pool = __ballot_sync(kFull, id >= 0 && id < a.num_blocks) & 0xFFu;
            }
            if (walk.f == 0) {
                for (int i = threadIdx.x; i < kTile * 8; i += 128) {
                    const int t = walk.i * kTile + i / 8;
                    uint4 x = make_uint4(0, 0, 0, 0);
                    if (t < walk.ctx) {
                        const int id = a.table[static_cast<size_t>(walk.b) * a.max_blocks + t / TTS_BLOCK_TOKENS];
                        if (id >= 0 && id < a.num_blocks)
                            x = *(reinterpret_cast<const uint4 *>(
                                      a.pool + (static_cast<size_t>(id) * TTS_BLOCK_TOKENS + t % TTS_BLOCK_TOKENS) *
                                                   (a.L + kLatentRope) + a.L) + i % 8);
                    }
                    reinterpret_cast<uint4 *>(a.kr)[static_cast<size_t>(walk.t) * kTile * 8 + i] = x;
                }
            }
            const uint32_t buf = done & 1;
            const bool is_k = walk.f < k_tiles;
            const int f0 = (is_k ? walk.f : walk.f - k_tiles) * features, all = a.Hq * (is_k ? a.nope : a.v);
            ok = warp_wait(&sh.acc_full[buf], (done / 2) & 1);
            tc_fence_after();
            // a head's values are written as they are, and again scaled if f16
            // does not hold them (rare; known with the barrier that the stores
            // wait for)
            const int token = walk.i * kTile + r;
            bool scaled = false;
            float largest = 0.0f;  // of this token's finite values of the head
            for (int q = 0; q < features / 64;) {
                // the staging half is free once the stores before the last have read it
                if (threadIdx.x == 0) asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory");
                if (epilogue_any(!ok)) {  // (all four warps leave together)
                    ok = false;
                    break;
                }
                uint32_t x[64];
                tmem_ld32_nowait(tl + buf * kFeatures + q * 64, x);
                tmem_ld32_nowait(tl + buf * kFeatures + q * 64 + 32, x + 32);
                tmem_wait_ld();
                float here = largest64(x);
                // A latent that is not finite makes every key and value of its
                // token so.  In the values it would spread to rows that do not
                // see the token (NaN times a zero weight): the values become
                // zero and the keys NaN, and the rows that see it are NaN from
                // their scores.  Values that are not finite by their weights
                // are so for every token: they stay.
                if (!(here < INFINITY)) {
                    const bool weights = latent_finite(a, walk.b, token, walk.ctx);
                    here = 0.0f;
#pragma unroll
                    for (int i = 0; i < 64; ++i) {
                        if (!weights) x[i] = is_k ? 0x7FFFFFFFu : 0u;
                        const float size = fabsf(__uint_as_float(x[i]));
                        if (size < INFINITY) here = fmaxf(here, size);
                    }
                }
                if (!scaled) largest = fmaxf(largest, here);
                if (scaled) {
                    const float by = __uint_as_float(static_cast<uint32_t>(127 - value_exp(largest)) << 23);  // 2^-e
#pragma unroll
                    for (int i = 0; i < 64; ++i) x[i] = __float_as_uint(__uint_as_float(x[i]) * by);
                }
                const float *v = reinterpret_cast<const float *>(x);
                const uint32_t to = stage + half * kChunkBytes + r * 128;
                // 16-byte chunk j of row r at j ^ (r % 8), the stores' swizzle
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    uint32_t p[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        p[i] = is_k ? pack_bf16(v[8 * j + 2 * i], v[8 * j + 2 * i + 1])
                                    : pack_f16(v[8 * j + 2 * i], v[8 * j + 2 * i + 1]);
                    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(to + ((j ^ (r & 7)) << 4)), "r"(p[0]),
                                 "r"(p[1]), "r"(p[2]), "r"(p[3]));
                }
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                const bool ends = !is_k && (a.v == 64 || q % 2);  // a head's values end
                const bool again = epilogue_any(ends && !scaled && f0 + q * 64 < all && token < walk.ctx && !f16_holds(largest));
                if (threadIdx.x == 0) {
                    if (f0 + q * 64 < all)
                        tma_store_2d(is_k ? &map_k : &map_v, f0 + q * 64, walk.t * kTile, stage + half * kChunkBytes);
                    asm volatile("cp.async.bulk.commit_group;" ::: "memory");
                }
                half ^= 1;
                ++q;
                if (!ends) continue;
                const size_t head = (f0 + q * 64) / a.v - 1;
                if (again) {
                    scaled = true;
                    q -= a.v / 64;
                    a.exps[(head * a.max_tiles + walk.t) * kTile + r] = static_cast<int8_t>(value_exp(largest));
                    // (the same places are written once more)
                    if (threadIdx.x == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
                } else {
                    if (threadIdx.x == 0 && f0 + q * 64 <= all)
                        a.info[head * a.max_tiles + walk.t] = in_pool | (scaled ? kScaled : 0u);
                    scaled = false;
                    largest = 0.0f;
                }
            }
            if (!ok) break;
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_addr(&sh.acc_empty[buf]));
        }
        if (threadIdx.x == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
    }
    else if (warp == 6 && blockIdx.x == 0) {
        // ---- the query tiles by the tokens that they see, most first (64
        // buckets): the attention's CTAs start in this order, so that the last
        // ones to run are short (16 prompts of 61 to 700 rows, 8 heads: 18.4 us
        // against 24 us in the streams' order)
        const int shift = max(0, 26 - __clz(max(1, token_tiles(most))));
        auto each_tile = [&](auto &&f) {
            for (int b = lane; b < limit; b += 32) {
                int rows, c;
                if (!prefill_stream(a, b, &rows, &c)) continue;
                for (int q = 0; q * kRows < rows; ++q)
                    f(b, q, 63 - min(63, token_tiles(c - rows + min(rows, (q + 1) * kRows)) >> shift));
            }
            __syncwarp();
        };
        sh.bucket[lane] = sh.bucket[lane + 32] = 0;
        __syncwarp();
        each_tile([&](int, int, int k) { atomicAdd(&sh.bucket[k], 1); });
        const int lo = sh.bucket[2 * lane], hi = sh.bucket[2 * lane + 1];
        int upto = lo + hi;
#pragma unroll
        for (int o = 1; o < 32; o *= 2) {
            const int x = __shfl_up_sync(kFull, upto, o);
            if (lane >= o) upto += x;
        }
        if (lane == 31) *a.num_qtiles = upto;
        sh.bucket[2 * lane] = upto - lo - hi;
        sh.bucket[2 * lane + 1] = upto - hi;
        __syncwarp();
        each_tile([&](int b, int q, int k) {
            const int to = atomicAdd(&sh.bucket[k], 1);
            if (to >= a.max_qtiles) return;  // (streams whose rows overlap)
            const int first = a.row_start[b];
            reinterpret_cast<int4 *>(a.qtiles + to)[0] =
                make_int4(first, a.row_start[b + 1] - first, a.ctx_lens[b], a.tile_start[b]);
            reinterpret_cast<int4 *>(a.qtiles + to)[1] = make_int4(q, 0, 0, 0);
        });
    }
    if (!ok) flag_error(a.err, TTS_ERRBIT_TIMEOUT);
    tc_fence_before();
    __syncthreads();
    if (warp == 6) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
    }
}

// --------------------------------------------------------------- attention

constexpr int kSlots = 8;           // ring slots of [128 tokens][64 values]: 1.6 tiles of keys and values
constexpr int kTiles = 4;           // barriers for the keys, and the values, of as many tiles
constexpr int kAttnThreads = 384;   // two softmax warpgroups; producer, MMA issuer and two spare warps
// A softmax thread holds a row's 128 scores: the registers that the others do not
// need go to it (8191 rows after 700 tokens: 260 us without, 253 with; 16 prompts,
// the whole call, 32.2 and 30.9).  The block has to start with kStartRegs a
// thread; launch_prefill looks.
constexpr int kSoftmaxRegs = 224, kOtherRegs = 56, kStartRegs = 168;
static_assert(256 * kSoftmaxRegs + 128 * kOtherRegs <= kAttnThreads * kStartRegs);

struct PrefillShared {
    uint64_t k_full[kTiles], k_done[kTiles], v_full[kTiles], v_done[kTiles], q_full[2], s_full[2], p_full[2], o_done[2], done;
    uint32_t tmem;
};

// A tile of scaled values (rare): the scores in log2 units with the tokens' e.
__device__ __forceinline__ void add_exps(uint32_t *x, float unit, const int8_t *exps) {
#pragma unroll
    for (int i = 0; i < kTile; i += 16) {
        const int4 e = reinterpret_cast<const int4 *>(exps)[i / 16];
        const int w[4] = {e.x, e.y, e.z, e.w};
#pragma unroll
        for (int k = 0; k < 16; ++k)
            x[i + k] = __float_as_uint(fmaf(static_cast<float>(static_cast<int8_t>(w[k / 4] >> (8 * (k % 4)))), unit, __uint_as_float(x[i + k])));
    }
}
// The sum of the weights without them.
__device__ __forceinline__ float sum_unscaled(const uint32_t *x, float scale_log2, float m, const int8_t *exps) {
    float sum[2] = {0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < kTile; i += 16) {
        const int4 e = reinterpret_cast<const int4 *>(exps)[i / 16];
        const int w[4] = {e.x, e.y, e.z, e.w};
#pragma unroll
        for (int k = 0; k < 16; ++k)
            sum[k % 2] += hw_ex2(fmaf(__uint_as_float(x[i + k]), scale_log2, -m) - static_cast<float>(static_cast<int8_t>(w[k / 4] >> (8 * (k % 4)))));
    }
    return sum[0] + sum[1];
}

template <int kNope, int kV>
__global__ void __launch_bounds__(kAttnThreads, 1)
latent_prefill_kernel(const __grid_constant__ CUtensorMap map_qn, const __grid_constant__ CUtensorMap map_qr,
                      const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_kr,
                      const __grid_constant__ CUtensorMap map_v, const PrefillArgs a) {
    constexpr int kQc = kNope / 64 + 1;   // chunks of a query or key row
    constexpr int kVc = kV / 64;          // chunks of a value row
    extern __shared__ __align__(1024) uint8_t raw[];
    const uint32_t q_base = smem_addr(raw);                       // [2][kQc] chunks
    const uint32_t ring = q_base + 2 * kQc * kChunkBytes;
    PrefillShared &sh = *reinterpret_cast<PrefillShared *>(raw + (2 * kQc + kSlots) * kChunkBytes);
    const int warp = uniform(threadIdx.x / 32), lane = threadIdx.x % 32;
    if (warp == 9 && lane == 0) {
        for (int i = 0; i < kTiles; ++i) {
            mbar_init(smem_addr(&sh.k_full[i]), 1);
            mbar_init(smem_addr(&sh.k_done[i]), 1);
            mbar_init(smem_addr(&sh.v_full[i]), 1);
            mbar_init(smem_addr(&sh.v_done[i]), 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_addr(&sh.q_full[i]), 1);
            mbar_init(smem_addr(&sh.s_full[i]), 1);
            mbar_init(smem_addr(&sh.p_full[i]), 4);
            mbar_init(smem_addr(&sh.o_done[i]), 1);
        }
        mbar_init(smem_addr(&sh.done), 1);
        fence_mbar_init();
        prefetch_tensormap(&map_qn);
        prefetch_tensormap(&map_qr);
        prefetch_tensormap(&map_k);
        prefetch_tensormap(&map_kr);
        prefetch_tensormap(&map_v);
    }
    if (warp == 8) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_addr(&sh.tmem))
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = uniform(sh.tmem);   // S0, S1, O0, O1: 128 columns each
    pdl_wait_prerequisites();
    pdl_allow_dependents();
    const int h = blockIdx.x % a.Hq, qt = blockIdx.x / a.Hq;
    const bool mine = qt < __ldcg(a.num_qtiles);
    const int4 of = __ldcg(reinterpret_cast<const int4 *>(a.qtiles + qt));  // (the list has room for every CTA)
    const int4 which = __ldcg(reinterpret_cast<const int4 *>(a.qtiles + qt) + 1);
    bool ok = true;
    if (uniform(mine)) {
        const int first = uniform(of.x), n = uniform(of.y), ctx = uniform(of.z), tile0 = uniform(of.w);
        const int q = uniform(which.x);
        const int r0 = q * kRows;                          // first row in the stream
        const bool two = r0 + kTile < n;
        // tokens either half sees, in tiles
        const int seen0 = ctx - n + min(n, r0 + kTile), seen1 = ctx - n + min(n, r0 + kRows);
        const int nt0 = (seen0 + kTile - 1) / kTile, nt1 = two ? (seen1 + kTile - 1) / kTile : 0;
        const int nt = max(nt0, nt1);
        if (warp >= 8) {
            asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
            if (warp == 8) {
                // ---- producer (one lane): the queries, then K and V of every tile
                if (lane == 0) {
                    for (int s = 0; s < (two ? 2 : 1); ++s) {
                        const uint32_t bar = smem_addr(&sh.q_full[s]), at = q_base + s * kQc * kChunkBytes;
                        mbar_arrive_expect_tx(bar, kQc * kChunkBytes);
                        for (int c = 0; c < kQc - 1; ++c)
                            tma_load_2d(at + c * kChunkBytes, &map_qn, h * kNope + c * 64, first + r0 + s * kTile, bar);
                        tma_load_2d(at + (kQc - 1) * kChunkBytes, &map_qr, h * kLatentRope, first + r0 + s * kTile, bar);
                    }
                    // a slot is free once the keys or values that it held are done with
                    uint32_t pos = 0;
                    auto slot_free = [&]() {
                        if (pos < kSlots) return true;
                        const uint32_t j = (pos - kSlots) / (kQc + kVc), c = (pos - kSlots) % (kQc + kVc);
                        return mbar_wait(smem_addr((c < kQc ? sh.k_done : sh.v_done) + j % kTiles), (j / kTiles) & 1, a.wait_limit);
                    };
                    int j = 0;
                    for (; ok && j < nt; ++j) {
                        const int y = (tile0 + j) * kTile;
                        for (int c = 0; ok && c < kQc + kVc; ++c, ++pos) {
                            const uint32_t bar = smem_addr((c < kQc ? sh.k_full : sh.v_full) + j % kTiles);
                            if (c == 0 || c == kQc) mbar_arrive_expect_tx(bar, (c ? kVc : kQc) * kChunkBytes + (a.stall && j == 0 && c == 0 ? 16 : 0));
                            ok = slot_free();
                            const uint32_t at = ring + pos % kSlots * kChunkBytes;
                            if (!ok) break;
                            if (c < kQc - 1) tma_load_2d(at, &map_k, h * kNope + c * 64, y, bar);
                            else if (c == kQc - 1) tma_load_2d(at, &map_kr, 0, y, bar);
                            else tma_load_2d(at, &map_v, h * kV + (c - kQc) * 64, y, bar);
                        }
                    }
                    for (int i = max(0, j - kTiles); i < j; ++i) {  // (the ring holds parts of at most kTiles tiles)
                        mbar_wait(smem_addr(&sh.k_full[i % kTiles]), (i / kTiles) & 1);
                        mbar_wait(smem_addr(&sh.v_full[i % kTiles]), (i / kTiles) & 1);
                    }
                    for (int s = 0; s < (two ? 2 : 1); ++s) mbar_wait(smem_addr(&sh.q_full[s]), 0);
                }
            } else if (warp == 9) {
                // ---- MMA issuer: S0(0) S1(0) | O0(j) S0(j+1) | O1(j) S1(j+1) ...
                // S of a half is overwritten right after the O product that reads
                // the weights kept in it; the tensor core runs them in order.
                // Barriers are by tile: a wait or commit takes the issuing warp about
                // 0.1 us.
                const uint32_t leader = elect_leader();
                bool go = true;
                auto scores = [&](auto half, int j) {
                    constexpr int s = decltype(half)::value;
                    const uint32_t pos = static_cast<uint32_t>(j) * (kQc + kVc);
#pragma unroll
                    for (int c = 0; c < kQc; ++c) {
                        const uint32_t sa = q_base + (s * kQc + c) * kChunkBytes, sb = ring + (pos + c) % kSlots * kChunkBytes;
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk)
                            mma_bf16_by(leader, tmem + s * kTile, sw128_desc(sa + kk * 32), sw128_desc(sb + kk * 32),
                                        mma_idesc(kTile, kTile), (c | kk) != 0);
                    }
                    mma_commit_by(leader, smem_addr(&sh.s_full[s]));
                };
                auto output = [&](auto half, int j) {
                    constexpr int s = decltype(half)::value;
                    const uint32_t pos = static_cast<uint32_t>(j) * (kQc + kVc) + kQc;
#pragma unroll
                    for (int c = 0; c < kVc; ++c) {
                        const uint32_t sb = ring + (pos + c) % kSlots * kChunkBytes;
#pragma unroll
                        for (int kk = 0; kk < kTile / 16; ++kk)
                            mma_ts_by(leader, tmem + (2 + s) * kTile + c * 64, tmem + s * kTile + kk * 8,
                                      sw128_mn_desc(sb + kk * 2048, kChunkBytes), mma_idesc_f16(kTile, 64) | kTransposeB,
                                      (j | kk) != 0);
                    }
                };
                constexpr std::integral_constant<int, 0> h0{};
                constexpr std::integral_constant<int, 1> h1{};
                {
                    WarpWaits<3> w;
                    w.set(0, &sh.k_full[0], 0);
                    w.set(1, &sh.q_full[0], 0);
                    w.none(2);
                    if (two) w.set(2, &sh.q_full[1], 0);
                    go = w.wait(a.wait_limit);
                    tc_fence_after();
                    if (go) {
                        scores(h0, 0);
                        if (two) scores(h1, 0);
                        mma_commit_by(leader, smem_addr(&sh.k_done[0]));
                    }
                }
                for (int j = 0; go && j < nt; ++j) {
                    // (a half beyond its last tile is passed over; the first half ends first)
                    auto turn = [&](auto half, int mine) {
                        constexpr int s = decltype(half)::value;
                        const bool last = s == 1 || !two;  // to use this tile's values and the next one's keys
                        WarpWaits<2> w;
                        w.set(0, &sh.p_full[s], j & 1);
                        w.set(1, &sh.v_full[j % kTiles], (j / kTiles) & 1);
                        go = w.wait(a.wait_limit);
                        if (!go) return;
                        tc_fence_after();
                        output(half, j);
                        if (last) mma_commit_by(leader, smem_addr(&sh.v_done[j % kTiles]));
                        if (j + 1 < mine) {
                            go = warp_wait(&sh.k_full[(j + 1) % kTiles], ((j + 1) / kTiles) & 1, a.wait_limit);
                            if (!go) return;
                            tc_fence_after();
                            scores(half, j + 1);
                            if (last) mma_commit_by(leader, smem_addr(&sh.k_done[(j + 1) % kTiles]));
                        } else {
                            mma_commit_by(leader, smem_addr(&sh.o_done[s]));
                        }
                    };
                    if (j < nt0) turn(h0, nt0);
                    if (go && two) turn(h1, nt1);
                }
                mma_commit_by(leader, smem_addr(&sh.done));
                ok = warp_wait(&sh.done, 0) && go;
            }
        } else {
            asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
            if (warp < 4 || two) {
                // ---- softmax warpgroups: thread = query row
                const int s = warp / 4, w = warp % 4;
                const int r = r0 + s * kTile + w * 32 + lane;          // row in the stream
                const int limit = ctx - n + min(n - 1, r) + 1;         // tokens it sees
                const int low = ctx - n + r0 + s * kTile + 1;          // tokens every row of the half sees
                const int tiles = s ? nt1 : nt0;
                const uint32_t lanes = static_cast<uint32_t>(w * 32) << 16;
                const uint32_t ts = tmem + lanes + s * kTile, to = tmem + lanes + (2 + s) * kTile;
                float m = kNoScore, l = 0.0f;
                const uint32_t *info = a.info + static_cast<size_t>(h) * a.max_tiles + tile0;
                const int8_t *exps = a.exps + (static_cast<size_t>(h) * a.max_tiles + tile0) * kTile;
                uint32_t mask = info[0];
                for (int j = 0; j < tiles; ++j) {
                    const uint32_t next_mask = j + 1 < tiles ? info[j + 1] : 0;
                    if (!warp_wait(&sh.s_full[s], j & 1, a.wait_limit)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    uint32_t x[kTile];
#pragma unroll
                    for (int c = 0; c < kTile; c += 32) tmem_ld32_nowait(ts + c, x + c);
                    tmem_wait_ld();
                    const bool scaled = mask & kScaled;
                    if ((j + 1) * kTile > low || mask != 0xFFu) {
                        const int left = limit - j * kTile;
#pragma unroll
                        for (int i = 0; i < kTile; ++i)
                            if (i >= left || !((mask >> (i / TTS_BLOCK_TOKENS)) & 1)) x[i] = 0xFF800000u;  // -inf
                        if (scaled) add_exps(x, 1.0f / a.scale_log2, exps + j * kTile);
                    }
                    mask = next_mask;
                    float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                    for (int i = 0; i < kTile; ++i) top[i % 4] = fmaxf(top[i % 4], __uint_as_float(x[i]));
                    const float t = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])) * a.scale_log2;
                    if (__any_sync(kFull, t > m + kSlack || scaled)) {
                        // (S(j) complete means that O(j - 1) is too; where values
                        // are scaled the sum may be far larger than 2^m's own weight:
                        // the factor in two steps)
                        const float now = fmaxf(m, t), root = hw_ex2(0.5f * (m - now)), f = root * root;
                        m = now;
                        l = l * root * root;
                        if (j > 0)
                            for (int c = 0; c < kV; c += 16) {
                                uint32_t o[16];
                                tmem_ld16_nowait(to + c, o);
                                tmem_wait_ld();
#pragma unroll
                                for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
                                tmem_st16(to + c, o);
                            }
                        if (scaled) l += sum_unscaled(x, a.scale_log2, m, exps + j * kTile);
                    }
                    float sum[2] = {0.0f, 0.0f};
#pragma unroll
                    for (int c = 0; c < kTile; c += 64) {
                        uint32_t p[32];
#pragma unroll
                        for (int i = 0; i < 32; ++i) {
                            const float p0 = hw_ex2(fmaf(__uint_as_float(x[c + 2 * i]), a.scale_log2, -m));
                            const float p1 = hw_ex2(fmaf(__uint_as_float(x[c + 2 * i + 1]), a.scale_log2, -m));
                            sum[0] += p0;
                            sum[1] += p1;
                            p[i] = pack_f16(p0, p1);
                        }
                        tmem_st32(ts + c / 2, p);
                    }
                    l += scaled ? 0.0f : sum[0] + sum[1];
                    tmem_wait_st();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(smem_addr(&sh.p_full[s]));
                }
                if (ok) ok = warp_wait(&sh.o_done[s], 0, a.wait_limit);
                if (ok) {
                    tc_fence_after();
                    const float inv = l == 0.0f ? 0.0f : 1.0f / l;  // no token left: zeros
                    uint4 *dst = reinterpret_cast<uint4 *>(a.out + (static_cast<size_t>(first + r) * a.Hq + h) * kV);
                    for (int c = 0; c < kV; c += 32) {
                        uint32_t o[32];
                        tmem_ld32_nowait(to + c, o);
                        tmem_wait_ld();
                        const float *f = reinterpret_cast<const float *>(o);
                        if (r < n)
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                dst[c / 8 + i] = make_uint4(pack_bf16(f[8 * i] * inv, f[8 * i + 1] * inv),
                                                            pack_bf16(f[8 * i + 2] * inv, f[8 * i + 3] * inv),
                                                            pack_bf16(f[8 * i + 4] * inv, f[8 * i + 5] * inv),
                                                            pack_bf16(f[8 * i + 6] * inv, f[8 * i + 7] * inv));
                    }
                }
            }
        }
        if (!ok) flag_error(a.err, TTS_ERRBIT_TIMEOUT);
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 8) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
    }
}

// -------------------------------------------------------------------- host

bool prefill_shape_ok(int B, int T, int Hq, int L, int nope, int v, int max_total) {
    return B >= 0 && T >= 0 && Hq >= 1 && Hq <= kLatentMaxHeads && L >= 64 && L <= kLatentMaxDim && L % 64 == 0 &&
           latent_head_dim_ok(nope) && latent_head_dim_ok(v) && max_total >= 0 && B <= (1 << 20);
}

// Workspace: keys, values and rotated key parts of the padded tokens, then
// the plan's arrays.
struct PrefillPlan {
    int64_t tiles, qtiles;   // at most
    size_t k_bytes, v_bytes, kr_bytes, start_bytes, qtile_bytes, info_bytes, exp_bytes;
    size_t total() const { return k_bytes + v_bytes + kr_bytes + start_bytes + qtile_bytes + info_bytes + exp_bytes + 256; }
};

PrefillPlan prefill_plan(int B, int T, int Hq, int nope, int v, int max_total) {
    PrefillPlan p;
    p.tiles = static_cast<int64_t>(max_total) / kTile + B;
    p.qtiles = static_cast<int64_t>(T) / kRows + B;
    const size_t rows = static_cast<size_t>(p.tiles) * kTile;
    p.k_bytes = rows * Hq * nope * 2;
    p.v_bytes = rows * Hq * v * 2;
    p.kr_bytes = rows * kLatentRope * 2;
    p.start_bytes = align_up((static_cast<size_t>(B) + 1) * 4, 256);
    p.qtile_bytes = align_up(static_cast<size_t>(p.qtiles) * sizeof(QueryTile), 256);
    p.info_bytes = align_up(static_cast<size_t>(p.tiles) * Hq * 4, 256);
    p.exp_bytes = rows * Hq;
    return p;
}

template <int kNope, int kV>
int launch_prefill(const CUtensorMap *m, const PrefillArgs &a, unsigned grid, cudaStream_t stream) {
    constexpr int kSmem = (2 * (kNope / 64 + 1) + kSlots) * kChunkBytes + static_cast<int>(sizeof(PrefillShared));
    auto kernel = latent_prefill_kernel<kNope, kV>;
    if (!allow_smem(kernel, kSmem)) return TTS_ERR_CUDA;
    static std::atomic<int> regs{0};  // (a compiler's choice, the same on every device)
    if (regs.load(std::memory_order_relaxed) == 0) {
        cudaFuncAttributes attr;
        if (cudaFuncGetAttributes(&attr, reinterpret_cast<const void *>(kernel)) != cudaSuccess) {
            cudaGetLastError();
            return TTS_ERR_CUDA;
        }
        regs.store(attr.numRegs, std::memory_order_relaxed);
    }
    if (regs.load(std::memory_order_relaxed) < kStartRegs) return TTS_ERR_UNSUPPORTED;
    return launch_kernel(kernel, dim3(grid), dim3(kAttnThreads), kSmem, {stream, true}, m[0], m[1], m[2], m[3], m[4], a);
}

}  // namespace
}  // namespace tts

extern "C" size_t tts_latent_prefill_attn_workspace_size(int32_t B, int32_t num_rows, int32_t num_q_heads,
                                                         int32_t latent_dim, int32_t nope_dim, int32_t v_dim,
                                                         int32_t max_total_ctx) {
    if (!tts::prefill_shape_ok(B, num_rows, num_q_heads, latent_dim, nope_dim, v_dim, max_total_ctx)) return 0;
    return tts::prefill_plan(B, num_rows, num_q_heads, nope_dim, v_dim, max_total_ctx).total();
}

extern "C" int tts_latent_prefill_attn(const tts_latent_cache *cache, const int32_t *d_block_table,
                                       int32_t max_blocks_per_seq, const int32_t *d_ctx_lens, int32_t max_total_ctx,
                                       int32_t B, const int32_t *d_row_start, int32_t num_rows, int32_t num_q_heads,
                                       int32_t nope_dim, int32_t v_dim, float scale, const void *d_q_nope,
                                       const void *d_q_rope, const void *d_w_uk, const void *d_w_uv, void *d_out,
                                       void *d_ws, size_t ws_bytes, int32_t *d_err, void *stream) {
    using namespace tts;
    const int st = check_latent_cache(cache, d_block_table, max_blocks_per_seq);
    if (st != TTS_OK) return st;
    if (!d_ctx_lens || !d_row_start || !d_q_nope || !d_q_rope || !d_w_uk || !d_w_uv || !d_out) return TTS_ERR_INVALID;
    if (B < 0 || num_rows < 0 || num_q_heads < 1 || max_total_ctx < 0 || nope_dim < 1 || v_dim < 1)
        return TTS_ERR_INVALID;
    if (!(scale > 0.0f) || std::isinf(scale)) return TTS_ERR_INVALID;
    const int L = cache->latent_dim, Hq = num_q_heads;
    if (!prefill_shape_ok(B, num_rows, Hq, L, nope_dim, v_dim, max_total_ctx)) return TTS_ERR_UNSUPPORTED;
    if (!aligned16(d_q_nope) || !aligned16(d_q_rope) || !aligned16(d_w_uk) || !aligned16(d_w_uv) || !aligned16(d_out))
        return TTS_ERR_INVALID;
    if (B == 0 || num_rows == 0) return TTS_OK;
    const PrefillPlan pl = prefill_plan(B, num_rows, Hq, nope_dim, v_dim, max_total_ctx);
    if (!d_ws || !aligned16(d_ws) || ws_bytes < pl.total()) return TTS_ERR_WORKSPACE;
    // the grid, GEMM units and token rows are 32-bit
    const int64_t unit_tiles = static_cast<int64_t>(Hq) * (nope_dim + v_dim) / kFeatures + 2;
    if (pl.tiles * unit_tiles > 0x20000000 || pl.qtiles * Hq > 0x7FFFFFFF) return TTS_ERR_UNSUPPORTED;

    uint8_t *ws = static_cast<uint8_t *>(d_ws);
    PrefillArgs a{};
    a.table = d_block_table;
    a.max_blocks = max_blocks_per_seq;
    a.num_blocks = cache->num_blocks;
    a.ctx_lens = d_ctx_lens;
    a.row_start = d_row_start;
    a.max_total = max_total_ctx;
    a.B = B;
    a.num_rows = num_rows;
    a.Hq = Hq;
    a.L = L;
    a.nope = nope_dim;
    a.v = v_dim;
    a.scale_log2 = scale * kLog2e;
    void *k = ws, *v = ws + pl.k_bytes;
    a.kr = reinterpret_cast<__nv_bfloat16 *>(ws + pl.k_bytes + pl.v_bytes);
    uint8_t *at = ws + pl.k_bytes + pl.v_bytes + pl.kr_bytes;
    a.tile_start = reinterpret_cast<int32_t *>(at);
    a.qtiles = reinterpret_cast<QueryTile *>(at + pl.start_bytes);
    a.max_qtiles = static_cast<int>(pl.qtiles);
    a.info = reinterpret_cast<uint32_t *>(at + pl.start_bytes + pl.qtile_bytes);
    a.max_tiles = static_cast<int>(pl.tiles);
    a.exps = reinterpret_cast<int8_t *>(at + pl.start_bytes + pl.qtile_bytes + pl.info_bytes);
    a.num_qtiles = reinterpret_cast<int32_t *>(at + pl.start_bytes + pl.qtile_bytes + pl.info_bytes + pl.exp_bytes);
    a.pool = static_cast<const __nv_bfloat16 *>(cache->pool);
    a.out = static_cast<__nv_bfloat16 *>(d_out);
    a.err = d_err;
    a.wait_limit = thread_opts().wait_limit;
    a.stall = thread_opts().stall == TTS_TEST_STALL_LATENT_PREFILL;
    const uint64_t kv_rows = static_cast<uint64_t>(pl.tiles) * kTile, T = num_rows;
    const uint64_t fk = static_cast<uint64_t>(Hq) * nope_dim, fv = static_cast<uint64_t>(Hq) * v_dim;
    CUtensorMap pool, uk, uv, qkv[5];
    if (!make_tma_2d_bf16(&pool, cache->pool, static_cast<uint64_t>(cache->num_blocks) * TTS_BLOCK_TOKENS,
                          L + kLatentRope, TTS_BLOCK_TOKENS, 64) ||
        !make_tma_2d_bf16(&uk, d_w_uk, fk, L, kWeightRows, 64) || !make_tma_2d_bf16(&uv, d_w_uv, fv, L, kWeightRows, 64) ||
        !make_tma_2d_bf16(&qkv[0], d_q_nope, T, fk, kTile, 64) ||
        !make_tma_2d_bf16(&qkv[1], d_q_rope, T, static_cast<uint64_t>(Hq) * kLatentRope, kTile, 64) ||
        !make_tma_2d_bf16(&qkv[2], k, kv_rows, fk, kTile, 64) ||
        !make_tma_2d_bf16(&qkv[3], a.kr, kv_rows, kLatentRope, kTile, 64) ||
        !make_tma_2d_bf16(&qkv[4], v, kv_rows, fv, kTile, 64))
        return TTS_ERR_CUDA;

    const cudaStream_t cs = static_cast<cudaStream_t>(stream);
    if (!allow_smem(latent_expand_kernel, kExpandSmem)) return TTS_ERR_CUDA;
    const int rc = launch_kernel(latent_expand_kernel, dim3(kExpandCtas), dim3(kExpandThreads), kExpandSmem,
                                 {cs, thread_pdl()}, pool, uk, uv, qkv[2], qkv[4], a);
    if (rc != TTS_OK) return rc;
    const unsigned grid = static_cast<unsigned>(pl.qtiles * Hq);
    if (nope_dim == 128)
        return v_dim == 128 ? launch_prefill<128, 128>(qkv, a, grid, cs) : launch_prefill<128, 64>(qkv, a, grid, cs);
    return v_dim == 128 ? launch_prefill<64, 128>(qkv, a, grid, cs) : launch_prefill<64, 64>(qkv, a, grid, cs);
}
