// Attention of whole prompts over the latent cache, expanded form: every
// head's keys (w_uk[h] c, kr) and values w_uv[h] c are multiplied out once,
// then ordinary causal attention.  Per (row, token, head) that costs
// 2 (nope + 64 + v) flop where the absorbed form costs 2 (2 latent_dim + 64):
// 640 against 2176 at 128, 128 and 512, for 2 latent_dim (nope + v) more per
// (token, head).  Three kernels, each a programmatic dependent of the one
// before:
//
//  1. latent_plan_kernel (one CTA): checks the streams, lays out their tokens
//     in the workspace (each stream from a 128-token boundary) and their query
//     tiles.
//  2. latent_expand_kernel: a tcgen05 GEMM per 128 tokens x 128 features,
//     latents fetched through the block table.
//  3. latent_prefill_kernel: attention of 256 rows of one head per CTA (two
//     128-row tiles that take turns on the tensor core: while one's weights
//     are computed, the other's products run).  S and O are in tensor memory;
//     the weights go back into S's columns as bf16 and are the A operand of
//     the second product.
#include <cuda_bf16.h>

#include <cmath>

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
constexpr float kNoScore = -1e30f;         // running maximum before any token (log2 units)
constexpr float kSlack = 8.0f;             // scores may pass it by this much before it moves (log2 units)

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    const __nv_bfloat162 p = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&p);
}

struct PrefillArgs {
    const int32_t *table;
    int max_blocks, num_blocks;
    const int32_t *ctx_lens;
    const int32_t *row_start;
    int max_total, B, num_rows, Hq, L, nope, v;
    float scale_log2;
    int32_t *tile_start;   // [B + 1] first token tile of each stream
    int32_t *qtile_start;  // [B + 1] first query tile
    uint32_t *blocks_ok;   // [token tiles] bit i: block i of the tile is in the pool
    const __nv_bfloat16 *pool;
    __nv_bfloat16 *kr;     // [token tiles * 128][64]
    __nv_bfloat16 *out;
    int32_t *err;
};

// -------------------------------------------------------------------- plan

constexpr int kPlanThreads = 256;

__global__ void __launch_bounds__(kPlanThreads) latent_plan_kernel(const PrefillArgs a) {
    __shared__ long long sums[3][kPlanThreads / 32];
    pdl_wait_prerequisites();
    pdl_allow_dependents();
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    const int per = (a.B + kPlanThreads - 1) / kPlanThreads;
    const int b0 = min(a.B, tid * per), b1 = min(a.B, b0 + per);
    // rows and context of stream b; false: its rows or its length are out of range
    auto stream = [&](int b, int *n, int *ctx) {
        const int first = a.row_start[b], end = a.row_start[b + 1];
        *ctx = a.ctx_lens[b];
        *n = 0;
        if (first == end) return true;
        if (first < 0 || end < first || end > a.num_rows) return false;
        *n = end - first;
        if (*ctx < *n || *ctx > a.max_blocks * TTS_BLOCK_TOKENS) {
            *n = 0;
            return false;
        }
        return true;
    };
    auto zero_rows = [&](int b) {
        const int first = max(0, a.row_start[b]), end = min(a.num_rows, a.row_start[b + 1]);
        flag_error(a.err, TTS_ERRBIT_CTX_LEN);
        uint4 *o = reinterpret_cast<uint4 *>(a.out);
        const size_t w = static_cast<size_t>(a.Hq) * a.v / 8;
        for (size_t i = first * w; first < end && i < end * w; ++i) o[i] = make_uint4(0, 0, 0, 0);
    };
    // exclusive scans over the streams: contexts (against max_total), then tiles
    auto scan = [&](long long mine, int which) {
        long long incl = mine;
#pragma unroll
        for (int o = 1; o < 32; o *= 2) {
            const long long x = __shfl_up_sync(kFull, incl, o);
            if (lane >= o) incl += x;
        }
        if (lane == 31) sums[which][warp] = incl;
        __syncthreads();
        long long at = incl - mine;
        for (int w = 0; w < warp; ++w) at += sums[which][w];
        return at;
    };
    long long mine = 0;
    for (int b = b0; b < b1; ++b) {
        int n, ctx;
        if (stream(b, &n, &ctx) && n) mine += ctx;
    }
    long long ctx_at = scan(mine, 0);
    const long long ctx_first = ctx_at;
    long long tiles = 0, qtiles = 0;
    for (int b = b0; b < b1; ++b) {
        int n, ctx;
        if (stream(b, &n, &ctx) && n) {
            ctx_at += ctx;
            if (ctx_at <= a.max_total) {
                tiles += (ctx + kTile - 1) / kTile;
                qtiles += (n + kRows - 1) / kRows;
            }
        }
    }
    long long t_at = scan(tiles, 1), q_at = scan(qtiles, 2);
    ctx_at = ctx_first;
    for (int b = b0; b < b1; ++b) {
        int n, ctx;
        const bool good = stream(b, &n, &ctx);
        bool taken = good;
        a.tile_start[b] = static_cast<int>(t_at);
        a.qtile_start[b] = static_cast<int>(q_at);
        if (good && n) {
            ctx_at += ctx;
            taken = ctx_at <= a.max_total;
            if (taken) {
                t_at += (ctx + kTile - 1) / kTile;
                q_at += (n + kRows - 1) / kRows;
            }
        }
        if (!taken) zero_rows(b);
    }
    if (b0 < b1 && b1 == a.B) {
        a.tile_start[a.B] = static_cast<int>(t_at);
        a.qtile_start[a.B] = static_cast<int>(q_at);
    }
}

// ------------------------------------------------------------------ expand

// K[t][h nope + d] = w_uk[h][d] . c_t and V likewise, bf16.  One CTA per 128
// tokens x 128 features (two fit an SM, so one's epilogue runs beside the
// other's products): A = latents through the block table, B = weights, both
// K-major; the accumulator leaves through shared memory as bf16 by TMA.
// The first feature tile's CTA also copies the tokens' rotated key parts and
// records which blocks are in the pool.
constexpr int kExpandStages = 3;
constexpr int kExpandThreads = 192;
constexpr int kExpandSmem = 1024 + kExpandStages * 2 * kChunkBytes;

struct ExpandShared {
    uint64_t full[kExpandStages], empty[kExpandStages], acc;
    uint32_t tmem;
};

__global__ void __launch_bounds__(kExpandThreads)
latent_expand_kernel(const __grid_constant__ CUtensorMap map_pool, const __grid_constant__ CUtensorMap map_uk,
                     const __grid_constant__ CUtensorMap map_uv, const __grid_constant__ CUtensorMap map_k,
                     const __grid_constant__ CUtensorMap map_v, const PrefillArgs a, int k_tiles) {
    extern __shared__ uint8_t raw[];
    __shared__ ExpandShared sh;
    const uint32_t base = (smem_addr(raw) + 1023u) & ~1023u;
    const int warp = uniform(threadIdx.x / 32), lane = threadIdx.x % 32;
    const int chunks = a.L / 64;
    if (warp == 5 && lane == 0) {
        for (int i = 0; i < kExpandStages; ++i) {
            mbar_init(smem_addr(&sh.full[i]), 1);
            mbar_init(smem_addr(&sh.empty[i]), 1);
        }
        mbar_init(smem_addr(&sh.acc), 1);
        fence_mbar_init();
    }
    if (warp == 4) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 128;" ::"r"(smem_addr(&sh.tmem))
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = uniform(sh.tmem);
    pdl_wait_prerequisites();
    pdl_allow_dependents();
    const bool is_k = static_cast<int>(blockIdx.x) < k_tiles;
    const int f0 = (is_k ? blockIdx.x : blockIdx.x - k_tiles) * kTile;
    const int features = a.Hq * (is_k ? a.nope : a.v);
    const int tile = blockIdx.y;
    const int b = uniform(stream_of_row(a.tile_start, a.B, tile, lane));  // (every warp)
    bool ok = true;
    if (b >= 0) {
        const int ctx = uniform(a.ctx_lens[b]);
        const int t0 = uniform((tile - a.tile_start[b]) * kTile);
        const int end = min(kTile, ctx - t0);  // tokens of the context in this tile
        const int32_t *row = a.table + static_cast<size_t>(b) * a.max_blocks;
        if (warp == 4) {
            // ---- producer: lanes 0-7 fetch a block each, lane 8 the weights
            int y = a.num_blocks * TTS_BLOCK_TOKENS;  // out of range: zeros
            bool in_pool = false;
            if (lane < 8 && lane * TTS_BLOCK_TOKENS < end) {
                const int id = row[t0 / TTS_BLOCK_TOKENS + lane];
                in_pool = id >= 0 && id < a.num_blocks;
                if (in_pool) y = id * TTS_BLOCK_TOKENS;
                else if (blockIdx.x == 0) flag_error(a.err, TTS_ERRBIT_BLOCK_ID);
            }
            const uint32_t mask = __ballot_sync(kFull, in_pool);
            if (blockIdx.x == 0 && lane == 0) a.blocks_ok[tile] = mask;
            int c = 0;
            for (; c < chunks; ++c) {
                const int s = c % kExpandStages;
                if (c >= kExpandStages && !warp_wait(&sh.empty[s], (c / kExpandStages - 1) & 1)) {
                    ok = false;
                    break;
                }
                const uint32_t bar = smem_addr(&sh.full[s]), at = base + s * 2 * kChunkBytes;
                if (lane == 0) mbar_arrive_expect_tx(bar, 2 * kChunkBytes);
                __syncwarp();
                if (lane < 8) tma_load_2d(at + lane * 2048, &map_pool, c * 64, y, bar);
                if (lane == 8) tma_load_2d(at + kChunkBytes, is_k ? &map_uk : &map_uv, c * 64, f0, bar);
            }
            if (lane == 0)
                for (int i = c > kExpandStages ? c - kExpandStages : 0; i < c; ++i)
                    mbar_wait(smem_addr(&sh.full[i % kExpandStages]), (i / kExpandStages) & 1);
        } else if (warp == 5) {
            // ---- MMA issuer; rows behind the context in its last block hold
            // anything and are cleared: their keys and values become zero
            const int stale = (TTS_BLOCK_TOKENS - end % TTS_BLOCK_TOKENS) % TTS_BLOCK_TOKENS;
            const uint32_t leader = elect_leader();
            for (int c = 0; c < chunks; ++c) {
                const int s = c % kExpandStages;
                if (!warp_wait(&sh.full[s], (c / kExpandStages) & 1)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t at = base + s * 2 * kChunkBytes;
                if (stale) {
                    for (int i = lane; i < stale * 8; i += 32)
                        asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(at + end * 128 + i * 16), "r"(0)
                                     : "memory");
                    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                    __syncwarp();
                }
#pragma unroll
                for (int kk = 0; kk < 4; ++kk)
                    mma_bf16_by(leader, tmem, sw128_desc(at + kk * 32), sw128_desc(at + kChunkBytes + kk * 32),
                                mma_idesc(kTile, kTile), (c | kk) != 0);
                mma_commit_by(leader, smem_addr(&sh.empty[s]));
            }
            mma_commit_by(leader, smem_addr(&sh.acc));
            if (!warp_wait(&sh.acc, 0)) ok = false;
        } else {
            // ---- rotated key parts, then the accumulator
            if (blockIdx.x == 0) {
                for (int i = threadIdx.x; i < kTile * 8; i += 128) {
                    const int t = i / 8;
                    uint4 x = make_uint4(0, 0, 0, 0);
                    if (t < end) {
                        const int id = row[(t0 + t) / TTS_BLOCK_TOKENS];
                        if (id >= 0 && id < a.num_blocks)
                            x = *(reinterpret_cast<const uint4 *>(
                                      a.pool + (static_cast<size_t>(id) * TTS_BLOCK_TOKENS + t % TTS_BLOCK_TOKENS) *
                                                   (a.L + kLatentRope) + a.L) + i % 8);
                    }
                    reinterpret_cast<uint4 *>(a.kr)[static_cast<size_t>(tile) * kTile * 8 + i] = x;
                }
            }
            ok = warp_wait(&sh.acc, 0);
            if (ok) {
                tc_fence_after();
                // every MMA has read the ring: stage the tile there, in the
                // stores' swizzle (row r: 16-byte chunk j at j ^ (r % 8))
                const int r = warp * 32 + lane;
                const uint32_t tl = tmem + (static_cast<uint32_t>(warp * 32) << 16);
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    uint32_t x[32];
                    tmem_ld32_nowait(tl + c * 32, x);
                    tmem_wait_ld();
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const int k = (c % 2) * 4 + j;
                        const uint32_t at = base + (c / 2) * kChunkBytes + r * 128 + ((k ^ (r & 7)) << 4);
                        const float *f = reinterpret_cast<const float *>(x) + 8 * j;
                        asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(pack_bf16(f[0], f[1])),
                                     "r"(pack_bf16(f[2], f[3])), "r"(pack_bf16(f[4], f[5])), "r"(pack_bf16(f[6], f[7]))
                                     : "memory");
                    }
                }
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            }
            asm volatile("barrier.cta.sync 1, 128;" ::: "memory");
            if (threadIdx.x == 0 && ok) {
                const CUtensorMap *m = is_k ? &map_k : &map_v;
                tma_store_2d(m, f0, tile * kTile, base);
                if (f0 + 64 < features) tma_store_2d(m, f0 + 64, tile * kTile, base + kChunkBytes);
                asm volatile("cp.async.bulk.commit_group;\n\tcp.async.bulk.wait_group 0;" ::: "memory");
            }
        }
        if (!ok) flag_error(a.err, TTS_ERRBIT_TIMEOUT);
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 4) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 128;" ::"r"(tmem) : "memory");
    }
}

// --------------------------------------------------------------- attention

constexpr int kSlots = 8;           // ring slots of [128 tokens][64 values]
constexpr int kAttnThreads = 320;   // two softmax warpgroups, producer, MMA issuer

struct PrefillShared {
    uint64_t full[kSlots], empty[kSlots], q_full[2], s_full[2], p_full[2], o_done[2], done;
    uint32_t tmem;
};

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
        for (int i = 0; i < kSlots; ++i) {
            mbar_init(smem_addr(&sh.full[i]), 1);
            mbar_init(smem_addr(&sh.empty[i]), 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_addr(&sh.q_full[i]), 1);
            mbar_init(smem_addr(&sh.s_full[i]), 1);
            mbar_init(smem_addr(&sh.p_full[i]), 4);
            mbar_init(smem_addr(&sh.o_done[i]), 1);
        }
        mbar_init(smem_addr(&sh.done), 1);
        fence_mbar_init();
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
    const int b = uniform(stream_of_row(a.qtile_start, a.B, qt, lane));
    bool ok = true;
    if (b >= 0) {
        const int first = uniform(a.row_start[b]), n = uniform(a.row_start[b + 1]) - first, ctx = uniform(a.ctx_lens[b]);
        // a stream's last tiles, which see the most tokens, come first
        const int q = uniform(a.qtile_start[b + 1]) - 1 - qt;
        const int tile0 = uniform(a.tile_start[b]);
        const int r0 = q * kRows;                          // first row in the stream
        const bool two = r0 + kTile < n;
        // tokens either half sees, in tiles
        const int seen0 = ctx - n + min(n, r0 + kTile), seen1 = ctx - n + min(n, r0 + kRows);
        const int nt0 = (seen0 + kTile - 1) / kTile, nt1 = two ? (seen1 + kTile - 1) / kTile : 0;
        const int nt = max(nt0, nt1);
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
                uint32_t pos = 0;
                for (int j = 0; ok && j < nt; ++j) {
                    const int y = (tile0 + j) * kTile;
                    for (int c = 0; c < kQc + kVc; ++c, ++pos) {
                        const uint32_t s = pos % kSlots;
                        if (pos >= kSlots && !mbar_wait(smem_addr(&sh.empty[s]), (pos / kSlots - 1) & 1)) {
                            ok = false;
                            break;
                        }
                        const uint32_t bar = smem_addr(&sh.full[s]), at = ring + s * kChunkBytes;
                        mbar_arrive_expect_tx(bar, kChunkBytes);
                        if (c < kQc - 1) tma_load_2d(at, &map_k, h * kNope + c * 64, y, bar);
                        else if (c == kQc - 1) tma_load_2d(at, &map_kr, 0, y, bar);
                        else tma_load_2d(at, &map_v, h * kV + (c - kQc) * 64, y, bar);
                    }
                }
                for (uint32_t i = pos > kSlots ? pos - kSlots : 0; i < pos; ++i)
                    mbar_wait(smem_addr(&sh.full[i % kSlots]), (i / kSlots) & 1);
                for (int s = 0; s < (two ? 2 : 1); ++s) mbar_wait(smem_addr(&sh.q_full[s]), 0);
            }
        } else if (warp == 9) {
            // ---- MMA issuer: S0(0) S1(0) | O0(j) S0(j+1) O1(j) S1(j+1) ...
            // S of a half is overwritten right after the O product that reads
            // the weights kept in it; the tensor core runs them in order.
            const uint32_t leader = elect_leader();
            bool go = true;
            auto scores = [&](int s, int j, bool last_use) {
                const uint32_t pos = static_cast<uint32_t>(j) * (kQc + kVc);
                WarpWaits<kQc + 1> w;
#pragma unroll
                for (int c = 0; c < kQc; ++c) w.set(c, &sh.full[(pos + c) % kSlots], ((pos + c) / kSlots) & 1);
                w.set(kQc, &sh.q_full[s], 0);
                if (!w.wait()) {
                    go = false;
                    return;
                }
                tc_fence_after();
#pragma unroll
                for (int c = 0; c < kQc; ++c) {
                    const uint32_t slot = (pos + c) % kSlots;
                    const uint32_t sa = q_base + (s * kQc + c) * kChunkBytes, sb = ring + slot * kChunkBytes;
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)
                        mma_bf16_by(leader, tmem + s * kTile, sw128_desc(sa + kk * 32), sw128_desc(sb + kk * 32),
                                    mma_idesc(kTile, kTile), (c | kk) != 0);
                    if (last_use) mma_commit_by(leader, smem_addr(&sh.empty[slot]));
                }
                mma_commit_by(leader, smem_addr(&sh.s_full[s]));
            };
            auto output = [&](int s, int j, bool last_use) {
                const uint32_t pos = static_cast<uint32_t>(j) * (kQc + kVc) + kQc;
                WarpWaits<kVc + 1> w;
#pragma unroll
                for (int c = 0; c < kVc; ++c) w.set(c, &sh.full[(pos + c) % kSlots], ((pos + c) / kSlots) & 1);
                w.set(kVc, &sh.p_full[s], j & 1);
                if (!w.wait()) {
                    go = false;
                    return;
                }
                tc_fence_after();
#pragma unroll
                for (int c = 0; c < kVc; ++c) {
                    const uint32_t slot = (pos + c) % kSlots, sb = ring + slot * kChunkBytes;
#pragma unroll
                    for (int kk = 0; kk < kTile / 16; ++kk)
                        mma_bf16_ts_by(leader, tmem + (2 + s) * kTile + c * 64, tmem + s * kTile + kk * 8,
                                       sw128_mn_desc(sb + kk * 2048, kChunkBytes), mma_idesc(kTile, 64) | kTransposeB,
                                       (j | kk) != 0);
                    if (last_use) mma_commit_by(leader, smem_addr(&sh.empty[slot]));
                }
            };
            scores(0, 0, !two);
            if (go && two) scores(1, 0, true);
            for (int j = 0; go && j < nt; ++j) {
                if (j < nt0) {
                    output(0, j, !two);
                    if (go && j + 1 < nt0) scores(0, j + 1, !two);
                    if (go && j + 1 == nt0) mma_commit_by(leader, smem_addr(&sh.o_done[0]));
                }
                if (go && two) {
                    output(1, j, true);
                    if (go && j + 1 < nt1) scores(1, j + 1, true);
                    if (go && j + 1 == nt1) mma_commit_by(leader, smem_addr(&sh.o_done[1]));
                }
            }
            mma_commit_by(leader, smem_addr(&sh.done));
            ok = warp_wait(&sh.done, 0) && go;
        } else if (warp < 4 || two) {
            // ---- softmax warpgroups: thread = query row
            const int s = warp / 4, w = warp % 4;
            const int r = r0 + s * kTile + w * 32 + lane;          // row in the stream
            const int limit = ctx - n + min(n - 1, r) + 1;         // tokens it sees
            const int low = ctx - n + r0 + s * kTile + 1;          // tokens every row of the half sees
            const int tiles = s ? nt1 : nt0;
            const uint32_t lanes = static_cast<uint32_t>(w * 32) << 16;
            const uint32_t ts = tmem + lanes + s * kTile, to = tmem + lanes + (2 + s) * kTile;
            float m = kNoScore, l = 0.0f;
            uint32_t mask = a.blocks_ok[tile0];
            for (int j = 0; j < tiles; ++j) {
                const uint32_t next_mask = j + 1 < tiles ? a.blocks_ok[tile0 + j + 1] : 0;
                if (!warp_wait(&sh.s_full[s], j & 1)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                uint32_t x[kTile];
#pragma unroll
                for (int c = 0; c < kTile; c += 32) tmem_ld32_nowait(ts + c, x + c);
                tmem_wait_ld();
                if ((j + 1) * kTile > low || mask != 0xFFu) {
                    const int left = limit - j * kTile;
#pragma unroll
                    for (int i = 0; i < kTile; ++i)
                        if (i >= left || !((mask >> (i / TTS_BLOCK_TOKENS)) & 1)) x[i] = 0xFF800000u;  // -inf
                }
                mask = next_mask;
                float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                for (int i = 0; i < kTile; ++i) top[i % 4] = fmaxf(top[i % 4], __uint_as_float(x[i]));
                const float t = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])) * a.scale_log2;
                if (__any_sync(kFull, t > m + kSlack)) {
                    // (S(j) complete means that O(j - 1) is too)
                    const float now = fmaxf(m, t), f = hw_ex2(m - now);
                    m = now;
                    l *= f;
                    if (j > 0)
                        for (int c = 0; c < kV; c += 16) {
                            uint32_t o[16];
                            tmem_ld16_nowait(to + c, o);
                            tmem_wait_ld();
#pragma unroll
                            for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
                            tmem_st16(to + c, o);
                        }
                }
                float sum[2] = {0.0f, 0.0f};
#pragma unroll
                for (int c = 0; c < kTile; c += 64) {
                    uint32_t p[32];
#pragma unroll
                    for (int i = 0; i < 32; ++i) {
                        const float p0 = hw_ex2(fmaf(__uint_as_float(x[c + 2 * i]), a.scale_log2, -m));
                        const float p1 = hw_ex2(fmaf(__uint_as_float(x[c + 2 * i + 1]), a.scale_log2, -m));
                        sum[0] += p0;  // fp32; only the weights that enter the MMA are rounded
                        sum[1] += p1;
                        p[i] = pack_bf16(p0, p1);
                    }
                    tmem_st32(ts + c / 2, p);
                }
                l += sum[0] + sum[1];
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_addr(&sh.p_full[s]));
            }
            if (ok) ok = warp_wait(&sh.o_done[s], 0);
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
    size_t k_bytes, v_bytes, kr_bytes, start_bytes, ok_bytes;
    size_t total() const { return k_bytes + v_bytes + kr_bytes + 2 * start_bytes + ok_bytes; }
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
    p.ok_bytes = align_up(static_cast<size_t>(p.tiles) * 4, 256);
    return p;
}

template <int kNope, int kV>
int launch_prefill(const CUtensorMap *m, const PrefillArgs &a, unsigned grid, cudaStream_t stream) {
    constexpr int kSmem = (2 * (kNope / 64 + 1) + kSlots) * kChunkBytes + static_cast<int>(sizeof(PrefillShared));
    auto kernel = latent_prefill_kernel<kNope, kV>;
    if (!ensure_dynamic_smem(reinterpret_cast<const void *>(kernel), kSmem)) return TTS_ERR_CUDA;
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
    // grids, and token rows in the maps' 32-bit coordinates
    if (pl.tiles > 65535 || pl.qtiles * Hq > 0x7FFFFFFF) return TTS_ERR_UNSUPPORTED;

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
    a.qtile_start = reinterpret_cast<int32_t *>(at + pl.start_bytes);
    a.blocks_ok = reinterpret_cast<uint32_t *>(at + 2 * pl.start_bytes);
    a.pool = static_cast<const __nv_bfloat16 *>(cache->pool);
    a.out = static_cast<__nv_bfloat16 *>(d_out);
    a.err = d_err;
    const uint64_t kv_rows = static_cast<uint64_t>(pl.tiles) * kTile, T = num_rows;
    const uint64_t fk = static_cast<uint64_t>(Hq) * nope_dim, fv = static_cast<uint64_t>(Hq) * v_dim;
    CUtensorMap pool, uk, uv, qkv[5];
    if (!make_tma_2d_bf16(&pool, cache->pool, static_cast<uint64_t>(cache->num_blocks) * TTS_BLOCK_TOKENS,
                          L + kLatentRope, TTS_BLOCK_TOKENS, 64) ||
        !make_tma_2d_bf16(&uk, d_w_uk, fk, L, kTile, 64) || !make_tma_2d_bf16(&uv, d_w_uv, fv, L, kTile, 64) ||
        !make_tma_2d_bf16(&qkv[0], d_q_nope, T, fk, kTile, 64) ||
        !make_tma_2d_bf16(&qkv[1], d_q_rope, T, static_cast<uint64_t>(Hq) * kLatentRope, kTile, 64) ||
        !make_tma_2d_bf16(&qkv[2], k, kv_rows, fk, kTile, 64) ||
        !make_tma_2d_bf16(&qkv[3], a.kr, kv_rows, kLatentRope, kTile, 64) ||
        !make_tma_2d_bf16(&qkv[4], v, kv_rows, fv, kTile, 64))
        return TTS_ERR_CUDA;

    const cudaStream_t cs = static_cast<cudaStream_t>(stream);
    int rc = launch_kernel(latent_plan_kernel, dim3(1), dim3(kPlanThreads), 0, {cs, thread_pdl()}, a);
    if (rc != TTS_OK) return rc;
    const int k_tiles = static_cast<int>((fk + kTile - 1) / kTile), v_tiles = static_cast<int>((fv + kTile - 1) / kTile);
    if (!ensure_dynamic_smem(reinterpret_cast<const void *>(latent_expand_kernel), kExpandSmem)) return TTS_ERR_CUDA;
    rc = launch_kernel(latent_expand_kernel, dim3(k_tiles + v_tiles, static_cast<unsigned>(pl.tiles)),
                       dim3(kExpandThreads), kExpandSmem, {cs, true}, pool, uk, uv, qkv[2], qkv[4], a, k_tiles);
    if (rc != TTS_OK) return rc;
    const unsigned grid = static_cast<unsigned>(pl.qtiles * Hq);
    if (nope_dim == 128)
        return v_dim == 128 ? launch_prefill<128, 128>(qkv, a, grid, cs) : launch_prefill<128, 64>(qkv, a, grid, cs);
    return v_dim == 128 ? launch_prefill<64, 128>(qkv, a, grid, cs) : launch_prefill<64, 64>(qkv, a, grid, cs);
}
