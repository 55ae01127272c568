// Decode attention over the latent cache, absorbed form: with q~ = w_uk[h]^T
// q_nope a head's scores and sums run over the latents themselves,
//   s_t = scale (q~ . c_t + q_rope . kr_t),   o~ = sum_t softmax(s)_t c_t,
//   out = w_uv[h] o~,
// so every head of a stream reads the same 2 (latent_dim + 64) bytes a token.
// Three kernels, each a programmatic dependent of the one before:
//
//  1. latent_absorb_kernel: q~ (bf16) and q_rope side by side, one row per
//     (query row, head).
//  2. latent_attn_kernel: split-KV attention on tcgen05, persistent, one CTA
//     per SM.  The query rows are the MMA's N side (N = 16..64 of a stream's
//     q_len x Hq rows), as in the codebook head, so that a few rows still use
//     whole MMAs: S^T[64 tokens][N] = KV . Q~^T and
//     O^T[latent_dim][N] += C^T . P^T, where C is the latent part of the same
//     shared-memory tile (read K-major for S^T, MN-major for O^T): a token's
//     row is fetched once.
//  3. latent_out_kernel: joins the splits and multiplies by w_uv.
//
// Bound: HBM at one query row a stream (16 heads: 30 flop a byte).  The MMAs
// of a 64-token tile read 9 x 8 KB (S^T) + 4 x 16 KB (O^T) of shared memory,
// about 1100 cycles at N <= 32, where HBM delivers the tile's 73.7 KB to an SM
// in about 3100.
#include <cuda_bf16.h>

#include <cmath>

#include "latent_common.cuh"
#include "tcgen05.cuh"
#include "tts_common.cuh"
#include "tts_internal.h"

namespace tts {
namespace {

constexpr unsigned kFull = 0xFFFFFFFFu;
constexpr int kTile = 64;              // tokens per tile (4 blocks)
constexpr int kChunkBytes = kTile * 128;       // [64 tokens][64 values] bf16, 128-byte swizzle
constexpr int kPairBytes = 2 * kChunkBytes;    // 128 latent dimensions: one MMA M block of O^T
constexpr int kMaxGroup = 64;          // query rows per work unit
constexpr int kCtas = 152;             // one per SM
constexpr int kAttnThreads = 224;      // 4 softmax warps, KV producer, MMA issuer, Q loader
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kNoScore = -1e30f;     // running maximum before any token (log2 units)
// The running maximum is moved only when a score passes it by this much (log2
// units): weights then reach 2^8, which fp32 sums and bf16 weights hold as
// well as 1, and O in tensor memory is rarely rescaled.
constexpr float kSlack = 8.0f;

// ---------------------------------------------------------------- mma.sync

__device__ __forceinline__ void mma16816(float *c, const uint32_t *a, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9},"
        " {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    const __nv_bfloat162 p = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&p);
}

// ------------------------------------------------------------------ absorb

// q~[r][h][l] = sum_d q_nope[r][h][d] w_uk[h][d][l], rounded to bf16 (the MMA
// that follows takes bf16), then q_rope[r][h] behind it.  A CTA holds the
// [nope][64] slice of one head's weights in registers (each of its 4 warps a
// quarter of d) and runs over 16-row chunks; the warps' sums meet in shared
// memory.  The contraction's and the columns' order inside an MMA is free, so
// a lane's weights are 16-byte loads: its 4 contraction rows are 4 adjacent d,
// its 8 column blocks 8 adjacent l.
// Latency-bound (2 MB of weights at 16 heads): the weights are in flight
// before the wait for the previous kernel.
constexpr int kAbsorbChunks = 4;  // 16-row chunks per CTA

template <int kSteps>  // 16-deep MMA steps per warp: nope / 64
__global__ void __launch_bounds__(128)
latent_absorb_kernel(const __nv_bfloat16 *__restrict__ q_nope, const __nv_bfloat16 *__restrict__ q_rope,
                     const __nv_bfloat16 *__restrict__ w_uk, __nv_bfloat16 *__restrict__ qt, int R, int Hq, int L) {
    constexpr int kNope = 64 * kSteps;
    __shared__ float red[4][16][68];
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, g = lane / 4, c = lane % 4;
    const int l0 = blockIdx.x * 64, h = blockIdx.y;
    uint32_t b[kSteps][8][2];
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
        const int d = (warp * kSteps + s) * 16 + 4 * c;
        uint4 w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            w[i] = __ldg(reinterpret_cast<const uint4 *>(w_uk + (static_cast<size_t>(h) * kNope + d + i) * L + l0 + 8 * g));
        const uint32_t *w0 = &w[0].x, *w1 = &w[1].x, *w2 = &w[2].x, *w3 = &w[3].x;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const uint32_t sel = (j & 1) ? 0x7632u : 0x5410u;
            b[s][j][0] = __byte_perm(w0[j / 2], w1[j / 2], sel);
            b[s][j][1] = __byte_perm(w2[j / 2], w3[j / 2], sel);
        }
    }
    pdl_wait_prerequisites();
    pdl_allow_dependents();  // only now: the attention reads the pool as soon as it starts
    const int W = L + kLatentRope;
    const int r_end = min(R, (static_cast<int>(blockIdx.z) + 1) * kAbsorbChunks * 16);
    for (int r0 = blockIdx.z * kAbsorbChunks * 16; r0 < r_end; r0 += 16) {
        float acc[8][4] = {};
#pragma unroll
        for (int s = 0; s < kSteps; ++s) {
            const int d = (warp * kSteps + s) * 16 + 4 * c;
            uint2 lo = make_uint2(0, 0), hi = make_uint2(0, 0);
            if (r0 + g < R)
                lo = *reinterpret_cast<const uint2 *>(q_nope + (static_cast<size_t>(r0 + g) * Hq + h) * kNope + d);
            if (r0 + g + 8 < R)
                hi = *reinterpret_cast<const uint2 *>(q_nope + (static_cast<size_t>(r0 + g + 8) * Hq + h) * kNope + d);
            const uint32_t a[4] = {lo.x, hi.x, lo.y, hi.y};
#pragma unroll
            for (int j = 0; j < 8; ++j) mma16816(acc[j], a, b[s][j][0], b[s][j][1]);
        }
        // column 2c (+1) of block j is l0 + 16 c (+ 8) + j
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            red[warp][g][16 * c + j] = acc[j][0];
            red[warp][g][16 * c + 8 + j] = acc[j][1];
            red[warp][g + 8][16 * c + j] = acc[j][2];
            red[warp][g + 8][16 * c + 8 + j] = acc[j][3];
        }
        __syncthreads();
        const int row = threadIdx.x / 8, col = threadIdx.x % 8 * 8;
        if (r0 + row < R) {
            float x[8];
#pragma unroll
            for (int i = 0; i < 8; ++i)
                x[i] = (red[0][row][col + i] + red[1][row][col + i]) + (red[2][row][col + i] + red[3][row][col + i]);
            __nv_bfloat16 *dst = qt + (static_cast<size_t>(r0 + row) * Hq + h) * W;
            *reinterpret_cast<uint4 *>(dst + l0 + col) =
                make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7]));
            if (blockIdx.x == 0)
                *reinterpret_cast<uint4 *>(dst + L + col) = *reinterpret_cast<const uint4 *>(
                    q_rope + (static_cast<size_t>(r0 + row) * Hq + h) * kLatentRope + col);
        }
        __syncthreads();
    }
}

// -------------------------------------------------------------- work split

// The work units are the 64-token tiles of every (stream, row group), group
// bg = b * G + g, in order; CTA c of P takes units [U c / P, U (c + 1) / P).
// The part of a group that a CTA takes is a segment; its partial result goes
// to slot c + bg (unique: going on to the next segment raises one of the two).
struct LatentPlan {
    int G, N;       // row groups a stream, rows per group (a multiple of 16)
    int P;          // CTAs
    size_t slots;   // P + B * G
    size_t qt_bytes, part_bytes, ml_bytes, starts_bytes;
    size_t total() const { return qt_bytes + part_bytes + ml_bytes + starts_bytes; }
};

LatentPlan latent_plan(int B, int q_len, int Hq, int L, int max_ctx) {
    LatentPlan p;
    const int rows = q_len * Hq;
    p.G = (rows + kMaxGroup - 1) / kMaxGroup;
    p.N = ((rows + p.G - 1) / p.G + 15) / 16 * 16;
    const long units = static_cast<long>(B) * p.G * ((static_cast<long>(max_ctx) + kTile - 1) / kTile);
    p.P = units < kCtas ? static_cast<int>(units < 1 ? 1 : units) : kCtas;
    p.slots = static_cast<size_t>(p.P) + static_cast<size_t>(B) * p.G;
    p.qt_bytes = align_up(static_cast<size_t>(B) * rows * (L + kLatentRope) * 2, 256);
    p.part_bytes = align_up(p.slots * p.N * L * 4, 256);
    p.ml_bytes = align_up(p.slots * p.N * 8, 256);
    p.starts_bytes = align_up((static_cast<size_t>(B) + 1) * 8, 256);
    return p;
}

// (of the CTAs launched, as many as there are units take part, so that every
// one of them has a unit and a group's CTAs are consecutive)
__device__ __forceinline__ int active_ctas(long long U, int launched) {
    return U < launched ? static_cast<int>(U) : launched;
}
__device__ __forceinline__ long long unit_begin(long long U, int c, int P) { return U * c / P; }
__device__ __forceinline__ int unit_owner(long long U, long long u, int P) {
    return static_cast<int>(((u + 1) * P - 1) / U);
}

struct LatentAttnArgs {
    const int32_t *table;
    int max_blocks, num_blocks;
    const int32_t *ctx_lens;
    int max_ctx, B, q_len, Hq, L;
    int G;
    float scale_log2;  // scale * log2(e)
    int causal;
    float *part;       // [slots][N][L] unnormalised o~
    float2 *ml;        // [slots][N] running maximum (log2 units), sum
    long long *starts; // [B + 1] first unit of each stream, U last
    int32_t *err;
    int pairs, ropes;  // ring slots
};

// Tiles of stream b (0: its length is out of range).
__device__ __forceinline__ int stream_tiles(const LatentAttnArgs &a, int b, int *ctx_out = nullptr) {
    const int ctx = a.ctx_lens[b];
    if (ctx_out) *ctx_out = ctx;
    if (ctx < a.q_len || ctx > a.max_ctx || ctx > a.max_blocks * TTS_BLOCK_TOKENS) return 0;
    return (ctx + kTile - 1) / kTile;
}

// Walks a CTA's segments; every role keeps its own copy.
struct Segments {
    int b, g, tile;        // next segment's start
    long long left;        // units left
    // current segment
    int ctx, first, count; // first tile, tiles
    int bg;
    __device__ __forceinline__ bool next(const LatentAttnArgs &a) {
        while (left > 0) {
            const int n = stream_tiles(a, b, &ctx);
            if (n == 0) {  // (never the CTA's first stream)
                ++b;
                continue;
            }
            first = tile;
            count = static_cast<int>(min(static_cast<long long>(n - tile), left));
            bg = b * a.G + g;
            left -= count;
            cur_b = b;
            cur_g = g;
            tile = 0;
            if (++g == a.G) {
                g = 0;
                ++b;
            }
            return true;
        }
        return false;
    }
    int cur_b, cur_g;
};

// ------------------------------------------------------------- attention

// Barrier of the four softmax warps with an OR over their threads.
__device__ __forceinline__ bool softmax_any(bool pred) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.b32 p, %1, 0;\n\t"
        "barrier.cta.red.or.pred q, 1, 128, p;\n\t"
        "selp.b32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"(static_cast<uint32_t>(pred))
        : "memory");
    return r != 0;
}
__device__ __forceinline__ void softmax_sync() { asm volatile("barrier.cta.sync 1, 128;" ::: "memory"); }

constexpr int kMaxPairs = 16, kMaxRopes = 4;

struct AttnShared {
    uint64_t full_l[kMaxPairs], empty_l[kMaxPairs], full_r[kMaxRopes], empty_r[kMaxRopes];
    uint64_t s_full[2], s_empty[2], p_full, p_empty, o_empty, q_full, q_empty, done;
    long long U;
    int start_b, start_g, start_tile;
    uint32_t tmem;
    long long sums[8];
    float mref[kMaxGroup], fac[kMaxGroup];
    int limit[kMaxGroup];
    union {
        uint32_t wmax[4][kMaxGroup];  // within a tile
        float lsum[4][kMaxGroup];     // at a segment's end
    };
};

// mbar_wait by a whole warp, with one answer.
__device__ __forceinline__ bool warp_wait(const uint64_t *bar, uint32_t parity) {
    return __all_sync(kFull, mbar_wait(smem_addr(bar), parity));
}

template <int N>
__global__ void __launch_bounds__(kAttnThreads, 1)
latent_attn_kernel(const __grid_constant__ CUtensorMap map_kv, const __grid_constant__ CUtensorMap map_q,
                   const LatentAttnArgs a) {
    extern __shared__ __align__(1024) uint8_t raw[];
    const uint32_t base = smem_addr(raw);
    const int chunks = a.L / 64, nb = (a.L + 127) / 128;
    const uint32_t q_base = base;                                       // [chunks + 1][N][128 B]
    const uint32_t p_base = q_base + (chunks + 1) * N * 128;            // [N][128 B]
    const uint32_t r_base = p_base + N * 128;                           // rope ring
    const uint32_t l_base = r_base + a.ropes * kChunkBytes;             // latent ring
    AttnShared &sh = *reinterpret_cast<AttnShared *>(raw + (l_base - base) + a.pairs * kPairBytes);
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;

    if (warp == 5 && lane == 0) {
        for (int i = 0; i < a.pairs; ++i) {
            mbar_init(smem_addr(&sh.full_l[i]), 1);
            mbar_init(smem_addr(&sh.empty_l[i]), 1);
        }
        for (int i = 0; i < a.ropes; ++i) {
            mbar_init(smem_addr(&sh.full_r[i]), 1);
            mbar_init(smem_addr(&sh.empty_r[i]), 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_addr(&sh.s_full[i]), 1);
            mbar_init(smem_addr(&sh.s_empty[i]), 4);
        }
        mbar_init(smem_addr(&sh.p_full), 4);
        mbar_init(smem_addr(&sh.p_empty), 1);
        mbar_init(smem_addr(&sh.o_empty), 4);
        mbar_init(smem_addr(&sh.q_full), 1);
        mbar_init(smem_addr(&sh.q_empty), 1);
        mbar_init(smem_addr(&sh.done), 1);
        fence_mbar_init();
        prefetch_tensormap(&map_kv);
        prefetch_tensormap(&map_q);
    }
    uint32_t cols = 32;
    while (cols < static_cast<uint32_t>((nb + 2) * N)) cols *= 2;
    if (warp == 6) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(&sh.tmem)),
                     "r"(cols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    // ---- this CTA's units: a scan of the streams' tile counts
    const int per = (a.B + kAttnThreads - 1) / kAttnThreads;
    const int b0 = min(a.B, static_cast<int>(threadIdx.x) * per), b1 = min(a.B, b0 + per);
    long long mine = 0;
    for (int b = b0; b < b1; ++b) {
        const int n = stream_tiles(a, b);
        mine += n;
        if (n == 0 && blockIdx.x == 0) flag_error(a.err, TTS_ERRBIT_CTX_LEN);
    }
    long long incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
        const long long x = __shfl_up_sync(kFull, incl, o);
        if (lane >= o) incl += x;
    }
    if (lane == 31) sh.sums[warp] = incl;
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    long long before = incl - mine, total = 0;
    for (int w = 0; w < kAttnThreads / 32; ++w) {
        if (w < warp) before += sh.sums[w];
        total += sh.sums[w];
    }
    const long long U = total * a.G;
    const int P = active_ctas(U, gridDim.x), me = blockIdx.x;
    const long long u0 = me < P ? unit_begin(U, me, P) : U, u1 = me < P ? unit_begin(U, me + 1, P) : U;
    {
        long long at = before * a.G;
        for (int b = b0; b < b1; ++b) {
            const long long n = stream_tiles(a, b);
            if (blockIdx.x == 0) a.starts[b] = at;
            if (u0 < u1 && u0 >= at && u0 < at + n * a.G) {
                sh.start_b = b;
                sh.start_g = static_cast<int>((u0 - at) / n);
                sh.start_tile = static_cast<int>((u0 - at) % n);
            }
            at += n * a.G;
        }
        if (blockIdx.x == 0 && threadIdx.x == 0) a.starts[a.B] = U;
    }
    __syncthreads();
    const uint32_t tmem = sh.tmem;
    Segments seg;
    seg.left = u1 - u0;
    seg.b = sh.start_b;
    seg.g = sh.start_g;
    seg.tile = sh.start_tile;
    pdl_allow_dependents();
    bool ok = true;

    if (warp == 4) {
        // ---- KV producer: per tile the rope chunk, then the latent pairs;
        // lanes 0-3 each fetch one block's 16 rows.  A block outside the pool
        // (or past the context) is read out of range, which fills zeros.
        const int oob = a.num_blocks * TTS_BLOCK_TOKENS;
        uint32_t it = 0, lpos = 0;
        const uint32_t ropes = a.ropes, pairs = a.pairs;
        while (ok && seg.next(a)) {
            const int32_t *row = a.table + static_cast<size_t>(seg.cur_b) * a.max_blocks;
            const int blocks = (seg.ctx + TTS_BLOCK_TOKENS - 1) / TTS_BLOCK_TOKENS;
            auto fetch = [&](int tile) {
                const int i = tile * 4 + lane;
                return lane < 4 && i < blocks ? row[i] : -1;
            };
            int id = fetch(seg.first);
            for (int k = 0; ok && k < seg.count; ++k, ++it) {
                const int tile = seg.first + k;
                int y = oob;
                if (lane < 4 && tile * 4 + lane < blocks) {
                    if (id >= 0 && id < a.num_blocks) y = id * TTS_BLOCK_TOKENS;
                    else flag_error(a.err, TTS_ERRBIT_BLOCK_ID);
                }
                if (k + 1 < seg.count) id = fetch(tile + 1);
                const uint32_t rs = it % ropes;
                const uint32_t fr = smem_addr(&sh.full_r[rs]);
                if (it >= ropes && !warp_wait(&sh.empty_r[rs], (it / ropes - 1) & 1)) {
                    ok = false;
                    break;
                }
                if (lane == 0) mbar_arrive_expect_tx(fr, kChunkBytes);
                __syncwarp();
                if (lane < 4) tma_load_2d(r_base + rs * kChunkBytes + lane * 2048, &map_kv, a.L, y, fr);
                for (int p = 0; p < nb; ++p, ++lpos) {
                    const uint32_t ls = lpos % pairs;
                    const uint32_t fl = smem_addr(&sh.full_l[ls]);
                    if (lpos >= pairs && !warp_wait(&sh.empty_l[ls], (lpos / pairs - 1) & 1)) {
                        ok = false;
                        break;
                    }
                    const int halves = min(2, chunks - 2 * p);
                    if (lane == 0) mbar_arrive_expect_tx(fl, halves * kChunkBytes);
                    __syncwarp();
                    if (lane < 4)
                        for (int i = 0; i < halves; ++i)
                            tma_load_2d(l_base + ls * kPairBytes + i * kChunkBytes + lane * 2048, &map_kv,
                                        (2 * p + i) * 64, y, fl);
                }
            }
        }
        // every copy lands before the CTA ends
        if (lane == 0) {
            for (uint32_t i = it > ropes ? it - ropes : 0; i < it; ++i)
                mbar_wait(smem_addr(&sh.full_r[i % ropes]), (i / ropes) & 1);
            for (uint32_t i = lpos > pairs ? lpos - pairs : 0; i < lpos; ++i)
                mbar_wait(smem_addr(&sh.full_l[i % pairs]), (i / pairs) & 1);
        }
    } else if (warp == 6) {
        // ---- Q loader: a segment's q~ rows, once the S MMAs of the one before are done
        pdl_wait_prerequisites();
        if (lane == 0) {
            uint32_t s = 0;
            for (; seg.next(a); ++s) {
                if (s > 0 && !mbar_wait(smem_addr(&sh.q_empty), (s - 1) & 1)) {
                    ok = false;
                    break;
                }
                const uint32_t bar = smem_addr(&sh.q_full);
                mbar_arrive_expect_tx(bar, (chunks + 1) * N * 128);
                const int y = seg.cur_b * a.q_len * a.Hq + seg.cur_g * N;
                for (int c = 0; c <= chunks; ++c) tma_load_2d(q_base + c * N * 128, &map_q, c * 64, y, bar);
            }
            if (s > 0) mbar_wait(smem_addr(&sh.q_full), (s - 1) & 1);
        }
    } else if (warp == 5) {
        // ---- MMA issuer (one lane issues; the warp clears stale rows).  S^T of
        // tile i + 1 goes before O^T of tile i, so the tensor core works on it
        // while the softmax warps turn S^T of tile i into weights.
        constexpr uint32_t idesc_s = mma_idesc(64, N);
        constexpr uint32_t idesc_o = mma_idesc(128, N) | kTransposeA;
        uint32_t it = 0, lpos = 0, segs = 0;
        const uint32_t ropes = a.ropes, pairs = a.pairs;
        // the tile whose O^T is outstanding
        bool pending = false, pend_first = false;
        uint32_t pend_lpos = 0, pend_seg = 0;
        auto issue_o = [&]() -> bool {
            // the outstanding tile is it - 1, before and after the loop
            if (!warp_wait(&sh.p_full, (it - 1) & 1)) return false;
            if (pend_first && pend_seg > 0 && !warp_wait(&sh.o_empty, (pend_seg - 1) & 1)) return false;
            tc_fence_after();
            if (lane == 0) {
                for (int p = 0; p < nb; ++p) {
                    const uint32_t ls = (pend_lpos + p) % pairs;
                    const uint32_t sa = l_base + ls * kPairBytes;
#pragma unroll
                    for (int k = 0; k < kTile / 16; ++k)
                        mma_bf16(tmem + (2 + p) * N, sw128_mn_desc(sa + k * 2048, kChunkBytes),
                                 sw128_desc(p_base + k * 32), idesc_o, !(pend_first && k == 0));
                    mma_commit(smem_addr(&sh.empty_l[ls]));
                }
                mma_commit(smem_addr(&sh.p_empty));
            }
            __syncwarp();
            return true;
        };
        while (ok && seg.next(a)) {
            if (!warp_wait(&sh.q_full, segs & 1)) {
                ok = false;
                break;
            }
            for (int k = 0; ok && k < seg.count; ++k) {
                const uint32_t buf = it & 1;
                if (it >= 2 && !warp_wait(&sh.s_empty[buf], (it / 2 - 1) & 1)) {
                    ok = false;
                    break;
                }
                const uint32_t rs = it % ropes;
                if (!warp_wait(&sh.full_r[rs], (it / ropes) & 1)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                if (lane == 0) {
                    const uint32_t sa = r_base + rs * kChunkBytes, sb = q_base + chunks * N * 128;
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)
                        mma_bf16(tmem + buf * N, sw128_desc(sa + kk * 32), sw128_desc(sb + kk * 32), idesc_s, kk != 0);
                    mma_commit(smem_addr(&sh.empty_r[rs]));
                }
                // rows behind the context in its last block hold anything (NaN
                // times a zero weight would spread): clear them
                const int end = seg.ctx - (seg.first + k) * kTile;  // tokens of the context in this tile
                const int stale = end < kTile ? (TTS_BLOCK_TOKENS - end % TTS_BLOCK_TOKENS) % TTS_BLOCK_TOKENS : 0;
                for (int p = 0; p < nb; ++p) {
                    const uint32_t ls = (lpos + p) % pairs;
                    if (!warp_wait(&sh.full_l[ls], ((lpos + p) / pairs) & 1)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t sa = l_base + ls * kPairBytes;
                    const int halves = min(2, chunks - 2 * p);
                    if (stale) {
                        for (int i = lane; i < halves * stale * 8; i += 32) {
                            const uint32_t at = sa + (i / (stale * 8)) * kChunkBytes + end * 128 + i % (stale * 8) * 16;
                            asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(at), "r"(0) : "memory");
                        }
                        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                        __syncwarp();
                    }
                    if (lane == 0)
                        for (int i = 0; i < halves; ++i)
#pragma unroll
                            for (int kk = 0; kk < 4; ++kk)
                                mma_bf16(tmem + buf * N, sw128_desc(sa + i * kChunkBytes + kk * 32),
                                         sw128_desc(q_base + (2 * p + i) * N * 128 + kk * 32), idesc_s, 1);
                }
                if (!ok) break;
                if (lane == 0) {
                    mma_commit(smem_addr(&sh.s_full[buf]));
                    if (k + 1 == seg.count) mma_commit(smem_addr(&sh.q_empty));
                }
                __syncwarp();
                if (pending && !issue_o()) {
                    ok = false;
                    break;
                }
                pending = true;
                pend_first = k == 0;
                pend_lpos = lpos;
                pend_seg = segs;
                lpos += nb;
                ++it;
            }
            ++segs;
        }
        if (ok && pending && !issue_o()) ok = false;
        if (lane == 0) {
            mma_commit(smem_addr(&sh.done));
            if (!mbar_wait(smem_addr(&sh.done), 0)) ok = false;
        }
    } else {
        // ---- softmax warps: lane l < 16 of warp w has token 16 w + l of the
        // tile (a 64-row accumulator's rows 16 w.. sit in lanes 32 w..), so a
        // warp's tokens are one block
        uint32_t it = 0;
        const uint32_t tl = tmem + (static_cast<uint32_t>(warp * 32) << 16);
        const int tok = warp * 16 + lane;
        const bool live = lane < 16;
        const int tid = threadIdx.x;
        while (ok && seg.next(a)) {
            const int32_t *row = a.table + static_cast<size_t>(seg.cur_b) * a.max_blocks;
            const int blocks = (seg.ctx + TTS_BLOCK_TOKENS - 1) / TTS_BLOCK_TOKENS;
            auto block_ok = [&](int tile) {
                const int i = tile * 4 + warp;
                if (i >= blocks) return false;
                const int id = row[i];
                return id >= 0 && id < a.num_blocks;
            };
            const int low = a.causal ? seg.ctx - a.q_len + 1 : seg.ctx;  // tokens every row sees
            softmax_sync();  // the last segment's reads of these are over
            if (tid < N) {
                sh.mref[tid] = kNoScore;
                const int j = (seg.cur_g * N + tid) / a.Hq;
                sh.limit[tid] = j >= a.q_len ? 0 : a.causal ? seg.ctx - a.q_len + j + 1 : seg.ctx;
            }
            softmax_sync();
            float l[N];
#pragma unroll
            for (int n = 0; n < N; ++n) l[n] = 0.0f;
            bool valid = block_ok(seg.first);
            for (int k = 0; k < seg.count; ++k, ++it) {
                const int tile = seg.first + k;
                const uint32_t buf = it & 1;
                const bool next_valid = k + 1 < seg.count && block_ok(tile + 1);
                if (!warp_wait(&sh.s_full[buf], (it / 2) & 1)) ok = false;
                tc_fence_after();
                uint32_t sr[N];
#pragma unroll
                for (int c = 0; c < N; c += 16) tmem_ld16_nowait(tl + buf * N + c, sr + c);
                tmem_wait_ld();
                tc_fence_before();
                if (lane == 0) mbar_arrive(smem_addr(&sh.s_empty[buf]));
                const int t = tile * kTile + tok;
                if (!valid || !live) {
#pragma unroll
                    for (int n = 0; n < N; ++n) sr[n] = 0xFF800000u;  // -inf
                } else if ((tile + 1) * kTile > low) {
#pragma unroll
                    for (int n = 0; n < N; ++n)
                        if (t >= sh.limit[n]) sr[n] = 0xFF800000u;
                }
                float top = -INFINITY;
#pragma unroll
                for (int n = 0; n < N; ++n) top = fmaxf(top, fmaf(__uint_as_float(sr[n]), a.scale_log2, -sh.mref[n]));
                if (softmax_any(top > kSlack || !ok)) {
                    // rare: raise the running maxima to this tile's, rescale sums and O
                    if (softmax_any(!ok)) {
                        ok = false;
                        break;
                    }
#pragma unroll
                    for (int n = 0; n < N; ++n) {
                        const uint32_t m = __reduce_max_sync(kFull, float_order_key(__uint_as_float(sr[n]) * a.scale_log2));
                        if (lane == 0) sh.wmax[warp][n] = m;
                    }
                    softmax_sync();
                    if (tid < N) {
                        const uint32_t m = max(max(sh.wmax[0][tid], sh.wmax[1][tid]), max(sh.wmax[2][tid], sh.wmax[3][tid]));
                        const float old = sh.mref[tid], now = fmaxf(old, order_key_float(m));
                        sh.mref[tid] = now;
                        sh.fac[tid] = hw_ex2(old - now);
                    }
                    softmax_sync();
#pragma unroll
                    for (int n = 0; n < N; ++n) l[n] *= sh.fac[n];
                    if (k > 0) {
                        if (!warp_wait(&sh.p_empty, (it - 1) & 1)) ok = false;
                        tc_fence_after();
                        for (int p = 0; p < nb; ++p)
                            for (int c = 0; c < N; c += 16) {
                                uint32_t o[16];
                                tmem_ld16_nowait(tl + (2 + p) * N + c, o);
                                tmem_wait_ld();
#pragma unroll
                                for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * sh.fac[c + i]);
                                tmem_st16(tl + (2 + p) * N + c, o);
                            }
                        tmem_wait_st();
                    }
                }
                float x[N];
#pragma unroll
                for (int n = 0; n < N; ++n) {
                    x[n] = hw_ex2(fmaf(__uint_as_float(sr[n]), a.scale_log2, -sh.mref[n]));
                    l[n] += x[n];  // fp32; only the weights that enter the MMA are rounded
                }
                // P of the tile before has been read (and its O^T added)
                if (it > 0 && !warp_wait(&sh.p_empty, (it - 1) & 1)) ok = false;
                if (live) {
#pragma unroll
                    for (int n = 0; n < N; ++n) {
                        const uint32_t at = p_base + n * 128 + (((tok >> 3) ^ (n & 7)) << 4) + (tok & 7) * 2;
                        asm volatile("st.shared.b16 [%0], %1;" ::"r"(at),
                                     "h"(__bfloat16_as_ushort(__float2bfloat16_rn(x[n])))
                                     : "memory");
                    }
                }
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_addr(&sh.p_full));
                valid = next_valid;
            }
            // ---- the segment's partial result
            if (!warp_wait(&sh.p_empty, (it - 1) & 1)) ok = false;
            if (softmax_any(!ok)) {  // (all four warps leave together)
                ok = false;
                break;
            }
#pragma unroll
            for (int n = 0; n < N; ++n) {
                float s = l[n];
#pragma unroll
                for (int o = 8; o > 0; o >>= 1) s += __shfl_xor_sync(kFull, s, o);
                if (lane == 0) sh.lsum[warp][n] = s;
            }
            const size_t slot = static_cast<size_t>(blockIdx.x) + seg.bg;
            softmax_sync();
            if (tid < N)
                a.ml[slot * N + tid] = make_float2(
                    sh.mref[tid], (sh.lsum[0][tid] + sh.lsum[1][tid]) + (sh.lsum[2][tid] + sh.lsum[3][tid]));
            tc_fence_after();
            for (int p = 0; p < nb; ++p) {
                const int d = p * 128 + warp * 32 + lane;
                for (int c = 0; c < N; c += 16) {
                    uint32_t o[16];
                    tmem_ld16_nowait(tl + (2 + p) * N + c, o);
                    tmem_wait_ld();
                    if (d < a.L) {
                        float *dst = a.part + (slot * N + c) * a.L + d;
#pragma unroll
                        for (int i = 0; i < 16; ++i) dst[static_cast<size_t>(i) * a.L] = __uint_as_float(o[i]);
                    }
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_addr(&sh.o_empty));
        }
    }
    if (!ok) flag_error(a.err, TTS_ERRBIT_TIMEOUT);
    tc_fence_before();
    __syncthreads();
    if (warp == 6) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(cols) : "memory");
    }
}

// ------------------------------------------------------------------ output

// out[r][h] = w_uv[h] o~[r][h], o~ the join of the row's splits (weights
// 2^(m_s - max m)), rounded to bf16 for the MMA.  A CTA takes one head and 16
// query rows; each of its v / 8 warps holds 8 of w_uv's rows in registers
// (loaded before the wait for the attention).  The contraction's order inside
// an MMA is free: a lane takes 8 adjacent l per 32, one 16-byte load.
template <int kV>
__global__ void __launch_bounds__(kV * 4)
latent_out_kernel(const LatentAttnArgs a, int N, int launched, const __nv_bfloat16 *__restrict__ w_uv,
                  __nv_bfloat16 *__restrict__ out) {
    constexpr int kWarps = kV / 8;
    constexpr int kMaxK = kLatentMaxDim / 32;
    extern __shared__ float4 raw4[];
    const int L = a.L, R = a.B * a.q_len;
    float *sums = reinterpret_cast<float *>(raw4);                 // [kWarps][L]
    uint8_t *at = reinterpret_cast<uint8_t *>(sums + kWarps * L);  // [16] rows of L bf16 + 64 bytes
    const int row_bytes = 2 * L + 64;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, g = lane / 4, c = lane % 4;
    const int r0 = blockIdx.x * 16, h = blockIdx.y;
    uint4 w[kMaxK];
#pragma unroll
    for (int k = 0; k < kMaxK; ++k)
        if (32 * k < L)
            w[k] = __ldg(reinterpret_cast<const uint4 *>(w_uv + (static_cast<size_t>(h) * kV + warp * 8 + g) * L + 32 * k + 8 * c));
    pdl_wait_prerequisites();
    pdl_allow_dependents();

    // ---- join: rows in turn to groups of `share` warps, which split the row's slots
    const int rows = min(16, R - r0);
    int share = kWarps;
    while (share > 1 && kWarps / share < rows) share /= 2;
    const long long U = a.starts[a.B];
    const int P = active_ctas(U, launched);
    for (int rr = 0; rr < 16; rr += kWarps / share) {
        const int i = rr + warp / share, sub = warp % share;
        if (i < rows) {
            const int r = r0 + i, b = r / a.q_len, idx = (r % a.q_len) * a.Hq + h;
            const int grp = idx / N, n = idx % N, bg = b * a.G + grp;
            float o[kLatentMaxDim / 32] = {};
            float inv = 0.0f;
            const long long s0 = a.starts[b], len = (a.starts[b + 1] - s0) / a.G;
            if (len > 0) {
                const int c0 = unit_owner(U, s0 + grp * len, P), c1 = unit_owner(U, s0 + (grp + 1) * len - 1, P);
                float M = kNoScore, S = 0.0f;
                for (int s = c0 + lane; s <= c1; s += 32) M = fmaxf(M, a.ml[(static_cast<size_t>(s) + bg) * N + n].x);
#pragma unroll
                for (int k = 16; k > 0; k >>= 1) M = fmaxf(M, __shfl_xor_sync(kFull, M, k));
                for (int s = c0 + lane; s <= c1; s += 32) {
                    const float2 v = a.ml[(static_cast<size_t>(s) + bg) * N + n];
                    S += v.y * hw_ex2(v.x - M);
                }
#pragma unroll
                for (int k = 16; k > 0; k >>= 1) S += __shfl_xor_sync(kFull, S, k);
                inv = S == 0.0f ? 0.0f : 1.0f / S;  // no token left: zeros
#pragma unroll 4
                for (int s = c0 + sub; s <= c1; s += share) {
                    const size_t at_row = (static_cast<size_t>(s) + bg) * N + n;
                    const float f = hw_ex2(a.ml[at_row].x - M);
                    const float2 *src = reinterpret_cast<const float2 *>(a.part + at_row * L);
#pragma unroll
                    for (int k = 0; k < kLatentMaxDim / 64; ++k)
                        if (64 * k < L) {
                            const float2 v = src[32 * k + lane];
                            o[2 * k] = fmaf(f, v.x, o[2 * k]);
                            o[2 * k + 1] = fmaf(f, v.y, o[2 * k + 1]);
                        }
                }
            }
#pragma unroll
            for (int k = 0; k < kLatentMaxDim / 64; ++k)
                if (64 * k < L) {
                    if (share == 1)
                        *reinterpret_cast<uint32_t *>(at + i * row_bytes + 128 * k + 4 * lane) =
                            pack_bf16(o[2 * k] * inv, o[2 * k + 1] * inv);
                    else
                        reinterpret_cast<float2 *>(sums + warp * L)[32 * k + lane] =
                            make_float2(o[2 * k] * inv, o[2 * k + 1] * inv);
                }
        }
        if (share > 1) {
            __syncthreads();
            for (int e = threadIdx.x; e < kWarps / share * (L / 2); e += blockDim.x) {
                const int which = e / (L / 2), l2 = e % (L / 2), i2 = rr + which;
                if (i2 < rows) {
                    float x = 0.0f, y = 0.0f;
                    for (int s = 0; s < share; ++s) {
                        const float2 v = reinterpret_cast<const float2 *>(sums + (which * share + s) * L)[l2];
                        x += v.x;
                        y += v.y;
                    }
                    *reinterpret_cast<uint32_t *>(at + i2 * row_bytes + 4 * l2) = pack_bf16(x, y);
                }
            }
            __syncthreads();
        }
        if (rr + kWarps / share >= rows) break;
    }
    __syncthreads();
    float acc[4] = {};
#pragma unroll
    for (int k = 0; k < kMaxK; ++k)
        if (32 * k < L) {
            uint4 lo = make_uint4(0, 0, 0, 0), hi = lo;
            if (g < rows) lo = *reinterpret_cast<const uint4 *>(at + g * row_bytes + 64 * k + 16 * c);
            if (g + 8 < rows) hi = *reinterpret_cast<const uint4 *>(at + (g + 8) * row_bytes + 64 * k + 16 * c);
            const uint32_t a0[4] = {lo.x, hi.x, lo.y, hi.y}, a1[4] = {lo.z, hi.z, lo.w, hi.w};
            mma16816(acc, a0, w[k].x, w[k].y);
            mma16816(acc, a1, w[k].z, w[k].w);
        }
    const int col = warp * 8 + 2 * c;
    if (g < rows)
        *reinterpret_cast<uint32_t *>(out + (static_cast<size_t>(r0 + g) * a.Hq + h) * kV + col) = pack_bf16(acc[0], acc[1]);
    if (g + 8 < rows)
        *reinterpret_cast<uint32_t *>(out + (static_cast<size_t>(r0 + g + 8) * a.Hq + h) * kV + col) =
            pack_bf16(acc[2], acc[3]);
}

// -------------------------------------------------------------------- host

bool decode_shape_ok(int B, int q_len, int Hq, int L, int nope, int v, int max_ctx) {
    return B >= 0 && q_len >= 1 && Hq >= 1 && static_cast<long>(q_len) * Hq <= 1024 && L >= 64 && L <= kLatentMaxDim &&
           L % 64 == 0 && latent_head_dim_ok(nope) && latent_head_dim_ok(v) && max_ctx >= 1 &&
           static_cast<long>(B) * q_len <= (1 << 20);
}

constexpr int kSmemLimit = 232448;

template <int N>
int launch_attention(const CUtensorMap &kv, const CUtensorMap &q, LatentAttnArgs a, int P, cudaStream_t stream) {
    // shared memory: q~, P, the rope slots, and latent pairs to the brim
    const int chunks = a.L / 64;
    a.ropes = N <= 32 ? 3 : 2;
    const int fixed = (chunks + 2) * N * 128 + a.ropes * kChunkBytes + static_cast<int>(sizeof(AttnShared));
    a.pairs = (kSmemLimit - fixed) / kPairBytes;
    if (a.pairs > kMaxPairs) a.pairs = kMaxPairs;
    const int smem = fixed + a.pairs * kPairBytes;
    // S^T of one tile is issued while the tile before still holds its pairs
    if (a.pairs < 2 * ((a.L + 127) / 128)) return TTS_ERR_UNSUPPORTED;
    if (!ensure_dynamic_smem(reinterpret_cast<const void *>(latent_attn_kernel<N>), smem)) return TTS_ERR_CUDA;
    return launch_kernel(latent_attn_kernel<N>, dim3(P), dim3(kAttnThreads), smem, {stream, true}, kv, q, a);
}

}  // namespace
}  // namespace tts

extern "C" size_t tts_latent_decode_attn_workspace_size(int32_t B, int32_t q_len, int32_t num_q_heads,
                                                        int32_t latent_dim, int32_t nope_dim, int32_t v_dim,
                                                        int32_t max_ctx_len) {
    if (!tts::decode_shape_ok(B, q_len, num_q_heads, latent_dim, nope_dim, v_dim, max_ctx_len)) return 0;
    return tts::latent_plan(B, q_len, num_q_heads, latent_dim, max_ctx_len).total();
}

extern "C" int tts_latent_decode_attn(const tts_latent_cache *cache, const int32_t *d_block_table,
                                      int32_t max_blocks_per_seq, const int32_t *d_ctx_lens, int32_t max_ctx_len,
                                      int32_t B, int32_t q_len, int32_t num_q_heads, int32_t nope_dim, int32_t v_dim,
                                      float scale, int32_t causal, const void *d_q_nope, const void *d_q_rope,
                                      const void *d_w_uk, const void *d_w_uv, void *d_out, void *d_ws, size_t ws_bytes,
                                      int32_t *d_err, void *stream) {
    using namespace tts;
    const int st = check_latent_cache(cache, d_block_table, max_blocks_per_seq);
    if (st != TTS_OK) return st;
    if (!d_ctx_lens || !d_q_nope || !d_q_rope || !d_w_uk || !d_w_uv || !d_out) return TTS_ERR_INVALID;
    if (B < 0 || q_len < 1 || num_q_heads < 1 || max_ctx_len < 1 || nope_dim < 1 || v_dim < 1) return TTS_ERR_INVALID;
    if (!(scale > 0.0f) || std::isinf(scale)) return TTS_ERR_INVALID;
    const int L = cache->latent_dim;
    if (!decode_shape_ok(B, q_len, num_q_heads, L, nope_dim, v_dim, max_ctx_len)) return TTS_ERR_UNSUPPORTED;
    if (!aligned16(d_q_nope) || !aligned16(d_q_rope) || !aligned16(d_w_uk) || !aligned16(d_w_uv) || !aligned16(d_out))
        return TTS_ERR_INVALID;
    if (B == 0) return TTS_OK;
    const LatentPlan pl = latent_plan(B, q_len, num_q_heads, L, max_ctx_len);
    if (!d_ws || !aligned16(d_ws) || ws_bytes < pl.total()) return TTS_ERR_WORKSPACE;

    using bf = const __nv_bfloat16 *;
    uint8_t *ws = static_cast<uint8_t *>(d_ws);
    __nv_bfloat16 *qt = reinterpret_cast<__nv_bfloat16 *>(ws);
    LatentAttnArgs a{};
    a.table = d_block_table;
    a.max_blocks = max_blocks_per_seq;
    a.num_blocks = cache->num_blocks;
    a.ctx_lens = d_ctx_lens;
    a.max_ctx = max_ctx_len;
    a.B = B;
    a.q_len = q_len;
    a.Hq = num_q_heads;
    a.L = L;
    a.G = pl.G;
    a.scale_log2 = scale * kLog2e;
    a.causal = causal != 0;
    a.part = reinterpret_cast<float *>(ws + pl.qt_bytes);
    a.ml = reinterpret_cast<float2 *>(ws + pl.qt_bytes + pl.part_bytes);
    a.starts = reinterpret_cast<long long *>(ws + pl.qt_bytes + pl.part_bytes + pl.ml_bytes);
    a.err = d_err;
    const int R = B * q_len, W = L + kLatentRope;
    CUtensorMap map_kv, map_q;
    if (!make_tma_2d_bf16(&map_kv, cache->pool, static_cast<uint64_t>(cache->num_blocks) * TTS_BLOCK_TOKENS, W,
                          TTS_BLOCK_TOKENS, 64) ||
        !make_tma_2d_bf16(&map_q, qt, static_cast<uint64_t>(R) * num_q_heads, W, pl.N, 64))
        return TTS_ERR_CUDA;

    const cudaStream_t cs = static_cast<cudaStream_t>(stream);
    const dim3 agrid(L / 64, num_q_heads, (R + 16 * kAbsorbChunks - 1) / (16 * kAbsorbChunks));
    int rc = launch_kernel(nope_dim == 128 ? latent_absorb_kernel<2> : latent_absorb_kernel<1>, agrid, dim3(128), 0,
                           {cs, thread_pdl()}, static_cast<bf>(d_q_nope), static_cast<bf>(d_q_rope),
                           static_cast<bf>(d_w_uk), qt, R, num_q_heads, L);
    if (rc != TTS_OK) return rc;
    switch (pl.N) {
        case 16: rc = launch_attention<16>(map_kv, map_q, a, pl.P, cs); break;
        case 32: rc = launch_attention<32>(map_kv, map_q, a, pl.P, cs); break;
        case 48: rc = launch_attention<48>(map_kv, map_q, a, pl.P, cs); break;
        default: rc = launch_attention<64>(map_kv, map_q, a, pl.P, cs); break;
    }
    if (rc != TTS_OK) return rc;
    const int smem = (v_dim / 8) * L * 4 + 16 * (2 * L + 64);
    auto out_kernel = v_dim == 128 ? latent_out_kernel<128> : latent_out_kernel<64>;
    if (!ensure_dynamic_smem(reinterpret_cast<const void *>(out_kernel), smem)) return TTS_ERR_CUDA;
    return launch_kernel(out_kernel, dim3((R + 15) / 16, num_q_heads), dim3(v_dim * 4), smem, {cs, true}, a, pl.N, pl.P,
                         static_cast<bf>(d_w_uv), static_cast<__nv_bfloat16 *>(d_out));
}
