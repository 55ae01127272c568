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
// Bound: HBM at one query row a stream (16 heads: 30 flop a byte).  HBM
// delivers a 64-token tile's 73.7 KB to an SM in 1.65 us; its 36 + 16 MMAs take
// 1.1 us at N <= 32 (an M = 64 MMA of 16 to 64 columns 38 to 42 cycles, an M =
// 128 one 48 to 52), and the ring holds 2.75 tiles, so that a tile takes
// 2.0 us.  With 48 rows (a verify step's 80 in two groups) the second
// group's reads come from L2, and the two tiles that fit beside the queries
// turn loads and MMAs into a chain of 1.6 us a tile; ending a segment costs
// another 2 to 3 us (98 KB of partial sums).  Measured, 16 heads, latent 512:
// 256 streams of 32 to 4096 tokens 52 us (4.8 TB/s), 64 streams of 50 to 1500
// 15 us, 64 x 5 causal rows over 256 to 2048 tokens 41 us, one stream of 65533
// tokens 16 us, one of 17 tokens 6.7 us.
#include <cuda_bf16.h>

#include <algorithm>
#include <cfloat>
#include <climits>
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
// Running maximum before any token (log2 units): no finite score is below it, so
// that a row whose scores are all far below zero still has weights.
constexpr float kNoScore = -FLT_MAX;
// The running maximum is moved only when a score passes it by this much (log2
// units): weights then reach 2^8, which fp32 sums and bf16 weights hold as
// well as 1, and O in tensor memory is rarely rescaled.
constexpr float kSlack = 8.0f;

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    const __nv_bfloat162 p = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&p);
}

// ------------------------------------------------------------------ absorb

// q~[r][h][l] = sum_d q_nope[r][h][d] w_uk[h][d][l], rounded to bf16 (the MMA
// that follows takes bf16).  A CTA takes one head, 128 of l and 128 query rows:
// one tcgen05 product of nope / 16 steps (q K-major, the weights MN-major as
// they lie), its result staged in shared memory and stored by TMA, which clips
// the rows past R.  Latency-bound (2 MB of weights at 16 heads): the weights
// are in flight before the wait for the previous kernel.  4.2 us at one row,
// 5.8 us at 320.
constexpr int kRowTile = 128;

__global__ void __launch_bounds__(128)
latent_absorb_kernel(const __grid_constant__ CUtensorMap map_qn, const __grid_constant__ CUtensorMap map_uk,
                     const __grid_constant__ CUtensorMap map_qt, int nope, int L, int R, int32_t *err) {
    extern __shared__ __align__(1024) uint8_t raw[];
    __shared__ uint64_t full, acc;
    __shared__ uint32_t tslot;
    const int warp = uniform(threadIdx.x / 32), lane = threadIdx.x % 32;
    const int l0 = blockIdx.x * 128, h = blockIdx.y, r0 = blockIdx.z * kRowTile;
    const int halves = l0 + 64 < L ? 2 : 1;
    const uint32_t wb = smem_addr(raw), w_chunk = nope * 128;   // [2][nope][64 l]
    const uint32_t qb = wb + 2 * w_chunk, q_chunk = kRowTile * 128;  // [nope / 64][128 rows][64 d]
    bool ok = true;
    if (warp == 0) {
        const uint32_t leader = elect_leader();
        if (leader) {
            mbar_init(smem_addr(&full), 1);
            mbar_init(smem_addr(&acc), 1);
            fence_mbar_init();
        }
        __syncwarp();
        mbar_expect_tx_by(leader, smem_addr(&full), halves * w_chunk + nope / 64 * q_chunk);
        for (int i = 0; i < halves; ++i)
            tma_load_2d_by(leader, wb + i * w_chunk, &map_uk, l0 + 64 * i, h * nope, smem_addr(&full));
        pdl_wait_prerequisites();
        for (int i = 0; i < nope / 64; ++i)
            tma_load_2d_by(leader, qb + i * q_chunk, &map_qn, h * nope + 64 * i, r0, smem_addr(&full));
        // (tensor memory only after the wait: the kernel before may be one that
        // still has to allocate its own)
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 128;" ::"r"(smem_addr(&tslot))
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    pdl_allow_dependents();  // only now: the attention allocates tensor memory and reads the pool as soon as it starts
    const uint32_t tmem = uniform(tslot);
    if (warp == 0) {
        const uint32_t leader = elect_leader();
        ok = warp_wait(&full, 0);
        tc_fence_after();
        const uint32_t idesc = (halves == 2 ? mma_idesc(kRowTile, 128) : mma_idesc(kRowTile, 64)) | kTransposeB;
        for (int k = 0; k < nope / 16; ++k)
            mma_bf16_by(leader, tmem, sw128_desc(qb + k / 4 * q_chunk + k % 4 * 32), sw128_mn_desc(wb + k * 2048, w_chunk),
                        idesc, k != 0);
        mma_commit_by(leader, smem_addr(&acc));
    }
    if (!warp_wait(&acc, 0)) ok = false;
    tc_fence_after();
    // the products have read the shared memory: stage the rows there, 64
    // values of a row 128-byte swizzled
    const int row = warp * 32 + lane;
    if (ok && r0 + warp * 32 < R)
        for (int c = 0; c < 2 * halves; ++c) {
            uint32_t x[32];
            tmem_ld32_nowait(tmem + (static_cast<uint32_t>(warp * 32) << 16) + c * 32, x);
            tmem_wait_ld();
            const float *f = reinterpret_cast<const float *>(x);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const uint32_t at = wb + c / 2 * q_chunk + row * 128 + (((c % 2 * 4 + j) ^ (row & 7)) << 4);
                asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(pack_bf16(f[8 * j], f[8 * j + 1])),
                             "r"(pack_bf16(f[8 * j + 2], f[8 * j + 3])), "r"(pack_bf16(f[8 * j + 4], f[8 * j + 5])),
                             "r"(pack_bf16(f[8 * j + 6], f[8 * j + 7])));
            }
        }
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    if (!ok) flag_error(err, TTS_ERRBIT_TIMEOUT);
    tc_fence_before();
    ok = !__syncthreads_or(!ok);
    if (warp == 0) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 128;" ::"r"(tmem) : "memory");
        if (ok && lane == 0) {
            for (int i = 0; i < halves; ++i) tma_store_2d(&map_qt, h * L + l0 + 64 * i, r0, wb + i * q_chunk);
            asm volatile("cp.async.bulk.commit_group;\n\tcp.async.bulk.wait_group 0;" ::: "memory");
        }
    }
}

// -------------------------------------------------------------- work split

// The work units are the 64-token tiles of every (stream, row group), group
// bg = b * G + g, in order, cut evenly over the CTAs; each group has one unit
// before its tiles (two with 48 rows or more), which stands for what starting
// and ending a group costs, a tile's time or two (16 rows, 64 streams: 23.8 us
// the call with one, 24.3 with two; 48 rows 32.6 and 31.8, at latent 256 23.5 and
// 22.4; 64 rows 36.3 and 35.9).  The part of a group that a CTA takes is
// a segment; its partial result goes to slot c + bg (unique: going on to the
// next segment raises one of the two).
__host__ __device__ constexpr int start_units(int N) { return N >= 48 ? 2 : 1; }

struct LatentPlan {
    int G, N;       // row groups a stream, rows per group (a multiple of 16)
    int P;          // CTAs
    long units;     // at most
    size_t slots;   // P + B * G
    size_t qt_bytes, part_bytes, ml_bytes, owner_bytes;
    size_t total() const { return qt_bytes + part_bytes + ml_bytes + owner_bytes; }
};

LatentPlan latent_plan(int B, int q_len, int Hq, int L, int max_ctx) {
    LatentPlan p;
    const int rows = q_len * Hq;
    p.G = (rows + kMaxGroup - 1) / kMaxGroup;
    p.N = ((rows + p.G - 1) / p.G + 15) / 16 * 16;
    p.units = static_cast<long>(B) * p.G * ((static_cast<long>(max_ctx) + kTile - 1) / kTile + start_units(p.N));
    p.P = p.units < kCtas ? static_cast<int>(p.units < 1 ? 1 : p.units) : kCtas;
    p.slots = static_cast<size_t>(p.P) + static_cast<size_t>(B) * p.G;
    p.qt_bytes = align_up(static_cast<size_t>(B) * rows * L * 2, 256);
    p.part_bytes = align_up(p.slots * p.N * L * 4, 256);
    p.ml_bytes = align_up(p.slots * p.N * 8, 256);
    p.owner_bytes = align_up(static_cast<size_t>(B) * p.G * 8, 256);
    return p;
}

// U units over the launched CTAs: the first U % P get one more than the rest.
// With fewer units than CTAs only the first U take part, so that a group's
// CTAs are consecutive and every one of them has a unit.
struct UnitCut {
    int each, rem, wide;  // units per CTA, CTAs with one more, units in those
    __device__ __forceinline__ UnitCut(int U, int launched) {
        const int P = max(1, min(U, launched));
        each = U / P;
        rem = U - each * P;
        wide = rem * (each + 1);
    }
    __device__ __forceinline__ int begin(int c) const { return c * each + min(c, rem); }
    __device__ __forceinline__ int owner(int u) const { return u < wide ? u / (each + 1) : rem + (u - wide) / each; }
};

struct LatentAttnArgs {
    const int32_t *table;
    int max_blocks, num_blocks;
    const int32_t *ctx_lens;
    int max_ctx, B, q_len, Hq, L;
    int G, start;      // row groups a stream, units before a group's tiles
    float scale_log2;  // scale * log2(e)
    int causal;
    float *part;       // [slots][N][L] unnormalised o~
    float2 *ml;        // [slots][N] running maximum (log2 units), sum
    int2 *owner;       // [B * G] first CTA and number of splits of each group
    int32_t *err;
    int pairs, ropes;  // ring slots
    long long wait_limit;  // SM clock cycles per bounded wait
    int stall;         // test support: a CTA's first tile expects 16 bytes that never come
};

// Tiles of a stream of `ctx` tokens (0: out of range).
__device__ __forceinline__ int stream_tiles(const LatentAttnArgs &a, int ctx) {
    if (ctx < a.q_len || ctx > a.max_ctx || ctx > a.max_blocks * TTS_BLOCK_TOKENS) return 0;
    return (ctx + kTile - 1) / kTile;
}

// Units of one of stream b's groups (0: its length is out of range).  The
// lengths may be read through the read-only path: this kernel starts when every
// CTA of the absorb kernel is past its wait, so nothing writes them any more.
// (Plain loads: 64 streams 26.7 -> 27.1 us the call, verify 56.6 -> 57.1.)
__device__ __forceinline__ int group_units(const LatentAttnArgs &a, int b) {
    const int n = stream_tiles(a, __ldg(a.ctx_lens + b));
    return n ? n + a.start : 0;
}

// A block's scan of the streams: thread t has the streams b0..b1 - 1, the first
// of which starts at unit `at`; U units in all.  `sums` holds an entry per warp.
struct StreamScan {
    int b0, b1, at, U;
};
template <int kThreads>
__device__ __forceinline__ StreamScan scan_streams(const LatentAttnArgs &a, int *sums) {
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int per = (a.B + kThreads - 1) / kThreads;
    StreamScan s;
    s.b0 = min(a.B, static_cast<int>(threadIdx.x) * per);
    s.b1 = min(a.B, s.b0 + per);
    int mine = 0;
    for (int b = s.b0; b < s.b1; ++b) mine += group_units(a, b);
    int incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
        const int x = __shfl_up_sync(kFull, incl, o);
        if (lane >= o) incl += x;
    }
    if (lane == 31) sums[warp] = incl;
    __syncthreads();
    s.at = incl - mine;
    s.U = 0;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) {
        if (w < warp) s.at += sums[w];
        s.U += sums[w];
    }
    s.at *= a.G;
    s.U *= a.G;
    return s;
}

// Walks a CTA's segments; every warp keeps its own copy.  The length of the
// next stream is read a segment ahead (a read takes as long as half a tile).
struct Segments {
    int b, g, unit;        // next unit (0: the group's first, then its tiles)
    int left;              // units left
    int ahead;             // ctx_lens[b]
    // current segment
    int cur_b, cur_g, bg;
    int ctx, first, count; // first tile, tiles
    __device__ __forceinline__ void look(const LatentAttnArgs &a) { ahead = b < a.B ? __ldg(a.ctx_lens + b) : 0; }
    __device__ __forceinline__ bool next(const LatentAttnArgs &a) {
        while (left > 0) {
            ctx = uniform(ahead);
            const int n = stream_tiles(a, ctx);
            if (n == 0) {  // (never the CTA's first stream)
                ++b;
                look(a);
                continue;
            }
            const int units = min(n + a.start - unit, left);
            first = max(unit - a.start, 0);
            count = unit + units - a.start - first;
            cur_b = b;
            cur_g = g;
            bg = b * a.G + g;
            left -= units;
            unit = 0;
            if (++g == a.G) {
                g = 0;
                ++b;
                look(a);
            }
            if (count > 0) return true;
        }
        return false;
    }
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

// Sets the bf16 values in 16 bytes of shared memory that are not finite to zero;
// whether there were any.
__device__ __forceinline__ bool keep_finite(uint32_t at) {
    uint32_t x[4];
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3]) : "r"(at) : "memory");
    bool found = false;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const bool low = (x[i] & 0x7F80u) == 0x7F80u, high = (x[i] & 0x7F800000u) == 0x7F800000u;
        if (low) x[i] &= 0xFFFF0000u;
        if (high) x[i] &= 0xFFFFu;
        found = found || low || high;
    }
    if (found)
        asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(x[0]), "r"(x[1]), "r"(x[2]), "r"(x[3]) : "memory");
    return found;
}

// Position in a ring of shared-memory slots; phase is the parity of the
// slot's current filling.
struct Ring {
    uint32_t n, slot = 0, phase = 0;
    __device__ __forceinline__ explicit Ring(uint32_t slots) : n(slots) {}
    __device__ __forceinline__ void next() {
        if (++slot == n) {
            slot = 0;
            phase ^= 1;
        }
    }
    __device__ __forceinline__ void back() {
        if (slot == 0) {
            slot = n;
            phase ^= 1;
        }
        --slot;
    }
};

constexpr int kMaxPairs = 16, kMaxRopes = 8;

struct AttnShared {
    uint64_t full[kMaxRopes], empty_l[kMaxPairs], empty_r[kMaxRopes];
    uint64_t s_full[2], p_full[2], p_empty[2], o_empty, q_full, q_empty, done;
    int start_b, start_g, start_unit;
    uint32_t tmem;
    int sums[8];
    int failed;
    int spoilt;       // of the tokens that not every row sees, the first whose latent is not finite
    alignas(16) float mref[kMaxGroup];
    float fac[kMaxGroup];
    int limit[kMaxGroup];
    union {
        float wmax[4][kMaxGroup];  // within a tile
        float lsum[4][kMaxGroup];     // at a segment's end
    };
};

// Buffers for the weights P: with one, the softmax waits for the O^T of the
// tile before.  A second one pays at 48 rows (64 streams x 5 causal rows of 16
// heads 54.0 us the call against 54.5); with 16 it makes no difference (64 streams
// 23.8), with 32 its space is worth more to the ring (28.1 against 28.4), with 64
// it does not fit.
__host__ __device__ constexpr int p_buffers(int N) { return N == 48 ? 2 : 1; }

// P enters the product as two bf16 numbers, its rounding and the remainder:
// the weights are then held to 2^-17.  Up to 48 rows the remainders are N more
// columns of the same MMAs, which is nearly free (a 128-row MMA of 16 to 64
// columns takes 48 to 52 cycles, most of them reading A).  64 rows would need
// more than tensor memory's 512 columns: the remainders are then a second
// operand for the same accumulator, kept in the tile's rope slot, whose keys
// S^T is done with.
__host__ __device__ constexpr bool p_beside(int N) { return N <= 48; }
__host__ __device__ constexpr int p_rows(int N) { return p_beside(N) ? 2 * N : N; }

template <int N>
__global__ void __launch_bounds__(kAttnThreads, 1)
latent_attn_kernel(const __grid_constant__ CUtensorMap map_kv, const __grid_constant__ CUtensorMap map_q,
                   const __grid_constant__ CUtensorMap map_qr, const LatentAttnArgs a) {
    extern __shared__ __align__(1024) uint8_t raw[];
    const uint32_t base = smem_addr(raw);
    constexpr int kPBufs = p_buffers(N);
    constexpr int kO = p_rows(N), kPBytes = kO * 128;  // columns of O^T (rows of P), bytes of a P buffer
    const int chunks = a.L / 64, nb = (a.L + 127) / 128;
    const uint32_t q_base = base, q_bytes = (chunks + 1) * N * 128;     // [chunks + 1][N][128 B]
    const uint32_t p_base = q_base + q_bytes;                           // [kPBufs][kO][128 B]
    const uint32_t r_base = p_base + kPBufs * kPBytes;                         // rope ring
    const uint32_t l_base = r_base + a.ropes * kChunkBytes;             // latent ring
    AttnShared &sh = *reinterpret_cast<AttnShared *>(raw + (l_base - base) + a.pairs * kPairBytes);
    const int warp = uniform(threadIdx.x / 32), lane = threadIdx.x % 32;

    if (warp == 5 && lane == 0) {
        for (int i = 0; i < a.pairs; ++i) mbar_init(smem_addr(&sh.empty_l[i]), 1);
        for (int i = 0; i < a.ropes; ++i) {
            mbar_init(smem_addr(&sh.full[i]), 1);
            mbar_init(smem_addr(&sh.empty_r[i]), 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_addr(&sh.s_full[i]), 1);
            mbar_init(smem_addr(&sh.p_full[i]), 4);
            mbar_init(smem_addr(&sh.p_empty[i]), 1);
        }
        mbar_init(smem_addr(&sh.q_full), 1);
        mbar_init(smem_addr(&sh.q_empty), 1);
        mbar_init(smem_addr(&sh.o_empty), 4);
        mbar_init(smem_addr(&sh.done), 1);
        sh.failed = 0;
        fence_mbar_init();
        prefetch_tensormap(&map_kv);
        prefetch_tensormap(&map_q);
        prefetch_tensormap(&map_qr);
    }
    uint32_t cols = 32;
    while (cols < static_cast<uint32_t>(2 * N + nb * kO)) cols *= 2;
    if (warp == 6) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(&sh.tmem)),
                     "r"(cols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    // ---- this CTA's units
    tc_fence_before();
    const StreamScan scan = scan_streams<kAttnThreads>(a, sh.sums);
    tc_fence_after();
    const UnitCut cut(scan.U, gridDim.x);
    const int u0 = min(scan.U, cut.begin(blockIdx.x)), u1 = min(scan.U, cut.begin(blockIdx.x + 1));
    if (u0 < u1 || blockIdx.x == 0) {
        int at = scan.at;
        for (int b = scan.b0; b < scan.b1; ++b) {
            const int w = group_units(a, b);
            if (u0 < u1 && u0 >= at && u0 < at + w * a.G) {
                sh.start_b = b;
                sh.start_g = (u0 - at) / w;
                sh.start_unit = (u0 - at) % w;
            }
            if (blockIdx.x == 0) {
                if (w == 0) flag_error(a.err, TTS_ERRBIT_CTX_LEN);
                for (int g = 0; g < a.G; ++g) {
                    const int first = w ? cut.owner(at + g * w + a.start) : 0;
                    a.owner[b * a.G + g] = make_int2(first, w ? cut.owner(at + (g + 1) * w - 1) - first + 1 : 0);
                }
            }
            at += w * a.G;
        }
    }
    __syncthreads();
    const uint32_t tmem = uniform(sh.tmem);
    Segments seg;
    seg.left = uniform(u1 - u0);
    seg.b = uniform(sh.start_b);
    seg.g = uniform(sh.start_g);
    seg.unit = uniform(sh.start_unit);
    if (seg.left > 0) seg.look(a);
    pdl_allow_dependents();
    bool ok = true;

    if (warp == 4) {
        // ---- KV producer: per tile the rope chunk, then the latent pairs,
        // one copy per block of 16 rows and 64 values.  A block outside the
        // pool (or past the context) is read out of range, which fills zeros.
        const uint32_t leader = elect_leader();
        const int oob = a.num_blocks * TTS_BLOCK_TOKENS;
        Ring rope(a.ropes), lat(a.pairs);
        uint32_t it = 0, lpos = 0;
        auto fetch = [&](const Segments &s, int tile) {  // lanes 0-3 (and so on): the tile's block ids
            const int i = tile * 4 + (lane & 3);
            return i * TTS_BLOCK_TOKENS < s.ctx ? a.table[static_cast<size_t>(s.cur_b) * a.max_blocks + i] : -1;
        };
        bool more = seg.next(a);
        int id = more ? fetch(seg, seg.first) : 0;
        while (ok && more) {
            const Segments cur = seg;
            for (int k = 0; ok && k < cur.count; ++k) {
                const int tile = cur.first + k;
                int y = oob;
                if ((tile * 4 + (lane & 3)) * TTS_BLOCK_TOKENS < cur.ctx) {
                    if (id >= 0 && id < a.num_blocks) y = id * TTS_BLOCK_TOKENS;
                    else flag_error(a.err, TTS_ERRBIT_BLOCK_ID);
                }
                if (k + 1 < cur.count) {
                    id = fetch(cur, tile + 1);
                } else {
                    more = seg.next(a);
                    if (more) id = fetch(seg, seg.first);
                }
                int ys[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) ys[i] = __shfl_sync(kFull, y, i);
                if (it >= rope.n && !warp_wait(&sh.empty_r[rope.slot], rope.phase ^ 1, a.wait_limit)) {
                    ok = false;
                    break;
                }
                // (the tile's one barrier: the MMAs of S^T take the whole tile)
                const uint32_t bar = smem_addr(&sh.full[rope.slot]), at = r_base + rope.slot * kChunkBytes;
                mbar_expect_tx_by(leader, bar, (chunks + 1) * kChunkBytes + (a.stall && it == 0 ? 16 : 0));
#pragma unroll
                for (int i = 0; i < 4; ++i) tma_load_2d_by(leader, at + i * 2048, &map_kv, a.L, ys[i], bar);
                rope.next();
                ++it;
                for (int p = 0; p < nb; ++p) {
                    if (lpos >= lat.n && !warp_wait(&sh.empty_l[lat.slot], lat.phase ^ 1, a.wait_limit)) {
                        ok = false;
                        break;
                    }
                    const uint32_t to = l_base + lat.slot * kPairBytes;
#pragma unroll
                    for (int i = 0; i < 4; ++i) tma_load_2d_by(leader, to + i * 2048, &map_kv, p * 128, ys[i], bar);
                    if (2 * p + 1 < chunks)
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            tma_load_2d_by(leader, to + kChunkBytes + i * 2048, &map_kv, p * 128 + 64, ys[i], bar);
                    lat.next();
                    ++lpos;
                }
            }
        }
        // every copy lands before the CTA ends
        for (uint32_t i = min(it, rope.n); i > 0; --i) {
            rope.back();
            warp_wait(&sh.full[rope.slot], rope.phase);
        }
    } else if (warp == 6) {
        // ---- Q loader: a segment's q~ rows, once the S MMAs of the one before are done
        pdl_wait_prerequisites();
        const uint32_t leader = elect_leader();
        uint32_t s = 0;
        for (; seg.next(a); ++s) {
            if (s > 0 && !warp_wait(&sh.q_empty, (s - 1) & 1, a.wait_limit)) {
                ok = false;
                break;
            }
            const uint32_t bar = smem_addr(&sh.q_full);
            mbar_expect_tx_by(leader, bar, q_bytes);
            const int y = seg.cur_b * a.q_len * a.Hq + seg.cur_g * N;
            for (int c = 0; c < chunks; ++c) tma_load_2d_by(leader, q_base + c * N * 128, &map_q, c * 64, y, bar);
            tma_load_2d_by(leader, q_base + chunks * N * 128, &map_qr, 0, y, bar);
        }
        if (s > 0) warp_wait(&sh.q_full, (s - 1) & 1);
    } else if (warp == 5) {
        // ---- MMA issuer (the warp runs converged; it also clears stale rows).
        // S^T of tile i + 1 goes before O^T of tile i, so the tensor core works
        // on it while the softmax warps turn S^T of tile i into weights (the
        // ring holds both tiles' pairs).
        const uint32_t leader = elect_leader();
        constexpr uint32_t idesc_s = mma_idesc(64, N);
        constexpr uint32_t idesc_o = mma_idesc(128, kO) | kTransposeA;
        Ring rope(a.ropes), lat(a.pairs);
        uint32_t it = 0, segs = 0;
        // the tile whose O^T is outstanding: the one before `it`
        bool pending = false, pend_first = false;
        Ring pend(a.pairs);
        uint32_t pend_seg = 0, pend_rope = 0;
        auto weights = [&](uint32_t tile) {  // what O^T of `tile` waits for
            WarpWaits<2> w;
            w.set(0, &sh.p_full[tile % kPBufs], (tile / kPBufs) & 1);
            w.none(1);
            if (pend_first && pend_seg > 0) w.set(1, &sh.o_empty, (pend_seg - 1) & 1);
            return w;
        };
        auto issue_o = [&](uint32_t tile) {
            const uint32_t pb = tile % kPBufs;
            tc_fence_after();
            const uint32_t sb = p_base + pb * kPBytes;
            for (int p = 0; p < nb; ++p) {
                const uint32_t sa = l_base + pend.slot * kPairBytes;
#pragma unroll
                for (int k = 0; k < kTile / 16; ++k)
                    mma_bf16_by(leader, tmem + 2 * N + p * kO, sw128_mn_desc(sa + k * 2048, kChunkBytes),
                                sw128_desc(sb + k * 32), idesc_o, !(pend_first && k == 0));
                if constexpr (!p_beside(N))
#pragma unroll
                    for (int k = 0; k < kTile / 16; ++k)
                        mma_bf16_by(leader, tmem + 2 * N + p * kO, sw128_mn_desc(sa + k * 2048, kChunkBytes),
                                    sw128_desc(r_base + pend_rope * kChunkBytes + k * 32), idesc_o, 1);
                mma_commit_by(leader, smem_addr(&sh.empty_l[pend.slot]));
                pend.next();
            }
            mma_commit_by(leader, smem_addr(&sh.p_empty[pb]));
            if constexpr (!p_beside(N)) mma_commit_by(leader, smem_addr(&sh.empty_r[pend_rope]));
            pending = false;
        };
        while (ok && seg.next(a)) {
            const int count = seg.count, left = seg.ctx - seg.first * kTile;  // tokens from the first tile on
            for (int k = 0; k < count; ++k) {
                const uint32_t buf = it & 1;
                // the tile and the queries (S's buffer is free: the weights
                // of the tile before the last, which came from it, are in)
                WarpWaits<2> w;
                w.set(0, &sh.full[rope.slot], rope.phase);
                w.none(1);
                if (k == 0) w.set(1, &sh.q_full, segs & 1);
                const Ring first = lat;
                // a tile that is still landing lets O^T of the one before go
                // first, if its weights are there: that frees ring slots
                bool ready = w.poll();
                if (!ready && pending) {
                    const WarpWaits<2> wo = weights(it - 1);
                    const long long t0 = clock64();
                    while (!ready && pending && ok) {
                        if (wo.poll()) issue_o(it - 1);
                        ready = w.poll();
                        ok = uniform(clock64() - t0 < a.wait_limit);
                    }
                }
                if (!ok || (!ready && !w.wait(a.wait_limit))) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t sr = r_base + rope.slot * kChunkBytes;
#pragma unroll
                for (int kk = 0; kk < 4; ++kk)
                    mma_bf16_by(leader, tmem + buf * N, sw128_desc(sr + kk * 32),
                                sw128_desc(q_base + chunks * N * 128 + kk * 32), idesc_s, kk != 0);
                const uint32_t rope_slot = rope.slot;
                if constexpr (p_beside(N)) mma_commit_by(leader, smem_addr(&sh.empty_r[rope_slot]));
                rope.next();
                for (int p = 0; p < nb; ++p) {
                    const uint32_t sa = l_base + lat.slot * kPairBytes, sb = q_base + 2 * p * N * 128;
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)
                        mma_bf16_by(leader, tmem + buf * N, sw128_desc(sa + kk * 32), sw128_desc(sb + kk * 32), idesc_s, 1);
                    if (2 * p + 1 < chunks)
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk)
                            mma_bf16_by(leader, tmem + buf * N, sw128_desc(sa + kChunkBytes + kk * 32),
                                        sw128_desc(sb + N * 128 + kk * 32), idesc_s, 1);
                    lat.next();
                }
                mma_commit_by(leader, smem_addr(&sh.s_full[buf]));
                if (k + 1 == count) mma_commit_by(leader, smem_addr(&sh.q_empty));
                if (pending) {
                    if (!weights(it - 1).wait(a.wait_limit)) {
                        ok = false;
                        break;
                    }
                    issue_o(it - 1);
                }
                // rows behind the context in its last block hold anything (in
                // O^T, NaN times a zero weight would spread): clear them.  S^T
                // may read them before or after; its rows there are masked.
                const int end = left - k * kTile;  // tokens of the context in this tile
                const int stop = (end + TTS_BLOCK_TOKENS - 1) / TTS_BLOCK_TOKENS * TTS_BLOCK_TOKENS;
                if (end < kTile && end < stop) {
                    Ring r = first;
                    for (int p = 0; p < nb; ++p, r.next())
                        for (int t = end + lane / 8; t < stop; t += 4) {
                            const uint32_t at = l_base + r.slot * kPairBytes + t * 128 + lane % 8 * 16;
                            asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(at), "r"(0) : "memory");
                            asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(at + kChunkBytes), "r"(0)
                                         : "memory");
                        }
                    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                    __syncwarp();
                }
                pending = true;
                pend_first = k == 0;
                pend = first;
                pend_seg = segs;
                pend_rope = rope_slot;
                ++it;
            }
            ++segs;
        }
        if (ok && pending) {
            ok = weights(it - 1).wait(a.wait_limit);
            if (ok) issue_o(it - 1);
        }
        mma_commit_by(leader, smem_addr(&sh.done));
        if (!warp_wait(&sh.done, 0)) ok = false;
    } else {
        // ---- softmax warps: warp w has the tokens 16 w.. of the tile, one
        // block (a 64-row accumulator's rows 16 w.. sit in lanes 32 w..); lane
        // (g, c) has tokens g and g + 8 and of every 8 columns 2 c and 2 c + 1.
        // Value i of a lane: token g + 8 (i / 2 % 2), column col(i).
        uint32_t it = 0;
        const uint32_t tl = tmem + (static_cast<uint32_t>(warp * 32) << 16);
        constexpr int kVals = N / 2;
        const int g = lane / 4, c2 = lane % 4 * 2;
        auto col = [&](int i) { return i / 4 * 8 + c2 + i % 2; };
        // Eight tokens of a row n of P are the 16-byte chunk (t / 8) ^ (n % 8),
        // a row of a transposed 8 x 8 matrix: the lane's of a store of four,
        // rows 0-7 at tokens 0-7 and 8-15, then rows 8-15
        const uint32_t pat = p_base + (lane / 16 * 8 + lane % 8) * 128 + (((2 * warp + lane / 8 % 2) ^ (lane % 8)) << 4);
        auto o_added = [&](uint32_t tile) { return warp_wait(&sh.p_empty[tile % kPBufs], (tile / kPBufs) & 1, a.wait_limit); };
        const int tid = threadIdx.x;
        int lslot = 0, rslot = 0;  // the tile's ring slots: its first latent pair, its rope chunk
        auto block_ok = [&](const Segments &s, int tile) {
            const int i = tile * 4 + warp;
            if (i * TTS_BLOCK_TOKENS >= s.ctx) return false;
            const int id = a.table[static_cast<size_t>(s.cur_b) * a.max_blocks + i];
            return id >= 0 && id < a.num_blocks;
        };
        bool more = seg.next(a), valid = more && block_ok(seg, seg.first);
        while (ok && more) {
            const int low = a.causal ? seg.ctx - a.q_len + 1 : seg.ctx;  // tokens every row sees
            softmax_sync();  // the last segment's reads of these are over
            if (tid == 0) sh.spoilt = INT_MAX;
            if (tid < N) {
                sh.mref[tid] = kNoScore;
                const int j = (seg.cur_g * N + tid) / a.Hq;
                sh.limit[tid] = j >= a.q_len ? 0 : a.causal ? seg.ctx - a.q_len + j + 1 : seg.ctx;
            }
            softmax_sync();
            float l[N / 4];  // of columns col(4 j) and col(4 j + 1)
#pragma unroll
            for (int n = 0; n < N / 4; ++n) l[n] = 0.0f;
            for (int k = 0; k < seg.count; ++k, ++it) {
                const int tile = seg.first + k;
                const uint32_t buf = it & 1;
                const bool next_valid = k + 1 < seg.count && block_ok(seg, tile + 1);
                // (the tile that last used this P buffer has had its O^T added)
                if (it >= kPBufs && kPBufs > 1 && !o_added(it - kPBufs)) ok = false;
                float mr[N / 4];
#pragma unroll
                for (int j = 0; j < N / 8; ++j) {
                    const float2 m2 = *reinterpret_cast<const float2 *>(sh.mref + 8 * j + c2);
                    mr[2 * j] = m2.x;
                    mr[2 * j + 1] = m2.y;
                }
                if (!warp_wait(&sh.s_full[buf], (it / 2) & 1, a.wait_limit)) ok = false;
                tc_fence_after();
                uint32_t sr[kVals];
#pragma unroll
                for (int c = 0; c < N; c += 16) tmem_ld_half16_nowait(tl + buf * N + c, sr + c / 2);
                tmem_wait_ld();
                const int t = tile * kTile + warp * 16 + g;
                if (!valid) {
#pragma unroll
                    for (int i = 0; i < kVals; ++i) sr[i] = 0xFF800000u;  // -inf
                } else if ((tile + 1) * kTile > low) {
#pragma unroll
                    for (int i = 0; i < kVals; ++i)
                        if (t + (i & 2) * 4 >= sh.limit[col(i)]) sr[i] = 0xFF800000u;
                }
                auto score = [&](int i) {  // log2 units, over the running maximum
                    return fmaf(__uint_as_float(sr[i]), a.scale_log2, -mr[i / 4 * 2 + i % 2]);
                };
                float tops[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                for (int i = 0; i < kVals; ++i) tops[i % 4] = fmaxf(tops[i % 4], score(i));
                const float top = fmaxf(fmaxf(tops[0], tops[1]), fmaxf(tops[2], tops[3]));
                if (!ok) sh.failed = 1;
                if (softmax_any(top > kSlack || !ok)) {
                    // rare: raise the running maxima to this tile's, rescale sums and O
                    if (*static_cast<volatile int *>(&sh.failed)) {  // (all four warps leave together)
                        ok = false;
                        break;
                    }
#pragma unroll
                    for (int j = 0; j < N / 4; ++j) {
                        const int i = j / 2 * 4 + j % 2;
                        float m = fmaxf(__uint_as_float(sr[i]), __uint_as_float(sr[i + 2])) * a.scale_log2;
#pragma unroll
                        for (int o = 4; o < 32; o *= 2) m = fmaxf(m, __shfl_xor_sync(kFull, m, o));
                        if (g == 0) sh.wmax[warp][col(i)] = m;
                    }
                    softmax_sync();
                    if (tid < N) {
                        const float m = fmaxf(fmaxf(sh.wmax[0][tid], sh.wmax[1][tid]), fmaxf(sh.wmax[2][tid], sh.wmax[3][tid]));
                        const float old = sh.mref[tid], now = fmaxf(old, m);
                        sh.mref[tid] = now;
                        sh.fac[tid] = hw_ex2(old - now);
                    }
                    softmax_sync();
#pragma unroll
                    for (int j = 0; j < N / 4; ++j) {
                        const int n = col(j / 2 * 4 + j % 2);
                        l[j] *= sh.fac[n];
                        mr[j] = sh.mref[n];
                    }
                    if (k > 0) {
                        if (!o_added(it - 1)) ok = false;
                        tc_fence_after();
                        for (int p = 0; p < nb; ++p)
                            for (int c = 0; c < kO; c += 16) {
                                uint32_t o[16];
                                tmem_ld16_nowait(tl + 2 * N + p * kO + c, o);
                                tmem_wait_ld();
#pragma unroll
                                for (int i = 0; i < 16; ++i)
                                    o[i] = __float_as_uint(__uint_as_float(o[i]) * sh.fac[(c < N ? c : c - N) + i]);
                                tmem_st16(tl + 2 * N + p * kO + c, o);
                            }
                        tmem_wait_st();
                    }
                }
                if (it > 0 && kPBufs == 1 && !o_added(it - 1)) ok = false;
                const uint32_t at_hi = pat + it % kPBufs * kPBytes;
                const uint32_t at_lo = p_beside(N) ? at_hi + N * 128 : pat - p_base + r_base + rslot * kChunkBytes;
                rslot = rslot + 1 < a.ropes ? rslot + 1 : 0;
                // (no memory clobber: the values' chains overlap; the fence below orders the stores)
                auto store = [&](uint32_t at, const uint32_t *m) {
                    asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(at),
                                 "r"(m[0]), "r"(m[1]), "r"(m[2]), "r"(m[3]));
                };
#pragma unroll
                for (int i = 0; i < kVals; i += 8) {  // two times eight columns
                    uint32_t hi[4], lo[4];
#pragma unroll
                    for (int m = 0; m < 4; ++m) {
                        const float x = hw_ex2(score(i + 2 * m)), y = hw_ex2(score(i + 2 * m + 1));
                        hi[m] = pack_bf16(x, y);
                        lo[m] = pack_bf16(x - __uint_as_float(hi[m] << 16), y - __uint_as_float(hi[m] & 0xFFFF0000u));
                        l[(i / 4 + m / 2) * 2] += x;
                        l[(i / 4 + m / 2) * 2 + 1] += y;
                    }
                    store(at_hi + i * 256, hi);
                    store(at_lo + i * 256, lo);
                }
                // A later row's latent that is not finite would spread to the
                // rows that do not see it (NaN times a zero weight): the product
                // does without it, and the rows that do see it get a NaN sum
                // (their scores of it may be minus infinity, a weight of zero).
                const int hi = min(seg.ctx - tile * kTile, kTile), lo = max(low - tile * kTile, 0);
                if (lo < hi)
                    for (int p = 0; p < nb; ++p) {
                        const int slot = lslot + p < a.pairs ? lslot + p : lslot + p - a.pairs;
                        for (int i = tid; i < (hi - lo) * 16; i += 128) {
                            if (2 * p + i / 8 % 2 == chunks) continue;  // (an odd last chunk's other half is not loaded)
                            if (keep_finite(l_base + slot * kPairBytes + i / 8 % 2 * kChunkBytes + (lo + i / 16) * 128 + i % 8 * 16))
                                atomicMin(&sh.spoilt, tile * kTile + lo + i / 16);
                        }
                    }
                lslot = lslot + nb < a.pairs ? lslot + nb : lslot + nb - a.pairs;
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_addr(&sh.p_full[it % kPBufs]));
                valid = next_valid;
            }
            // ---- the segment's partial result; the next one is looked up meanwhile
            const int bg = seg.bg;
            more = seg.next(a);
            valid = more && block_ok(seg, seg.first);
            if (!o_added(it - 1)) ok = false;
            if (softmax_any(!ok)) {  // (all four warps leave together)
                ok = false;
                break;
            }
#pragma unroll
            for (int j = 0; j < N / 4; ++j) {
                float s = l[j];
#pragma unroll
                for (int o = 4; o < 32; o *= 2) s += __shfl_xor_sync(kFull, s, o);
                if (g == 0) sh.lsum[warp][col(j / 2 * 4 + j % 2)] = s;
            }
            const size_t slot = static_cast<size_t>(blockIdx.x) + bg;
            softmax_sync();
            if (tid < N) {
                const float sum = (sh.lsum[0][tid] + sh.lsum[1][tid]) + (sh.lsum[2][tid] + sh.lsum[3][tid]);
                a.ml[slot * N + tid] = make_float2(sh.mref[tid], sh.limit[tid] > sh.spoilt ? NAN : sum);
            }
            tc_fence_after();
            for (int p = 0; p < nb; ++p) {
                const int d = p * 128 + warp * 32 + lane;
                uint32_t o[N], rest[N];
#pragma unroll
                for (int c = 0; c < N; c += 16) tmem_ld16_nowait(tl + 2 * N + p * kO + c, o + c);
                if constexpr (p_beside(N))
#pragma unroll
                    for (int c = 0; c < N; c += 16) tmem_ld16_nowait(tl + 2 * N + p * kO + N + c, rest + c);
                tmem_wait_ld();
                if constexpr (p_beside(N))
#pragma unroll
                    for (int n = 0; n < N; ++n) o[n] = __float_as_uint(__uint_as_float(o[n]) + __uint_as_float(rest[n]));
                if (d < a.L) {
                    float *dst = a.part + slot * N * a.L + d;
#pragma unroll
                    for (int n = 0; n < N; ++n) dst[n * a.L] = __uint_as_float(o[n]);
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
// 2^(m_s - max m)).  A CTA takes one head and shares the rows evenly with the
// head's others; its warps join the rows' splits into the B operand, then one
// product D[v][rows] with the head's weights.  o~ enters as two bf16 numbers,
// its rounding in the first half of the columns and the remainder in the other,
// so that it is held to 2^-17 (the MMA's time is that of reading the weights).
// Latency-bound: the weights are in flight before the wait for the attention,
// and a row's partial results are read together with their maxima and sums.
// 6.3 us for one row of one split, 7 us for 64 rows, 9.4 us for one row of 152
// splits, 11.5 us for 320 rows (27 MB of partial sums, from L2).
// Up to 80 rows a CTA go through in one or two rounds, one after the other
// (latent_out_kernel; few rows share the warps).  More go through in rounds of
// 24 whose joins, products and stores overlap (latent_out_rounds_kernel).  The
// whole call, without and with: 512 rows of 16 heads (57 a CTA) 51.5 and 53.4
// us, 768 rows (86) 61.8 and 59.6 us, 1185 rows of 20 heads 112 and 106 us, 1128
// rows of short contexts 55.5 and 47.1 us.
constexpr int kOutThreads = 512, kOutWarps = kOutThreads / 32;
constexpr int kOutRows = 40;               // rows a round of latent_out_kernel, at most
constexpr int kJoinWarps = 12, kRoundRows = 24;
constexpr int kRoundThreads = (4 + kJoinWarps + 1) * 32;  // stores, joins, weights and MMAs
constexpr int kRoundCols = 2 * kRoundRows;

// Group of query row r's head h, and the row in it.
__device__ __forceinline__ int group_of(const LatentAttnArgs &a, int N, int r, int h, int &n) {
    const int b = r / a.q_len, idx = (r - b * a.q_len) * a.Hq + h, grp = idx / N;
    n = idx - grp * N;
    return b * a.G + grp;
}

// Two values of row i at dimensions l and l + 1 into the operand [L / 64][cols][64],
// 128-byte swizzled: roundings, remainders cols / 2 rows on.
__device__ __forceinline__ void put_joined(uint8_t *joined, int cols, int i, int l, float x, float y) {
    uint8_t *to = joined + (l / 64 * cols + i) * 128 + (((l % 64 / 8) ^ (i & 7)) << 4) + l % 8 * 2;
    const uint32_t hi = pack_bf16(x, y);
    *reinterpret_cast<uint32_t *>(to) = hi;
    *reinterpret_cast<uint32_t *>(to + cols * 64) = pack_bf16(x - bf16_lo(hi), y - bf16_hi(hi));
}

// D[v][cols] = the head's weights . the joined rows, by one warp.
__device__ __forceinline__ void out_product(uint32_t leader, uint32_t d, uint32_t weights, uint32_t joined, int chunks,
                                            int v_dim, int cols) {
    const uint32_t idesc = mma_idesc(v_dim, cols);
    for (int c = 0; c < chunks; ++c)
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
            mma_bf16_by(leader, d, sw128_desc(weights + c * v_dim * 128 + kk * 32), sw128_desc(joined + c * cols * 128 + kk * 32),
                        idesc, (c | kk) != 0);
}

// Stores `rows` rows from r0 on by four warps (`warp` 0-3), lane = output
// dimension: 32 w + lane of a 128-row accumulator, 16 w + lane (lane < 16) of a
// 64-row one; 2-byte stores, 64 bytes a warp.
__device__ __forceinline__ void store_rows(const LatentAttnArgs &a, int warp, uint32_t tmem, int cols, int v_dim, int h,
                                           int r0, int rows, __nv_bfloat16 *out) {
    const int lane = threadIdx.x % 32, d = v_dim == 128 ? warp * 32 + lane : warp * 16 + lane;
    const uint32_t tl = tmem + (static_cast<uint32_t>(warp * 32) << 16);
    for (int i = 0; i < rows; i += 8) {
        uint32_t x[8], y[8];
        tmem_ld8_nowait(tl + i, x);
        tmem_ld8_nowait(tl + cols / 2 + i, y);
        tmem_wait_ld();
        if (v_dim == 128 || lane < 16)
#pragma unroll
            for (int k = 0; k < 8; ++k)
                if (i + k < rows)
                    out[(static_cast<size_t>(r0 + i + k) * a.Hq + h) * v_dim + d] =
                        __float2bfloat16_rn(__uint_as_float(x[k]) + __uint_as_float(y[k]));
    }
}

// Joins `count` splits of one row by a warp, two read together: o (4 x 128
// dimensions) is scaled by 2^-M, M the largest of the splits' maxima, and S is
// the sum of their sums alike.  Every load is issued, past the last split or
// dimension from the last one (with weight zero, or to no use): under a
// condition each would wait for the one before.
__device__ __forceinline__ void join_row(const float *part, size_t part_step, const float2 *ml, size_t ml_step, int count,
                                         const int *dims, float4 *o, float &M, float &S) {
    constexpr int kQ = 4, kAtOnce = 2;
    for (int s0 = 0; s0 < count; s0 += kAtOnce) {
        float4 x[kAtOnce][kQ];
        float2 v[kAtOnce];
#pragma unroll
        for (int u = 0; u < kAtOnce; ++u) {
            const int s = min(s0 + u, count - 1);
            v[u] = __ldcg(ml + static_cast<size_t>(s) * ml_step);
#pragma unroll
            for (int k = 0; k < kQ; ++k) x[u][k] = __ldcg(reinterpret_cast<const float4 *>(part + static_cast<size_t>(s) * part_step + dims[k]));
        }
        float top = M;
#pragma unroll
        for (int u = 0; u < kAtOnce; ++u) {
            if (s0 + u >= count) v[u] = make_float2(-INFINITY, 0.0f);
            top = fmaxf(top, v[u].x);
        }
        const float f0 = hw_ex2(M - top);
        M = top;
        S *= f0;
#pragma unroll
        for (int k = 0; k < kQ; ++k) {
            o[k].x *= f0;
            o[k].y *= f0;
            o[k].z *= f0;
            o[k].w *= f0;
        }
#pragma unroll
        for (int u = 0; u < kAtOnce; ++u) {
            const float f = hw_ex2(v[u].x - top);
            S = fmaf(f, v[u].y, S);
#pragma unroll
            for (int k = 0; k < kQ; ++k) {
                o[k].x = fmaf(f, x[u][k].x, o[k].x);
                o[k].y = fmaf(f, x[u][k].y, o[k].y);
                o[k].z = fmaf(f, x[u][k].z, o[k].z);
                o[k].w = fmaf(f, x[u][k].w, o[k].w);
            }
        }
    }
}

// The same for 128 dimensions (`part` is this lane's four) of the splits first,
// first + stride, .. below `count`, which may be many: 32 at a time, each lane
// with one split's maximum and sum, sixteen splits' parts in flight.
__device__ __forceinline__ void join_part(const float *part, size_t part_step, const float2 *ml, size_t ml_step, int first,
                                          int stride, int count, float4 &o, float &M, float &S) {
    constexpr int kAtOnce = 16;
    const int lane = threadIdx.x % 32, mine = first < count ? (count - first + stride - 1) / stride : 0;
    for (int c0 = 0; c0 < mine; c0 += 32) {
        const int m = min(32, mine - c0);
        float4 x[kAtOnce];
        auto load = [&](int u0) {
#pragma unroll
            for (int u = 0; u < kAtOnce; ++u) {
                const size_t s = first + (c0 + min(u0 + u, m - 1)) * stride;
                x[u] = __ldcg(reinterpret_cast<const float4 *>(part + s * part_step));
            }
        };
        float2 v = __ldcg(ml + static_cast<size_t>(first + (c0 + min(lane, m - 1)) * stride) * ml_step);
        load(0);
        if (lane >= m) v = make_float2(-INFINITY, 0.0f);
        float top = fmaxf(M, v.x);
#pragma unroll
        for (int i = 16; i > 0; i >>= 1) top = fmaxf(top, __shfl_xor_sync(kFull, top, i));
        const float f0 = hw_ex2(M - top), f = hw_ex2(v.x - top);
        float sum = f * v.y;
#pragma unroll
        for (int i = 16; i > 0; i >>= 1) sum += __shfl_xor_sync(kFull, sum, i);
        M = top;
        S = fmaf(S, f0, sum);
        o.x *= f0;
        o.y *= f0;
        o.z *= f0;
        o.w *= f0;
        for (int u0 = 0; u0 < m; u0 += kAtOnce) {
#pragma unroll
            for (int u = 0; u < kAtOnce; ++u) {
                const float w = __shfl_sync(kFull, f, u0 + u);
                o.x = fmaf(w, x[u].x, o.x);
                o.y = fmaf(w, x[u].y, o.y);
                o.z = fmaf(w, x[u].z, o.z);
                o.w = fmaf(w, x[u].w, o.w);
            }
            if (u0 + kAtOnce < m) load(u0 + kAtOnce);
        }
    }
}

__global__ void __launch_bounds__(kOutThreads)
latent_out_kernel(const __grid_constant__ CUtensorMap map_uv, const LatentAttnArgs a, int N,
                  int rows_per_round, int v_dim, __nv_bfloat16 *__restrict__ out) {
    extern __shared__ __align__(1024) uint8_t raw[];
    __shared__ float2 ms[kOutWarps];
    __shared__ uint64_t full, acc;
    __shared__ uint32_t tslot;
    const int L = a.L, R = a.B * a.q_len, chunks = L / 64;
    const int cols = (rows_per_round + 7) / 8 * 16;                // columns: roundings, remainders
    const uint32_t wb = smem_addr(raw), w_chunk = v_dim * 128;     // [chunks][v][64 l]
    uint8_t *joined = raw + chunks * w_chunk;                      // [chunks][cols][64 l], 128-byte swizzle
    float *sums = reinterpret_cast<float *>(joined + chunks * cols * 128);  // [kOutWarps][128]
    const int warp = uniform(threadIdx.x / 32), lane = threadIdx.x % 32;
    const int h = blockIdx.y;
    bool ok = true;
    if (warp == 0) {
        const uint32_t leader = elect_leader();
        if (leader) {
            mbar_init(smem_addr(&full), 1);
            mbar_init(smem_addr(&acc), 1);
            fence_mbar_init();
        }
        __syncwarp();
        mbar_expect_tx_by(leader, smem_addr(&full), chunks * w_chunk);
        for (int c = 0; c < chunks; ++c)
            tma_load_2d_by(leader, wb + c * w_chunk, &map_uv, 64 * c, h * v_dim, smem_addr(&full));
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 128;" ::"r"(smem_addr(&tslot))
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = uniform(tslot);
    for (uint32_t round = 0;; ++round) {
        const int r0 = (blockIdx.x + round * gridDim.x) * rows_per_round, rows = min(rows_per_round, R - r0);
        if (rows <= 0) break;
        // ---- join: a warp a row; up to 4 rows a warp for every 128 of their
        // dimensions, the warps left over sharing the splits
        const int quarters = (L + 127) / 128, lq = quarters > 2 ? 2 : quarters - 1;  // log2, rounded up
        const int lshare = rows > 4 ? 0 : rows > 2 ? 2 : rows > 1 ? 3 : 4;           // log2 of a row's warps
        const int ldims = lshare ? lq : 0, lss = lshare - ldims, ss = 1 << lss;
        const int sub = warp & ((1 << lshare) - 1), i0 = warp >> lshare;
        const int first = sub >> ldims, d0 = (sub & ((1 << ldims) - 1)) * 128 + 4 * lane;
        if (round == 0) {
            pdl_wait_prerequisites();
            pdl_allow_dependents();
        }
        int n, bg = group_of(a, N, r0 + min(i0, rows - 1), h, n);
        int2 own = __ldcg(a.owner + bg);
        for (int rr = 0; rr < rows; rr += kOutWarps >> lshare) {
            const int i = rr + i0;
            // the next row's owner is read a row ahead
            int n_next;
            const int bg_next = group_of(a, N, r0 + min(i + (kOutWarps >> lshare), rows - 1), h, n_next);
            const int2 own_next = __ldcg(a.owner + bg_next);
            if (i < rows) {
                const size_t row = (static_cast<size_t>(own.x) + bg) * N + n;
                const float2 *ml = a.ml + row;  // split s: ml[s * N]
                const float *part = a.part + row * L;
                int dims[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) dims[k] = min(d0 + 128 * k, L - 4);
                const size_t step = static_cast<size_t>(N) * L;
                float4 o[4] = {};
                float M = kNoScore, S = 0.0f;
                if (lshare) join_part(part + dims[0], step, ml, N, first, ss, own.y, o[0], M, S);
                else join_row(part, step, ml, N, own.y, dims, o, M, S);
                if (lss == 0) {
                    const float inv = S == 0.0f ? 0.0f : 1.0f / S;  // no token left: zeros
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        if (d0 + 128 * k < L && (k == 0 || !lshare)) {
                            put_joined(joined, cols, i, d0 + 128 * k, o[k].x * inv, o[k].y * inv);
                            put_joined(joined, cols, i, d0 + 128 * k + 2, o[k].z * inv, o[k].w * inv);
                        }
                } else {
                    if (lane == 0) ms[warp] = make_float2(M, S);
                    if (d0 < L) *reinterpret_cast<float4 *>(sums + warp * 128 + 4 * lane) = o[0];
                }
            }
            if (lss > 0) {  // (one pass: every row has its warps)
                __syncthreads();
                if (i < rows && first == 0 && d0 < L) {
                    float M = kNoScore, S = 0.0f;
                    float4 x = {};
                    for (int s = 0; s < ss; ++s) M = fmaxf(M, ms[warp + (s << ldims)].x);
                    for (int s = 0; s < ss; ++s) {
                        const float2 v = ms[warp + (s << ldims)];
                        const float4 y = *reinterpret_cast<const float4 *>(sums + (warp + (s << ldims)) * 128 + 4 * lane);
                        const float f = hw_ex2(v.x - M);
                        S = fmaf(f, v.y, S);
                        x.x = fmaf(f, y.x, x.x);
                        x.y = fmaf(f, y.y, x.y);
                        x.z = fmaf(f, y.z, x.z);
                        x.w = fmaf(f, y.w, x.w);
                    }
                    const float inv = S == 0.0f ? 0.0f : 1.0f / S;
                    put_joined(joined, cols, i, d0, x.x * inv, x.y * inv);
                    put_joined(joined, cols, i, d0 + 2, x.z * inv, x.w * inv);
                }
            }
            own = own_next;
            n = n_next;
            bg = bg_next;
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        tc_fence_before();
        __syncthreads();
        tc_fence_after();
        if (warp == 0) {
            const uint32_t leader = elect_leader();
            if (!warp_wait(&full, 0)) ok = false;
            tc_fence_after();
            out_product(leader, tmem, wb, smem_addr(joined), chunks, v_dim, cols);
            mma_commit_by(leader, smem_addr(&acc));
        }
        if (warp < 4) {
            if (!warp_wait(&acc, round & 1)) ok = false;
            tc_fence_after();
            if (ok) store_rows(a, warp, tmem, cols, v_dim, h, r0, rows, out);
        }
        // the next rows' operand and accumulator take the places of these
        tc_fence_before();
        __syncthreads();
        tc_fence_after();
    }
    if (!ok) flag_error(a.err, TTS_ERRBIT_TIMEOUT);
    if (warp == 0) {
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 128;" ::"r"(tmem) : "memory");
    }
}

// The same for more rows a CTA (`per` of them, from per x blockIdx.x on), `each`
// (up to 24) a round: twelve warps join two rows each into one of two operands,
// one warp issues the products, four store.
__global__ void __launch_bounds__(kRoundThreads)
latent_out_rounds_kernel(const __grid_constant__ CUtensorMap map_uv, const LatentAttnArgs a, int N, int per, int each,
                         int v_dim, __nv_bfloat16 *__restrict__ out) {
    extern __shared__ __align__(1024) uint8_t raw[];
    __shared__ uint64_t full, joined_full[2], joined_empty[2], acc_full[2], acc_empty[2], fin;
    __shared__ uint32_t tslot;
    const int L = a.L, chunks = L / 64;
    const uint32_t w_chunk = v_dim * 128, j_bytes = chunks * kRoundCols * 128;
    uint8_t *joined = raw + chunks * w_chunk;                      // [2][chunks][48][64 l], after [chunks][v][64 l]
    const uint32_t wb = smem_addr(raw), jb = smem_addr(joined);
    const int warp = uniform(threadIdx.x / 32), lane = threadIdx.x % 32;
    const int h = blockIdx.y, begin = blockIdx.x * per, end = min(begin + per, a.B * a.q_len);
    const int rounds = (end - begin + each - 1) / each;
    constexpr int kIssuer = 4 + kJoinWarps;
    bool ok = true;
    if (warp == kIssuer) {
        const uint32_t leader = elect_leader();
        if (leader) {
            mbar_init(smem_addr(&full), 1);
            mbar_init(smem_addr(&fin), 1);
            for (int i = 0; i < 2; ++i) {
                mbar_init(smem_addr(&joined_full[i]), kJoinWarps);
                mbar_init(smem_addr(&joined_empty[i]), 1);
                mbar_init(smem_addr(&acc_full[i]), 1);
                mbar_init(smem_addr(&acc_empty[i]), 4);
            }
            fence_mbar_init();
        }
        __syncwarp();
        mbar_expect_tx_by(leader, smem_addr(&full), chunks * w_chunk);
        for (int c = 0; c < chunks; ++c)
            tma_load_2d_by(leader, wb + c * w_chunk, &map_uv, 64 * c, h * v_dim, smem_addr(&full));
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 128;" ::"r"(smem_addr(&tslot))
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = uniform(tslot);
    if (warp == kIssuer) {
        const uint32_t leader = elect_leader();
        ok = warp_wait(&full, 0);
        for (int k = 0; ok && k < rounds; ++k) {
            const int buf = k & 1;
            WarpWaits<2> w;
            w.set(0, &joined_full[buf], (k / 2) & 1);
            w.none(1);
            if (k >= 2) w.set(1, &acc_empty[buf], (k / 2 - 1) & 1);
            ok = w.wait();
            if (!ok) break;
            tc_fence_after();
            out_product(leader, tmem + buf * kRoundCols, wb, jb + buf * j_bytes, chunks, v_dim, kRoundCols);
            mma_commit_by(leader, smem_addr(&joined_empty[buf]));
            mma_commit_by(leader, smem_addr(&acc_full[buf]));
        }
        mma_commit_by(leader, smem_addr(&fin));
        if (!warp_wait(&fin, 0)) ok = false;
    } else if (warp >= 4) {
        const int i = warp - 4;
        int dims[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) dims[k] = min(4 * lane + 128 * k, L - 4);
        const size_t step = static_cast<size_t>(N) * L;
        pdl_wait_prerequisites();
        pdl_allow_dependents();
        int n, bg = group_of(a, N, min(begin + i, end - 1), h, n);
        int2 own = __ldcg(a.owner + bg);
        for (int k = 0; ok && k < rounds; ++k) {
            const int buf = k & 1, r0 = begin + k * each, rows = min(each, end - r0);
            for (int j = i; j < each; j += kJoinWarps) {
                // (the next row's owner is read a row ahead)
                int n_next;
                const int r_next = j + kJoinWarps < each ? r0 + j + kJoinWarps : r0 + each + i;
                const int bg_next = group_of(a, N, min(r_next, end - 1), h, n_next);
                const int2 own_next = __ldcg(a.owner + bg_next);
                const size_t row = (static_cast<size_t>(own.x) + bg) * N + n;
                float4 o[4] = {};
                float M = kNoScore, S = 0.0f;
                if (j < rows) join_row(a.part + row * L, step, a.ml + row, N, own.y, dims, o, M, S);
                if (j == i && k >= 2 && !warp_wait(&joined_empty[buf], (k / 2 - 1) & 1)) {
                    ok = false;
                    break;
                }
                if (j < rows) {
                    const float inv = S == 0.0f ? 0.0f : 1.0f / S;  // no token left: zeros
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const int d = 4 * lane + 128 * q;
                        if (d < L) {
                            put_joined(joined + buf * j_bytes, kRoundCols, j, d, o[q].x * inv, o[q].y * inv);
                            put_joined(joined + buf * j_bytes, kRoundCols, j, d + 2, o[q].z * inv, o[q].w * inv);
                        }
                    }
                }
                own = own_next;
                n = n_next;
                bg = bg_next;
            }
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            __syncwarp();
            if (ok && lane == 0) mbar_arrive(smem_addr(&joined_full[buf]));
        }
    } else {
        for (int k = 0; k < rounds; ++k) {
            const int buf = k & 1, r0 = begin + k * each;
            if (!warp_wait(&acc_full[buf], (k / 2) & 1)) {
                ok = false;
                break;
            }
            tc_fence_after();
            store_rows(a, warp, tmem + buf * kRoundCols, kRoundCols, v_dim, h, r0, min(each, end - r0), out);
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_addr(&acc_empty[buf]));
        }
    }
    if (!ok) flag_error(a.err, TTS_ERRBIT_TIMEOUT);
    tc_fence_before();
    __syncthreads();
    if (warp == kIssuer) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 128;" ::"r"(tmem) : "memory");
    }
}

// -------------------------------------------------------------------- host

bool decode_shape_ok(int B, int q_len, int Hq, int L, int nope, int v, int max_ctx) {
    return B >= 0 && q_len >= 1 && Hq >= 1 && static_cast<long>(q_len) * Hq <= 1024 && L >= 64 && L <= kLatentMaxDim &&
           L % 64 == 0 && latent_head_dim_ok(nope) && latent_head_dim_ok(v) && max_ctx >= 1 &&
           static_cast<long>(B) * q_len <= (1 << 20);
}

constexpr int kSmemLimit = 232448;

template <int N>
int launch_attention(const CUtensorMap &kv, const CUtensorMap &q, const CUtensorMap &qr, LatentAttnArgs a, int P,
                     cudaStream_t stream) {
    // shared memory: q~, P, the rope slots, and latent pairs to the brim
    const int chunks = a.L / 64;
    const int fixed = ((chunks + 1) * N + p_buffers(N) * p_rows(N)) * 128 + static_cast<int>(sizeof(AttnShared));
    const int nb = (a.L + 127) / 128, tiles = (kSmemLimit - fixed) / (kChunkBytes + nb * kPairBytes);
    a.ropes = std::min(std::max(tiles, 2), kMaxRopes);  // a rope slot for every tile on its way
    a.pairs = std::min((kSmemLimit - fixed - a.ropes * kChunkBytes) / kPairBytes, kMaxPairs);
    if (a.pairs < 2 * nb) return TTS_ERR_UNSUPPORTED;  // (S^T goes one tile ahead of O^T)
    const int smem = fixed + a.ropes * kChunkBytes + a.pairs * kPairBytes;
    if (!allow_smem(latent_attn_kernel<N>, smem)) return TTS_ERR_CUDA;
    return launch_kernel(latent_attn_kernel<N>, dim3(P), dim3(kAttnThreads), smem, {stream, true}, kv, q, qr, a);
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
    // units are 32-bit (contexts end at the table's last block)
    const int most_ctx = std::min(max_ctx_len, max_blocks_per_seq * TTS_BLOCK_TOKENS);
    if (latent_plan(B, q_len, num_q_heads, L, most_ctx).units > 0x40000000L) return TTS_ERR_UNSUPPORTED;
    if (!d_ws || !aligned16(d_ws) || ws_bytes < pl.total()) return TTS_ERR_WORKSPACE;

    uint8_t *ws = static_cast<uint8_t *>(d_ws);
    void *qt = ws;  // q~ [R][Hq][L]
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
    a.start = start_units(pl.N);
    a.scale_log2 = scale * kLog2e;
    a.causal = causal != 0;
    a.part = reinterpret_cast<float *>(ws + pl.qt_bytes);
    a.ml = reinterpret_cast<float2 *>(ws + pl.qt_bytes + pl.part_bytes);
    a.owner = reinterpret_cast<int2 *>(ws + pl.qt_bytes + pl.part_bytes + pl.ml_bytes);
    a.err = d_err;
    a.wait_limit = thread_opts().wait_limit;
    a.stall = thread_opts().stall == TTS_TEST_STALL_LATENT_DECODE;
    const int R = B * q_len, Hq = num_q_heads;
    const uint64_t qrows = static_cast<uint64_t>(R) * Hq;
    CUtensorMap map_kv, map_q, map_qr, map_qn, map_uk, map_qt, map_uv;
    if (!make_tma_2d_bf16(&map_kv, cache->pool, static_cast<uint64_t>(cache->num_blocks) * TTS_BLOCK_TOKENS,
                          L + kLatentRope, TTS_BLOCK_TOKENS, 64) ||
        !make_tma_2d_bf16(&map_q, qt, qrows, L, pl.N, 64) ||
        !make_tma_2d_bf16(&map_qr, d_q_rope, qrows, kLatentRope, pl.N, 64) ||
        !make_tma_2d_bf16(&map_qn, d_q_nope, R, static_cast<uint64_t>(Hq) * nope_dim, kRowTile, 64) ||
        !make_tma_2d_bf16(&map_uk, d_w_uk, static_cast<uint64_t>(Hq) * nope_dim, L, nope_dim, 64) ||
        !make_tma_2d_bf16(&map_qt, qt, R, static_cast<uint64_t>(Hq) * L, kRowTile, 64) ||
        !make_tma_2d_bf16(&map_uv, d_w_uv, static_cast<uint64_t>(Hq) * v_dim, L, v_dim, 64))
        return TTS_ERR_CUDA;

    const cudaStream_t cs = static_cast<cudaStream_t>(stream);
    const int absorb_smem = 2 * nope_dim * 128 + nope_dim / 64 * kRowTile * 128;
    if (!allow_smem(latent_absorb_kernel, absorb_smem)) return TTS_ERR_CUDA;
    int rc = launch_kernel(latent_absorb_kernel, dim3((L + 127) / 128, Hq, (R + kRowTile - 1) / kRowTile), dim3(128),
                           absorb_smem, {cs, thread_pdl()}, map_qn, map_uk, map_qt, static_cast<int>(nope_dim), L, R,
                           d_err);
    if (rc != TTS_OK) return rc;
    switch (pl.N) {
        case 16: rc = launch_attention<16>(map_kv, map_q, map_qr, a, pl.P, cs); break;
        case 32: rc = launch_attention<32>(map_kv, map_q, map_qr, a, pl.P, cs); break;
        case 48: rc = launch_attention<48>(map_kv, map_q, map_qr, a, pl.P, cs); break;
        default: rc = launch_attention<64>(map_kv, map_q, map_qr, a, pl.P, cs); break;
    }
    if (rc != TTS_OK) return rc;
    // one CTA fits an SM: as many as there are SMs share the rows evenly
    const int most = std::max(1, kCtas / Hq), cta_rows = (R + most - 1) / most;
    auto *o = static_cast<__nv_bfloat16 *>(d_out);
    const int v = v_dim;
    if (cta_rows <= 2 * kOutRows) {
        const int rounds = cta_rows > kOutRows ? 2 : 1;
        const int per = (R + most * rounds - 1) / (most * rounds), gx = std::min(most, (R + per - 1) / per);
        const int smem = L / 64 * (v + (per + 7) / 8 * 16) * 128 + kOutWarps * 512;
        if (!allow_smem(latent_out_kernel, smem)) return TTS_ERR_CUDA;
        return launch_kernel(latent_out_kernel, dim3(gx, Hq), dim3(kOutThreads), smem, {cs, true}, map_uv, a, pl.N, per, v, o);
    }
    const int rounds = (cta_rows + kRoundRows - 1) / kRoundRows, each = (cta_rows + rounds - 1) / rounds;
    const int smem = L / 64 * (v + 2 * kRoundCols) * 128;
    if (!allow_smem(latent_out_rounds_kernel, smem)) return TTS_ERR_CUDA;
    return launch_kernel(latent_out_rounds_kernel, dim3((R + cta_rows - 1) / cta_rows, Hq), dim3(kRoundThreads), smem,
                         {cs, true}, map_uv, a, pl.N, cta_rows, each, v, o);
}
