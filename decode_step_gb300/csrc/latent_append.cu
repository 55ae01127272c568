// Latent append: this step's (or prompt's) rows go to the paged latent pool,
// a row being a latent c (copied) and a rotated key part kr, and the same
// tokens' query parts are rotated at the same positions.
//
// A row's work is a list of 16-byte items: (Hq + 1) x 4 rotary items (8 pairs
// (i, i + 32) each: 16 bytes of either half; the last head is the key part) and
// latent_dim / 8 copies.  Pure data movement: the bytes are each row's 2
// (latent_dim + 64) + 2 x 64 Hq, read once and written once.
// A CTA takes one row, or four where there are more rows than CTAs fit at once
// (a CTA's time is latency): 12 prompts of 8409 rows in all, 16 heads, take 11.9
// us, 4.5 TB/s, 64 rows 2.5 us.
// The rows' first items are loaded before their positions are known (they do
// not depend on them); meanwhile a warp per row finds the stream and the block
// and computes the 32 angles, shared through shared memory.
#include <cuda_bf16.h>

#include <cmath>

#include "latent_common.cuh"
#include "tts_common.cuh"
#include "tts_internal.h"

namespace tts {
namespace {

constexpr int kThreads = 128;
constexpr int kAhead = 2;  // items per thread and row loaded before the position is known
// One-row CTAs that run at once (42 registers a thread: ten an SM).  Up to so
// many rows the one-row kernel is ahead (1520 rows 3.7 us against 4.2), beyond
// them its second wave is not (1600 rows 4.6 against 4.2, 2432 rows 5.2 against
// 4.55; 16 heads, latent 512).
constexpr int kAtOnce = 152 * 10;
constexpr int kHalf = kLatentRope / 2;

// Rotary frequencies base^(-2i/64) in turns a token, scaled by 2^64: a
// position's angle modulo one turn is then the low half of a 64-bit product,
// exact but for the frequency's own rounding (2^-53: 2^-32 turns at position
// 2^20).  Double arithmetic would bound the kernel: this part does two double
// operations a cycle and SM, and 32 reduced angles a row take some 400.
struct HalfFreqs {
    uint64_t turns[kHalf];
};

// cos and sin of s * turns 2 pi: the leading 24 bits by sincospif, the rest to
// first order (an error of a few 2^-24).
__device__ __forceinline__ float2 turn_cos_sin(int s, uint64_t turns) {
    const int64_t a = static_cast<int64_t>(static_cast<uint64_t>(s) * turns);  // [-1/2, 1/2) turn
    const float hi = __ll2float_rn(a);
    const float lo = __ll2float_rn(a - __float2ll_rn(hi));
    float sn, cs;
    sincospif(hi * 0x1.0p-63f, &sn, &cs);  // (2^-64 turns are 2^-63 half turns)
    const float d = lo * (6.2831853f * 0x1.0p-64f);
    return make_float2(fmaf(-sn, d, cs), fmaf(cs, d, sn));
}

struct LatentAppendArgs {
    const int32_t *table;
    int max_blocks;
    const int32_t *ctx_before;
    int B, num_rows;
    const int32_t *row_start;  // null: rows_per_stream rows each
    int rows_per_stream;
    int Hq, L, num_blocks;
    const __nv_bfloat16 *c_new, *kr_new;
    const __nv_bfloat16 *q;
    __nv_bfloat16 *q_out;
    __nv_bfloat16 *pool;
    int32_t *err;
};

template <int kRows>
__global__ void __launch_bounds__(kThreads) latent_append_kernel(const LatentAppendArgs a, const HalfFreqs freqs) {
    __shared__ float2 cs[kRows][kHalf];
    __shared__ int where[kRows][2];  // block (-1: skip the row), slot
    pdl_wait_prerequisites();
    pdl_allow_dependents();
    const int row0 = blockIdx.x * kRows;
    const int rope_items = 4 * (a.Hq + 1), items = rope_items + a.L / 8;
    auto load = [&](int row, int it, uint4 &lo, uint4 &hi) {
        if (it < rope_items) {
            const int h = it >> 2;
            const __nv_bfloat16 *x = h < a.Hq ? a.q + (static_cast<size_t>(row) * a.Hq + h) * kLatentRope
                                              : a.kr_new + static_cast<size_t>(row) * kLatentRope;
            lo = reinterpret_cast<const uint4 *>(x)[it & 3];
            hi = reinterpret_cast<const uint4 *>(x)[(it & 3) + 4];
        } else {
            lo = __ldcs(reinterpret_cast<const uint4 *>(a.c_new + static_cast<size_t>(row) * a.L) + it - rope_items);
        }
    };
    uint4 lo[kRows][kAhead], hi[kRows][kAhead];
#pragma unroll
    for (int i = 0; i < kRows; ++i)
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            const int it = threadIdx.x + u * kThreads;
            if (it < items && row0 + i < a.num_rows) load(row0 + i, it, lo[i][u], hi[i][u]);
        }

    if (threadIdx.x < 32 * kRows) {
        const int i = threadIdx.x / 32, lane = threadIdx.x % 32, row = row0 + i;
        int b = -1, j = 0;
        if (row < a.num_rows) {
            if (a.row_start) {
                b = stream_of_row(a.row_start, a.B, row, lane);
                j = b < 0 ? 0 : row - a.row_start[b];
            } else {
                b = row / a.rows_per_stream;
                j = row - b * a.rows_per_stream;
            }
        }
        int blk = -1, s = 0;
        if (b >= 0) {
            const int before = a.ctx_before[b];
            const int cap = a.max_blocks * TTS_BLOCK_TOKENS;
            if (before < 0 || before >= cap || j >= cap - before) {
                if (lane == 0) flag_error(a.err, TTS_ERRBIT_CTX_LEN);
            } else {
                s = before + j;
                blk = a.table[static_cast<size_t>(b) * a.max_blocks + s / TTS_BLOCK_TOKENS];
                if (blk < 0 || blk >= a.num_blocks) {
                    if (lane == 0) flag_error(a.err, TTS_ERRBIT_BLOCK_ID);
                    blk = -1;
                }
            }
        }
        if (lane == 0) {
            where[i][0] = blk;
            where[i][1] = s % TTS_BLOCK_TOKENS;
        }
        cs[i][lane] = turn_cos_sin(s, freqs.turns[lane]);
    }
    __syncthreads();

#pragma unroll
    for (int i = 0; i < kRows; ++i) {
        const int blk = where[i][0], row = row0 + i;
        if (blk < 0) continue;
        uint4 *dst = reinterpret_cast<uint4 *>(
            a.pool + (static_cast<size_t>(blk) * TTS_BLOCK_TOKENS + where[i][1]) * (a.L + kLatentRope));
        auto emit = [&](int it, const uint4 &vlo, const uint4 &vhi) {
            if (it >= rope_items) {
                dst[it - rope_items] = vlo;
                return;
            }
            float x1[8], x2[8];
            Chunk<__nv_bfloat16>::unpack(vlo, x1);
            Chunk<__nv_bfloat16>::unpack(vhi, x2);
            const int p = it & 3;
            uint32_t o1[4], o2[4];
#pragma unroll
            for (int e = 0; e < 8; e += 2) {
                const float2 c0 = cs[i][8 * p + e], c1 = cs[i][8 * p + e + 1];
                const __nv_bfloat162 r1 = __floats2bfloat162_rn(fmaf(-x2[e], c0.y, x1[e] * c0.x),
                                                                fmaf(-x2[e + 1], c1.y, x1[e + 1] * c1.x));
                const __nv_bfloat162 r2 = __floats2bfloat162_rn(fmaf(x1[e], c0.y, x2[e] * c0.x),
                                                                fmaf(x1[e + 1], c1.y, x2[e + 1] * c1.x));
                o1[e / 2] = *reinterpret_cast<const uint32_t *>(&r1);
                o2[e / 2] = *reinterpret_cast<const uint32_t *>(&r2);
            }
            const int h = it >> 2;
            uint4 *o = h < a.Hq
                           ? reinterpret_cast<uint4 *>(a.q_out + (static_cast<size_t>(row) * a.Hq + h) * kLatentRope)
                           : dst + a.L / 8;
            o[p] = make_uint4(o1[0], o1[1], o1[2], o1[3]);
            o[p + 4] = make_uint4(o2[0], o2[1], o2[2], o2[3]);
        };
#pragma unroll
        for (int u = 0; u < kAhead; ++u)
            if (threadIdx.x + u * kThreads < items) emit(threadIdx.x + u * kThreads, lo[i][u], hi[i][u]);
        for (int it = threadIdx.x + kAhead * kThreads; it < items; it += kThreads) {
            uint4 vlo, vhi;
            load(row, it, vlo, vhi);
            emit(it, vlo, vhi);
        }
    }
}

}  // namespace
}  // namespace tts

extern "C" int tts_latent_append(const tts_latent_cache *cache, const int32_t *d_block_table,
                                 int32_t max_blocks_per_seq, const int32_t *d_ctx_before, int32_t B,
                                 const int32_t *d_row_start, int32_t num_rows, int32_t num_q_heads, float rope_base,
                                 const void *d_c_new, const void *d_kr_new, const void *d_q_rope, void *d_q_rope_out,
                                 int32_t *d_err, void *stream) {
    using namespace tts;
    const int st = check_latent_cache(cache, d_block_table, max_blocks_per_seq);
    if (st != TTS_OK) return st;
    if (!d_ctx_before || !d_c_new || !d_kr_new || B < 0 || num_rows < 0) return TTS_ERR_INVALID;
    if (num_q_heads < 0 || num_q_heads > kLatentMaxHeads || (num_q_heads > 0 && (!d_q_rope || !d_q_rope_out)))
        return TTS_ERR_INVALID;
    if (!(rope_base > 1.0f) || rope_base == INFINITY) return TTS_ERR_INVALID;
    if (!d_row_start && (B == 0 ? num_rows != 0 : num_rows % B != 0)) return TTS_ERR_INVALID;
    if (!aligned16(d_c_new) || !aligned16(d_kr_new) || !aligned16(d_q_rope) || !aligned16(d_q_rope_out))
        return TTS_ERR_INVALID;
    if (B == 0 || num_rows == 0) return TTS_OK;

    LatentAppendArgs a{};
    a.table = d_block_table;
    a.max_blocks = max_blocks_per_seq;
    a.ctx_before = d_ctx_before;
    a.B = B;
    a.num_rows = num_rows;
    a.row_start = d_row_start;
    a.rows_per_stream = num_rows / B;
    a.Hq = num_q_heads;
    a.L = cache->latent_dim;
    a.num_blocks = cache->num_blocks;
    a.c_new = static_cast<const __nv_bfloat16 *>(d_c_new);
    a.kr_new = static_cast<const __nv_bfloat16 *>(d_kr_new);
    a.q = static_cast<const __nv_bfloat16 *>(d_q_rope);
    a.q_out = static_cast<__nv_bfloat16 *>(d_q_rope_out);
    a.pool = static_cast<__nv_bfloat16 *>(cache->pool);
    a.err = d_err;
    HalfFreqs f;
    for (int i = 0; i < kHalf; ++i) {
        const double turns = pow(static_cast<double>(rope_base), -2.0 * i / kLatentRope) * 0.15915494309189535;  // 1 / (2 pi)
        f.turns[i] = static_cast<uint64_t>(turns * 0x1.0p64);
    }
    const LaunchOpts o{static_cast<cudaStream_t>(stream), thread_pdl()};
    if (num_rows > kAtOnce)
        return launch_kernel(latent_append_kernel<4>, dim3((num_rows + 3) / 4), dim3(kThreads), 0, o, a, f);
    return launch_kernel(latent_append_kernel<1>, dim3(num_rows), dim3(kThreads), 0, o, a, f);
}
