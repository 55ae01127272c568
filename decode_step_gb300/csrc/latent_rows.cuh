// Attention of one (query row, head) over the latent cache, a CTA each: the
// definition in its absorbed form, in fp32 on CUDA cores.
//   q~ = w_uk[h]^T q_nope;  s_t = scale (q~ . c_t + q_rope . kr_t)
//   o~ = sum_t softmax(s)_t c_t;  out = w_uv[h] o~
// Warps take tokens in turn, each with a running maximum and sum (online
// softmax) and 16 dimensions of o~ per lane; the warps' results are joined
// through shared memory.
#pragma once

#include <cuda_bf16.h>

#include "latent_common.cuh"
#include "tts_common.cuh"

namespace tts {

struct LatentRowsArgs {
    const int32_t *table;
    int max_blocks, num_blocks;
    const int32_t *ctx_lens;
    int max_ctx, B, q_len, Hq, L, nope, v;
    const int32_t *row_start;  // null: q_len rows per stream
    int num_rows;
    float scale;
    int causal;
    const __nv_bfloat16 *pool, *q_nope, *q_rope, *w_uk, *w_uv;
    __nv_bfloat16 *out;
    int32_t *err;
};

constexpr int kRowWarps = 8;

static __global__ void __launch_bounds__(kRowWarps * 32) latent_rows_kernel(const LatentRowsArgs a) {
    __shared__ float qs[kLatentMaxDim + kLatentRope];
    __shared__ float os[kRowWarps][kLatentMaxDim];
    __shared__ float ml[kRowWarps][2];
    const int row = blockIdx.x, h = blockIdx.y;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int b = a.row_start ? stream_of_row(a.row_start, a.B, row, lane) : row / a.q_len;
    if (b < 0) return;
    const int first = a.row_start ? a.row_start[b] : b * a.q_len;
    const int n = a.row_start ? a.row_start[b + 1] - first : a.q_len;
    const int ctx = a.ctx_lens[b];
    __nv_bfloat16 *out = a.out + (static_cast<size_t>(row) * a.Hq + h) * a.v;
    long total = ctx;  // of the streams up to this one that have rows
    for (int i = 0; a.row_start && i < b; ++i) {
        const int ni = a.row_start[i + 1] - a.row_start[i], ci = a.ctx_lens[i];
        if (ni > 0 && a.row_start[i] >= 0 && a.row_start[i + 1] <= a.num_rows && ci >= ni &&
            ci <= a.max_blocks * TTS_BLOCK_TOKENS)
            total += ci;
    }
    const bool rows_ok = first >= 0 && first + n <= a.num_rows;
    if (!rows_ok || ctx < n || total > a.max_ctx || ctx > a.max_blocks * TTS_BLOCK_TOKENS) {
        if (threadIdx.x == 0) flag_error(a.err, TTS_ERRBIT_CTX_LEN);
        for (int i = threadIdx.x; i < a.v; i += blockDim.x) out[i] = __float2bfloat16_rn(0.0f);
        return;
    }
    const int limit = a.causal ? ctx - n + (row - first) + 1 : ctx;
    const __nv_bfloat16 *qn = a.q_nope + (static_cast<size_t>(row) * a.Hq + h) * a.nope;
    for (int l = threadIdx.x; l < a.L; l += blockDim.x) {
        float s = 0.0f;
        for (int d = 0; d < a.nope; ++d)
            s += __bfloat162float(qn[d]) * __bfloat162float(a.w_uk[(static_cast<size_t>(h) * a.nope + d) * a.L + l]);
        qs[l] = s * a.scale;
    }
    for (int i = threadIdx.x; i < kLatentRope; i += blockDim.x)
        qs[a.L + i] = __bfloat162float(a.q_rope[(static_cast<size_t>(row) * a.Hq + h) * kLatentRope + i]) * a.scale;
    __syncthreads();
    const int W = a.L + kLatentRope;
    float m = -INFINITY, l_sum = 0.0f, o[kLatentMaxDim / 32] = {};
    for (int t = warp; t < limit; t += kRowWarps) {
        const int blk = a.table[static_cast<size_t>(b) * a.max_blocks + t / TTS_BLOCK_TOKENS];
        if (blk < 0 || blk >= a.num_blocks) {
            if (lane == 0) flag_error(a.err, TTS_ERRBIT_BLOCK_ID);
            continue;
        }
        const __nv_bfloat16 *kv = a.pool + (static_cast<size_t>(blk) * TTS_BLOCK_TOKENS + t % TTS_BLOCK_TOKENS) * W;
        float s = 0.0f;
        for (int i = lane; i < W; i += 32) s += qs[i] * __bfloat162float(kv[i]);
#pragma unroll
        for (int k = 16; k > 0; k >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, k);
        const float m2 = fmaxf(m, s);
        const float f = m == -INFINITY ? 0.0f : expf(m - m2), p = expf(s - m2);
        l_sum = l_sum * f + p;
#pragma unroll
        for (int i = 0; i < kLatentMaxDim / 32; ++i)
            if (lane + 32 * i < a.L) o[i] = o[i] * f + p * __bfloat162float(kv[lane + 32 * i]);
        m = m2;
    }
    if (lane == 0) {
        ml[warp][0] = m;
        ml[warp][1] = l_sum;
    }
    for (int i = 0; i < kLatentMaxDim / 32; ++i)
        if (lane + 32 * i < a.L) os[warp][lane + 32 * i] = o[i];
    __syncthreads();
    float M = -INFINITY, S = 0.0f;
    for (int w = 0; w < kRowWarps; ++w) M = fmaxf(M, ml[w][0]);
    for (int w = 0; w < kRowWarps; ++w) S += ml[w][0] == -INFINITY ? 0.0f : ml[w][1] * expf(ml[w][0] - M);
    __syncthreads();
    for (int l = threadIdx.x; l < a.L; l += blockDim.x) {
        float x = 0.0f;
        for (int w = 0; w < kRowWarps; ++w) x += ml[w][0] == -INFINITY ? 0.0f : os[w][l] * expf(ml[w][0] - M);
        qs[l] = S == 0.0f ? 0.0f : x / S;
    }
    __syncthreads();
    for (int i = warp; i < a.v; i += kRowWarps) {
        float s = 0.0f;
        for (int l = lane; l < a.L; l += 32)
            s += qs[l] * __bfloat162float(a.w_uv[(static_cast<size_t>(h) * a.v + i) * a.L + l]);
#pragma unroll
        for (int k = 16; k > 0; k >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, k);
        if (lane == 0) out[i] = __float2bfloat16_rn(s);
    }
}

}  // namespace tts
