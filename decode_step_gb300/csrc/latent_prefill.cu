// Attention of whole prompts over the latent cache.
#include <cmath>

#include "latent_common.cuh"
#include "latent_rows.cuh"
#include "tts_internal.h"

namespace tts {
namespace {

bool prefill_shape_ok(int B, int T, int Hq, int L, int nope, int v, int max_total) {
    return B >= 0 && T >= 0 && Hq >= 1 && Hq <= kLatentMaxHeads && L >= 64 && L <= kLatentMaxDim && L % 64 == 0 &&
           latent_head_dim_ok(nope) && latent_head_dim_ok(v) && max_total >= 0;
}

}  // namespace
}  // namespace tts

extern "C" size_t tts_latent_prefill_attn_workspace_size(int32_t B, int32_t num_rows, int32_t num_q_heads,
                                                         int32_t latent_dim, int32_t nope_dim, int32_t v_dim,
                                                         int32_t max_total_ctx) {
    if (!tts::prefill_shape_ok(B, num_rows, num_q_heads, latent_dim, nope_dim, v_dim, max_total_ctx)) return 0;
    return 256;
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
    if (!prefill_shape_ok(B, num_rows, num_q_heads, cache->latent_dim, nope_dim, v_dim, max_total_ctx))
        return TTS_ERR_UNSUPPORTED;
    if (!aligned16(d_q_nope) || !aligned16(d_q_rope) || !aligned16(d_w_uk) || !aligned16(d_w_uv) || !aligned16(d_out))
        return TTS_ERR_INVALID;
    if (B == 0 || num_rows == 0) return TTS_OK;
    if (!d_ws || !aligned16(d_ws) ||
        ws_bytes < tts_latent_prefill_attn_workspace_size(B, num_rows, num_q_heads, cache->latent_dim, nope_dim, v_dim,
                                                          max_total_ctx))
        return TTS_ERR_WORKSPACE;
    using bf = const __nv_bfloat16 *;
    const LatentRowsArgs a{d_block_table, max_blocks_per_seq, cache->num_blocks, d_ctx_lens, max_total_ctx, B, 0,
                           num_q_heads, cache->latent_dim, nope_dim, v_dim, d_row_start, num_rows, scale, 1,
                           static_cast<bf>(cache->pool), static_cast<bf>(d_q_nope), static_cast<bf>(d_q_rope),
                           static_cast<bf>(d_w_uk), static_cast<bf>(d_w_uv), static_cast<__nv_bfloat16 *>(d_out), d_err};
    return launch_kernel(latent_rows_kernel, dim3(num_rows, num_q_heads), dim3(kRowWarps * 32), 0,
                         {static_cast<cudaStream_t>(stream), false}, a);
}
