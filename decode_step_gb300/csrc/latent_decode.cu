// Decode attention over the latent cache (absorbed form).
#include <cmath>

#include "latent_common.cuh"
#include "latent_rows.cuh"
#include "tts_internal.h"

namespace tts {
namespace {

bool decode_shape_ok(int B, int q_len, int Hq, int L, int nope, int v, int max_ctx) {
    return B >= 0 && q_len >= 1 && Hq >= 1 && static_cast<long>(q_len) * Hq <= 1024 && L >= 64 && L <= kLatentMaxDim &&
           L % 64 == 0 && latent_head_dim_ok(nope) && latent_head_dim_ok(v) && max_ctx >= 1 &&
           static_cast<long>(B) * q_len <= (1 << 20);
}

}  // namespace
}  // namespace tts

extern "C" size_t tts_latent_decode_attn_workspace_size(int32_t B, int32_t q_len, int32_t num_q_heads,
                                                        int32_t latent_dim, int32_t nope_dim, int32_t v_dim,
                                                        int32_t max_ctx_len) {
    if (!tts::decode_shape_ok(B, q_len, num_q_heads, latent_dim, nope_dim, v_dim, max_ctx_len)) return 0;
    return 256;
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
    if (!decode_shape_ok(B, q_len, num_q_heads, cache->latent_dim, nope_dim, v_dim, max_ctx_len))
        return TTS_ERR_UNSUPPORTED;
    if (!aligned16(d_q_nope) || !aligned16(d_q_rope) || !aligned16(d_w_uk) || !aligned16(d_w_uv) || !aligned16(d_out))
        return TTS_ERR_INVALID;
    if (B == 0) return TTS_OK;
    if (!d_ws || !aligned16(d_ws) ||
        ws_bytes < tts_latent_decode_attn_workspace_size(B, q_len, num_q_heads, cache->latent_dim, nope_dim, v_dim,
                                                         max_ctx_len))
        return TTS_ERR_WORKSPACE;
    using bf = const __nv_bfloat16 *;
    const LatentRowsArgs a{d_block_table, max_blocks_per_seq, cache->num_blocks, d_ctx_lens, max_ctx_len, B, q_len,
                           num_q_heads, cache->latent_dim, nope_dim, v_dim, nullptr, B * q_len, scale, causal,
                           static_cast<bf>(cache->pool), static_cast<bf>(d_q_nope), static_cast<bf>(d_q_rope),
                           static_cast<bf>(d_w_uk), static_cast<bf>(d_w_uv), static_cast<__nv_bfloat16 *>(d_out), d_err};
    return launch_kernel(latent_rows_kernel, dim3(B * q_len, num_q_heads), dim3(kRowWarps * 32), 0,
                         {static_cast<cudaStream_t>(stream), false}, a);
}
