// Page moves of a paged cache: whole blocks copied to others, streams forked
// from others (full blocks shared, the last, partly filled one copied), and a
// pool's blocks moved together with the tables that name them.  The same
// kernels serve the KV cache (two pools, or the one of FP8 records) and the
// latent cache: a block is so many 16-byte words of each pool.
//
// No arithmetic: the floor is 2 x the moved blocks' bytes at the copy
// bandwidth.  A block (32 KB of keys and 32 KB of values for 8 heads of 128)
// is cut into pieces of 8 KB, so that a few blocks already occupy every SM and
// many are spread evenly.  Closing up 4,096 blocks of which 2,700 are in use (916
// move, 120 MB of traffic): 20.6 us, 5.8 TB/s; 48 blocks copied 2.6 us and 64 forks
// 3.3 us, a launch and one chain of dependent reads.
#include "tts_common.cuh"
#include "tts_internal.h"

namespace tts {
namespace {

constexpr int kThreads = 256;
constexpr int kPieceWords = 512;  // 16-byte words a piece
constexpr int kAhead = 4;         // words a thread has on their way
constexpr int kCtasPerSm = 8;

struct Pools {
    uint4 *pool[2];
    int words;       // of a block, a pool
    int pieces;      // of a block, all pools
    int num_blocks;
};

struct Piece {
    const uint4 *from;
    uint4 *to;
    int words;
};
__device__ __forceinline__ Piece piece_of(const Pools &p, int from, int to, int piece) {
    const int each = (p.words + kPieceWords - 1) / kPieceWords;
    const int which = piece >= each;
    const int at = (piece - which * each) * kPieceWords;
    uint4 *base = p.pool[which] + at;
    return {base + static_cast<size_t>(from) * p.words, base + static_cast<size_t>(to) * p.words,
            min(kPieceWords, p.words - at)};
}
__device__ __forceinline__ bool in_pool(const Pools &p, int id) { return id >= 0 && id < p.num_blocks; }

// Copies `count` pieces of a list in shared memory, by every thread of the CTA;
// words of several pieces are on their way at once.
__device__ __forceinline__ void copy_pieces(const Piece *list, int count) {
    const int all = count * kPieceWords;
    for (int i0 = threadIdx.x; i0 < all; i0 += kAhead * kThreads) {
        uint4 x[kAhead];
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            const int i = i0 + u * kThreads;
            if (i < all) {
                const Piece &p = list[i / kPieceWords];
                if (i % kPieceWords < p.words) x[u] = p.from[i % kPieceWords];
            }
        }
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            const int i = i0 + u * kThreads;
            if (i < all) {
                const Piece &p = list[i / kPieceWords];
                if (i % kPieceWords < p.words) p.to[i % kPieceWords] = x[u];
            }
        }
    }
}

// Each thread's piece, if it has one, joins the CTA's list; then all are copied.
__device__ __forceinline__ void gather_and_copy(Piece *list, int *count, bool has, const Piece &piece) {
    if (threadIdx.x == 0) *count = 0;
    __syncthreads();
    if (has) list[atomicAdd(count, 1)] = piece;
    __syncthreads();
    copy_pieces(list, *count);
    __syncthreads();
}

// ------------------------------------------------------------------- copies

__global__ void __launch_bounds__(kThreads)
copy_blocks_kernel(const Pools pools, const int32_t *src, const int32_t *dst, long long units, int32_t *err) {
    __shared__ Piece list[kThreads];
    __shared__ int count;
    pdl_wait_prerequisites();
    pdl_allow_dependents();
    // unit = (pair, piece); CTA c takes units c, c + grid, ...
    const long long grid = gridDim.x, round = grid * kThreads;
    for (long long base = blockIdx.x; base < units; base += round) {
        const long long unit = base + threadIdx.x * grid;
        bool has = unit < units;
        Piece piece{};
        if (has) {
            const int i = static_cast<int>(unit / pools.pieces), part = static_cast<int>(unit % pools.pieces);
            const int from = src[i], to = dst[i];
            has = in_pool(pools, from) && in_pool(pools, to);
            if (has) piece = piece_of(pools, from, to, part);
            else flag_error(err, TTS_ERRBIT_BLOCK_ID);
        }
        gather_and_copy(list, &count, has, piece);
    }
}

// -------------------------------------------------------------------- forks

// CTA (fork, piece) copies a piece of the last block; piece 0's also writes
// the child's row.  (Parents are only read: no child of the call is one.)
__global__ void __launch_bounds__(kThreads)
fork_kernel(const Pools pools, int32_t *table, int max_blocks, int32_t *ctx_lens, int B, const int32_t *parent,
            const int32_t *child, const int32_t *new_block, int32_t *err) {
    __shared__ Piece piece;
    pdl_wait_prerequisites();
    const int f = blockIdx.x / pools.pieces, part = blockIdx.x % pools.pieces;
    const int p = parent[f], c = child[f];
    const bool first = part == 0 && threadIdx.x == 0;
    if (p < 0 || p >= B || c < 0 || c >= B || p == c) {
        if (first) flag_error(err, TTS_ERRBIT_STREAM);
        return;
    }
    const int ctx = ctx_lens[p];
    if (ctx < 0 || ctx > max_blocks * TTS_BLOCK_TOKENS) {
        if (first) flag_error(err, TTS_ERRBIT_CTX_LEN);
        return;
    }
    const int full = ctx / TTS_BLOCK_TOKENS;
    const int32_t *from_row = table + static_cast<size_t>(p) * max_blocks;
    int32_t *to_row = table + static_cast<size_t>(c) * max_blocks;
    if (ctx % TTS_BLOCK_TOKENS) {
        const int from = from_row[full], to = new_block[f];
        if (!in_pool(pools, from) || !in_pool(pools, to)) {
            if (first) flag_error(err, TTS_ERRBIT_BLOCK_ID);
            return;
        }
        if (threadIdx.x == 0) piece = piece_of(pools, from, to, part);
        __syncthreads();
        copy_pieces(&piece, 1);
        if (first) to_row[full] = to;
    }
    if (part == 0) {
        for (int i = threadIdx.x; i < full; i += kThreads) to_row[i] = from_row[i];
        if (threadIdx.x == 0) ctx_lens[c] = ctx;
    }
}

// --------------------------------------------------------------- compaction

// Where block `id` goes (itself: it stays), or -1: its destination is outside
// the pool or moves itself.
__device__ __forceinline__ int destination(const int32_t *map, int num_blocks, int id) {
    const int to = map[id];
    if (to == id) return id;
    if (to < 0 || to >= num_blocks || map[to] != to) return -1;
    return to;
}

__global__ void __launch_bounds__(kThreads)
compact_kernel(const Pools pools, const int32_t *map, int32_t *table, long long entries, int32_t *err) {
    __shared__ Piece list[kThreads];
    __shared__ int count;
    pdl_wait_prerequisites();
    const long long grid = gridDim.x, round = grid * kThreads;
    for (long long i = static_cast<long long>(blockIdx.x) * kThreads + threadIdx.x; i < entries; i += round) {
        const int id = table[i];
        if (!in_pool(pools, id)) continue;
        const int to = destination(map, pools.num_blocks, id);
        if (to >= 0 && to != id) table[i] = to;
    }
    // unit = (block, piece), CTA c takes units c, c + grid, ...: neighbouring
    // blocks (the ones that move are the last) go to different CTAs
    const long long units = static_cast<long long>(pools.num_blocks) * pools.pieces;
    for (long long base = blockIdx.x; base < units; base += round) {
        const long long unit = base + threadIdx.x * grid;
        bool has = unit < units;
        Piece piece{};
        if (has) {
            const int id = static_cast<int>(unit / pools.pieces), part = static_cast<int>(unit % pools.pieces);
            const int to = destination(map, pools.num_blocks, id);
            if (to < 0 && part == 0) flag_error(err, TTS_ERRBIT_BLOCK_ID);
            has = to >= 0 && to != id;
            if (has) piece = piece_of(pools, id, to, part);
        }
        gather_and_copy(list, &count, has, piece);
    }
}

// --------------------------------------------------------------------- host

// The pools of a cache as blocks of 16-byte words.
int pools_of(const tts_kv_cache *cache, Pools *out) {
    if (!cache || !cache->k_pool || cache->num_blocks < 1 || cache->num_kv_heads < 1 || cache->head_dim < 1)
        return TTS_ERR_INVALID;
    if (cache->block_size != TTS_BLOCK_TOKENS) return TTS_ERR_UNSUPPORTED;
    const bool fp8 = cache->dtype == TTS_FP8_E4M3;
    if (!fp8 && cache->dtype != TTS_F32 && cache->dtype != TTS_BF16) return TTS_ERR_UNSUPPORTED;
    if (fp8 && cache->head_dim != 128) return TTS_ERR_UNSUPPORTED;
    if (!fp8 && !cache->v_pool) return TTS_ERR_INVALID;
    const int64_t tile = fp8 ? 4224 : static_cast<int64_t>(TTS_BLOCK_TOKENS) * cache->head_dim * (cache->dtype == TTS_F32 ? 4 : 2);
    const int64_t bytes = tile * cache->num_kv_heads;
    if (bytes % 16 != 0 || bytes > (int64_t(1) << 30)) return TTS_ERR_UNSUPPORTED;
    if (!aligned16(cache->k_pool) || (!fp8 && !aligned16(cache->v_pool))) return TTS_ERR_INVALID;
    out->pool[0] = static_cast<uint4 *>(cache->k_pool);
    out->pool[1] = fp8 ? nullptr : static_cast<uint4 *>(cache->v_pool);
    out->words = static_cast<int>(bytes / 16);
    out->pieces = (out->words + kPieceWords - 1) / kPieceWords * (fp8 ? 1 : 2);
    out->num_blocks = cache->num_blocks;
    return TTS_OK;
}

int pools_of(const tts_latent_cache *cache, Pools *out) {
    if (!cache || !cache->pool || cache->num_blocks < 1) return TTS_ERR_INVALID;
    if (cache->block_size != TTS_BLOCK_TOKENS || cache->dtype != TTS_BF16 || cache->rope_dim != 64 ||
        cache->latent_dim < 64 || cache->latent_dim > 512 || cache->latent_dim % 64 != 0)
        return TTS_ERR_UNSUPPORTED;
    if (!aligned16(cache->pool)) return TTS_ERR_INVALID;
    out->pool[0] = static_cast<uint4 *>(cache->pool);
    out->pool[1] = nullptr;
    out->words = TTS_BLOCK_TOKENS * (cache->latent_dim + cache->rope_dim) / 8;
    out->pieces = (out->words + kPieceWords - 1) / kPieceWords;
    out->num_blocks = cache->num_blocks;
    return TTS_OK;
}

template <typename... P, typename... A>
int launch_pages(void (*kernel)(P...), long long ctas, void *stream, A &&...args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(ctas));
    cfg.blockDim = dim3(kThreads);
    cfg.stream = static_cast<cudaStream_t>(stream);
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = thread_pdl() ? 1 : 0;
    if (cudaLaunchKernelEx(&cfg, kernel, static_cast<A &&>(args)...) != cudaSuccess) {
        cudaGetLastError();
        return TTS_ERR_CUDA;
    }
    return TTS_OK;
}

template <typename Cache>
int copy_blocks(const Cache *cache, const int32_t *d_src, const int32_t *d_dst, int32_t n, int32_t *d_err, void *stream) {
    Pools pools;
    const int st = pools_of(cache, &pools);
    if (st != TTS_OK) return st;
    if (n < 0 || (n > 0 && (!d_src || !d_dst))) return TTS_ERR_INVALID;
    if (n == 0) return TTS_OK;
    const long long units = static_cast<long long>(n) * pools.pieces, most = static_cast<long long>(kCtasPerSm) * sm_count();
    return launch_pages(copy_blocks_kernel, units < most || most == 0 ? units : most, stream, pools, d_src, d_dst, units, d_err);
}

template <typename Cache>
int fork_streams(const Cache *cache, int32_t *d_block_table, int32_t max_blocks_per_seq, int32_t *d_ctx_lens, int32_t B,
                 const int32_t *d_parent, const int32_t *d_child, const int32_t *d_new_block, int32_t n, int32_t *d_err,
                 void *stream) {
    Pools pools;
    const int st = pools_of(cache, &pools);
    if (st != TTS_OK) return st;
    if (!d_block_table || !d_ctx_lens || B < 0 || max_blocks_per_seq < 1 || max_blocks_per_seq > (1 << 20) || n < 0 ||
        (n > 0 && (!d_parent || !d_child || !d_new_block)))
        return TTS_ERR_INVALID;
    if (n == 0) return TTS_OK;
    const long long ctas = static_cast<long long>(n) * pools.pieces;
    if (ctas > 0x7FFFFFFF) return TTS_ERR_UNSUPPORTED;
    return launch_pages(fork_kernel, ctas, stream, pools, d_block_table, max_blocks_per_seq, d_ctx_lens, B, d_parent,
                        d_child, d_new_block, d_err);
}

template <typename Cache>
int compact_blocks(const Cache *cache, const int32_t *d_map, int32_t *d_block_table, int32_t max_blocks_per_seq, int32_t B,
                   int32_t *d_err, void *stream) {
    Pools pools;
    const int st = pools_of(cache, &pools);
    if (st != TTS_OK) return st;
    if (!d_map || B < 0 || max_blocks_per_seq < 1 || max_blocks_per_seq > (1 << 20) || (B > 0 && !d_block_table))
        return TTS_ERR_INVALID;
    const long long entries = static_cast<long long>(B) * max_blocks_per_seq;
    const long long units = static_cast<long long>(pools.num_blocks) * pools.pieces;
    const long long most = static_cast<long long>(kCtasPerSm) * sm_count();
    return launch_pages(compact_kernel, units < most || most == 0 ? units : most, stream, pools, d_map, d_block_table,
                        entries, d_err);
}

}  // namespace
}  // namespace tts

extern "C" int tts_kv_copy_blocks(const tts_kv_cache *cache, const int32_t *d_src, const int32_t *d_dst, int32_t n,
                                  int32_t *d_err, void *stream) {
    return tts::copy_blocks(cache, d_src, d_dst, n, d_err, stream);
}
extern "C" int tts_latent_copy_blocks(const tts_latent_cache *cache, const int32_t *d_src, const int32_t *d_dst, int32_t n,
                                      int32_t *d_err, void *stream) {
    return tts::copy_blocks(cache, d_src, d_dst, n, d_err, stream);
}
extern "C" int tts_kv_fork(const tts_kv_cache *cache, int32_t *d_block_table, int32_t max_blocks_per_seq,
                           int32_t *d_ctx_lens, int32_t B, const int32_t *d_parent, const int32_t *d_child,
                           const int32_t *d_new_block, int32_t n, int32_t *d_err, void *stream) {
    return tts::fork_streams(cache, d_block_table, max_blocks_per_seq, d_ctx_lens, B, d_parent, d_child, d_new_block, n,
                             d_err, stream);
}
extern "C" int tts_latent_fork(const tts_latent_cache *cache, int32_t *d_block_table, int32_t max_blocks_per_seq,
                               int32_t *d_ctx_lens, int32_t B, const int32_t *d_parent, const int32_t *d_child,
                               const int32_t *d_new_block, int32_t n, int32_t *d_err, void *stream) {
    return tts::fork_streams(cache, d_block_table, max_blocks_per_seq, d_ctx_lens, B, d_parent, d_child, d_new_block, n,
                             d_err, stream);
}
extern "C" int tts_kv_compact(const tts_kv_cache *cache, const int32_t *d_map, int32_t *d_block_table,
                              int32_t max_blocks_per_seq, int32_t B, int32_t *d_err, void *stream) {
    return tts::compact_blocks(cache, d_map, d_block_table, max_blocks_per_seq, B, d_err, stream);
}
extern "C" int tts_latent_compact(const tts_latent_cache *cache, const int32_t *d_map, int32_t *d_block_table,
                                  int32_t max_blocks_per_seq, int32_t B, int32_t *d_err, void *stream) {
    return tts::compact_blocks(cache, d_map, d_block_table, max_blocks_per_seq, B, d_err, stream);
}
