// Shared by the latent-cache kernels: limits, argument checks and launching
// (sm_103a).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "tts_common.cuh"
#include "tts_decode.h"
#include "tts_internal.h"

namespace tts {

constexpr int kLatentRope = 64;        // rotary values of a query or key
constexpr int kLatentMaxDim = 512;
constexpr int kLatentMaxHeads = 1024;

inline int check_latent_cache(const tts_latent_cache *cache, const int32_t *d_block_table, int32_t max_blocks) {
    if (!cache || !cache->pool || !d_block_table) return TTS_ERR_INVALID;
    if (cache->num_blocks < 1 || max_blocks < 1 || max_blocks > (1 << 20)) return TTS_ERR_INVALID;
    if (cache->num_blocks > 0x7FFFFFFF / TTS_BLOCK_TOKENS) return TTS_ERR_UNSUPPORTED;  // token rows are 32-bit
    if (cache->block_size != TTS_BLOCK_TOKENS || cache->dtype != TTS_BF16 || cache->rope_dim != kLatentRope ||
        cache->latent_dim < 64 || cache->latent_dim > kLatentMaxDim || cache->latent_dim % 64 != 0)
        return TTS_ERR_UNSUPPORTED;
    return aligned16(cache->pool) ? TTS_OK : TTS_ERR_INVALID;
}

inline bool latent_head_dim_ok(int d) { return d == 64 || d == 128; }

// Dynamic shared memory of a kernel that has static shared memory too: the two
// together pass the 48 KB that need no leave before the dynamic part does.
template <typename... P>
inline bool allow_smem(void (*kernel)(P...), int bytes) {
    constexpr int kNoLeave = 48 * 1024;
    return ensure_dynamic_smem(reinterpret_cast<const void *>(kernel), bytes > kNoLeave ? bytes : kNoLeave + 16);
}

// Launches a kernel, as a programmatic dependent of the one before it if o.pdl.
template <typename... P, typename... A>
inline int launch_kernel(void (*kernel)(P...), dim3 grid, dim3 block, size_t smem, LaunchOpts o, A &&...args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = o.stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = o.pdl ? 1 : 0;
    if (cudaLaunchKernelEx(&cfg, kernel, static_cast<A &&>(args)...) != cudaSuccess) {
        cudaGetLastError();
        return TTS_ERR_CUDA;
    }
    return TTS_OK;
}

// Lane 0's value, which the compiler then knows to be the same in every lane:
// code that depends on nothing else is compiled for the uniform registers that
// tcgen05 and TMA instructions take their operands from.
__device__ __forceinline__ int uniform(int x) { return __shfl_sync(0xFFFFFFFFu, x, 0); }

// Bounded mbarrier wait by a whole converged warp, with one answer.  Waits for
// copies and products that are on their way when a kernel gives up take the
// default limit.
__device__ __forceinline__ bool warp_wait(const uint64_t *bar, uint32_t parity, long long limit = kWaitLimitCycles) {
    const bool ok = __all_sync(0xFFFFFFFFu, mbar_wait(smem_addr(bar), parity, limit));
    __syncwarp();
    return ok;
}
// Whether the phase has completed, without waiting (try_wait may suspend the
// thread for a while).
__device__ __forceinline__ bool mbar_test(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.b32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0;
}
// The same for several barriers at once.  A wait that succeeds at once still
// takes about 0.1 us, in which a warp that issues MMAs leaves the tensor core
// idle: every barrier is polled before the first answer is used.
template <int kMax>
struct WarpWaits {
    uint32_t bar[kMax], parity[kMax];  // bar 0: none
    __device__ __forceinline__ void set(int i, const uint64_t *b, uint32_t par) {
        bar[i] = smem_addr(b);
        parity[i] = par;
    }
    __device__ __forceinline__ void none(int i) { bar[i] = 0; }
    __device__ __forceinline__ bool poll() const {
        bool ok[kMax];
#pragma unroll
        for (int i = 0; i < kMax; ++i) ok[i] = bar[i] == 0 || mbar_test(bar[i], parity[i]);
        bool all = true;
#pragma unroll
        for (int i = 0; i < kMax; ++i) all = all && ok[i];
        all = __all_sync(0xFFFFFFFFu, all);
        __syncwarp();
        return all;
    }
    // Polls until all have: where a wait stands in a chain of short steps
    // (try_wait's wake-up takes a few hundred cycles).
    __device__ __forceinline__ bool spin(long long limit = kWaitLimitCycles) const {
        if (poll()) return true;
        const long long t0 = clock64();
        for (uint32_t n = 1;; ++n) {
            if (poll()) return true;
            // (one answer for the warp: the lanes' clocks may differ)
            if ((n & 63u) == 0 && __any_sync(0xFFFFFFFFu, clock64() - t0 > limit)) return false;
        }
    }
    __device__ __forceinline__ bool wait(long long limit = kWaitLimitCycles) const {
        if (poll()) return true;
        bool all = true;
#pragma unroll
        for (int i = 0; i < kMax; ++i) all = all && (bar[i] == 0 || mbar_wait(bar[i], parity[i], limit));
        all = __all_sync(0xFFFFFFFFu, all);
        __syncwarp();
        return all;
    }
};

}  // namespace tts
