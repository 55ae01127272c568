// Attention of chunks of new tokens (prompts, or pieces of them) over the paged
// KV cache, causal, with an optional sliding window and sinks:
//   out[r][h] = sum_t softmax_t(scale * q[r][h] . k_t) v_t
// over the tokens t <= p (p the row's position) with t < sinks or t > p - window.
//
// Work.  A query tile is two halves of 128 matrix rows; a half holds 128 /
// group tokens with all `group` query heads of one KV head (so that a KV tile is
// read once for the group).  A segment is a query tile and a KV head; its work is
// the 80-token tiles of the context that some row sees.  The flat list of all
// segments, each kPartCost and then its tiles long, is split into equal contiguous
// ranges, one a CTA: long and short segments, prompts and few rows over a long
// context all spread over the SMs alike (without the kPartCost the CTAs with many
// short segments ran 40% longer).  A range boundary that falls within kSnap tiles of
// a segment's end moves there; a segment that is split all the same is published in
// parts (m, l, o), and the last CTA to finish one (an atomic ticket, never a wait)
// joins them in the order of the CTAs, so that results do not depend on who is
// last; more than kJoinHere parts are left to a second kernel.  Every CTA finds its
// range by itself from the streams' lengths.
//
// A CTA: two softmax warpgroups, one a half (or, where one half has no rows and the
// context is long, both on the one half's, tile by tile in turns); an MMA issuer a
// half (a commit or a wait takes its warp about 190 cycles: one issuer was the
// bound); a producer of keys and queries and one of values (TMA through the table, a
// box of 16 tokens x 64 dimensions of keys, 16 x 128 of values; FP8: bulk copies of
// codes and scales).  bf16: two guards, warps that look at the values of the tiles that not
// every row sees whole (below).  FP8: four warps that turn codes into f16, which is
// exact, where the MMAs want them; the keys' scales go to the scores, the values' to
// the weights.
//
// A tile.  S = Q K^T is a tcgen05 MMA of 128 x 80 x 128 from shared memory, O += P V
// one of 128 x 128 x 80 with P from tensor memory.  80 tokens, because 80 columns of
// scores, 40 of weights and 128 of output fit a half's 256 columns side by side: the
// next scores need only that the last ones were read.  (With 128 tokens P lies in S's
// columns, and scores, softmax and product are one chain of 3,300 cycles a tile.)  P
// is bf16 (FP8: f16, times the value's scale); the softmax sum is of the fp32 weights
// before that rounding (2^-8 of a weight at most; f16 2^-11).  The running maximum
// moves only when a score passes it by more than prompt_slack.
//
// What bounds it.  Long prompts (8,191 rows after 700, 16 query and 8 KV heads): 248
// us, 1.30 PFLOP/s, 0.68 of a dense product's measured rate; the softmax warps take
// about 2,000 cycles a tile for both halves, the MMAs 1,435 of them (the first, with
// both operands in shared memory, 417 a half, bound by their 128 bytes a cycle; the
// second 320).  61 rows after 65,472: 58 us, 4.6 TB/s.  333 rows: 18 us, latency.
// FP8 takes twice the bf16 time (8,191 rows 520 us) with no unit near its limit (4,095
// rows: issue slots 45%, matrix unit 24%, shared memory's pipe 30%): chains of waits
// between converters, MMAs and softmax, and in short contexts O is scaled in nearly
// every tile, since the maximum moves with any score that passes it.  A CTA
// does not have 16 softmax warps (two threads a row: 386 us, spills and twice the
// reads of scores).
//
// Values that are not finite.  A weight of zero times NaN is NaN, so a token that
// a row does not see must not meet it in the matrix product.  Tiles that every
// row sees need no care.  In the others the guards (FP8: the converters) clear such
// values in shared memory, and the rows that do see them get them at the end.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cfloat>
#include <cmath>

#include "latent_common.cuh"
#include "tcgen05.cuh"
#include "tts_common.cuh"
#include "tts_internal.h"

namespace tts {
namespace {

constexpr unsigned kFull = 0xFFFFFFFFu;
constexpr int kDim = 128;
constexpr int kRows = 128;                  // matrix rows of a half
constexpr int kBlocks = 5, kTile = kBlocks * TTS_BLOCK_TOKENS;  // blocks and tokens a tile
constexpr int kQueryBytes = kRows * 128;    // [128 rows][64 values], 128-byte swizzle; two a half
constexpr int kChunkBytes = kTile * 128;    // [80 tokens][64 values]
constexpr int kSlotBytes = 2 * kChunkBytes; // a tile of keys, or of values block by block: [5][2][16 tokens][64 values]
constexpr int kBlockBytes = 4096;           // a block's values of a head
__host__ __device__ constexpr int prompt_slots(bool fp8) { return fp8 ? 2 : 4; }  // tiles of keys, and of values, in the ring
constexpr int kRawSlots = 3, kRawBytes = kBlocks * 2048;       // FP8: tiles of codes on their way, of keys and of values
constexpr int kRecordBytes = 4224, kScaleStages = 8, kScaleBytes = kBlocks * 128;
// FP8: the weights are 2^8 times what they are else, so that times their values'
// scales they stay clear of f16's subnormals, as tts_decode_attn has them; so is
// their sum
constexpr float kFp8Log2 = 8.0f;
// Tensor memory: a half's S, its P (two weights a column), and both halves' O
constexpr int kS = 0, kP = kTile, kHalf = 128, kO = 256;
static_assert(kP + kTile / 2 <= kHalf);
// Two softmax warpgroups; two issuers, two guards, two producers; FP8: four
// converters instead of the guards
__host__ __device__ constexpr int prompt_threads(bool fp8) { return fp8 ? 512 : 448; }
constexpr int kMostThreads = 512;
constexpr int kFewTiles = 128;              // query tiles that one warp looks at
constexpr int kMaxStreams = 4096;           // (their lengths are staged in shared memory)
constexpr int kSnap = 2;                    // tiles
constexpr int kPartCost = 2;                // what a segment costs beside its tiles, in tiles
constexpr int kMinTiles = 6;                // tiles a CTA at least, where there are more CTAs than segments
constexpr float kLog2e = 1.4426950408889634f;
// Running maximum before any token (log2 units): no finite score is below it.
constexpr float kNoScore = -FLT_MAX;
// Maxima whose exponents are taken by another way: half a step of fp32 is 2^-4 from here on.
__device__ __forceinline__ bool large_score(float m) { return fabsf(m) > 1 << 20 && fabsf(m) < FLT_MAX; }
// In the place of a part's maximum: there is no such part.  (One without weights, all
// its scores -inf, has kNoScore, and may have values that are not finite.)
constexpr float kNoPart = -INFINITY;
// Scores may pass it by this much before it moves (log2 units); in FP8 weights stay
// at 1 at most, so that with a scale below 256 they are in f16's range.
__host__ __device__ constexpr float prompt_slack(bool fp8) { return fp8 ? 0.0f : 8.0f; }
constexpr int kPartFloats = kRows * kDim + 2 * kRows;  // o, m, l of a half
// Tiles of a part from which on half 1 stays half a step behind, its exponentials
// while half 0 waits and loads; short parts are a chain of latencies, which that would
// lengthen.
constexpr int kPairTiles = 10;
// One half's rows use both halves, tile by tile, in segments of at least so many
// tiles that are spread over more than two ranges: where a few rows meet a long
// context the chain of one tile is the bound (4 streams of 17 rows after 4,000: 23
// us, else 36).  Others gain nothing and would have parts to join (32 streams: 101
// us, with turns 114; after 1,000 tokens 42 and 58).
constexpr int kTakeTurns = 24;
constexpr int kSoloTiles = 10;
static_assert(kSoloTiles < kTakeTurns && (kSoloTiles - 2 * kSnap) / (kPartCost + 1) + 2 <= 4);
constexpr int kJoinHere = 4;                // parts that the last CTA joins; more are left to the second kernel

struct PromptArgs {
    const int32_t *table;
    int max_blocks, num_blocks;
    const int32_t *ctx_lens;
    const int32_t *row_start;
    int B, num_rows, Hq, Hkv, group, tokens;  // tokens: of a half
    int window, sinks;                        // window 0: none
    float scale_log2;
    const uint8_t *k_pool, *v_pool;           // FP8: the records, and none
    __nv_bfloat16 *out;
    float *part;          // [CTA][first, later part][half] partial results
    int32_t *tickets;     // [CTA][half] of a segment that begins in it
    int4 *jobs;           // [CTA][half] segments that the second kernel joins: rows (0: none), first row, KV head, parts
    int ctas, max_tiles;  // query tiles at most
    int few;              // B <= 32 and few query tiles: one warp finds the ranges
    int zero_row;         // a row behind the pool: reads as zeros
    int32_t *err;
    long long wait_limit; // SM clock cycles per bounded wait
    int stall;            // test support: the first keys expect 16 bytes that never come
};

// ---------------------------------------------------------------- the work

// Rows and context of stream b; false: out of range.
__device__ __forceinline__ bool prompt_stream(const PromptArgs &a, int b, int *first, int *n, int *ctx) {
    *first = __ldcg(a.row_start + b);
    const int end = __ldcg(a.row_start + b + 1);
    *ctx = __ldcg(a.ctx_lens + b);
    *n = 0;
    if (*first == end) return true;
    if (*first < 0 || end < *first || end > a.num_rows) return false;
    if (*ctx < end - *first || *ctx > a.max_blocks * TTS_BLOCK_TOKENS) return false;
    *n = end - *first;
    return true;
}
__device__ __forceinline__ int query_tiles(const PromptArgs &a, int n) { return (n + 2 * a.tokens - 1) / (2 * a.tokens); }

// What a query tile sees: the tokens below `high`, of which those from `low` on
// (the first row's window) and the sinks; in tiles: the first `head`
// ones and, `skip` further on, the others.
struct Span {
    int low, high, tiles, head, skip;
};
__device__ __forceinline__ Span span_of(const PromptArgs &a, int n, int ctx, int i) {
    Span s;
    const int r0 = i * 2 * a.tokens;
    s.high = ctx - n + min(n, r0 + 2 * a.tokens);
    s.low = a.window ? max(0, ctx - n + r0 + 1 - a.window) : 0;
    s.head = (min(a.sinks, s.high) + kTile - 1) / kTile;
    s.skip = max(0, s.low / kTile - s.head);
    s.tiles = (s.high + kTile - 1) / kTile - s.skip;
    return s;
}

// Equal ranges of the flat list, each segment kPartCost and then its tiles long
// (T in all, W CTAs, T >= W).
struct Ranges {
    int q, rem;
    __device__ __forceinline__ int start(int c) const { return c * q + min(c, rem); }
    __device__ __forceinline__ int of(int t) const {
        const int big = rem * (q + 1);
        return t < big ? t / (q + 1) : rem + (t - big) / q;
    }
};

// Whether some row does not see some token of the tile (`first`, `last`: tokens up
// to the first and the last row's own).
__device__ __forceinline__ bool tile_edge(const PromptArgs &a, int t0, int first, int last) {
    return !(t0 + kTile <= first && (!a.window || t0 + kTile <= a.sinks || t0 >= last - a.window));
}

// How a part's tiles are worked on: by the first half, by both (both have rows), or
// by the two halves in turns (for the first one's rows).
constexpr int kBoth = 1, kTurns = 2;

// Walks a CTA's range: part after part of a segment, tile after tile.
struct Walk {
    int left;                  // tiles of the range left, this one among them
    int b, i, g, k;            // stream, query tile, KV head, tile of the segment
    int s0;                    // the segment's place in the flat list
    int first, n, ctx;         // of the stream
    Span span;
    __device__ __forceinline__ int r0(const PromptArgs &a) const { return i * 2 * a.tokens; }
    __device__ __forceinline__ bool two(const PromptArgs &a) const { return r0(a) + a.tokens < n; }
    __device__ __forceinline__ int tiles() const { return min(left, span.tiles - k); }  // of the part, from its first one on
    __device__ __forceinline__ int mode(const PromptArgs &a, int range) const {
        return two(a) ? kBoth : span.tiles >= kTakeTurns && span.tiles > 2 * range ? kTurns : 0;
    }
    __device__ __forceinline__ void seek(const PromptArgs &a) {  // b: the next stream that has rows
        for (; b < a.B; ++b) {
            const bool good = prompt_stream(a, b, &first, &n, &ctx);
            n = uniform(good ? n : 0);
            ctx = uniform(ctx);
            first = uniform(first);
            if (n) return;
        }
    }
    __device__ __forceinline__ void settle(const PromptArgs &a) {  // k may be behind the segment's last tile
        if (k < span.tiles) return;
        k = 0;
        s0 += kPartCost + span.tiles;
        if (++g < a.Hkv) return;
        g = 0;
        if (++i == query_tiles(a, n)) {
            i = 0;
            ++b;
            seek(a);
        }
        span = span_of(a, n, ctx, i);
    }
    __device__ __forceinline__ void advance(const PromptArgs &a) {
        ++k;
        if (--left > 0 && k == span.tiles) settle(a);
    }
};

// A place in a ring of slots and its barriers' parity.
template <int kSlots>
struct Place {
    uint32_t slot = 0, phase = 0;
    bool again = false;  // the ring has been through once
    __device__ __forceinline__ void next() {
        if (++slot == kSlots) {
            slot = 0;
            phase ^= 1;
            again = true;
        }
    }
    // Waits for what the slots were last filled with.
    __device__ __forceinline__ void drain(const uint64_t *full) {
        for (int i = again ? kSlots : slot; i > 0; --i) {
            if (slot == 0) {
                slot = kSlots;
                phase ^= 1;
            }
            --slot;
            warp_wait(&full[slot], phase);
        }
    }
};

// What the producer tells the other warps: of a part (a segment's tiles in this
// CTA), and of a tile that a half works on.
struct PartInfo {
    int first, n, ctx, b;         // of the stream
    int r0, g, number, tiles;     // first row of the query tile, KV head, from 1, tiles of the part
    int k, head, skip;            // first tile of the part; Span
    int high, shares, more, mode; // first CTA of the segment, CTAs that follow
};
// The same of a part's values, by their producer, which may be ahead of the keys'.
struct ValueInfo {
    int tiles, first, high, k, head, skip;  // first, high: tokens up to the first and the last row's own
};
struct __align__(8) TileInfo {
    int flags, t0;  // bits 0-4: blocks in the pool; then its part's note, its slot and its scales' stage; first token
};
constexpr int kAllBlocks = (1 << kBlocks) - 1, kPair = 0x80, kMasked = 0x100, kFresh = 0x200, kLast = 0x400, kEnd = 0x800, kPartShift = 12, kSlotShift = 16, kStageShift = 18;
// (The producers are at most six tiles ahead of a half that works, and of one that
// has no part in a tile but is still at the end of an earlier part.)
constexpr int kInfos = 8;
constexpr int kLookups = 6;  // tiles whose blocks a warp looks up at once
static_assert(kLookups * kBlocks <= 32);

struct PromptShared {
    uint64_t k_full[4], k_empty[4], v_full[4], v_empty[4], checked[4], behind[4];
    uint64_t raw_full[2][kRawSlots], raw_empty[2][kRawSlots], q_raw[2];  // FP8: of keys, values; the queries before f16
    uint64_t q_full[2], q_empty, s_full[2], s_empty[2], p_full[2], o_done[2], o_empty[2], stored[2], told[2], done[2];
    __align__(16) PartInfo parts[kInfos];
    ValueInfo values[kInfos];
    TileInfo tiles[2][kInfos];  // by use of the half
    int4 jobs[2];
    int v_valid[kInfos];   // FP8: blocks of a tile of values in the pool
    uint32_t tmem;
    int odd[8];            // number of the part whose tiles held values that are not finite, by number % 8
    int last[2];           // whether the half's part was the last one
    long long scan[2][kMostThreads / 32];
    int b, i, g, k, s0, first, n, ctx, from, to, q, rem, refused;
};
// Shared memory: the queries, the ring of keys, of values, in FP8 the codes of
// either and the scales, and PromptShared.
template <bool kFp8>
struct PromptSmem {
    static constexpr int keys = 4 * kQueryBytes, values = keys + prompt_slots(kFp8) * kSlotBytes;
    static constexpr int raw = values + prompt_slots(kFp8) * kSlotBytes, scales = raw + (kFp8 ? 2 * kRawSlots * kRawBytes : 0);
    static constexpr int shared = scales + (kFp8 ? kScaleStages * kScaleBytes : 0);
    static constexpr int total = shared + static_cast<int>(sizeof(PromptShared));
    static_assert(total <= 227 * 1024);
    static_assert(kMaxStreams * 16 <= scales - keys);
};

// Zeros in the rows of the refused streams (rare), by every thread of the grid.
__device__ __noinline__ void zero_refused(const PromptArgs &a) {
    const size_t width = static_cast<size_t>(a.Hq) * kDim / 8;  // 16-byte pieces a row
    const size_t me = static_cast<size_t>(blockIdx.x) * blockDim.x + threadIdx.x, all = static_cast<size_t>(gridDim.x) * blockDim.x;
    for (int b = 0; b < a.B; ++b) {
        int first, n, ctx;
        if (prompt_stream(a, b, &first, &n, &ctx)) continue;
        if (me == 0) flag_error(a.err, TTS_ERRBIT_CTX_LEN);
        const int from = max(0, first), to = min(a.num_rows, __ldcg(a.row_start + b + 1));
        if (from >= to) continue;
        for (size_t i = from * width + me; i < to * width; i += all) reinterpret_cast<uint4 *>(a.out)[i] = make_uint4(0, 0, 0, 0);
    }
}

// Sum over the threads before this one, and over all.
template <int kThreads>
__device__ __forceinline__ long long scan_before(long long mine, long long *warps, long long *all) {
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    long long incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
        const long long x = __shfl_up_sync(kFull, incl, o);
        if (lane >= o) incl += x;
    }
    if (lane == 31) warps[warp] = incl;
    __syncthreads();
    long long before = incl - mine, total = 0;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) {
        if (w < warp) before += warps[w];
        total += warps[w];
    }
    *all = total;
    return before;
}

// What the CTA does, of T in all and of so many segments, into sh.q, rem and, where
// it has no segment to look up, sh.from and to.  False: the CTA has nothing to do.
__device__ __forceinline__ bool split_work(const PromptArgs &a, PromptShared &sh, int T, int segments, bool write, int *x0, int *x1) {
    const int W = min(min(a.ctas, T), max((T + kMinTiles - 1) / kMinTiles, segments)), c = blockIdx.x;
    const Ranges ranges{W ? T / W : 0, W ? T - T / W * W : 0};
    if (write) {
        sh.q = ranges.q;
        sh.rem = ranges.rem;
        if (c >= W) sh.from = sh.to = 0;
        else if (c + 1 == W) sh.to = T - kPartCost * segments;
    }
    *x0 = ranges.start(c);
    *x1 = ranges.start(c + 1);
    return c < W;
}
// Where the range's ends x lie in query tile t (the i-th of stream b), whose
// segments of n tiles begin at `at` in the list.
__device__ __forceinline__ void look_up(const PromptArgs &a, PromptShared &sh, int x0, int x1, int at, int b, int t, int i, int n,
                                        const int4 &stream) {
    const int each = kPartCost + n;
#pragma unroll 1
    for (int which = 0; which < 2; ++which) {
        const int x = which ? x1 : x0;
        if (x < at || x >= at + each * a.Hkv) continue;
        const int g = (x - at) / each, s0 = at + g * each;
        int k = x - s0 - kPartCost;
        if (k <= kSnap) k = 0;
        else if (n - k <= kSnap) k = n;
        const int before = s0 - kPartCost * (t * a.Hkv + g) + k;  // tiles
        if (which) {
            sh.to = before;
        } else {
            sh.from = before;
            sh.b = b;
            sh.i = i;
            sh.g = g;
            sh.k = k;
            sh.s0 = s0;
            sh.first = stream.x;
            sh.n = stream.y;
            sh.ctx = stream.z;
        }
    }
}

// find_range by one warp, without a barrier, for up to 32 streams (a lane each)
// and few query tiles: what a small call waits for before its first copy.
__device__ __forceinline__ void find_range_few(const PromptArgs &a, PromptShared &sh) {
    const int lane = threadIdx.x % 32;
    int first = 0, n = 0, ctx = 0;
    const bool good = lane >= a.B || prompt_stream(a, lane, &first, &n, &ctx);
    const int refused = __any_sync(kFull, !good), mine = query_tiles(a, n);
    int upto = mine;
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
        const int x = __shfl_up_sync(kFull, upto, o);
        if (lane >= o) upto += x;
    }
    int tiles = __shfl_sync(kFull, upto, 31);
    const int from = upto - mine;  // the stream's first query tile
    const bool apart = tiles >= 0 && tiles <= a.max_tiles;  // (else the streams' rows overlap)
    if (!apart) {
        if (blockIdx.x == 0 && lane == 0) flag_error(a.err, TTS_ERRBIT_CTX_LEN);
        tiles = 0;
    }
    if (lane == 0) sh.refused = refused;
    int total = 0, x0 = 0, x1 = 0;
    bool work = true;
#pragma unroll 1
    for (int pass = 0; work && pass < 2; ++pass) {
        int at = 0;
#pragma unroll 1
        for (int t0 = 0; t0 < tiles; t0 += 32) {
            const int t = t0 + lane;
            int b = 0;  // the last stream that begins at or before tile t
#pragma unroll
            for (int step = 16; step > 0; step /= 2)
                if (__shfl_sync(kFull, from, b + step) <= t) b += step;
            const int4 s = make_int4(__shfl_sync(kFull, first, b), __shfl_sync(kFull, n, b), __shfl_sync(kFull, ctx, b),
                                     __shfl_sync(kFull, from, b));
            const int here = t < tiles ? span_of(a, s.y, s.z, t - s.w).tiles : -kPartCost;
            int incl = kPartCost + here;
#pragma unroll
            for (int o = 1; o < 32; o *= 2) {
                const int x = __shfl_up_sync(kFull, incl, o);
                if (lane >= o) incl += x;
            }
            if (pass && t < tiles) look_up(a, sh, x0, x1, (at + incl - kPartCost - here) * a.Hkv, b, t, t - s.w, here, s);
            at += __shfl_sync(kFull, incl, 31);
        }
        total = at;
        if (!pass) work = split_work(a, sh, total * a.Hkv, tiles * a.Hkv, lane == 0, &x0, &x1);
    }
}

// Finds the CTA's range: sh.from, to (tiles before its ends), its first stream,
// query tile, KV head, tile (sh.b, i, g, k, s0, first, n, ctx), and sh.q, rem.
// `streams`: room for kMaxStreams.  Every thread calls it; a barrier has to follow.
template <int kThreads>
__device__ __forceinline__ void find_range(const PromptArgs &a, PromptShared &sh, int4 *streams) {
    const int per = (a.B + kThreads - 1) / kThreads;
    const int b0 = min(a.B, static_cast<int>(threadIdx.x) * per), b1 = min(a.B, b0 + per);
    long long mine = 0;
    bool refused = false;
    for (int b = b0; b < b1; ++b) {
        int first, n, ctx;
        refused = !prompt_stream(a, b, &first, &n, &ctx) || refused;
        mine += query_tiles(a, n);
        streams[b] = make_int4(first, n, ctx, 0);
    }
    long long all_tiles;
    long long at = scan_before<kThreads>(mine, sh.scan[0], &all_tiles);
    // (more than these only if the streams' rows overlap)
    const bool apart = all_tiles <= a.max_tiles;
    const int tiles = apart ? static_cast<int>(all_tiles) : 0;
    if (!apart && blockIdx.x == 0 && threadIdx.x == 0) flag_error(a.err, TTS_ERRBIT_CTX_LEN);
    for (int b = b0; b < b1; ++b) {
        streams[b].w = static_cast<int>(at);
        at += query_tiles(a, streams[b].y);
    }
    if (__syncthreads_or(refused)) zero_refused(a);
    // the tiles of this thread's share of the query tiles
    const int each = (tiles + kThreads - 1) / kThreads;
    const int t0 = min(tiles, static_cast<int>(threadIdx.x) * each), t1 = min(tiles, t0 + each);
    int start_b = 0;
    if (t0 < t1) {
        int hi = a.B;  // streams[start_b].w <= t0 < streams[hi].w
        while (hi - start_b > 1) {
            const int mid = (start_b + hi) / 2;
            if (streams[mid].w <= t0) start_b = mid;
            else hi = mid;
        }
    }
    auto each_tile = [&](auto &&f) {
        int b = start_b;
        int4 s = t0 < t1 ? streams[b] : make_int4(0, 0, 0, 0);
#pragma unroll 1
        for (int t = t0; t < t1; ++t) {
            while (b + 1 < a.B && streams[b + 1].w <= t) s = streams[++b];
            f(b, t, t - s.w, span_of(a, s.y, s.z, t - s.w).tiles);
        }
    };
    long long sum = 0, total;
    each_tile([&](int, int, int, int n) { sum += kPartCost + n; });
    const long long before = scan_before<kThreads>(sum, sh.scan[1], &total) * a.Hkv;
    const int T = static_cast<int>(total) * a.Hkv;  // (below 2^30, as the host has seen to)
    int x0, x1;
    if (split_work(a, sh, T, tiles * a.Hkv, threadIdx.x == 0, &x0, &x1)) {
        int at_tile = static_cast<int>(before);
        each_tile([&](int b, int t, int i, int n) {
            look_up(a, sh, x0, x1, at_tile, b, t, i, n, streams[b]);
            at_tile += (kPartCost + n) * a.Hkv;
        });
    }
}

// CTAs that share a segment: its first part's and how many follow.
struct Shares {
    int first, more;
};
__device__ __forceinline__ Shares shares_of(const Ranges &r, int s0, int tiles) {
    if (tiles <= 2 * kSnap) return {0, 0};
    s0 += kPartCost;
    const int lo = r.of(s0 + kSnap) + 1, hi = r.of(s0 + tiles - kSnap - 1);  // boundaries inside that stay
    return {lo - 1, max(0, hi - lo + 1)};
}

// A block's rows, both halves (make_tma_rows_in_halves_bf16), by a converged warp's leader.
__device__ __forceinline__ void tma_load_rows_by(uint32_t leader, uint32_t dst, const CUtensorMap *map, int y, uint32_t bar) {
    asm volatile(
        "{\n\t.reg .pred q;\n\t"
        "setp.ne.b32 q, %5, 0;\n\t"
        "@q cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %2}], [%4];\n\t}" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(0), "r"(y), "r"(bar), "r"(leader)
        : "memory");
}

// ------------------------------------------------------------- the softmax

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    const __nv_bfloat162 p = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&p);
}
// Four E4M3 codes as two f16 pairs: exact.
__device__ __forceinline__ void codes_to_f16(uint32_t w, uint32_t &lo, uint32_t &hi) {
    asm("{\n\t.reg .b16 l, h;\n\t"
        "mov.b32 {l, h}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, l;\n\t"
        "cvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(w));
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
    const __half2 p = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&p);
}
__device__ __forceinline__ uint32_t bf16_to_f16(uint32_t w) { return pack_f16(bf16_lo(w), bf16_hi(w)); }
__device__ __forceinline__ void sts128(uint32_t at, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
}
// Codes of 0x7F or 0xFF (not a number) of a word become 0.
__device__ __forceinline__ void drop_odd(uint32_t &w) {
    const uint32_t bad = ((w & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u;  // 0x80 in such a byte
    w &= ~((bad >> 7) * 0xFFu);
}
// Operand whose 8 x 16-byte pieces are contiguous (no swizzle), the contraction
// side's next eight values `lead` bytes on, the other side's next eight rows `stride`.
__device__ __forceinline__ uint64_t plain_desc(uint32_t addr, uint32_t lead, uint32_t stride) {
    return static_cast<uint64_t>((addr & 0x3FFFFu) >> 4) | (static_cast<uint64_t>(lead >> 4) << 16) |
           (static_cast<uint64_t>(stride >> 4) << 32) | (static_cast<uint64_t>(1) << 46);
}
// Two fp32 operations an instruction, and the largest of three.
__device__ __forceinline__ uint64_t pack2(float lo, float hi) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ void unpack2(uint64_t x, float &lo, float &hi) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(x));
}
__device__ __forceinline__ uint64_t fma2(uint64_t x, uint64_t y, uint64_t z) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(x), "l"(y), "l"(z));
    return r;
}
__device__ __forceinline__ void times2(uint32_t &x, uint32_t &y, float a, float b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(pack2(__uint_as_float(x), __uint_as_float(y))), "l"(pack2(a, b)));
    float lo, hi;
    unpack2(r, lo, hi);
    x = __float_as_uint(lo);
    y = __float_as_uint(hi);
}
__device__ __forceinline__ uint64_t add2(uint64_t x, uint64_t y) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(x), "l"(y));
    return r;
}
__device__ __forceinline__ float max3(float x, float y, float z) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(x), "f"(y), "f"(z));
    return r;
}
// Bits 15 and 31: whether the halves' exponents (bf16) are all ones.
__device__ __forceinline__ uint32_t ones(uint32_t w) { return (w & 0x7F807F80u) + 0x00800080u; }
// warp_wait where the phase has mostly completed.
__device__ __forceinline__ bool quick_wait(const uint64_t *bar, uint32_t parity, long long limit) {
    return __all_sync(kFull, mbar_test(smem_addr(bar), parity)) || warp_wait(bar, parity, limit);
}
// Bits of the tokens of word w (32 tokens from `base` on) before token t.
__device__ __forceinline__ uint32_t bits_before(int t, int base) {
    const int n = t - base;
    return n <= 0 ? 0u : n >= 32 ? kFull : (1u << n) - 1u;
}

// Values of this row's tokens that are not finite, of 32 dimensions from d on,
// added up in o (rare): those of the tiles that the guards cleared.
template <bool kFp8>
__device__ __noinline__ void find_odd(const PromptArgs &a, const PartInfo &part, int step, int j, int limit, int d, float *o) {
    const int first_limit = part.ctx - part.n + part.r0 + 1;
    for (; j < part.tiles; j += step) {
        const int k = part.k + j, t0 = (k < part.head ? k : k + part.skip) * kTile;
        if (!tile_edge(a, t0, first_limit, part.high)) continue;
        for (int t = t0; t < t0 + kTile && t < limit; ++t) {
            if (a.window && t >= a.sinks && t < limit - a.window) continue;
            const int id = __ldcg(a.table + static_cast<size_t>(part.b) * a.max_blocks + t / TTS_BLOCK_TOKENS);
            if (id < 0 || id >= a.num_blocks) continue;
            const size_t tile = static_cast<size_t>(id) * a.Hkv + part.g;
            const int slot = t % TTS_BLOCK_TOKENS;
#pragma unroll 1
            for (int e = 0; e < 32; ++e) {
                if constexpr (kFp8) {
                    const uint8_t code = a.k_pool[tile * kRecordBytes + 2048 + 16 * (d + e) + 4 * (slot % 8 / 2) + slot % 2 + 2 * (slot / 8)];
                    if ((code & 0x7F) == 0x7F) o[e] = __uint_as_float(0x7FC00000u);
                } else {
                    const uint32_t w = reinterpret_cast<const uint16_t *>(a.v_pool)[(tile * TTS_BLOCK_TOKENS + slot) * kDim + d + e];
                    if ((w & 0x7F80u) == 0x7F80u) o[e] += __uint_as_float(w << 16);
                }
            }
        }
    }
}
template <bool kFp8>
__device__ __forceinline__ void add_odd(const PromptArgs &a, const PartInfo &part, int step, int j, int limit, int d, float *f) {
    float o[32];
    for (int i = 0; i < 32; ++i) o[i] = 0.0f;
    find_odd<kFp8>(a, part, step, j, limit, d, o);
#pragma unroll
    for (int i = 0; i < 32; ++i) f[i] += o[i];
}

// o / l as 32 bf16 values.
__device__ __forceinline__ void store_row(__nv_bfloat16 *out, const float *f, float inv) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
        reinterpret_cast<uint4 *>(out)[i] =
            make_uint4(pack_bf16(f[8 * i] * inv, f[8 * i + 1] * inv), pack_bf16(f[8 * i + 2] * inv, f[8 * i + 3] * inv),
                       pack_bf16(f[8 * i + 4] * inv, f[8 * i + 5] * inv), pack_bf16(f[8 * i + 6] * inv, f[8 * i + 7] * inv));
}
__device__ __forceinline__ float inverse(float l) { return l == 0.0f ? 0.0f : 1.0f / l; }  // no token left: zeros

// Slot of a part: CTA, whether the segment begins in it, half.  [32][128 rows][4]
// floats o, then m and l of the rows.  (A CTA's parts of split segments are its
// first one, of a segment that began in an earlier CTA, and its last one.)
__device__ __forceinline__ float *part_slot(float *parts, int cta, bool begins, int half) {
    return parts + static_cast<size_t>((cta * 2 + (begins ? 0 : 1)) * 2 + half) * kPartFloats;
}
// Part i of a segment whose first CTA is `first`: one a CTA (of half s), or with
// both halves' in turns two.
__device__ __forceinline__ float *segment_part(float *parts, int first, int i, bool turns, int s) {
    const int c = turns ? i / 2 : i;
    return part_slot(parts, first + c, c == 0, turns ? i % 2 : s);
}

template <bool kFp8>
__global__ void __launch_bounds__(prompt_threads(kFp8), 1)
prompt_attn_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
                   const __grid_constant__ CUtensorMap map_v, const PromptArgs a) {
    constexpr int kThreads = prompt_threads(kFp8), kSlots = prompt_slots(kFp8);
    using Smem = PromptSmem<kFp8>;
    extern __shared__ __align__(1024) uint8_t raw[];
    const uint32_t q_base = smem_addr(raw), k_base = q_base + Smem::keys, v_base = q_base + Smem::values;
    PromptShared &sh = *reinterpret_cast<PromptShared *>(raw + Smem::shared);
    const int warp = uniform(threadIdx.x / 32), lane = threadIdx.x % 32;
    if (warp == 11 && lane == 0) {
        for (int i = 0; i < kSlots; ++i) {
            mbar_init(smem_addr(&sh.k_full[i]), kFp8 ? 2 : 1);
            mbar_init(smem_addr(&sh.k_empty[i]), 2);  // (a half each, by who is done with the slot)
            mbar_init(smem_addr(&sh.v_full[i]), kFp8 ? 2 : 1);
            mbar_init(smem_addr(&sh.v_empty[i]), 2);
            mbar_init(smem_addr(&sh.checked[i]), 2);
            mbar_init(smem_addr(&sh.behind[i]), 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_addr(&sh.q_full[i]), kFp8 ? 4 : 1);
            mbar_init(smem_addr(&sh.q_raw[i]), 1);
            for (int j = 0; j < kRawSlots; ++j) {
                mbar_init(smem_addr(&sh.raw_full[i][j]), 1);
                mbar_init(smem_addr(&sh.raw_empty[i][j]), 2);
            }
            mbar_init(smem_addr(&sh.s_full[i]), 1);
            mbar_init(smem_addr(&sh.s_empty[i]), 4);
            mbar_init(smem_addr(&sh.p_full[i]), 4);
            mbar_init(smem_addr(&sh.o_done[i]), 1);
            mbar_init(smem_addr(&sh.o_empty[i]), 4);
            mbar_init(smem_addr(&sh.stored[i]), 4);
            mbar_init(smem_addr(&sh.told[i]), 1);
        }
        mbar_init(smem_addr(&sh.q_empty), 2);
        mbar_init(smem_addr(&sh.done[0]), 1);
        mbar_init(smem_addr(&sh.done[1]), 1);
        for (int i = 0; i < 8; ++i) sh.odd[i] = 0;
        sh.jobs[0] = sh.jobs[1] = make_int4(0, 0, 0, 0);
        fence_mbar_init();
    }
    if (warp == 8 && lane == 0) {
        prefetch_tensormap(&map_q);
        if constexpr (!kFp8) {
            prefetch_tensormap(&map_k);
            prefetch_tensormap(&map_v);
        }
    }
    pdl_wait_prerequisites();
    // (tensor memory only after the wait: the kernel before may be one that
    // still has to allocate its own)
    if (warp == 12) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_addr(&sh.tmem))
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    if (a.few) {
        if (warp == 13) find_range_few(a, sh);
    } else {
        find_range<kThreads>(a, sh, reinterpret_cast<int4 *>(raw + Smem::keys));
        // (the staged lengths make way for copies)
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (a.few && sh.refused) zero_refused(a);
    pdl_allow_dependents();
    const uint32_t tmem = uniform(sh.tmem);
    const Ranges ranges{uniform(sh.q), uniform(sh.rem)};
    const int all_tiles = uniform(sh.to - sh.from);
    bool ok = true;
    if (all_tiles > 0) {
        if (warp >= 8) {
            if (warp == 8 || warp == 13) {
                // ---- producers, of keys and of values.  Lane l looks up block l % 5 of the l / 5-th of the next six tiles
                const bool for_keys = warp == 8;
                const uint32_t leader = elect_leader();
                uint32_t part = 0, q_count[2] = {0, 0};
                Place<kFp8 ? kRawSlots : kSlots> at;
                uint64_t *full = kFp8 ? sh.raw_full[!for_keys] : for_keys ? sh.k_full : sh.v_full;
                uint64_t *empty = kFp8 ? sh.raw_empty[!for_keys] : for_keys ? sh.k_empty : sh.v_empty;
                uint32_t tile = 0;  // of the CTA
                // ids of the tiles from the part's j-th on (kNoBlock: no token of it is seen)
                constexpr int kNoBlock = -0x7FFFFFFF;
                auto lookup = [&](const Walk &w, int tiles, int j) {
                    j += lane / kBlocks;
                    const int k = w.k + j, t = ((k < w.span.head ? k : k + w.span.skip) * kBlocks + lane % kBlocks) * TTS_BLOCK_TOKENS;
                    // (blocks without a token that some row sees may hold anything)
                    if (lane >= kLookups * kBlocks || j >= tiles || t >= w.span.high ||
                        (t >= a.sinks && t + TTS_BLOCK_TOKENS <= w.span.low))
                        return kNoBlock;
                    return __ldcg(a.table + static_cast<size_t>(w.b) * a.max_blocks + t / TTS_BLOCK_TOKENS);
                };
                Walk walk;
                walk.left = all_tiles;
                walk.b = uniform(sh.b);
                walk.i = uniform(sh.i);
                walk.g = uniform(sh.g);
                walk.k = uniform(sh.k);
                walk.s0 = uniform(sh.s0);
                walk.first = uniform(sh.first);
                walk.n = uniform(sh.n);
                walk.ctx = uniform(sh.ctx);
                walk.span = span_of(a, walk.n, walk.ctx, walk.i);
                walk.settle(a);
                int uses[2] = {0, 0};
                int tiles = walk.tiles(), id = lookup(walk, tiles, 0);
                for (bool begun = false; ok && walk.left > 0;) {
                    const int mode = walk.mode(a, ranges.q), note = part % kInfos, r0 = walk.r0(a), before = walk.ctx - walk.n;
                    if (for_keys && lane == 0) {
                        const Shares shares = shares_of(ranges, walk.s0, walk.span.tiles);
                        PartInfo &p = sh.parts[note];
                        p.first = walk.first; p.n = walk.n; p.ctx = walk.ctx; p.b = walk.b;
                        p.r0 = r0; p.g = walk.g; p.number = part + 1; p.tiles = tiles;
                        p.k = walk.k; p.head = walk.span.head; p.skip = walk.span.skip;
                        p.high = walk.span.high; p.shares = shares.first; p.more = shares.more; p.mode = mode;
                    }
                    if (!for_keys && lane == 0)
                        sh.values[note] = {tiles, before + r0 + 1, walk.span.high, walk.k, walk.span.head, walk.span.skip};
                    Walk next = walk;
                    next.left -= tiles - 1;
                    next.k += tiles - 1;
                    next.advance(a);
                    const int next_tiles = next.left > 0 ? next.tiles() : 0;
                    int ahead = lookup(walk, tiles, kLookups), after = next.left > 0 ? lookup(next, next_tiles, 0) : kNoBlock;
                    // the tiles that every row of a half sees whole begin in [from, to], or up to sinks
                    int whole_from[2], whole_to[2];
#pragma unroll
                    for (int s = 0; s < 2; ++s) {
                        const int row0 = r0 + (mode == kTurns ? 0 : s * a.tokens);
                        whole_from[s] = a.window ? before + min(walk.n, row0 + a.tokens) - a.window : 0;
                        whole_to[s] = before + row0 + 1 - kTile;
                    }
                    const int step = mode == kTurns ? 2 : 1;
                    const bool paired = mode == kBoth && tiles >= kPairTiles;
                    int y = 0, good = 0, from = kLookups * kBlocks;
#pragma unroll 1
                    for (int j = 0; ok && j < tiles; ++j) {
                        from += kBlocks;
                        if (from >= kLookups * kBlocks) {
                            from = 0;
                            if (j) {
                                id = ahead;
                                ahead = lookup(walk, tiles, j + kLookups);
                            }
                            const bool here = id >= 0 && id < a.num_blocks;
                            if (!here && id != kNoBlock) flag_error(a.err, TTS_ERRBIT_BLOCK_ID);
                            y = here ? (id * a.Hkv + walk.g) * TTS_BLOCK_TOKENS : a.zero_row;
                            good = static_cast<int>(__ballot_sync(kFull, here));
                        }
                        if (for_keys) {
                            const int mask = (good >> from) & kAllBlocks;
                            const int k = walk.k + j, t0 = (k < walk.span.head ? k : k + walk.span.skip) * kTile;
                            const int common = mask | (paired ? kPair : 0) | (j < step ? kFresh : 0) |
                                               (j >= tiles - step ? kLast : 0) | note << kPartShift |
                                               static_cast<int>(tile % kSlots) << kSlotShift |
                                               static_cast<int>(tile % kScaleStages) << kStageShift;
#pragma unroll
                            for (int s = 0; s < 2; ++s) {
                                if (mode == kTurns ? s != j % 2 : s == 1 && mode != kBoth) continue;
                                const bool whole = mask == kAllBlocks && t0 <= whole_to[s] &&
                                                   (t0 >= whole_from[s] || t0 + kTile <= a.sinks);
                                if (lane == 0) sh.tiles[s][uses[s] % kInfos] = {common | (whole ? 0 : kMasked), t0};
                                uses[s] += 1;
                            }
                        }
                        int ys[kBlocks];
#pragma unroll
                        for (int i = 0; i < kBlocks; ++i) ys[i] = __shfl_sync(kFull, y, from + i);
                        if (at.again && !quick_wait(&empty[at.slot], at.phase ^ 1, a.wait_limit)) {
                            ok = false;
                            break;
                        }
                        const uint32_t bar = smem_addr(&full[at.slot]), more = a.stall && for_keys && !begun ? 16 : 0;
                        begun = true;
                        if constexpr (kFp8) {
                            // codes (and with the keys' the scales) of the blocks that are in the pool
                            const int here = (good >> from) & kAllBlocks;
                            if (!for_keys && lane == 0) sh.v_valid[tile % kInfos] = here;
                            __syncwarp();
                            mbar_expect_tx_by(leader, bar, __popc(here) * (for_keys ? 2048 + 128 : 2048) + more);
                            const uint32_t to = q_base + Smem::raw + ((for_keys ? 0 : kRawSlots) + at.slot) * kRawBytes;
                            const uint32_t scales = q_base + Smem::scales + tile % kScaleStages * kScaleBytes;
#pragma unroll
                            for (int i = 0; i < kBlocks; ++i)
                                if ((here >> i) & 1 && leader) {
                                    const uint8_t *record = a.k_pool + static_cast<size_t>(ys[i] / TTS_BLOCK_TOKENS) * kRecordBytes;
                                    bulk_load_nohint(to + i * 2048, record + (for_keys ? 0 : 2048), 2048, bar);
                                    if (for_keys) bulk_load_nohint(scales + i * 128, record + 4096, 128, bar);
                                }
                            __syncwarp();
                        } else if (for_keys) {
                            mbar_expect_tx_by(leader, bar, kSlotBytes + more);
                            const uint32_t to = k_base + at.slot * kSlotBytes;
#pragma unroll
                            for (int i = 0; i < 2 * kBlocks; ++i)
                                tma_load_2d_by(leader, to + i / kBlocks * kChunkBytes + i % kBlocks * 2048, &map_k, i / kBlocks * 64,
                                               ys[i % kBlocks], bar);
                        } else {
                            mbar_expect_tx_by(leader, bar, kSlotBytes);
                            const uint32_t to = v_base + at.slot * kSlotBytes;
#pragma unroll
                            for (int i = 0; i < kBlocks; ++i) tma_load_rows_by(leader, to + i * kBlockBytes, &map_v, ys[i], bar);
                        }
                        at.next();
                        ++tile;
                        if (for_keys && j == 0) {
                            // the part's queries
                            ok = part == 0 || warp_wait(&sh.q_empty, (part - 1) & 1, a.wait_limit);
                            if (!ok) break;
                            const int halves = mode == kBoth ? 2 : 1;
                            ++q_count[0];
                            q_count[1] += halves - 1;
                            if (lane == 0)
                                for (int s = 0; s < halves; ++s) {
                                    const uint32_t q_bar = smem_addr(kFp8 ? &sh.q_raw[s] : &sh.q_full[s]);
                                    mbar_arrive_expect_tx(q_bar, 2 * a.tokens * a.group * 128);
                                    for (int c = 0; c < 2; ++c)
                                        asm volatile(
                                            "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes"
                                            " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(q_base + (2 * s + c) * kQueryBytes),
                                            "l"(reinterpret_cast<uint64_t>(&map_q)), "r"(c * 64), "r"(walk.g * a.group),
                                            "r"(walk.first + r0 + s * a.tokens), "r"(q_bar)
                                            : "memory");
                                }
                            __syncwarp();
                        }
                    }
                    ++part;
                    walk = next;
                    tiles = next_tiles;
                    id = after;
                }
                // every copy lands before the CTA ends
                at.drain(full);
                for (uint32_t s = 0; s < 2; ++s)
                    if (q_count[s]) warp_wait(kFp8 ? &sh.q_raw[s] : &sh.q_full[s], (q_count[s] - 1) & 1);
            } else if (warp == 9 || warp == 10) {
                // ---- MMA issuers, one a half: S(j + 1) O(j), or, where the halves take
                // turns, S(j + 2) O(j).  The next scores need only that the last ones were
                // read, so that the softmax warps find theirs when they come.  (A commit or
                // a wait takes the issuing warp about 0.1 us: one warp for both halves was
                // the bound.)  Every slot is waited for and given back by either half,
                // worked on or not: a barrier's parity tells one use from the next, not
                // from the one after.
                const int s = warp - 9;
                const uint32_t leader = elect_leader();
                Place<kSlots> keys, values;  // of the next scores, and outputs
                uint32_t uses = 0, outs = 0, parts = 0, left_parts = 0, both = 0, behind = 0;
                bool go = true;
                const uint32_t d_s = tmem + s * kHalf + kS, d_p = tmem + s * kHalf + kP, d_o = tmem + kO + s * kDim;
                uint64_t queries = 0;
                for (int left = all_tiles, part = 0; go && left > 0; ++part) {
                    // (the producer's notes are there once the part's first keys are)
                    go = quick_wait(&sh.k_full[keys.slot], keys.phase, a.wait_limit);
                    if (!go) break;
                    const volatile PartInfo &info = sh.parts[part % kInfos];
                    const int tiles = uniform(info.tiles), mode = uniform(info.mode);
                    left -= tiles;
                    // the first half's tiles are all, the second's all or none; in turns every other one
                    const int of = mode == kTurns ? 1 + s : s == 0 || mode == kBoth ? 3 : 0;  // bits: even, odd tiles
                    const int lag = mode == kTurns ? 2 : 1;
                    queries = sw128_desc(q_base + (mode == kTurns ? 0 : 2 * s * kQueryBytes));
                    {
                        WarpWaits<2> x;
                        x.set(0, &sh.q_full[0], part & 1);
                        x.none(1);
                        if (s == 1 && mode == kBoth) x.set(1, &sh.q_full[1], both++ & 1);
                        go = x.wait(a.wait_limit);
                    }
                    const bool paired = mode == kBoth && tiles >= kPairTiles;
                    bool fresh = true;
                    if (go && (of == 0 || (of == 2 && tiles == 1)) && lane == 0) mbar_arrive(smem_addr(&sh.q_empty));
#pragma unroll 1
                    for (int j = 0; go && j < tiles + lag; ++j) {
                        if (j < tiles) {
                            const bool work = (of >> (j & 1)) & 1;
                            WarpWaits<2> x;
                            x.set(0, &sh.k_full[keys.slot], keys.phase);
                            x.none(1);
                            if (work && uses) x.set(1, &sh.s_empty[s], (uses - 1) & 1);
                            go = x.spin(a.wait_limit);
                            if (go && s == 1 && paired) {
                                // half 1 stays half a step behind (its exponentials while half
                                // 0 waits and loads, not at the same time)
                                go = quick_wait(&sh.behind[keys.slot], behind >> keys.slot & 1, a.wait_limit);
                                behind ^= 1u << keys.slot;
                            }
                            if (!go) break;
                            if (work) {
                                ++uses;
                                tc_fence_after();
                                const uint64_t k0 = sw128_desc(k_base + keys.slot * kSlotBytes);
#pragma unroll
                                for (int kk = 0; kk < 8; ++kk)  // (descriptors count 16 bytes)
                                    mma_bf16_by(leader, d_s, queries + (kk / 4 * kQueryBytes + kk % 4 * 32) / 16,
                                                k0 + (kk / 4 * kChunkBytes + kk % 4 * 32) / 16,
                                                kFp8 ? mma_idesc_f16(kRows, kTile) : mma_idesc(kRows, kTile), kk != 0);
                                mma_commit_by(leader, smem_addr(&sh.s_full[s]));
                            } else {
                                mbar_arrive_by(leader, smem_addr(&sh.k_empty[keys.slot]));
                            }
                            keys.next();
                        }
                        if (j >= lag) {
                            const bool work = (of >> ((j - lag) & 1)) & 1;
                            WarpWaits<3> x;
                            x.set(0, &sh.v_full[values.slot], values.phase);
                            x.none(1);
                            x.none(2);
                            if constexpr (!kFp8) x.set(1, &sh.checked[values.slot], values.phase);
                            // (also where the half has no part in this one, before it gives a slot back:
                            // its softmax warps read the notes on the part that they are at the end of,
                            // and nothing else holds back the producers, which write over them)
                            if (fresh && left_parts != parts) x.set(2, &sh.o_empty[s], (parts - 1) & 1);
                            go = x.spin(a.wait_limit);
                            if (!go) break;
                            if (fresh) left_parts = parts;
                            if (work) {
                                WarpWaits<1> y;
                                y.set(0, &sh.p_full[s], outs++ & 1);
                                go = y.spin(a.wait_limit);
                                if (!go) break;
                                tc_fence_after();
                                // (FP8: a block's values as [2][128 dimensions][8 tokens])
                                const uint32_t v_at = v_base + values.slot * kSlotBytes;
                                const uint64_t v0 = kFp8 ? plain_desc(v_at, kBlockBytes / 2, 128) : sw128_mn_desc(v_at, kBlockBytes / 2);
#pragma unroll
                                for (int kk = 0; kk < kBlocks; ++kk)
                                    mma_ts_by(leader, d_o, d_p + kk * 8, v0 + kk * kBlockBytes / 16,
                                              kFp8 ? mma_idesc_f16(kRows, kDim) : mma_idesc(kRows, kDim) | kTransposeB,
                                              !fresh || kk != 0);
                                mma_commit_by(leader, smem_addr(&sh.o_done[s]));
                                if (fresh) ++parts;
                                fresh = false;
                            } else {
                                mbar_arrive_by(leader, smem_addr(&sh.v_empty[values.slot]));
                            }
                            values.next();
                        }
                    }
                }
                // nothing more for the softmax warps (their latest scores' barrier is
                // complete: their weights were waited for)
                if (go && lane == 0) {
                    reinterpret_cast<volatile int &>(sh.tiles[s][uses % kInfos].flags) = kEnd;
                    mbar_arrive(smem_addr(&sh.s_full[s]));
                }
                __syncwarp();
                mma_commit_by(leader, smem_addr(&sh.done[s]));
                ok = warp_wait(&sh.done[s], 0) && go;
            } else if constexpr (kFp8) {
                // ---- converters: warps 11 and 12 keys, 14 and 15 values; all the queries.
                // Codes are exact in f16; the scales go to the scores and the weights.
                const bool for_keys = warp < 13;
                const int me = (warp & 1) ^ (for_keys ? 1 : 0);  // of two
                Place<kRawSlots> from;
                Place<kSlots> to;
                uint64_t *empty = for_keys ? sh.k_empty : sh.v_empty, *full = for_keys ? sh.k_full : sh.v_full;
                uint32_t tile = 0, both = 0;
                auto give_up = [&](bool good) { return ok = good; };
                for (int left = all_tiles, part = 0; ok && left > 0; ++part) {
                    if (!give_up(quick_wait(&sh.raw_full[!for_keys][from.slot], from.phase, a.wait_limit))) break;
                    // (the notes on the queries come with them, those on the tiles with the codes)
                    if (!give_up(warp_wait(&sh.q_raw[0], part & 1, a.wait_limit))) break;
                    const int mode = uniform(static_cast<const volatile PartInfo &>(sh.parts[part % kInfos]).mode);
                    int tiles, first = 0, high = 0, k0 = 0, head = 0, skip = 0;
                    if (for_keys) {
                        tiles = uniform(static_cast<const volatile PartInfo &>(sh.parts[part % kInfos]).tiles);
                    } else {
                        const volatile ValueInfo &info = sh.values[part % kInfos];
                        tiles = uniform(info.tiles);
                        first = uniform(info.first);
                        high = uniform(info.high);
                        k0 = uniform(info.k);
                        head = uniform(info.head);
                        skip = uniform(info.skip);
                    }
                    left -= tiles;
                    for (int s = 0; s < (mode == kBoth ? 2 : 1); ++s) {
                        if (s == 1 && !give_up(warp_wait(&sh.q_raw[1], both++ & 1, a.wait_limit))) break;
                        const uint32_t q = q_base + 2 * s * kQueryBytes + ((for_keys ? 0 : 2) + me) * (kQueryBytes / 2) + lane * 16;
#pragma unroll 4
                        for (int e = 0; e < kQueryBytes / 2; e += 512) {
                            const uint4 x = lds128(q + e);
                            sts128(q + e, bf16_to_f16(x.x), bf16_to_f16(x.y), bf16_to_f16(x.z), bf16_to_f16(x.w));
                        }
                        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                        __syncwarp();
                        mbar_arrive_by(lane == 0, smem_addr(&sh.q_full[s]));
                    }
                    if (!ok) break;
#pragma unroll 1
                    for (int j = 0; j < tiles; ++j, ++tile) {
                        if (!give_up(quick_wait(&sh.raw_full[!for_keys][from.slot], from.phase, a.wait_limit))) break;
                        if (to.again && !give_up(quick_wait(&empty[to.slot], to.phase ^ 1, a.wait_limit))) break;
                        const uint32_t codes = q_base + Smem::raw + ((for_keys ? 0 : kRawSlots) + from.slot) * kRawBytes;
                        const uint32_t out = (for_keys ? k_base : v_base) + to.slot * kSlotBytes;
                        if (for_keys) {
                            // 16 codes of a token, 16-byte piece p of row r: dimensions 16 (p ^ r % 8) on.
                            // A lane's rows are eight apart.
                            const int r = me * 4 + lane / 8, c = lane % 8 ^ r;
                            const uint32_t in = codes + (me * 32 + lane) * 16;
                            const uint32_t at = out + c / 4 * kChunkBytes + r * 128, q = c % 4 * 2;
                            const uint32_t lo_at = at + ((q ^ r) << 4), hi_at = at + (((q + 1) ^ r) << 4);
#pragma unroll
                            for (int e = 0; e < kRawBytes; e += 1024) {
                                const uint4 x = lds128(in + e);
                                uint32_t h[8];
                                codes_to_f16(x.x, h[0], h[1]);
                                codes_to_f16(x.y, h[2], h[3]);
                                codes_to_f16(x.z, h[4], h[5]);
                                codes_to_f16(x.w, h[6], h[7]);
                                sts128(lo_at + e, h[0], h[1], h[2], h[3]);
                                sts128(hi_at + e, h[4], h[5], h[6], h[7]);
                            }
                        } else {
                            const int k = k0 + j, t0 = (k < head ? k : k + skip) * kTile;
                            const int valid = *reinterpret_cast<volatile int *>(&sh.v_valid[tile % kInfos]);
                            // (what the rows see alike meets them in the product: only tiles at an edge are
                            // cleared, and stale codes of blocks that are not in the pool)
                            const bool edge = tile_edge(a, t0, first, high);
                            bool odd = false;
                            // a dimension's 16 codes of a block: word i has slots 2i, 2i + 1, 2i + 8, 2i + 9
                            const uint32_t in = codes + (me * 32 + lane) * 16, at = out + (me * 32 + lane) * 16;
                            if (edge || valid != kAllBlocks) {
#pragma unroll 1
                                for (int e = 0; e < kRawBytes; e += 1024) {
                                    const bool held = (valid >> (e / 2048)) & 1;
                                    if (held && !edge) continue;
                                    const uint4 was = lds128(in + e);
                                    uint4 x = was;
                                    drop_odd(x.x);
                                    drop_odd(x.y);
                                    drop_odd(x.z);
                                    drop_odd(x.w);
                                    if (!((was.x ^ x.x) | (was.y ^ x.y) | (was.z ^ x.z) | (was.w ^ x.w))) continue;
                                    sts128(in + e, x.x, x.y, x.z, x.w);
                                    if (!held) continue;
#pragma unroll 1
                                    for (int i = 0; i < 16; ++i) {
                                        const uint32_t w = i / 4 == 0 ? was.x ^ x.x : i / 4 == 1 ? was.y ^ x.y : i / 4 == 2 ? was.z ^ x.z : was.w ^ x.w;
                                        const int b = i % 4, t = t0 + e / 2048 * TTS_BLOCK_TOKENS + i / 4 * 2 + b % 2 + b / 2 * 8;
                                        odd = odd || ((w >> (8 * b)) & 0xFF && t < high && (!a.window || t < a.sinks || t >= first - a.window));
                                    }
                                }
                            }
#pragma unroll
                            for (int e = 0; e < kRawBytes; e += 1024) {
                                const uint4 x = lds128(in + e);
                                uint32_t h[8];
                                codes_to_f16(x.x, h[0], h[4]);
                                codes_to_f16(x.y, h[1], h[5]);
                                codes_to_f16(x.z, h[2], h[6]);
                                codes_to_f16(x.w, h[3], h[7]);
                                const uint32_t to_at = at + e / 2048 * kBlockBytes + e % 2048;
                                sts128(to_at, h[0], h[1], h[2], h[3]);
                                sts128(to_at + kBlockBytes / 2, h[4], h[5], h[6], h[7]);
                            }
                            if (odd) sh.odd[(part + 1) % 8] = part + 1;
                        }
                        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                        __syncwarp();
                        mbar_arrive_by(lane == 0, smem_addr(&full[to.slot]));
                        mbar_arrive_by(lane == 0, smem_addr(&sh.raw_empty[!for_keys][from.slot]));
                        from.next();
                        to.next();
                    }
                }
            } else {
                // ---- guards: values that are not finite leave the tiles that some
                // row does not see whole.  (They keep step with every tile: a barrier's
                // parity tells one use of a slot from the next, not from the one after.)
                Place<kSlots> values;
                for (int left = all_tiles, part = 1; ok && left > 0; ++part) {
                    ok = quick_wait(&sh.v_full[values.slot], values.phase, a.wait_limit);
                    if (!ok) break;
                    const volatile ValueInfo &info = sh.values[(part - 1) % kInfos];
                    const int tiles = uniform(info.tiles), first = uniform(info.first), high = uniform(info.high);
                    const int k0 = uniform(info.k), head = uniform(info.head), skip = uniform(info.skip);
                    left -= tiles;
#pragma unroll 1
                    for (int j = 0; j < tiles; ++j) {
                        ok = quick_wait(&sh.v_full[values.slot], values.phase, a.wait_limit);
                        if (!ok) break;
                        const int k = k0 + j, t0 = (k < head ? k : k + skip) * kTile;
                        if (tile_edge(a, t0, first, high)) {
                            uint8_t *v = raw + Smem::values + values.slot * kSlotBytes;
                            const uint32_t from = smem_addr(v) + ((warp - 11) * 32 + lane) * 16;
                            // bit 15 or 31 of a word: an exponent of ones in that half
                            uint32_t any = 0;
#pragma unroll
                            for (int e = 0; e < kSlotBytes / 1024; ++e) {
                                const uint4 x = lds128(from + e * 1024);
                                any |= ones(x.x) | ones(x.y) | ones(x.z) | ones(x.w);
                            }
                            if (any & 0x80008000u) {  // rare
                                bool odd = false;
#pragma unroll 1
                                for (int e = (warp - 11) * 32 + lane; e < kSlotBytes / 16; e += 64) {
                                    uint16_t *h = reinterpret_cast<uint16_t *>(v + e * 16);
                                    const int t = t0 + e / (kBlockBytes / 16) * TTS_BLOCK_TOKENS + e / 8 % TTS_BLOCK_TOKENS;
#pragma unroll 1
                                    for (int i = 0; i < 8; ++i)
                                        if ((h[i] & 0x7F80u) == 0x7F80u) {
                                            h[i] = 0;
                                            odd = odd || (t < high && (!a.window || t < a.sinks || t >= first - a.window));
                                        }
                                }
                                if (odd) sh.odd[part % 8] = part;
                                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                            }
                            __syncwarp();
                        }
                        if (lane == 0) mbar_arrive(smem_addr(&sh.checked[values.slot]));
                        values.next();
                    }
                }
            }
        } else {
            // ---- softmax warpgroups: thread = matrix row
            const int s = warp / 4, w = warp % 4;
            const int row = w * 32 + lane, token = row / a.group;
            const uint32_t lanes = static_cast<uint32_t>(w * 32) << 16;
            const uint32_t ts = tmem + lanes + s * kHalf + kS, tp = ts - kS + kP, to = tmem + lanes + kO + s * kDim;
            uint32_t joins = 0;  // of this half's parts with others'
            int limit = 0;                  // tokens up to the row's own
            int held = -1;                  // slot of the values of the last use, until it is given back
            float m = kNoScore, l = 0.0f;
            const uint32_t first_lane = lane == 0, first_thread = threadIdx.x % 128 == 0;
            // (a barrier takes more than a hundred cycles to answer: it is asked before
            // other work, and waited for only where the answer was no)
            bool there = false;
            for (uint32_t use = 0;; ++use) {
                if (!__all_sync(kFull, there) && !warp_wait(&sh.s_full[s], use & 1, a.wait_limit)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const volatile TileInfo &info = sh.tiles[s][use % kInfos];
                const int flags = info.flags;
                if (flags & kEnd) break;
                if (flags & kFresh) {
                    const volatile PartInfo *p = &sh.parts[(flags >> kPartShift) % kInfos];
                    const int before = p->ctx - p->n, from = p->r0 + (s == 1 && p->mode == kBoth ? a.tokens : 0);
                    limit = before + min(from + token + 1, min(p->n, from + a.tokens));
                    // (matrix rows that are no query hold whatever is there, and have no say in the
                    // warp's maximum: the others' roundings would depend on it)
                    m = token < a.tokens && from + token < p->n ? kNoScore : INFINITY;
                    l = 0.0f;
                }
                uint32_t x[kTile];
                tmem_ld32_nowait(ts, x);
                tmem_ld32_nowait(ts + 32, x + 32);
                tmem_ld16_nowait(ts + 64, x + 64);
                tmem_wait_ld();
                tc_fence_before();
                __syncwarp();
                mbar_arrive_by(first_lane, smem_addr(&sh.s_empty[s]));
                mbar_arrive_by(first_thread, smem_addr(&sh.k_empty[(flags >> kSlotShift) % 4]));
                mbar_arrive_by(first_thread && (flags & kLast), smem_addr(&sh.q_empty));
                const bool free = use == 0 || mbar_test(smem_addr(&sh.o_done[s]), (use - 1) & 1);
                // FP8: the scales of the tile's keys and values, 16 and 16 a block
                const float *scales = nullptr;
                if constexpr (kFp8) {
                    scales = reinterpret_cast<const float *>(raw + Smem::scales + (flags >> kStageShift) % kScaleStages * kScaleBytes);
#pragma unroll
                    for (int i = 0; i < kTile; i += 4) {
                        const float4 k = *reinterpret_cast<const float4 *>(scales + i / 16 * 32 + i % 16);
                        times2(x[i], x[i + 1], k.x, k.y);
                        times2(x[i + 2], x[i + 3], k.z, k.w);
                    }
                }
                if (flags & kMasked) {
                    const int t0 = info.t0;
#pragma unroll
                    for (int c = 0; c < (kTile + 31) / 32; ++c) {
                        const int base = t0 + 32 * c;
                        uint32_t see = bits_before(limit, base);
                        if (a.window) see &= bits_before(a.sinks, base) | ~bits_before(limit - a.window, base);
                        see &= ((flags >> (2 * c)) & 1 ? 0xFFFFu : 0u) | ((flags >> (2 * c)) & 2 ? 0xFFFF0000u : 0u);
#pragma unroll
                        for (int i = 0; i < 32 && 32 * c + i < kTile; ++i)
                            if (!((see >> i) & 1)) x[32 * c + i] = 0xFF800000u;  // -inf
                    }
                }
                float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                for (int i = 0; i < kTile; i += 2)
                    top[i / 2 % 4] = max3(top[i / 2 % 4], __uint_as_float(x[i]), __uint_as_float(x[i + 1]));
                const float high = fmaxf(max3(top[0], top[1], top[2]), top[3]) * a.scale_log2;
                // (the product before this tile's has to be complete before O is scaled, and
                // before its weights are overwritten: waited for as late as possible)
                if (__any_sync(kFull, high > m + prompt_slack(kFp8))) {
                    if (use && !quick_wait(&sh.o_done[s], (use - 1) & 1, a.wait_limit)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const float now = fmaxf(m, high), f = hw_ex2(m - now);
                    m = now;
                    l *= f;
                    if (!(flags & kFresh))
#pragma unroll 1
                        for (int c = 0; c < kDim; c += 16) {
                            uint32_t o[16];
                            tmem_ld16_nowait(to + c, o);
                            tmem_wait_ld();
#pragma unroll
                            for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
                            tmem_st16(to + c, o);
                        }
                }
                // An exponent is scale * score - m by one fused operation, off by what m was
                // rounded by: one factor for all of the row's weights, which the end divides
                // out.  Where m is so large that the factor would leave the range, the
                // difference to m is taken first, of scores scaled and rounded as m was (a row
                // at a time: other rows keep their bits).  (In the branch above, where m moves,
                // this cost FP8 4%.)
                float minus = kFp8 ? kFp8Log2 - m : -m;
                if (__any_sync(kFull, large_score(m))) {  // rare
                    if (large_score(m)) {
                        const float back = 1.0f / a.scale_log2;
#pragma unroll
                        for (int i = 0; i < kTile; ++i)
                            x[i] = __float_as_uint((__fmul_rn(__uint_as_float(x[i]), a.scale_log2) - m) * back);
                        minus = kFp8 ? kFp8Log2 : 0.0f;
                    }
                }
                uint64_t sum[2] = {0, 0};
                const uint64_t scale2 = pack2(a.scale_log2, a.scale_log2), minus2 = pack2(minus, minus);
                uint32_t weights[kTile / 2];
#pragma unroll
                for (int i = 0; i < kTile / 2; ++i) {
                    float e0, e1;
                    unpack2(fma2(pack2(__uint_as_float(x[2 * i]), __uint_as_float(x[2 * i + 1])), scale2, minus2), e0, e1);
                    e0 = hw_ex2(e0);
                    e1 = hw_ex2(e1);
                    sum[i % 2] = add2(sum[i % 2], pack2(e0, e1));
                    if constexpr (kFp8) {
                        x[2 * i] = __float_as_uint(e0);
                        x[2 * i + 1] = __float_as_uint(e1);
                    } else {
                        weights[i] = pack_bf16(e0, e1);
                    }
                }
                if constexpr (kFp8) {
#pragma unroll
                    for (int i = 0; i < kTile; i += 4) {
                        float4 v = *reinterpret_cast<const float4 *>(scales + i / 16 * 32 + 16 + i % 16);
                        uint32_t *e = x + i;
                        if (flags & kMasked) {  // a token without weight may have any scale
                            v.x = e[0] ? v.x : 0.0f;
                            v.y = e[1] ? v.y : 0.0f;
                            v.z = e[2] ? v.z : 0.0f;
                            v.w = e[3] ? v.w : 0.0f;
                        }
                        times2(e[0], e[1], v.x, v.y);
                        times2(e[2], e[3], v.z, v.w);
                        weights[i / 2] = pack_f16(__uint_as_float(e[0]), __uint_as_float(e[1]));
                        weights[i / 2 + 1] = pack_f16(__uint_as_float(e[2]), __uint_as_float(e[3]));
                    }
                }
                if (!__all_sync(kFull, free) && !warp_wait(&sh.o_done[s], (use - 1) & 1, a.wait_limit)) {
                    ok = false;
                    break;
                }
                there = mbar_test(smem_addr(&sh.s_full[s]), (use + 1) & 1);
                tc_fence_after();
                mbar_arrive_by(first_thread && held >= 0, smem_addr(&sh.v_empty[max(held, 0)]));
                held = (flags >> kSlotShift) % 4;
                tmem_st32(tp, weights);
                tmem_st8(tp + 32, weights + 32);
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                mbar_arrive_by(first_lane, smem_addr(&sh.p_full[s]));
                mbar_arrive_by(threadIdx.x == 0 && (flags & kPair), smem_addr(&sh.behind[(flags >> kSlotShift) % 4]));
                float sum0, sum1;
                unpack2(add2(sum[0], sum[1]), sum0, sum1);
                l += sum0 + sum1;
                if (!(flags & kLast)) continue;
                // ---- the part's end: the rows, or what is joined with other parts
                ok = warp_wait(&sh.o_done[s], use & 1, a.wait_limit);
                if (!ok) break;
                tc_fence_after();
                mbar_arrive_by(first_thread, smem_addr(&sh.v_empty[held]));
                held = -1;
                // (the note is read until o_empty says that the rows have left the part, not after)
                const PartInfo &p = sh.parts[(flags >> kPartShift) % kInfos];
                const bool turns = p.mode == kTurns;
                const int r = p.r0 + (s == 1 && !turns ? a.tokens : 0) + token;  // row in the stream
                const bool odd = *reinterpret_cast<volatile int *>(&sh.odd[p.number % 8]) == p.number;
                const bool real = token < a.tokens && r < p.n;
                const int first = p.shares, count = (p.more + 1) * (turns ? 2 : 1);
                __nv_bfloat16 *out = a.out + (static_cast<size_t>(p.first + r) * a.Hq + p.g * a.group + row % a.group) * kDim;
                // (with both halves' parts in turns: half 1's tiles are the odd ones)
                const int step = turns ? 2 : 1, j0 = turns ? s : 0;
                if (count == 1) {
                    const float inv = inverse(l);
#pragma unroll 1
                    for (int c = 0; c < kDim; c += 32) {
                        float f[32];
                        tmem_ld32_nowait(to + c, reinterpret_cast<uint32_t *>(f));
                        tmem_wait_ld();
                        if (odd && real) add_odd<kFp8>(a, p, step, j0, limit, c, f);
                        if (real) store_row(out + c, f, inv);
                    }
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(smem_addr(&sh.o_empty[s]));
                    continue;
                }
                // (a part in turns is of a segment of several CTAs: their rule sees to that)
                const bool begins = static_cast<int>(blockIdx.x) == first, alone = turns && p.tiles == 1;
                float *mine = part_slot(a.part, blockIdx.x, begins, s);
                const int4 job = make_int4(min(p.n - (r - token), a.tokens) * a.group, p.first + r, p.g, turns ? -count : count);
#pragma unroll 1
                for (int c = 0; c < kDim; c += 32) {
                    float f[32];
                    tmem_ld32_nowait(to + c, reinterpret_cast<uint32_t *>(f));
                    tmem_wait_ld();
                    if (odd && real) add_odd<kFp8>(a, p, step, j0, limit, c, f);
                    if (real)
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            reinterpret_cast<float4 *>(mine)[(c / 4 + i) * kRows + row] =
                                make_float4(f[4 * i], f[4 * i + 1], f[4 * i + 2], f[4 * i + 3]);
                }
                if (real) {
                    mine[kRows * kDim + row] = m;
                    mine[kRows * kDim + kRows + row] = l;
                    if (alone) {  // no tile was half 1's
                        mine[kPartFloats + kRows * kDim + row] = kNoPart;
                        mine[kPartFloats + kRows * kDim + kRows + row] = 0.0f;
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_addr(&sh.o_empty[s]));
                if (count > kJoinHere) {
                    if (begins && row == 0 && (s == 0 || !turns)) sh.jobs[s] = job;
                    continue;
                }
                if (lane == 0) mbar_arrive(smem_addr(&sh.stored[s]));
                // (bounded waits, as everywhere: a warp may have given up)
                if (w == 0) ok = warp_wait(&sh.stored[s], joins & 1, a.wait_limit);
                if (row == 0 && ok) {
                    int old;
                    int32_t *ticket = a.tickets + 2 * first + (turns ? 0 : s);
                    const int add = alone ? 2 : 1;
                    asm volatile("atom.acq_rel.gpu.global.add.s32 %0, [%1], %2;" : "=r"(old) : "l"(ticket), "r"(add) : "memory");
                    sh.last[s] = old + add == count;
                    if (old + add == count) *ticket = 0;
                    mbar_arrive(smem_addr(&sh.told[s]));
                }
                __syncwarp();
                ok = ok && warp_wait(&sh.told[s], joins & 1, a.wait_limit);
                ++joins;
                if (!ok) break;
                if (!*reinterpret_cast<volatile int *>(&sh.last[s]) || !real) continue;
                float best = kNoScore, total = 0.0f;
#pragma unroll 1
                for (int i = 0; i < count; ++i) best = fmaxf(best, __ldcg(segment_part(a.part, first, i, turns, s) + kRows * kDim + row));
#pragma unroll 1
                for (int i = 0; i < count; ++i) {
                    const float *q = segment_part(a.part, first, i, turns, s) + kRows * kDim + row;
                    total = fmaf(hw_ex2(__ldcg(q) - best), __ldcg(q + kRows), total);
                }
                const float inv = inverse(total);
#pragma unroll 1
                for (int d = 0; d < kDim; d += 32) {
                    float o[32];
#pragma unroll
                    for (int i = 0; i < 32; ++i) o[i] = 0.0f;
#pragma unroll 1
                    for (int i = 0; i < count; ++i) {
                        const float *q = segment_part(a.part, first, i, turns, s);
                        const float mq = __ldcg(q + kRows * kDim + row);
                        const float f = hw_ex2(mq - best);
                        if (mq == kNoPart) continue;  // (o was not written)
                        float4 x[8];
#pragma unroll
                        for (int e = 0; e < 8; ++e) x[e] = __ldcg(reinterpret_cast<const float4 *>(q) + (d / 4 + e) * kRows + row);
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            o[4 * e] = fmaf(x[e].x, f, o[4 * e]);
                            o[4 * e + 1] = fmaf(x[e].y, f, o[4 * e + 1]);
                            o[4 * e + 2] = fmaf(x[e].z, f, o[4 * e + 2]);
                            o[4 * e + 3] = fmaf(x[e].w, f, o[4 * e + 3]);
                        }
                    }
                    store_row(out + d, o, inv);
                }
            }
        }
        if (!ok) flag_error(a.err, TTS_ERRBIT_TIMEOUT);
    }
    tc_fence_before();
    __syncthreads();
    if (threadIdx.x < 2) a.jobs[2 * blockIdx.x + threadIdx.x] = sh.jobs[threadIdx.x];
    if (warp == 12) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
    }
}

// ---------------------------------------------------------------- the join

// Segments of more than kJoinHere parts: one CTA's threads would read them at a
// few bytes a cycle (61 rows of 8 KV heads in 19 parts of 62 KB each: 54 us), so
// a second kernel spreads the work over every SM, 128 rows of 8 dimensions an
// item, four threads a row (that call whole: 95 us, with this kernel 59).  It runs
// wherever a table may hold more than kSoloTiles tiles, and finds that there is
// nothing to do by looking at one word a CTA and half.
constexpr int kJoinThreads = 512, kJoinItems = kDim / 8, kJoinGroups = kJoinThreads / kRows;

__global__ void __launch_bounds__(kJoinThreads)
prompt_join_kernel(float *parts, const int4 *jobs, int ctas, __nv_bfloat16 *out, int Hq, int group) {
    __shared__ int found[kJoinThreads / 32], entry;
    __shared__ float some[kJoinGroups][10][kRows];  // m, l and 8 dimensions of each group's parts
    pdl_wait_prerequisites();
    pdl_allow_dependents();
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    const int row = threadIdx.x % kRows, mine_of = threadIdx.x / kRows;
    int before = 0;  // jobs of the entries seen so far
    for (int base = 0; base < 2 * ctas; base += kJoinThreads) {
        const int e = base + threadIdx.x;
        const int mine = e < 2 * ctas ? __ldcg(&jobs[e].x) : 0;
        const unsigned any = __ballot_sync(kFull, mine != 0);
        if (lane == 0) found[warp] = __popc(any);
        __syncthreads();
        int total = 0;
        for (int w = 0; w < kJoinThreads / 32; ++w) total += found[w];
        // this CTA's items (job, 8 dimensions) of these entries
        const int lo = before * kJoinItems, hi = (before + total) * kJoinItems, grid = gridDim.x, me = blockIdx.x;
        for (int item = me + (max(lo - me, 0) + grid - 1) / grid * grid; item < hi; item += grid) {
            // the entry of the job: the warp that found it, then its lane
            int nth = item / kJoinItems - before;
            for (int w = 0; w < warp; ++w) nth -= found[w];
            if (mine != 0 && nth == __popc(any & ((1u << lane) - 1u))) entry = e;
            __syncthreads();
            const int4 job = __ldcg(jobs + entry);
            const int s = entry % 2, first = entry / 2, d = item % kJoinItems * 8;
            const bool turns = job.w < 0, real = row < job.x;
            const int count = abs(job.w);
            // a thread: parts mine_of, mine_of + 4, ... of a row
            float best = kNoScore, l = 0.0f, o[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) o[i] = 0.0f;
            constexpr int kAhead = 5;
            for (int i0 = mine_of; real && i0 < count; i0 += kAhead * kJoinGroups) {
                float mq[kAhead], lq[kAhead];
                float4 x[kAhead][2];
#pragma unroll
                for (int u = 0; u < kAhead; ++u) {
                    const int i = i0 + u * kJoinGroups;
                    mq[u] = kNoPart;
                    lq[u] = 0.0f;
                    x[u][0] = x[u][1] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                    if (i >= count) continue;
                    const float *q = segment_part(parts, first, i, turns, s);
                    mq[u] = __ldcg(q + kRows * kDim + row);
                    lq[u] = __ldcg(q + kRows * kDim + kRows + row);
                    x[u][0] = __ldcg(reinterpret_cast<const float4 *>(q) + d / 4 * kRows + row);
                    x[u][1] = __ldcg(reinterpret_cast<const float4 *>(q) + (d / 4 + 1) * kRows + row);
                }
                float now = best;
#pragma unroll
                for (int u = 0; u < kAhead; ++u) now = fmaxf(now, mq[u]);
                const float f0 = hw_ex2(best - now);
                best = now;
                l *= f0;
#pragma unroll
                for (int i = 0; i < 8; ++i) o[i] *= f0;
#pragma unroll
                for (int u = 0; u < kAhead; ++u) {
                    // (where a half had no tile o was not written)
                    const float f = hw_ex2(mq[u] - now);
                    const bool none = mq[u] == kNoPart;
                    const float v[8] = {x[u][0].x, x[u][0].y, x[u][0].z, x[u][0].w, x[u][1].x, x[u][1].y, x[u][1].z, x[u][1].w};
                    l = fmaf(f, lq[u], l);
#pragma unroll
                    for (int i = 0; i < 8; ++i) o[i] = none ? o[i] : fmaf(f, v[i], o[i]);
                }
            }
            some[mine_of][0][row] = best;
            some[mine_of][1][row] = l;
#pragma unroll
            for (int i = 0; i < 8; ++i) some[mine_of][2 + i][row] = o[i];
            __syncthreads();
            if (mine_of == 0 && real) {
                float top = kNoScore, sum = 0.0f, r[8];
                for (int k = 0; k < kJoinGroups; ++k) top = fmaxf(top, some[k][0][row]);
#pragma unroll
                for (int i = 0; i < 8; ++i) r[i] = 0.0f;
                for (int k = 0; k < kJoinGroups; ++k) {
                    const float f = hw_ex2(some[k][0][row] - top);
                    sum = fmaf(f, some[k][1][row], sum);
#pragma unroll
                    for (int i = 0; i < 8; ++i) r[i] = fmaf(f, some[k][2 + i][row], r[i]);
                }
                const float inv = inverse(sum);
                *reinterpret_cast<uint4 *>(out + (static_cast<size_t>(job.y + row / group) * Hq + job.z * group + row % group) * kDim + d) =
                    make_uint4(pack_bf16(r[0] * inv, r[1] * inv), pack_bf16(r[2] * inv, r[3] * inv),
                               pack_bf16(r[4] * inv, r[5] * inv), pack_bf16(r[6] * inv, r[7] * inv));
            }
            __syncthreads();
        }
        before += total;
        __syncthreads();
    }
}

// -------------------------------------------------------------------- host

int prompt_ctas() {
    const int n = sm_count();
    return n > 0 ? n : 160;  // no device visible (size queries on a build host)
}

bool prompt_shape_ok(int B, int T, int Hq, int Hkv) {
    return B >= 0 && T >= 0 && Hkv >= 1 && Hq >= Hkv && Hq % Hkv == 0;
}

size_t prompt_part_bytes() { return align_up(static_cast<size_t>(prompt_ctas()) * 4 * kPartFloats * sizeof(float), 256); }
size_t prompt_ticket_bytes() { return align_up(static_cast<size_t>(prompt_ctas()) * 2 * sizeof(int32_t), 256); }
size_t prompt_job_bytes() { return align_up(static_cast<size_t>(prompt_ctas()) * 2 * sizeof(int4), 256); }
// parts, jobs, and last the tickets
size_t prompt_workspace_bytes() { return prompt_part_bytes() + prompt_job_bytes() + prompt_ticket_bytes(); }

}  // namespace
}  // namespace tts

extern "C" size_t tts_prompt_attn_workspace_size(int32_t B, int32_t num_rows, int32_t num_q_heads, int32_t num_kv_heads,
                                                 int32_t head_dim) {
    using namespace tts;
    if (!prompt_shape_ok(B, num_rows, num_q_heads, num_kv_heads) || head_dim != kDim || B > kMaxStreams ||
        num_q_heads / num_kv_heads > kRows)
        return 0;
    return prompt_workspace_bytes();
}

extern "C" int tts_prompt_attn(const tts_kv_cache *cache, const int32_t *d_block_table, int32_t max_blocks_per_seq,
                               const int32_t *d_ctx_lens, int32_t B, const int32_t *d_row_start, int32_t num_rows,
                               int32_t num_q_heads, float scale, int32_t window, int32_t sinks, const void *d_q,
                               void *d_out, void *d_ws, size_t ws_bytes, int32_t *d_err, void *stream) {
    using namespace tts;
    const bool none = B == 0 || num_rows == 0;  // nothing is read or written: the tensors may be empty
    if (!cache || !d_row_start) return TTS_ERR_INVALID;
    if (!none && (!d_block_table || !d_ctx_lens || !d_q || !d_out)) return TTS_ERR_INVALID;
    if (!cache->k_pool || (!cache->v_pool && cache->dtype != TTS_FP8_E4M3) || cache->num_blocks < 1 ||
        cache->num_kv_heads < 1)
        return TTS_ERR_INVALID;
    if (max_blocks_per_seq < 1 || max_blocks_per_seq > (1 << 20) || window < 0 || sinks < 0 || !(scale > 0.0f) ||
        std::isinf(scale))
        return TTS_ERR_INVALID;
    const int Hq = num_q_heads, Hkv = cache->num_kv_heads;
    if (!prompt_shape_ok(B, num_rows, Hq, Hkv)) return TTS_ERR_INVALID;
    if (cache->block_size != TTS_BLOCK_TOKENS || cache->head_dim != kDim ||
        (cache->dtype != TTS_BF16 && cache->dtype != TTS_FP8_E4M3))
        return TTS_ERR_UNSUPPORTED;
    if (B > kMaxStreams || Hq / Hkv > kRows) return TTS_ERR_UNSUPPORTED;
    const uint64_t pool_rows = static_cast<uint64_t>(cache->num_blocks) * Hkv * TTS_BLOCK_TOKENS;
    if (pool_rows >= (1ULL << 31)) return TTS_ERR_UNSUPPORTED;
    const bool fp8 = cache->dtype == TTS_FP8_E4M3;
    if (!aligned16(cache->k_pool) || (!fp8 && !aligned16(cache->v_pool)) || !aligned16(d_q) || !aligned16(d_out)) return TTS_ERR_INVALID;
    if (none) return TTS_OK;
    if (!d_ws || ws_bytes < prompt_workspace_bytes() || (reinterpret_cast<uintptr_t>(d_ws) & 255u) != 0)
        return TTS_ERR_WORKSPACE;

    PromptArgs a{};
    a.table = d_block_table;
    a.max_blocks = max_blocks_per_seq;
    a.num_blocks = cache->num_blocks;
    a.ctx_lens = d_ctx_lens;
    a.row_start = d_row_start;
    a.B = B;
    a.num_rows = num_rows;
    a.Hq = Hq;
    a.Hkv = Hkv;
    a.group = Hq / Hkv;
    a.tokens = kRows / a.group;
    // (no context passes 2^24 tokens)
    a.window = window < (1 << 25) ? window : 0;
    a.sinks = sinks < (1 << 24) ? sinks : 1 << 24;
    if (!a.window) a.sinks = 0;
    a.scale_log2 = scale * kLog2e;
    a.k_pool = static_cast<const uint8_t *>(cache->k_pool);
    a.v_pool = static_cast<const uint8_t *>(cache->v_pool);
    a.out = static_cast<__nv_bfloat16 *>(d_out);
    a.ctas = prompt_ctas();
    a.part = static_cast<float *>(d_ws);
    a.jobs = reinterpret_cast<int4 *>(static_cast<uint8_t *>(d_ws) + prompt_part_bytes());
    a.tickets = reinterpret_cast<int32_t *>(static_cast<uint8_t *>(d_ws) + prompt_part_bytes() + prompt_job_bytes());
    a.zero_row = static_cast<int>(pool_rows);
    a.err = d_err;
    a.wait_limit = thread_opts().wait_limit;
    a.stall = thread_opts().stall == TTS_TEST_STALL_PROMPT;
    // the flat list of tiles is 32-bit
    const int64_t query_tiles = static_cast<int64_t>(num_rows) / (2 * a.tokens) + B;
    a.max_tiles = static_cast<int>(query_tiles);
    a.few = B <= 32 && query_tiles <= kFewTiles;
    if (query_tiles * Hkv * (max_blocks_per_seq / kBlocks + 1 + kPartCost) >= (1LL << 30)) return TTS_ERR_UNSUPPORTED;
    CUtensorMap map_q, map_k{}, map_v{};
    if (!make_tma_queries_bf16(&map_q, d_q, num_rows, Hq, a.group, a.tokens)) return TTS_ERR_CUDA;
    if (!fp8 && (!make_tma_2d_bf16(&map_k, cache->k_pool, pool_rows, kDim, TTS_BLOCK_TOKENS, 64) ||
        !make_tma_rows_in_halves_bf16(&map_v, cache->v_pool, pool_rows, TTS_BLOCK_TOKENS)))
        return TTS_ERR_CUDA;
    const auto kernel = fp8 ? prompt_attn_kernel<true> : prompt_attn_kernel<false>;
    const int smem = fp8 ? PromptSmem<true>::total : PromptSmem<false>::total;
    if (!allow_smem(kernel, smem)) return TTS_ERR_CUDA;
    const cudaStream_t cs = static_cast<cudaStream_t>(stream);
    const int rc = launch_kernel(kernel, dim3(a.ctas), dim3(prompt_threads(fp8)), smem, {cs, thread_pdl()}, map_q, map_k, map_v, a);
    // With at most kSoloTiles tiles no segment is worked on in turns, nor has it more
    // than kJoinHere parts (a range is at least kPartCost + 1 long): none is left over
    if (rc != TTS_OK || max_blocks_per_seq <= kSoloTiles * kBlocks) return rc;
    return launch_kernel(prompt_join_kernel, dim3(a.ctas), dim3(kJoinThreads), 0, {cs, true}, a.part, a.jobs, a.ctas, a.out,
                         a.Hq, a.group);
}
