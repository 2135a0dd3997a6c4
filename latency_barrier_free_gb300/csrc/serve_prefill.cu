// serve_prefill.cu -- attention over the 4-bit or 8-bit cache for prompts: many queries
// of a request at once (rra_serve.h), on the tensor cores' own memory.
//
// A row is one query of one head.  A CTA takes a segment: TILES x 128 rows of
// one request and KV head, and walks the keys that any of them sees, 128 at a
// time.  Four warps unpack a tile of the cache: V as binary16 (code * scale,
// rounded to 11 bits), K as two binary16 numbers whose sum is 2 * code * scale
// exactly (codes of 3 * 2^i times an 11-bit scale have 13 bits, and twice the
// smallest product's last one, 2^-25, is binary16's smallest number), so that
// scores keep the accuracy of their binary32 accumulation; the second costs half
// as much again in tensor work.  One thread issues
//     S_i = Q_i K_hi^T + Q_i K_lo^T,   O_i += P_i V      (tcgen05.mma, sums in TMEM)
// and a warpgroup for each tile i turns S_i into weights P_i, in place: a thread
// has a row, so maxima and sums need no exchange.  While one tile's scores are
// exponentiated the other's products run.
//
// The maximum that weights are taken against moves only when a score passes it by
// more than kPromptSlack (in units of log2); then O is scaled, in TMEM, which is
// rare after a row's first keys.  The code of every role is kept small (loops
// over 32 columns, one place for each product): four kinds of warps share the
// instruction cache, and with twice the code the issuing thread alone cost a
// third of the time.
//
// Work is cut into equal runs of key tiles, one per CTA, as in serve_attn.cu;
// what a run has of a segment it shares goes to the workspace, and the last CTA
// to arrive adds the parts in order.
//
// 3 requests of up to 1024 queries and 8192 keys, 64 heads over 8 of 128: 261
// GFLOP in 259.5 us, 1006 TFLOP/s, or 1509 with the second part of K.  Per 256
// rows and 128 keys that is about 4200 cycles, of which products at their full
// rate would take 3072.  Longest is the chain of one tile: its values' and next
// scores' products (1536 cycles alone, 1750 beside the stores and reads of the
// rest), a wait of 250, its softmax (2000: reading the scores, their maximum, and
// 128 exponentials a thread take about as long each).  TMEM has no room for the
// next scores beside the weights, so only the other tile fills the gap.
//
// Over the 8-bit cache K is one binary16 number, its code: 271 GFLOP (3 requests of up
// to 1024 queries) in 285 us, 950 TFLOP/s.  The products have 2048 of the 4150 cycles
// for 256 rows and 128 keys; the softmax, one thread a row and one warp a scheduler,
// takes 2300 to 3000 of one tile's chain, the products behind it 1070 and 340.
#include <algorithm>
#include <type_traits>

#include "serve_attn_rows8.cuh"
#include "serve_tc.cuh"

namespace rra {

constexpr float kPromptSlack = 8.f;    // log2 of how far weights may pass 1 before the maximum moves
// Weights enter their product with the values as binary16, which has few bits left below 2^-14 and none below 2^-25, while a
// row's sum counts them whole.  So they are taken 2^kPromptLift times as large: 2^(8 + 7) fits.  (131072 keys of one run, each
// 2^-25.3 of the largest: without it their share, 0.3 % of the values' size, was missing.)
constexpr float kPromptLift = 7.f, kPromptUnlift = 1.f / 128;
// 8-bit cache: what scores are multiplied with, times a block's 2^k, has to be a number of binary32, neither 0 nor infinite.  With
// less than 2^-90 scores (at most 2^50 before) are as good as 0; with more than 2^95 those that are not 0 (at least 2^-65 before)
// are larger than scores may be.
constexpr float kPromptLeast = 0x1p-90f, kPromptBeyond = 0x1p95f;
// A tile's blocks whose units of values are far apart (kKv8Apart), or far below those that maxima are against, do not enter one
// product: binary16 has no weights for both.  The blocks down to kKv8Apart below the highest unit come first, then those down to
// kKv8Apart below the highest that is left, and so on, each time with weights against their own maximum, O and l being brought to
// it: not below 2^-kPromptRange of the highest so far, so that they stay numbers of binary32.
constexpr float kPromptAbsent = -100.f;  // unit of a block that is not there
constexpr float kPromptRange = 56.f;
constexpr float kPromptMost = 32768.f;  // 8-bit cache: what a block's weights of a row may add up to before the maximum moves

template <typename F, int D, int TILES>
struct PromptShape {
    using B = typename F::template Block<D>;
    static constexpr int kParts = F::kBits == 4 ? 2 : 1;  // of K: high and low, or codes as they are
    static constexpr int kRows = TILES * kPromptRows;
    static constexpr int kPanel = 128 * 128;            // 128 rows of 64 binary16, swizzled in 128 bytes
    static constexpr int kTile = D / 64 * kPanel;       // 128 rows of D binary16
    static constexpr int kK = TILES * kTile;            // after the queries: two stages of K, all parts
    static constexpr int kV = kK + 2 * kParts * kTile;  // V
    static constexpr int kEnd = kV + kTile;
    static constexpr int kSums = kK;                    // before any tile: running sums of the requests' chunks
    static_assert(4 * (RRA_SERVE_MAX_REQUESTS + 1) <= kEnd - kSums, "the sums fit");
    // Warps: softmax (a warp reaches the TMEM lanes of its number modulo 4), then four that unpack, then one for each tile
    // that issues its products: one for both left the tensor cores idle for 300 to 500 cycles between products.  Of the two
    // left in the last warpgroup one looks up pages.
    // Whole warpgroups, for the registers: a softmax thread holds all 128 scores of its row (read back from TMEM in two
    // passes instead, their latency alone took 1200 cycles a tile).  The shares of a warpgroup's thread are those that
    // the launch gives (65536 over all threads, a multiple of 8), taken from the issuing one for the softmax.
    static constexpr int kSoftmaxWarps = 4 * TILES;
    static constexpr int kUnpack = kSoftmaxWarps;
    static constexpr int kIssue = kUnpack + 4;
    static constexpr int kWarps = kIssue + 4;
    static constexpr int kLaunchRegs = 65536 / (32 * kWarps) / 8 * 8;
    static constexpr int kSoftmaxRegs = TILES == 2 ? 184 : 216;
    static constexpr int kUnpackRegs = TILES == 2 ? 96 : 168;
    static constexpr int kIssueRegs = TILES == 2 ? 48 : 120;
    static_assert(TILES * kSoftmaxRegs + kUnpackRegs + kIssueRegs <= (TILES + 2) * kLaunchRegs, "what the launch has");
    static constexpr int kThreads = 32 * kWarps;
    static constexpr int kColumns = TILES == 2 ? 512 : 256;  // of TMEM: S of every tile, then O of every tile
    static constexpr int kPartFloats = kPromptRows * (D + 2);  // floats of a part: rows in columns of 4 channels, statistics
    static constexpr int kSmem = 1024 + kEnd;
};

// The work: chunks of kRows rows of every request and KV head.
template <int kRows>
struct CacheWork {
    const AttnParams& p;
    __device__ __forceinline__ int requests() const { return p.a.requests; }
    __device__ __forceinline__ int heads() const { return p.a.cache.kv_heads; }
    __device__ __forceinline__ AttnLengths lengths(int b) const { return attn_lengths(p, b); }
    __device__ __forceinline__ int chunks(const AttnLengths& n) const { return (n.qn * p.group + kRows - 1) / kRows; }
    __device__ __forceinline__ PromptItem item(const AttnLengths& n, int c) const {
        const int rows = n.qn * p.group, last = min(rows, (c + 1) * kRows) - 1;
        const int end = p.a.causal ? max(0, n.kv - n.qn + p.by_group(last) + 1) : n.kv;
        const int first = p.window > 0 ? max(0, n.kv - n.qn + p.by_group(c * kRows) - p.window + 1) : 0;
        return prompt_item(first, end);
    }
};

// The highest unit of a tile's values below those that a product takes; kPromptAbsent: none.
__device__ __forceinline__ float next_unit(const float4* ex, float unit) {
    float most = kPromptAbsent;
#pragma unroll
    for (int b = 0; b < 8; ++b) most = ex[b].y < unit - kKv8Apart ? fmaxf(most, ex[b].y) : most;
    return most;
}

template <typename F, int D, int TILES>
__global__ void __launch_bounds__(PromptShape<F, D, TILES>::kThreads, 1) kv_attention_prompt_kernel(const __grid_constant__ AttnParams p) {
    using Sh = PromptShape<F, D, TILES>;
    using B = typename F::template Block<D>;
    constexpr int J = D / kKvGroup;
    constexpr bool kEight = F::kBits == 8;
    extern __shared__ unsigned char raw_smem[];
    __shared__ __align__(8) uint64_t bar_mem[7 * TILES + 4 + 2 + 4 + 1 + 8];
    __shared__ int64_t part[Sh::kWarps];
    __shared__ volatile uint32_t seen_words[4][4];  // of the last four tiles, which keys are there
    __shared__ volatile int32_t places[4][9];  // of four tiles: the cache's blocks of its keys (-1: none), and how many keys there are
    // 8-bit cache, of eight tiles, of each block: 2^exponent of K, exponent of V, 2 to minus that, and infinity if the tile's units
    // are far apart, else 0.  And of each row its highest maximum in such a tile.
    __shared__ float4 exponents[8][8];
    __shared__ float highest[kEight ? TILES * kPromptRows : 1];
    __shared__ uint32_t tmem_base;
    __shared__ volatile uint32_t arrived[2][TILES];  // of the run's first and last segment
    __shared__ volatile uint32_t added[2][TILES];    // whether this CTA has counted itself there
    __shared__ PromptSegment start;
    const rra_kv_attention_args_t& a = p.a;
    const int tid = (int)threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t smem = (smem_u32(raw_smem) + 1023u) & ~1023u;
    int32_t* const chunk_sums = (int32_t*)(raw_smem + (smem - smem_u32(raw_smem)) + Sh::kSums);
    AttnWorkspace* const ws = (AttnWorkspace*)a.workspace;
    float* const parts = (float*)(ws + 1);

    const uint32_t bars = smem_u32(bar_mem);
    // q_full[i], pv_full[i]: what the next products of tile i wait for, with their turn; s_full[i], o_full[i]: done
    const uint32_t q_full = bars, s_full = q_full + 8 * TILES, pv_full = s_full + 8 * TILES, o_full = pv_full + 8 * TILES,
                   joined = o_full + 8 * TILES, k_full = joined + 8 * TILES, k_empty = k_full + 16, v_empty = k_empty + 16,
                   seen_full = v_empty + 16, drained = seen_full + 32, place_full = drained + 8, place_empty = place_full + 32,
                   part_full = place_empty + 32, part_done = part_full + 8 * TILES;  // of a tile's further products
    constexpr uint32_t kTurn = TILES == 2 ? 1 : 0;
    pdl_release_early();
    if (tid == 0) {
        for (int i = 0; i < TILES; ++i) {
            added[0][i] = added[1][i] = 0u;
            mbar_init(q_full + 8 * i, kPromptRows + kTurn);
            mbar_init(s_full + 8 * i, 1);
            mbar_init(pv_full + 8 * i, kPromptRows + 128 + kTurn);
            mbar_init(o_full + 8 * i, 1);
            mbar_init(joined + 8 * i, kPromptRows);
            mbar_init(part_full + 8 * i, kPromptRows);
            mbar_init(part_done + 8 * i, 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(v_empty + 8 * i, TILES);
            mbar_init(k_full + 8 * i, 128);
            mbar_init(k_empty + 8 * i, TILES);
        }
        for (int i = 0; i < 4; ++i) {
            mbar_init(seen_full + 8 * i, 4);
            mbar_init(place_full + 8 * i, 1);
            mbar_init(place_empty + 8 * i, 4);
        }
        mbar_init(drained, TILES);
        if (kTurn) mbar_arrive(q_full);  // the first turn
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        fence_proxy_async_smem();
    }
    pdl_wait();

    const CacheWork<Sh::kRows> work{p};
    int64_t r0, r1, run;
    if (!prompt_run<Sh::kWarps>(work, chunk_sums, part, start, r0, r1, run)) return;
    if (warp == Sh::kIssue) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" : : "r"(smem_u32(&tmem_base)), "r"(Sh::kColumns) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tc_before_sync();
    __syncthreads();
    tc_after_sync();
    const uint32_t tmem = tmem_base;
    PromptSegment seg = start;
    prompt_load(work, seg);
    auto first_of = [&](const PromptSegment& s) {
        const int64_t from = (s.begin > r0 ? s.begin : r0) - s.begin - kPromptSegmentCost;
        return (int)(from > 0 ? from : 0);
    };
    auto end_of = [&](const PromptSegment& s) {
        const int64_t to = (s.end < r1 ? s.end : r1) - s.begin - kPromptSegmentCost;
        return (int)(to > 0 ? to : 0);
    };
    auto wait = [&](uint32_t bar, uint32_t parity) {
        return __all_sync(0xffffffffu, attn_try(bar, parity & 1u) || attn_wait_slow(bar, parity & 1u, ws));
    };

    uint32_t n = 0;   // key tiles of this run so far
    uint32_t sn = 0;  // segments so far that had tiles
    uint32_t pn = 0;  // further products of a tile so far
    bool ok = true;
    if (warp < Sh::kSoftmaxWarps) {
        // =============================== softmax: a thread has a row ====
        set_registers<Sh::kSoftmaxRegs, Sh::kLaunchRegs>();
        const int i = warp >> 2, row = tid & 127;
        const uint32_t lanes = tmem + ((uint32_t)(warp & 3) << 21);  // this warp's quarter of the TMEM lanes
        const uint32_t s_at = lanes + 128 * i, o_at = lanes + 128 * (TILES + i);
        uint32_t joins = 0;
        while (ok) {
            const int t0 = first_of(seg), t1 = end_of(seg);
            const int all_rows = seg.n.qn * p.group, r = seg.c * Sh::kRows + i * kPromptRows + row;
            const bool live = r < all_rows;
            constexpr float kNone = -FLT_MAX;  // no key yet
            // (8-bit cache: m is in units of log2, and O and l are 2^-m as large; l has no 2^v)
            if (kEight) highest[tid] = kNone;
            float m = kEight && !live ? 0.f : kNone, limit = kNone, l = 0.f, factor = 1.f;
            if (t0 < t1) {
                // ---- the row's query, scaled, into shared memory; the keys that it sees ----
                int lo = 0, hi = 0;
                {
                    uint4 x[D / 8];
                    const int tok = live ? p.by_group(r) : 0;
                    if (live) {
                        const __nv_bfloat16* src = (const __nv_bfloat16*)a.q + (seg.n.q0 + tok) * a.q_token_stride +
                                                   (seg.h * p.group + r - tok * p.group) * a.q_head_stride;
#pragma unroll
                        for (int k = 0; k < D / 8; ++k) x[k] = *((const uint4*)src + k);
                        const int pos = seg.n.kv - seg.n.qn + tok;
                        hi = a.causal ? max(0, min(seg.n.kv, pos + 1)) : seg.n.kv;
                        lo = p.window > 0 ? max(0, pos - p.window + 1) : 0;
                    } else {
#pragma unroll
                        for (int k = 0; k < D / 8; ++k) x[k] = make_uint4(0u, 0u, 0u, 0u);
                    }
                    float most = 0.f, down;
#pragma unroll
                    for (int k = 0; k < D / 8; ++k) {
                        const uint32_t v[4] = {x[k].x, x[k].y, x[k].z, x[k].w};
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            most = fmaxf(most, fmaxf(fabsf(__uint_as_float(v[e] << 16)), fabsf(__uint_as_float(v[e] & 0xffff0000u))));
                    }
                    attn_row_scale(p, most, down, factor);
                    if constexpr (kEight) factor = fminf(fmaxf(factor, kPromptLeast), kPromptBeyond);
                    else factor *= 0.5f;  // K is held twice as large
#pragma unroll
                    for (int k = 0; k < D / 8; ++k) {
                        const uint32_t v[4] = {x[k].x, x[k].y, x[k].z, x[k].w};
                        uint32_t h[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            h[e] = pack_half2(__uint_as_float(v[e] << 16) * down, __uint_as_float(v[e] & 0xffff0000u) * down);
                        sts_v4(smem + i * Sh::kTile + (k >> 3) * Sh::kPanel + row * 128 + (((k & 7) ^ (row & 7)) << 4), h[0], h[1], h[2], h[3]);
                    }
                }
                fence_proxy_async_smem();
                mbar_arrive(q_full + 8 * i);

                const uint64_t factor2 = pair2(factor, factor), lift2 = pair2(kPromptLift, kPromptLift);
                for (int tl = t0; tl < t1 && ok; ++tl, ++n) {
                    ok = wait(seen_full + 8 * (n & 3), n >> 2) && wait(s_full + 8 * i, n);
                    if (!ok) break;
                    tc_after_sync();
                    const int key0 = (seg.first_tile + tl) * kPromptKeys;
                    const volatile uint32_t* const words = seen_words[n & 3];
                    const bool whole = __all_sync(0xffffffffu, key0 >= lo && key0 + kPromptKeys <= hi) &&
                                       (words[0] & words[1] & words[2] & words[3]) == 0xffffffffu;
                    uint32_t v[128];
#pragma unroll
                    for (int q = 0; q < 4; ++q) tc_ld32(s_at + 32 * q, v + 32 * q);
                    tc_wait_ld();
                    if (!whole) {
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            // keys lo..hi of these 32, as bits, and of them those that are there
                            const int from = min(max(lo - key0 - 32 * q, 0), 32), to = min(max(hi - key0 - 32 * q, 0), 32);
                            const uint32_t below = to == 32 ? 0xffffffffu : (1u << to) - 1u;
                            const uint32_t mask = words[q] & below & (from == 32 ? 0u : 0xffffffffu << from);
#pragma unroll
                            for (int k = 0; k < 32; ++k) v[32 * q + k] = mask >> k & 1u ? v[32 * q + k] : 0xff800000u;
                        }
                    }
                    if constexpr (kEight) {
                        // As in serve_attn_rows8.cuh: a block of 16 keys has the exponents k and v; scores are v[] 2^k, weights
                        // 2^(score factor + v - m), the sum's parts 2^-v as large.  m (kNone: no key yet) is the largest such
                        // exponent of the row's first tile, until weights get large, which their sum shows.
                        const float4* const ex = exponents[n & 7];
                        for (bool exact = __any_sync(0xffffffffu, m == kNone);; exact = true) {
                            if (exact && __any_sync(0xffffffffu, ex[0].w != 0.f)) {  // units that are far apart
                                float unit = next_unit(ex, INFINITY);
                                uint32_t to = pv_full;
                                tc_wait_st();  // of the weights that led here
#pragma unroll 1
                                while (true) {
                                    auto takes = [&](int b) { return ex[b].y <= unit && ex[b].y >= unit - kKv8Apart; };
                                    float now = -INFINITY;
#pragma unroll
                                    for (int b = 0; b < 8; ++b) {
                                        float top = -INFINITY;
#pragma unroll
                                        for (int k = 0; k < 16; ++k) top = fmaxf(top, __uint_as_float(v[16 * b + k]));
                                        if (takes(b)) now = fmaxf(now, fmaf(top, factor * ex[b].x, ex[b].y));
                                    }
                                    const float high = fmaxf(fmaxf(highest[tid], m), now);
                                    highest[tid] = high;
                                    now = fmaxf(now, high - kPromptRange);  // a row that sees none of the blocks is ready for any
                                    const float by = exp2_fast(m - now);
                                    m = now;
                                    l *= by;
                                    if (tl > t0 || to != pv_full)
#pragma unroll 1
                                        for (int q = 0; q < D / 16; ++q) {
                                            uint32_t o[16];
                                            tc_ld16(o_at + 16 * q, o);
                                            tc_wait_ld();
#pragma unroll
                                            for (int k = 0; k < 16; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * by);
                                            tc_st16(o_at + 16 * q, o);
                                        }
                                    const float less = m == kNone ? 0.f : kPromptLift - m;
#pragma unroll
                                    for (int b = 0; b < 8; b += 2) {
                                        uint32_t w[16];
#pragma unroll
                                        for (int c = b; c < b + 2; ++c) {
                                            const float up = factor * ex[c].x, off = takes(c) ? less + ex[c].y : -INFINITY;
                                            float sum = 0.f;
#pragma unroll
                                            for (int k = 0; k < 16; k += 2) {
                                                const float e0 = exp2_fast(fmaf(__uint_as_float(v[16 * c + k]), up, off));
                                                const float e1 = exp2_fast(fmaf(__uint_as_float(v[16 * c + k + 1]), up, off));
                                                sum += e0 + e1;
                                                w[8 * (c - b) + k / 2] = pack_half2(e0, e1);
                                            }
                                            l = fmaf(sum, ex[c].z, l);
                                        }
                                        tc_st16(s_at + 8 * b, w);
                                    }
                                    unit = next_unit(ex, unit);
                                    tc_wait_st();
                                    tc_before_sync();
                                    mbar_arrive(to + 8 * i);
                                    to = part_full;
                                    if (unit == kPromptAbsent) break;
                                    ok = wait(part_done + 8 * i, pn++);
                                    if (!ok) break;
                                    tc_after_sync();
                                }
                                goto given;
                            }
                            if (exact) {
                                float now = -INFINITY;
#pragma unroll
                                for (int b = 0; b < 8; ++b) {
                                    float top = -INFINITY;
#pragma unroll
                                    for (int k = 0; k < 16; ++k) top = fmaxf(top, __uint_as_float(v[16 * b + k]));
                                    now = fmaxf(now, fmaf(top, factor * ex[b].x, ex[b].y));
                                }
                                now = fmaxf(m, now);
                                const float by = exp2_fast(m - now);
                                m = now;
                                l *= by;
                                if (tl > t0 && __any_sync(0xffffffffu, by != 1.f)) {
#pragma unroll 1
                                    for (int q = 0; q < D / 16; ++q) {
                                        uint32_t o[16];
                                        tc_ld16(o_at + 16 * q, o);
                                        tc_wait_ld();
#pragma unroll
                                        for (int k = 0; k < 16; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * by);
                                        tc_st16(o_at + 16 * q, o);
                                    }
                                }
                            }
                            const float less = m == kNone ? 0.f : kPromptLift - m;
                            float most = ex[0].w, all = 0.f;
#pragma unroll
                            for (int q = 0; q < 2; ++q) {
                                uint32_t w[32];
#pragma unroll
                                for (int b = 4 * q; b < 4 * q + 4; ++b) {
                                    const float4 e = ex[b];
                                    const float by = factor * e.x, off = less + e.y;
                                    const uint64_t by2 = pair2(by, by), off2 = pair2(off, off);
                                    uint64_t sum = pair2(0.f, 0.f);
#pragma unroll
                                    for (int k = 16 * b; k < 16 * b + 16; k += 2) {
                                        float e0, e1;
                                        split2(fma2(pair2(__uint_as_float(v[k]), __uint_as_float(v[k + 1])), by2, off2), e0, e1);
                                        e0 = exp2_fast(e0);
                                        e1 = exp2_fast(e1);
                                        sum = add2(sum, pair2(e0, e1));
                                        w[k / 2 - 32 * q] = pack_half2(e0, e1);
                                    }
                                    float a0, a1;
                                    split2(sum, a0, a1);
                                    most = fmaxf(most, a0 + a1);
                                    all = fmaf(a0 + a1, e.z, all);
                                }
                                tc_st32(s_at + 32 * q, w);
                            }
                            if (exact || !__any_sync(0xffffffffu, most > kPromptMost)) {
                                l += all;
                                break;
                            }
                        }
                        tc_wait_st();
                        tc_before_sync();
                        mbar_arrive(pv_full + 8 * i);
                    given:
                        continue;
                    }
                    float tops[4] = {-FLT_MAX, -FLT_MAX, -FLT_MAX, -FLT_MAX};
#pragma unroll
                    for (int k = 0; k < 128; k += 2)
                        tops[k >> 1 & 3] = fmaxf(tops[k >> 1 & 3], fmaxf(__uint_as_float(v[k]), __uint_as_float(v[k + 1])));
                    const float top = fmaxf(fmaxf(tops[0], tops[1]), fmaxf(tops[2], tops[3]));
                    if (__any_sync(0xffffffffu, top > limit)) {  // a maximum moves: scale what was summed
                        const float now = top > limit ? top : m;
                        const float by = exp2_fast((m - now) * factor);
                        m = now;
                        limit = now + __fdividef(kPromptSlack, factor);
                        l *= by;
                        if (tl > t0) {
#pragma unroll 1
                            for (int q = 0; q < D / 16; ++q) {
                                uint32_t o[16];
                                tc_ld16(o_at + 16 * q, o);
                                tc_wait_ld();
#pragma unroll
                                for (int k = 0; k < 16; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * by);
                                tc_st16(o_at + 16 * q, o);
                            }
                        }
                    }
                    // ---- weights, where the scores were ----
                    const uint64_t off = pair2(-m, -m);
                    uint64_t sums[2] = {pair2(0.f, 0.f), pair2(0.f, 0.f)};
#pragma unroll
                    for (int q = 0; q < 2; ++q) {
#pragma unroll
                        for (int k = 64 * q; k < 64 * q + 64; k += 2) {
                            float e0, e1;
                            split2(fma2(add2(pair2(__uint_as_float(v[k]), __uint_as_float(v[k + 1])), off), factor2, lift2), e0, e1);
                            e0 = exp2_fast(e0);
                            e1 = exp2_fast(e1);
                            sums[k >> 1 & 1] = add2(sums[k >> 1 & 1], pair2(e0, e1));
                            v[k / 2] = pack_half2(e0, e1);
                        }
                        tc_st32(s_at + 32 * q, v + 32 * q);
                    }
                    float a0, a1;
                    split2(add2(sums[0], sums[1]), a0, a1);
                    l += a0 + a1;
                    tc_wait_st();
                    tc_before_sync();
                    mbar_arrive(pv_full + 8 * i);
                }
                if (ok) ok = wait(o_full + 8 * i, sn);
                if (!ok) break;
                tc_after_sync();
                ++sn;
            }
            // ---- the segment's end in this run ----
            const bool starts = seg.begin >= r0, ends = seg.end <= r1;
            const float top = kEight ? m : m * factor;
            l *= kPromptUnlift;  // O stays lifted until it is divided by its sum
            auto put = [&](__nv_bfloat16* to, const float* o, float inv) {  // 32 channels
#pragma unroll
                for (int k = 0; k < 32; k += 8) {
                    uint4 u;
                    uint32_t* const w = (uint32_t*)&u;
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const __nv_bfloat162 z = __floats2bfloat162_rn(o[k + 2 * e] * inv, o[k + 2 * e + 1] * inv);
                        w[e] = *(const uint32_t*)&z;
                    }
                    *(uint4*)(to + k) = u;
                }
            };
            if (starts && ends) {
                float inv = 0.f;
                __nv_bfloat16* const to = live ? attn_row(p, seg.n.q0, seg.h, r, top, l, true, inv) : nullptr;
                inv *= kPromptUnlift;
#pragma unroll
                for (int q = 0; q < D / 32; ++q) {
                    uint32_t v[32];
                    tc_ld32(o_at + 32 * q, v);
                    tc_wait_ld();
                    if (live) put(to + 32 * q, (const float*)v, inv);
                }
            } else {
                // The last CTA to arrive adds the parts in order; its own, if it finds all others there, from where it is.
                const int i0 = (int)(seg.begin / run), i1 = (int)((seg.end - 1) / run);
                uint32_t* const count = &ws->arrived[i0 * TILES + i];
                volatile uint32_t& others = arrived[starts ? 1 : 0][i];
                auto meet = [&]() {
                    mbar_arrive(joined + 8 * i);
                    return wait(joined + 8 * i, joins++);
                };
                if (row == 0) others = ld_acquire_u32(count);
                ok = meet();
                if (!ok) break;
                int mine = (int)blockIdx.x;
                if (others != (uint32_t)(i1 - i0)) {
                    mine = -1;
                    float4* const to = (float4*)(parts + (((int64_t)blockIdx.x * 2 + (starts ? 1 : 0)) * TILES + i) * Sh::kPartFloats);
                    if (t0 < t1) {
#pragma unroll 1
                        for (int q = 0; q < D / 32; ++q) {
                            uint32_t v[32];
                            tc_ld32(o_at + 32 * q, v);
                            tc_wait_ld();
#pragma unroll
                            for (int k = 0; k < 8; ++k)
                                to[(8 * q + k) * kPromptRows + row] =
                                    make_float4(__uint_as_float(v[4 * k]), __uint_as_float(v[4 * k + 1]), __uint_as_float(v[4 * k + 2]),
                                                __uint_as_float(v[4 * k + 3]));
                        }
                    }
                    ((float2*)(to + D / 4 * kPromptRows))[row] = make_float2(top, l);
                    __threadfence();
                    ok = meet();
                    if (ok && row == 0) {
                        others = atomicAdd(count, 1u);
                        added[starts ? 1 : 0][i] = 1u;
                    }
                    ok = ok && meet();
                    if (!ok) break;
                }
                if (others == (uint32_t)(i1 - i0)) {
                    __threadfence();
                    auto part_of = [&](int x) {
                        return (const float4*)(parts + (((int64_t)x * 2 + (x == i0 ? 1 : 0)) * TILES + i) * Sh::kPartFloats);
                    };
                    auto stats_of = [&](int x) {
                        return x == mine ? make_float2(top, l) : __ldcg((const float2*)(part_of(x) + D / 4 * kPromptRows) + row);
                    };
                    float best = -FLT_MAX, sum = 0.f;
#pragma unroll 4
                    for (int x = i0; x <= i1; ++x) best = fmaxf(best, stats_of(x).x);
#pragma unroll 4
                    for (int x = i0; x <= i1; ++x) {
                        const float2 st = stats_of(x);
                        sum += st.y * exp2_fast(st.x - best);
                    }
                    float inv = 0.f;
                    __nv_bfloat16* const to = live ? attn_row(p, seg.n.q0, seg.h, r, best, sum, true, inv) : nullptr;
                    inv *= kPromptUnlift;
#pragma unroll 1
                    for (int q = 0; q < D / 32; ++q) {
                        float o[32];
#pragma unroll
                        for (int k = 0; k < 32; ++k) o[k] = 0.f;
#pragma unroll 1
                        for (int x = i0; x <= i1; ++x) {
                            const float2 st = stats_of(x);
                            uint32_t v[32];
                            if (x == mine) {
                                tc_ld32(o_at + 32 * q, v);
                                tc_wait_ld();
                            } else {
#pragma unroll
                                for (int k = 0; k < 8; ++k) *(float4*)(v + 4 * k) = __ldcg(part_of(x) + (8 * q + k) * kPromptRows + row);
                            }
                            if (st.y != 0.f) {  // else nothing was seen there, and its channels may not have been written
                                const float by = exp2_fast(st.x - best);
#pragma unroll
                                for (int k = 0; k < 32; ++k) o[k] = fmaf(__uint_as_float(v[k]), by, o[k]);
                            }
                        }
                        if (live) put(to + 32 * q, o, inv);
                    }
                    if (row == 0) *count = 0u;
                }
            }
            if (seg.end >= r1) break;
            tc_before_sync();
            prompt_next(work, seg);
        }
        // A wait ran out: the results are lost, but the counters of the segments from here on have to be zero for the next
        // call.  So this CTA still counts itself, and whoever is last there clears them.
        if (!ok && row == 0)
#pragma unroll 1
            while (true) {
                const int which = seg.begin >= r0 ? 1 : 0;
                if (which == 0 || seg.end > r1) {
                    const int i0 = (int)(seg.begin / run), i1 = (int)((seg.end - 1) / run);
                    uint32_t* const count = &ws->arrived[i0 * TILES + i];
                    const uint32_t before = added[which][i] != 0u ? arrived[which][i] : atomicAdd(count, 1u);
                    if (before == (uint32_t)(i1 - i0)) *count = 0u;
                }
                if (seg.end >= r1) break;
                prompt_next(work, seg);
            }
    } else if (warp < Sh::kIssue) {
        // =============================== unpacking: a thread has half a row of two keys, 64 apart ====
        // so that a half of V's keys is unpacked while products still read the other
        set_registers<Sh::kUnpackRegs, Sh::kLaunchRegs>();
        int64_t left = 0;  // tiles of this run
        for (PromptSegment s = seg;;) {
            left += max(0, end_of(s) - first_of(s));
            if (s.end >= r1) break;
            prompt_next(work, s);
        }
        if constexpr (kEight) {
            // Pieces of 16 codes: eight lanes read a row of 128 (four one of 64), the warps 16 rows (32) at a time.
            constexpr int kLanes = D / 16, kStep = 128 / kLanes, kTurns = kPromptKeys / kStep;
            const int thread = tid & 127, piece = thread % kLanes, key0 = thread / kLanes, unpacker = warp - Sh::kUnpack;
            uint4 k[kTurns], v[kTurns];  // K of tile n, V of tile n - 1
            uint32_t there = 0u;         // which keys of this warp's word are there
            int32_t blocks[8], count = 0;
            auto places_of = [&](uint32_t t) {
                const volatile int32_t* const from = places[t & 3];
                count = from[8];
#pragma unroll
                for (int b = 0; b < 8; ++b) blocks[b] = from[b];
            };
            auto load = [&](uint4* x, int codes) {
#pragma unroll
                for (int i = 0; i < kTurns; ++i) {
                    const int key = key0 + kStep * i, block = D == 128 ? blocks[i] : key0 >> 4 ? blocks[2 * i + 1] : blocks[2 * i];
                    const bool here = block >= 0 && key < count;
                    x[i] = here ? *(const uint4*)((const char*)a.cache.pages + (int64_t)block * B::kBytes + codes + B::at(key & 15, piece)) : make_uint4(0u, 0u, 0u, 0u);
                }
            };
            auto look = [&]() {  // of the tile whose places are at hand
                int low = -1, high = -1;
#pragma unroll
                for (int w = 0; w < 4; ++w)
                    if (w == unpacker) low = blocks[2 * w], high = blocks[2 * w + 1];
                const int keys = min(max(count - 32 * unpacker, 0), 32);
                there = ((low >= 0 ? 0xffffu : 0u) | (high >= 0 ? 0xffff0000u : 0u)) & (keys == 32 ? 0xffffffffu : (1u << keys) - 1u);
            };
            auto unpack = [&](const uint4& c, int key, uint32_t to) {
                const uint32_t w[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    const int e = x ^ (piece >> 2 & 1);  // panels are as far apart as all banks: their pieces take turns
                    uint32_t h[4];
                    from_e4m3x4(e ? w[2] : w[0], h[0], h[1]);
                    from_e4m3x4(e ? w[3] : w[1], h[2], h[3]);
                    sts_v4(to + (piece >> 2) * Sh::kPanel + key * 128 + ((((piece & 3) * 2 + e) ^ (key & 7)) << 4), h[0], h[1], h[2], h[3]);
                }
            };
            if (left > 0) {
                ok = wait(place_full, 0);
                if (ok) {
                    places_of(0);
                    load(k, 0);
                    look();
                }
            }
#pragma unroll 1
            for (int64_t tile = 0; ok && tile <= left && left > 0; ++tile) {
                const uint32_t t = (uint32_t)tile, stage = t & 1;
                if (tile < left) {
                    if (lane == 0) {
                        seen_words[t & 3][unpacker] = there;
                        mbar_arrive(seen_full + 8 * (t & 3));
                    }
                    if (tile >= 2) ok = wait(k_empty + 8 * stage, (t >> 1) - 1);
                    if (!ok) break;
#pragma unroll
                    for (int i = 0; i < kTurns; ++i) unpack(k[i], key0 + kStep * i, smem + Sh::kK + stage * Sh::kParts * Sh::kTile);
                    fence_proxy_async_smem();
                    mbar_arrive(k_full + 8 * stage);
                    if (tile + 1 < left) {
                        ok = wait(place_full + 8 * ((t + 1) & 3), (t + 1) >> 2);
                        if (!ok) break;
                        places_of(t + 1);
                        load(k, 0);
                        look();
                    }
                }
                if (tile > 0) {  // V of the tile before
#pragma unroll
                    for (int i = 0; i < kTurns; ++i) {
                        if (i % (kTurns / 2) == 0 && tile > 1) ok = ok && wait(v_empty + 8 * (i / (kTurns / 2)), t - 2);
                        if (ok) unpack(v[i], key0 + kStep * i, smem + Sh::kV);
                    }
                    if (!ok) break;
                    fence_proxy_async_smem();
                    for (int i = 0; i < TILES; ++i) mbar_arrive(pv_full + 8 * i);
                }
                if (tile < left) {
                    places_of(t);
                    load(v, B::kV);
                    __syncwarp();
                    if (lane == 0) mbar_arrive(place_empty + 8 * (t & 3));
                }
            }
        } else {
        const int unpacker = warp - Sh::kUnpack, side = unpacker >> 1, key_in = 32 * (unpacker & 1) + lane;
        constexpr int kLoads = D / 64;  // 16-byte loads of half a row of codes
        struct Codes {  // of half a row, and the row's scales
            uint4 c[kLoads];
            uint32_t s[J / 2];
        };
        struct Places {  // the keys' blocks; null if they are not there
            const char* block[2];
        };
        const int row = key_in % kKvBlockTokens;  // of both keys in their blocks: tiles and pages are whole blocks
        auto places_of = [&](uint32_t t) {
            Places at;
            ok = wait(place_full + 8 * (t & 3), t >> 2);
            const volatile int32_t* const from = places[t & 3];
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                const int block = from[(key_in + 64 * x) / kKvBlockTokens];
                at.block[x] = ok && block >= 0 && key_in + 64 * x < from[8] ? (const char*)a.cache.pages + (int64_t)block * B::kBytes : nullptr;
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(place_empty + 8 * (t & 3));
            return at;
        };
        auto load = [&](Codes (&x)[2], const Places& at, int codes, int scales) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const bool here = at.block[i] != nullptr;
#pragma unroll
                for (int k = 0; k < kLoads; ++k)
                    x[i].c[k] = here ? *((const uint4*)(at.block[i] + codes + row * B::kRow + side * (B::kRow / 2)) + k) : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
                for (int k = 0; k < J / 2; ++k)
                    x[i].s[k] = here ? *((const uint32_t*)(at.block[i] + scales + row * B::kScaleRow) + k) : 0u;
            }
        };
        // Half a row's codes as binary16 into their place of a swizzled tile; with_rest twice as large, and the part that
        // rounding lost into `rest`.
        const uint32_t row_at = key_in * 128;
        auto unpack = [&](const Codes& x, uint32_t to, uint32_t rest, auto with_rest) {
            uint32_t wd[4 * kLoads];
#pragma unroll
            for (int k = 0; k < kLoads; ++k) wd[4 * k] = x.c[k].x, wd[4 * k + 1] = x.c[k].y, wd[4 * k + 2] = x.c[k].z, wd[4 * k + 3] = x.c[k].w;
            // word (c - 4 side) * J/2 + jh: channels 4 c.. of group 2 jh in its low half, of group 2 jh + 1 in its high one
#pragma unroll
            for (int c = 0; c < 4; c += 2)
#pragma unroll
                for (int jh = 0; jh < J / 2; ++jh) {
                    uint32_t even[4], odd[4];
                    const uint32_t s = decltype(with_rest)::value ? half2_mul(x.s[jh], 0x40004000u) : x.s[jh];
                    from_e2m1x8(wd[c * (J / 2) + jh], even);
                    from_e2m1x8(wd[(c + 1) * (J / 2) + jh], odd);
#pragma unroll
                    for (int jj = 0; jj < 2; ++jj) {
                        const uint32_t s2 = __byte_perm(s, 0u, jj ? 0x3232u : 0x1010u);
                        const uint32_t v[4] = {even[2 * jj], even[2 * jj + 1], odd[2 * jj], odd[2 * jj + 1]};
                        uint32_t h[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e) h[e] = half2_mul(v[e], s2);
                        const uint32_t at = jh * Sh::kPanel + row_at + (((jj * 4 + 2 * side + c / 2) ^ (key_in & 7)) << 4);
                        sts_v4(to + at, h[0], h[1], h[2], h[3]);
                        if constexpr (decltype(with_rest)::value) {
                            uint32_t g[4];
#pragma unroll
                            for (int e = 0; e < 4; ++e) g[e] = half2_rest(v[e], s2, h[e]);
                            sts_v4(rest + at, g[0], g[1], g[2], g[3]);
                        }
                    }
                }
        };
        constexpr uint32_t kHalf = 64 * 128;  // from a tile's first key to its 65th
        // K is unpacked a tile ahead of V: its two stages are free before V's one
        Codes k[2], v[2];        // K of tile n, V of tile n - 1
        Places here = {{nullptr, nullptr}};  // of tile n
        if (left > 0) {
            here = places_of(0);
            load(k, here, 0, B::kScaleK);
        }
#pragma unroll 1
        for (int64_t tile = 0; ok && tile <= left && left > 0; ++tile) {
            const Places now = here;
            const uint32_t t = (uint32_t)tile, stage = t & 1;
            if (tile < left) {
                const uint32_t there = __ballot_sync(0xffffffffu, (side == 0 ? now.block[0] : now.block[1]) != nullptr);
                if (lane == 0) {
                    seen_words[t & 3][unpacker] = there;
                    mbar_arrive(seen_full + 8 * (t & 3));
                }
                if (tile >= 2) ok = wait(k_empty + 8 * stage, (t >> 1) - 1);
                if (!ok) break;
                const uint32_t to = smem + Sh::kK + stage * Sh::kParts * Sh::kTile;
#pragma unroll
                for (int i = 0; i < 2; ++i) unpack(k[i], to + i * kHalf, to + Sh::kTile + i * kHalf, std::true_type{});
                fence_proxy_async_smem();
                mbar_arrive(k_full + 8 * stage);
                if (tile + 1 < left) {
                    here = places_of(t + 1);
                    if (!ok) break;
                    load(k, here, 0, B::kScaleK);
                }
            }
            if (tile > 0) {  // V of the tile before
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    if (tile > 1) ok = wait(v_empty + 8 * i, t - 2);
                    if (!ok) break;
                    unpack(v[i], smem + Sh::kV + i * kHalf, 0u, std::false_type{});
                }
                if (!ok) break;
                fence_proxy_async_smem();
                for (int i = 0; i < TILES; ++i) mbar_arrive(pv_full + 8 * i);
            }
            if (tile < left) load(v, now, B::kV, B::kScaleV);
        }
        }
    } else {
        // =============================== products of tile i: one thread issues ====
        set_registers<Sh::kIssueRegs, Sh::kLaunchRegs>();
        const int i = warp - Sh::kIssue;
        if (i == 2) {
            // =============================== another warp looks up pages, up to four tiles ahead of the unpacking ====
            // (by the unpacking warps themselves, lookups and addresses took a quarter of a tile's time: 270 us against 259)
            const int ps = a.cache.page_tokens, blocks = ps / kKvBlockTokens;
            constexpr int kAhead = kEight ? 4 : 1;  // tiles looked up at once: the exponents are another round trip
            uint32_t t = 0;
            for (PromptSegment s = seg; ok;) {
                const int end = end_of(s);
                float unit = kPromptAbsent;  // of values, that maxima are against or about to be
                for (int tl = first_of(s); ok && tl < end; tl += kAhead) {
                    const int key0 = (s.first_tile + tl) * kPromptKeys, key = key0 + kKvBlockTokens * lane;
                    int block = -1;
                    if (lane < kAhead * 8 && tl + (lane >> 3) < end && key < s.n.kv) {
                        const int at = p.by_page(key), page = a.block_table[s.b * a.table_stride + at];
                        if (page >= 0 && page < a.cache.num_pages) block = (page * a.cache.kv_heads + s.h) * blocks + (key - at * ps) / kKvBlockTokens;
                    }
                    float4 ex = make_float4(1.f, kPromptAbsent, 1.f, 0.f);
                    if constexpr (kEight) {
                        if (block >= 0) {
                            const uint32_t w = *(const uint32_t*)((const char*)a.cache.pages + (int64_t)block * B::kBytes + B::kExponents);
                            ex = make_float4(two_to(kv8_exponent(w, 0)), (float)kv8_exponent(w, 1), two_to(-kv8_exponent(w, 1)), 0.f);
                        }
                    }
                    for (int x = 0; x < kAhead && tl + x < end; ++x, ++t) {
                        const bool mine = lane >> 3 == x;
                        if (kEight) {
                            const bool here = mine && ex.y != kPromptAbsent;
                            auto highest_below = [&](float y) { return (float)__reduce_max_sync(0xffffffffu, here && ex.y < y ? (int)ex.y : (int)kPromptAbsent); };
                            const float most = highest_below(INFINITY), least = (float)__reduce_min_sync(0xffffffffu, here ? (int)ex.y : -(int)kPromptAbsent);
                            unit = fmaxf(unit, most);
                            if (unit - least > kKv8Apart) {  // (no block: least is above all)
                                ex.w = mine ? INFINITY : ex.w;
                                for (float next = most; next != kPromptAbsent; next = highest_below(unit - kKv8Apart)) unit = next;
                            }
                        }
                        if (t >= 4) ok = wait(place_empty + 8 * (t & 3), (t >> 2) - 1);
                        if (!ok) break;
                        if (mine) {
                            places[t & 3][lane & 7] = block;
                            if (kEight) exponents[t & 7][lane & 7] = ex;
                        }
                        if (lane == 0) places[t & 3][8] = min(kPromptKeys, s.n.kv - key0 - x * kPromptKeys);
                        __syncwarp();
                        if (lane == 0) mbar_arrive(place_full + 8 * (t & 3));
                    }
                }
                if (s.end >= r1) break;
                prompt_next(work, s);
            }
        }
        ok = i < TILES;
        constexpr uint32_t kQk = mma_desc(kPromptKeys, false), kPv = mma_desc(D, true);
        const uint32_t q_desc = tile_desc(smem + i * Sh::kTile, 16), k_desc = tile_desc(smem + Sh::kK, 16),
                       v_desc = tile_desc(smem + Sh::kV, Sh::kPanel);
        constexpr uint32_t kStep = Sh::kTile >> 4;  // from one tile to the next, in a descriptor
        const uint32_t s_at = tmem + 128 * i, o_at = tmem + 128 * (TILES + i);
        // The tiles' warps take turns: left alone they fall into step, and products and softmax of both alternate instead
        // of overlapping (394 us against 330 us, measured when the rest was slower).  The turn arrives at the barrier that the warp waits on for its
        // operands: each further wait cost it 200 to 400 cycles (with two more, for halves of P and V: 381 us).
        while (ok) {
            const int t0 = first_of(seg), t1 = end_of(seg);
            if (t0 < t1) {
                bool far = false;  // whether the units of the tile whose products come next are far apart
#pragma unroll 1
                for (int tl = t0 - 1; tl < t1; ++tl) {  // products of tile tl, scores of the next
                    const bool values = tl >= t0, next = tl + 1 < t1;
                    const uint32_t then = n + (values ? 1 : 0);  // the tile whose scores come next
                    // K is ready long before: first its wait, so that nothing comes between the products
                    ok = (!next || wait(k_full + 8 * (then & 1), then >> 1)) && (values ? wait(pv_full + 8 * i, n) : wait(q_full + 8 * i, sn));
                    if (!ok) break;
                    tc_after_sync();
                    const uint32_t k_at = k_desc + (then & 1) * Sh::kParts * kStep;
                    bool sums = tl > t0;
                    if (far) {  // all but the last of its products
                        const float4* const ex = exponents[n & 7];
                        for (float unit = next_unit(ex, next_unit(ex, INFINITY)); ok && unit != kPromptAbsent; unit = next_unit(ex, unit)) {
                            if (elected()) {
#pragma unroll 1
                                for (int k = 0; k < kPromptKeys / 16; ++k) tc_mma_ts(o_at, s_at + 8 * k, v_desc + k * (2048 >> 4), kPv, sums || k > 0);
                                tc_commit(part_done + 8 * i);
                            }
                            __syncwarp();
                            ok = wait(part_full + 8 * i, pn++);
                            tc_after_sync();
                            sums = true;
                        }
                        if (!ok) break;
                    }
                    if (elected()) {
                        if (values) {  // O_i += P_i V
#pragma unroll
                            for (int k = 0; k < kPromptKeys / 16; ++k) {
                                tc_mma_ts(o_at, s_at + 8 * k, v_desc + k * (2048 >> 4), kPv, sums || k > 0);
                                if (k == kPromptKeys / 32 - 1) tc_commit(v_empty);
                            }
                            tc_commit(v_empty + 8);
                        }
                        if (next) {  // S_i = Q_i K^T, all parts of K
#pragma unroll
                            for (int k = 0; k < Sh::kParts * (D / 16); ++k) {
                                constexpr auto at = [](int x) { return (uint32_t)((x % (D / 16) >> 2) * Sh::kPanel + (x & 3) * 32) >> 4; };
                                tc_mma(s_at, q_desc + at(k), k_at + k / (D / 16) * kStep + at(k), kQk, k > 0);
                            }
                            tc_commit(s_full + 8 * i);
                            tc_commit(k_empty + 8 * (then & 1));
                            if (kTurn) mbar_arrive(i == 1 ? pv_full : values ? pv_full + 8 : q_full + 8);
                        } else {
                            tc_commit(o_full + 8 * i);
                            if (kTurn) mbar_arrive(i == 0 ? pv_full + 8 : q_full);
                        }
                    }
                    __syncwarp();
                    n = then;
                    far = kEight && next && __any_sync(0xffffffffu, exponents[n & 7][0].w != 0.f);
                }
                ++sn;
            }
            if (!ok || seg.end >= r1) break;
            prompt_next(work, seg);
        }
        // nothing is in flight when TMEM goes back
        if (i < TILES) {
            if (elected()) tc_commit(drained);
            __syncwarp();
            attn_wait_quiet(drained, 0);
        }
    }
    tc_before_sync();
    __syncthreads();
    if (warp == Sh::kIssue)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" : : "r"(tmem), "r"(Sh::kColumns) : "memory");
}

template <typename F, int D, int TILES>
static rra_status_t prompt_launch(const AttnParams& p, int ctas, rra_stream_t stream) {
    using Sh = PromptShape<F, D, TILES>;
    const void* k = (const void*)kv_attention_prompt_kernel<F, D, TILES>;
    static_assert(Sh::kSmem <= 227 * 1024 - 1024, "shared memory");
    if (configure_cluster_kernel(k, Sh::kSmem) != cudaSuccess) {
        cudaGetLastError();
        return RRA_ERR_CUDA;
    }
    // The shares of the registers are of what the launch has: a build that launches with fewer would wait for them forever.
    static const bool enough = [k] {
        cudaFuncAttributes f;
        return cudaFuncGetAttributes(&f, k) == cudaSuccess && f.numRegs == Sh::kLaunchRegs;
    }();
    if (!enough) return RRA_ERR_CUDA;
    void* args[] = {(void*)&p};
    return serve_launch(k, dim3((unsigned)ctas), Sh::kThreads, Sh::kSmem, 1, stream, args);
}

size_t prefill_partial_bytes(int head_dim) {
    return (size_t)kPromptMaxCtas * 2 * 2 * kPromptRows * ((size_t)head_dim + 2) * sizeof(float);
}

template <typename F>
static rra_status_t prefill_launch(const AttnParams& p, int tiles, int ctas, rra_stream_t stream) {
    if (p.a.cache.head_dim == 128) return tiles == 2 ? prompt_launch<F, 128, 2>(p, ctas, stream) : prompt_launch<F, 128, 1>(p, ctas, stream);
    return tiles == 2 ? prompt_launch<F, 64, 2>(p, ctas, stream) : prompt_launch<F, 64, 1>(p, ctas, stream);
}

rra_status_t launch_prefill(const AttnParams& p, int bits, int tiles, int sms, rra_stream_t stream) {
    const int ctas = std::min(sms, kPromptMaxCtas);
    return bits == 8 ? prefill_launch<Cache8>(p, tiles, ctas, stream) : prefill_launch<Cache4>(p, tiles, ctas, stream);
}

}  // namespace rra
