// serve_prefill.cu -- attention over the 4-bit cache for prompts: many queries
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
#include <algorithm>
#include <type_traits>

#include "serve_attn.cuh"

namespace rra {

constexpr int kPromptKeys = 128;       // keys of a tile
constexpr int kPromptRows = 128;       // rows of a tile: the TMEM lanes
constexpr int kPromptMinRun = 4;       // key tiles a CTA takes at least
// What starting and ending a segment costs, in key tiles (3 requests of up to 1024 queries and 8192 keys, 64 heads over 8 of 128:
// 2, 3, 4, 5 and 6 take 304, 276, 259, 262 and 265 us: with less, a CTA that gets the shortest segments ends last).
constexpr int kPromptSegmentCost = 4;
constexpr int kPromptMaxCtas = 192;    // CTAs that the workspace has room for
constexpr float kPromptSlack = 8.f;    // log2 of how far weights may pass 1 before the maximum moves
// Weights enter their product with the values as binary16, which has few bits left below 2^-14 and none below 2^-25, while a
// row's sum counts them whole.  So they are taken 2^kPromptLift times as large: 2^(8 + 7) fits.  (131072 keys of one run, each
// 2^-25.3 of the largest: without it their share, 0.3 % of the values' size, was missing.)
constexpr float kPromptLift = 7.f, kPromptUnlift = 1.f / 128;
static_assert(kPromptMaxCtas * 2 <= kAttnMaxCtas, "a counter for each tile of a CTA's last segment");

template <int D, int TILES>
struct PromptShape {
    using B = KvBlock<D>;
    static constexpr int kRows = TILES * kPromptRows;
    static constexpr int kPanel = 128 * 128;            // 128 rows of 64 binary16, swizzled in 128 bytes
    static constexpr int kTile = D / 64 * kPanel;       // 128 rows of D binary16
    static constexpr int kK = TILES * kTile;            // after the queries: two stages of K, high and low parts
    static constexpr int kV = kK + 4 * kTile;           // V
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
    static constexpr int kPart = kPromptRows * (D + 2);      // floats of a part: rows in columns of 4 channels, statistics
    static constexpr int kSmem = 1024 + kEnd;
};

// ------------------------------------------------------------- tcgen05 ----
// A tile in shared memory as an operand.  Low word: start and, for the operand whose rows are keys, the distance of its
// panels of 64 columns, in 16 bytes; a step along the tile adds to the start.  High word: 8 rows apart by 1024 bytes,
// 128-byte swizzle.
__device__ __forceinline__ uint32_t tile_desc(uint32_t addr, uint32_t panels) { return addr >> 4 | panels >> 4 << 16; }
constexpr uint32_t kTileDescHigh = 1024u >> 4 | 1u << 14 | 2u << 29;
// binary32 sums of binary16 products, 128 rows, n columns; b_keys: B's rows are the summed index
constexpr uint32_t mma_desc(int n, bool b_keys) {
    return 1u << 4 | (b_keys ? 1u << 16 : 0u) | (uint32_t)(n >> 3) << 17 | (uint32_t)(128 >> 4) << 24;
}
__device__ __forceinline__ void tc_mma(uint32_t d, uint32_t a, uint32_t b, uint32_t desc, bool add) {
    asm volatile("{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\tsetp.ne.b32 p, %4, 0;\n\tmov.b64 a, {%1, %5};\n\t"
                 "mov.b64 b, {%2, %5};\n\ttcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, p;\n\t}"
                 : : "r"(d), "r"(a), "r"(b), "r"(desc), "r"(add ? 1 : 0), "r"(kTileDescHigh) : "memory");
}
__device__ __forceinline__ void tc_mma_ts(uint32_t d, uint32_t a, uint32_t b, uint32_t desc, bool add) {
    asm volatile("{\n\t.reg .pred p;\n\t.reg .b64 b;\n\tsetp.ne.b32 p, %4, 0;\n\tmov.b64 b, {%2, %5};\n\t"
                 "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %3, p;\n\t}"
                 : : "r"(d), "r"(a), "r"(b), "r"(desc), "r"(add ? 1 : 0), "r"(kTileDescHigh) : "memory");
}
// This warpgroup's registers a thread, from what it was launched with.
template <int N, int FROM>
__device__ __forceinline__ void set_registers() {
    if constexpr (N > FROM) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" : : "n"(N));
    if constexpr (N < FROM) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" : : "n"(N));
}
// One lane of the warp, the same for every call.
__device__ __forceinline__ bool elected() {
    uint32_t one;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(one));
    return one != 0;
}
__device__ __forceinline__ void tc_commit(uint32_t bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" : : "r"(bar) : "memory");
}
__device__ __forceinline__ void tc_before_sync() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_after_sync() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tc_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
// 32 columns of this warp's 32 lanes
__device__ __forceinline__ void tc_ld32(uint32_t a, uint32_t* v) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,"
        "%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
          "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15]), "=r"(v[16]),
          "=r"(v[17]), "=r"(v[18]), "=r"(v[19]), "=r"(v[20]), "=r"(v[21]), "=r"(v[22]), "=r"(v[23]), "=r"(v[24]),
          "=r"(v[25]), "=r"(v[26]), "=r"(v[27]), "=r"(v[28]), "=r"(v[29]), "=r"(v[30]), "=r"(v[31])
        : "r"(a));
}
__device__ __forceinline__ void tc_st32(uint32_t a, const uint32_t* v) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,"
        "%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31};"
        :
        : "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
          "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15]), "r"(v[16]), "r"(v[17]), "r"(v[18]),
          "r"(v[19]), "r"(v[20]), "r"(v[21]), "r"(v[22]), "r"(v[23]), "r"(v[24]), "r"(v[25]), "r"(v[26]), "r"(v[27]),
          "r"(v[28]), "r"(v[29]), "r"(v[30]), "r"(v[31]), "r"(a)
        : "memory");
}
__device__ __forceinline__ void tc_ld16(uint32_t a, uint32_t* v) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
          "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
        : "r"(a));
}
__device__ __forceinline__ void tc_st16(uint32_t a, const uint32_t* v) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15};"
        :
        : "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
          "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15]), "r"(a)
        : "memory");
}
__device__ __forceinline__ void mbar_arrive(uint32_t bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" : : "r"(bar) : "memory");
}
__device__ __forceinline__ void sts_v4(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" : : "r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}
__device__ __forceinline__ uint64_t pair2(float a, float b) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ void split2(uint64_t v, float& a, float& b) { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v)); }
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint32_t half2_mul(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
// a * b - c, rounded once: with c the rounded product, what its rounding lost
__device__ __forceinline__ uint32_t half2_rest(uint32_t a, uint32_t b, uint32_t c) {
    const __half2 r = __hfma2(*(const __half2*)&a, *(const __half2*)&b, __hneg2(*(const __half2*)&c));
    return *(const uint32_t*)&r;
}

// --------------------------------------------------------- work as a row ----
// Chunk c of request b: its rows' key tiles.
struct PromptItem {
    int32_t first_tile, tiles;
};
template <int kRows>
__device__ __forceinline__ PromptItem prompt_item(const AttnParams& p, const AttnLengths& n, int c) {
    const int rows = n.qn * p.group, last = min(rows, (c + 1) * kRows) - 1;
    const int end = p.a.causal ? max(0, n.kv - n.qn + p.by_group(last) + 1) : n.kv;
    const int first = p.window > 0 ? max(0, n.kv - n.qn + p.by_group(c * kRows) - p.window + 1) : 0;
    PromptItem t;
    t.first_tile = first / kPromptKeys;
    t.tiles = max(1, (end + kPromptKeys - 1) / kPromptKeys - t.first_tile);
    return t;
}
template <int kRows>
__device__ __forceinline__ int prompt_chunks(const AttnParams& p, const AttnLengths& n) {
    return (n.qn * p.group + kRows - 1) / kRows;
}

// A segment: chunk c of request b, KV head h, at begin..end of the row of all segments: first its cost, then its tiles.
struct PromptSegment {
    AttnLengths n;
    int32_t b, c, h, chunks, first_tile;
    int64_t begin, end;
};
template <int kRows>
__device__ __forceinline__ void prompt_load(const AttnParams& p, PromptSegment& s) {
    s.n = attn_lengths(p, s.b);
    s.chunks = prompt_chunks<kRows>(p, s.n);
    const PromptItem t = prompt_item<kRows>(p, s.n, s.c);
    s.first_tile = t.first_tile;
    s.end = s.begin + t.tiles + kPromptSegmentCost;
}
template <int kRows>
__device__ __forceinline__ void prompt_next(const AttnParams& p, PromptSegment& s) {
    s.begin = s.end;
    if (++s.c >= s.chunks) {
        s.c = 0;
        do {
            if (++s.b == p.a.requests) s.b = 0, ++s.h;
            s.n = attn_lengths(p, s.b);
        } while (s.n.qn == 0 && s.h < p.a.cache.kv_heads);  // some request has queries: there is a segment
    }
    prompt_load<kRows>(p, s);
}

// Exclusive sum over the block, and the total.
template <int kWarps>
__device__ __forceinline__ int64_t block_sum(int64_t v, int64_t& total, int64_t* part) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int64_t inc = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t up = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += up;
    }
    __syncthreads();
    if (lane == 31) part[warp] = inc;
    __syncthreads();
    int64_t before = 0;
    total = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        if (w < warp) before += part[w];
        total += part[w];
    }
    return before + inc - v;
}

template <int D, int TILES>
__global__ void __launch_bounds__(PromptShape<D, TILES>::kThreads, 1) kv_attention_prompt_kernel(const __grid_constant__ AttnParams p) {
    using Sh = PromptShape<D, TILES>;
    using B = KvBlock<D>;
    constexpr int J = B::kGroups;
    extern __shared__ unsigned char raw_smem[];
    __shared__ __align__(8) uint64_t bar_mem[5 * TILES + 4 + 2 + 4 + 1 + 8];
    __shared__ int64_t part[Sh::kWarps];
    __shared__ volatile uint32_t seen_words[4][4];  // of the last four tiles, which keys are there
    __shared__ volatile int32_t places[4][9];  // of four tiles: the cache's blocks of its keys (-1: none), and how many keys there are
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
                   seen_full = v_empty + 16, drained = seen_full + 32, place_full = drained + 8, place_empty = place_full + 32;
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

    // ---- this CTA's run: chunks of the requests, then the chunks' tiles, the same for every head ----
    int64_t total_chunks = 0;
    for (int b0 = 0; b0 < a.requests; b0 += Sh::kThreads) {
        const int b = b0 + tid;
        int64_t all;
        const int64_t at = block_sum<Sh::kWarps>(b < a.requests ? prompt_chunks<Sh::kRows>(p, attn_lengths(p, b)) : 0, all, part);
        if (b < a.requests) chunk_sums[b] = (int32_t)(total_chunks + at);
        total_chunks += all;
    }
    // Chunks are counted in 32 bits, which the rows of any batch fit.  More of them are the same rows over and over: cu_q does
    // not ascend, and there is no result to give.
    if (total_chunks > INT32_MAX) return;
    if (tid == 0) chunk_sums[a.requests] = (int32_t)total_chunks;
    __syncthreads();
    auto owner = [&](int n, int& b, int& c) {
        int low = 0, high = a.requests;
        while (high - low > 1) {
            const int mid = (low + high) >> 1;
            if (chunk_sums[mid] <= n) low = mid;
            else high = mid;
        }
        b = low;
        c = n - chunk_sums[low];
    };
    auto cost_of = [&](int n) {
        int b, c;
        owner(n, b, c);
        return prompt_item<Sh::kRows>(p, attn_lengths(p, b), c).tiles + kPromptSegmentCost;
    };
    int64_t per_head = 0;
    for (int n0 = 0; n0 < total_chunks; n0 += Sh::kThreads) {
        int64_t all;
        block_sum<Sh::kWarps>(n0 + tid < total_chunks ? cost_of(n0 + tid) : 0, all, part);
        per_head += all;
    }
    const int64_t total = per_head * a.cache.kv_heads;
    int64_t run = (total + gridDim.x - 1) / gridDim.x;
    run = run < kPromptMinRun + kPromptSegmentCost ? kPromptMinRun + kPromptSegmentCost : run;
    const int64_t r0 = (int64_t)blockIdx.x * run, r1 = r0 + run < total ? r0 + run : total;
    if (r0 >= r1) return;
    {
        const int64_t h = r0 / per_head, w = r0 - h * per_head;
        int64_t before = 0;
        for (int n0 = 0; n0 < total_chunks && before <= w; n0 += Sh::kThreads) {
            int64_t all;
            const int n = n0 + tid, cost = n < total_chunks ? cost_of(n) : 0;
            const int64_t at = before + block_sum<Sh::kWarps>(cost, all, part);
            if (at <= w && w < at + cost) {
                owner(n, start.b, start.c);
                start.h = (int)h;
                start.begin = h * per_head + at;
            }
            before += all;
        }
    }
    if (warp == Sh::kIssue) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" : : "r"(smem_u32(&tmem_base)), "r"(Sh::kColumns) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tc_before_sync();
    __syncthreads();
    tc_after_sync();
    const uint32_t tmem = tmem_base;
    PromptSegment seg = start;
    prompt_load<Sh::kRows>(p, seg);
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
            float m = -FLT_MAX, limit = -FLT_MAX, l = 0.f, factor = 1.f;
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
                    factor *= 0.5f;  // K is held twice as large
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
            const float top = m * factor;
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
                    float4* const to = (float4*)(parts + (((int64_t)blockIdx.x * 2 + (starts ? 1 : 0)) * TILES + i) * Sh::kPart);
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
                        return (const float4*)(parts + (((int64_t)x * 2 + (x == i0 ? 1 : 0)) * TILES + i) * Sh::kPart);
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
            prompt_next<Sh::kRows>(p, seg);
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
                prompt_next<Sh::kRows>(p, seg);
            }
    } else if (warp < Sh::kIssue) {
        // =============================== unpacking: a thread has half a row of two keys, 64 apart ====
        // so that a half of V's keys is unpacked while products still read the other
        set_registers<Sh::kUnpackRegs, Sh::kLaunchRegs>();
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
        int64_t left = 0;  // tiles of this run
        for (PromptSegment s = seg;;) {
            left += max(0, end_of(s) - first_of(s));
            if (s.end >= r1) break;
            prompt_next<Sh::kRows>(p, s);
        }
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
                const uint32_t to = smem + Sh::kK + stage * 2 * Sh::kTile;
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
    } else {
        // =============================== products of tile i: one thread issues ====
        set_registers<Sh::kIssueRegs, Sh::kLaunchRegs>();
        const int i = warp - Sh::kIssue;
        if (i == 2) {
            // =============================== another warp looks up pages, up to four tiles ahead of the unpacking ====
            // (by the unpacking warps themselves, lookups and addresses took a quarter of a tile's time: 270 us against 259)
            const int ps = a.cache.page_tokens, blocks = ps / kKvBlockTokens;
            uint32_t t = 0;
            for (PromptSegment s = seg; ok;) {
                const int end = end_of(s);
                for (int tl = first_of(s); ok && tl < end; ++tl, ++t) {
                    const int key0 = (s.first_tile + tl) * kPromptKeys, key = key0 + kKvBlockTokens * lane;
                    int block = -1;
                    if (lane < kPromptKeys / kKvBlockTokens && key < s.n.kv) {
                        const int at = p.by_page(key), page = a.block_table[s.b * a.table_stride + at];
                        if (page >= 0 && page < a.cache.num_pages) block = (page * a.cache.kv_heads + s.h) * blocks + (key - at * ps) / kKvBlockTokens;
                    }
                    if (t >= 4) ok = wait(place_empty + 8 * (t & 3), (t >> 2) - 1);
                    if (!ok) break;
                    if (lane < kPromptKeys / kKvBlockTokens) places[t & 3][lane] = block;
                    if (lane == 0) places[t & 3][8] = min(kPromptKeys, s.n.kv - key0);
                    __syncwarp();
                    if (lane == 0) mbar_arrive(place_full + 8 * (t & 3));
                }
                if (s.end >= r1) break;
                prompt_next<Sh::kRows>(p, s);
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
#pragma unroll 1
                for (int tl = t0 - 1; tl < t1; ++tl) {  // products of tile tl, scores of the next
                    const bool values = tl >= t0, next = tl + 1 < t1;
                    const uint32_t then = n + (values ? 1 : 0);  // the tile whose scores come next
                    // K is ready long before: first its wait, so that nothing comes between the products
                    ok = (!next || wait(k_full + 8 * (then & 1), then >> 1)) && (values ? wait(pv_full + 8 * i, n) : wait(q_full + 8 * i, sn));
                    if (!ok) break;
                    tc_after_sync();
                    const uint32_t k_at = k_desc + (then & 1) * 2 * kStep;
                    if (elected()) {
                        if (values) {  // O_i += P_i V
#pragma unroll
                            for (int k = 0; k < kPromptKeys / 16; ++k) {
                                tc_mma_ts(o_at, s_at + 8 * k, v_desc + k * (2048 >> 4), kPv, tl > t0 || k > 0);
                                if (k == kPromptKeys / 32 - 1) tc_commit(v_empty);
                            }
                            tc_commit(v_empty + 8);
                        }
                        if (next) {  // S_i = Q_i K^T, both parts of K
#pragma unroll
                            for (int k = 0; k < 2 * (D / 16); ++k) {
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
                }
                ++sn;
            }
            if (!ok || seg.end >= r1) break;
            prompt_next<Sh::kRows>(p, seg);
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

template <int D, int TILES>
static rra_status_t prompt_launch(const AttnParams& p, int ctas, rra_stream_t stream) {
    using Sh = PromptShape<D, TILES>;
    const void* k = (const void*)kv_attention_prompt_kernel<D, TILES>;
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

rra_status_t launch_prefill(const AttnParams& p, int tiles, int sms, rra_stream_t stream) {
    const int ctas = std::min(sms, kPromptMaxCtas);
    if (p.a.cache.head_dim == 128) return tiles == 2 ? prompt_launch<128, 2>(p, ctas, stream) : prompt_launch<128, 1>(p, ctas, stream);
    return tiles == 2 ? prompt_launch<64, 2>(p, ctas, stream) : prompt_launch<64, 1>(p, ctas, stream);
}

}  // namespace rra
