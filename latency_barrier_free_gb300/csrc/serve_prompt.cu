// serve_prompt.cu -- attention of whole prompts over their own keys and values
// (rra_serve.h), on the tensor cores' own memory.
//
// A tile is 128 rows: `group` query heads of one KV head, of 128 / group neighbouring
// tokens, so that heads share their keys and values and few tokens fill a tile.
// A CTA takes a segment, TILES tiles of one request and KV head, and walks the
// keys that any of their rows sees, 128 at a time: queries, keys and values come
// by TMA, one thread for each tile issues
//     S_i = Q_i K^T,   O_i += P_i V        (tcgen05.mma, sums in TMEM)
// and two warpgroups for each tile turn S_i into weights P_i, in place.  A warp has
// 16 rows, four threads a row (the layout of an accumulator of mma): one thread a row
// would take twice as long from scores to weights, and the tensor cores have nothing
// but the other tile's products to do meanwhile (TMEM: 128 columns of S and D of O a
// tile, twice).
//
// The maximum that weights are taken against is that of a row's first tile, until
// weights get large: their sum, which is needed anyway, shows it (an earlier form
// looked for each tile's maximum first, 400 of the 1350 cycles from scores to
// weights).  Only then the tile's maximum is found, and O scaled, in TMEM.
//
// A value that is infinite or NaN would spoil rows that do not see it: 0 times it
// is NaN.  So in tiles that some row does not see whole, a warp looks values over in
// shared memory before products may read them; such elements become 0 there, and
// rows that see them get them at their end.
//
// Few segments are dealt out whole, the longest first, to and fro over the CTAs.
// Many, or where that leaves CTAs idle (a few long ones), are cut into equal runs
// of key tiles, one per CTA (serve_tc.cuh); what a run has of a segment it shares
// goes to the workspace, and the last CTA to arrive adds the parts in order.
//
// 64 heads over 8 of 128, bfloat16, prompts of 8192 and 78 tokens, 1.1 TFLOP:
// 775 us among other calls, 1420 TFLOP/s, at the power limit; 8 over 1, one of 16384
// 359 us, 1530 TFLOP/s (large library products reach 1937).  The products of 256 rows
// and 128 keys take 2080 cycles at their full rate; the pipe is 55 to 70 % busy.  The
// rest is the chain of one tile, scores to weights (about 1000 cycles) and its two
// products, where the other tile's products do not cover it.  Few short ones are
// latency: 5 prompts, 14 heads over 2 of 64, take 7.6 us.
#include <algorithm>
#include <cmath>

#include <cuda.h>

#include "serve_tc.cuh"

namespace rra {


constexpr int kDealRequests = 1024;  // up to so many requests segments are dealt out: their order is found in shared memory
// And up to so many segments a CTA.  With more, runs are as even, and a CTA's next segment mostly reads the keys that the one
// before it read (32 heads over 32: 16 requests of 1024 tokens, 14 segments a CTA, 228 us, in runs 206; 64 of 300, 27, 277 and 257.
// 64 heads over 8: 64 of 512, 54, 541 and 481; 3 of 2000, 10, 184 and 193; one of 500, 1, 16.6 and 31.6).
constexpr int kDealItems = 10, kDealChunks = kDealItems * kPromptMaxCtas;
constexpr int kDealExcess = 10;  // key tiles that a CTA may have above the mean: about what finding runs and joining parts costs

struct PromptParams {
    CUtensorMap q, k, v;  // [channels][heads][tokens]; boxes of 64 channels, q: group heads of `span` tokens, k, v: 128 tokens
    rra_prompt_attention_args_t a;
    float factor;         // |scale| log2(e), above 0
    float flip;           // what scores are multiplied with first: 1, or -1 or 0 with the scale
    int32_t heads_of_kv;  // query heads of a KV head
    int32_t group, parts; // query heads of a tile; tiles for all heads of a KV head (1 up to 128 heads)
    int32_t span;         // tokens of a tile
    int32_t window;       // a.window, at most 2^30
    Divisor by_group, by_parts, by_chunk;  // by_chunk: tokens of a CTA
};

template <typename T, int D, int TILES>
struct WholeShape {
    static constexpr bool kHalf = std::is_same<T, __half>::value;
    // Weights are 2^kLift times as large as they are; a thread's share of a row in a tile may add up to kMost: more is no
    // binary16, and sums of large values stay far from binary32's end.
    static constexpr float kLift = kHalf ? 7.f : 0.f, kUnlift = kHalf ? 1.f / 128 : 1.f, kMost = kHalf ? 32768.f : 1024.f;
    static constexpr int kPanel = 128 * 128;       // 128 rows of 64 channels, swizzled in 128 bytes
    static constexpr int kTile = D / 64 * kPanel;
    static constexpr int kStages = 2;              // of K, and of V
    static constexpr int kK = TILES * kTile, kV = kK + kStages * kTile, kEnd = kV + kStages * kTile;
    static constexpr int kSums = kK;               // before any tile: running sums of the requests' chunks
    static_assert(4 * (RRA_SERVE_MAX_REQUESTS + 1) <= kEnd - kSums, "the sums fit");
    // Warps: eight of softmax for each tile (a warp reaches the 32 TMEM lanes of its number modulo 4; the first four have the
    // first 16 of them), then one for each tile that issues its products, one for the copies, and one that looks values over.
    static constexpr int kSoftmaxWarps = 8 * TILES, kIssue = kSoftmaxWarps, kCopy = kIssue + 2, kLook = kIssue + 3, kWarps = kIssue + 4;
    static constexpr int kThreads = 32 * kWarps;
    static constexpr int kLaunchRegs = 65536 / kThreads / 8 * 8;
    // The softmax holds 64 scores a thread (two tiles, 96 for all warps: 5 % slower).
    static constexpr int kSoftmaxRegs = TILES == 2 ? 104 : 184;
    static constexpr int kIssueRegs = TILES == 2 ? 64 : 128;
    static_assert(2 * TILES * kSoftmaxRegs + kIssueRegs <= (2 * TILES + 1) * kLaunchRegs, "what the launch has");
    static constexpr int kColumns = TILES == 2 ? 512 : 256;    // of TMEM: S of every tile, then O of every tile
    static constexpr int kPartFloats = kPromptRows * (D + 2);  // of a part: rows in columns of 4 channels, statistics
    static constexpr int kSmem = 1024 + kEnd;
    static_assert(20 * kDealRequests + 4 * (kDealChunks + 1) <= kEnd - kSums, "and what dealing out needs");
};

// The work: chunks of TILES * span tokens of every request, for every head (a KV head and the part of its query heads).
template <int TILES>
struct WholeWork {
    const PromptParams& p;
    __device__ __forceinline__ int requests() const { return p.a.requests; }
    __device__ __forceinline__ int heads() const { return p.a.kv_heads * p.parts; }
    __device__ __forceinline__ AttnLengths lengths(int b) const {
        const int most = (int)p.a.tokens;
        AttnLengths r;
        r.q0 = min(max(p.a.cu[b], 0), most);
        r.kv = r.qn = max(0, min(max(p.a.cu[b + 1], 0), most) - r.q0);
        return r;
    }
    __device__ __forceinline__ int chunks(const AttnLengths& n) const { return n.qn > 0 ? p.by_chunk(n.qn - 1) + 1 : 0; }
    __device__ __forceinline__ PromptItem item(const AttnLengths& n, int c) const {
        const int first = c * TILES * p.span, last = min(n.qn, first + TILES * p.span) - 1;
        return prompt_item(p.window > 0 ? max(0, first - p.window + 1) : 0, p.a.causal ? last + 1 : n.qn);
    }
};

// Exclusive sum over the block, and the total, in 32 bits; part: a word for each warp.
template <int kWarps>
__device__ __forceinline__ int short_sum(int v, int& total, int32_t* part) {
    static_assert(kWarps <= 32, "a lane for each warp");
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int inc = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int up = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += up;
    }
    if (lane == 31) part[warp] = inc;
    __syncthreads();
    int w = lane < kWarps ? part[lane] : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int up = __shfl_up_sync(0xffffffffu, w, o);
        if (lane >= o) w += up;
    }
    total = __shfl_sync(0xffffffffu, w, 31);
    const int before = __shfl_sync(0xffffffffu, w, warp > 0 ? warp - 1 : 0);
    __syncthreads();
    return inc - v + (warp > 0 ? before : 0);
}

// Deals the segments out: this CTA's in items[] as (first token, tokens, chunk, head), their number; 0 if there is nothing to
// do, -1 if the work is better cut into runs.  Segment i of all, by number of chunk from the last down, then by request, those
// with most chunks first, then by head, goes to CTA i of the first round, to CTA gridDim - 1 - i of the second, and so on:
// where later chunks see more keys that is the longest first.  scratch: 20 kDealRequests + 4 (kDealChunks + 1) bytes, sums: a
// word for each warp; the whole block.
template <int kWarps, typename W>
__device__ __forceinline__ int prompt_deal(const W& work, int32_t* scratch, int64_t* sums, int4* items) {
    constexpr int kThreads = 32 * kWarps;
    const int tid = (int)threadIdx.x, requests = work.requests(), heads = work.heads(), ctas = (int)gridDim.x;
    if (requests > kDealRequests) return -1;
    int32_t *const q0 = scratch, *const qn = q0 + kDealRequests, *const chunks = qn + kDealRequests, *const sorted = chunks + kDealRequests,
                   *const order = sorted + kDealRequests, *const levels = order + kDealRequests;
    int mine = 0, longest = 0, before;
    for (int b = tid; b < requests; b += kThreads) {
        const AttnLengths n = work.lengths(b);
        q0[b] = n.q0, qn[b] = n.qn;
        mine += min(chunks[b] = work.chunks(n), kDealChunks + 1);
        longest = max(longest, n.qn);
    }
    short_sum<kWarps>(mine, before, (int32_t*)sums);
    const int64_t total = (int64_t)before * heads;
    if (total == 0) return 0;
    if (total > (int64_t)kDealItems * ctas) return -1;
    for (int b = tid; b < requests; b += kThreads) {
        const int c = chunks[b];
        int rank = 0;
        for (int x = 0; x < requests; ++x) rank += chunks[x] > c || (chunks[x] == c && x < b);
        sorted[rank] = c;
        order[rank] = b;
    }
    // CTAs' shares differ by no more than the longest segment's cost
    const bool uneven = __syncthreads_or(longest > (kDealExcess - kPromptSegmentCost) * kPromptKeys);
    // level i is the chunks sorted[0] - 1 - i: how many there are at lower levels
    const int most = sorted[0];
    before = 0;
    for (int i0 = 0; i0 < most; i0 += kThreads) {
        const int i = i0 + tid, c = most - 1 - i;
        int low = 0, high = requests;  // requests with more than c chunks
        while (i < most && low < high) {
            const int mid = (low + high) >> 1;
            if (sorted[mid] > c) low = mid + 1;
            else high = mid;
        }
        int all;
        const int at = before + short_sum<kWarps>(i < most ? low : 0, all, (int32_t*)sums);  // up to kDealRequests * kThreads
        if (i < most) levels[i] = at;
        before += all;
    }
    if (tid == 0) levels[most] = before;
    __syncthreads();
    const int rounds = (int)((total + ctas - 1) / ctas);
    // segment of CTA x in round k
    auto item = [&](int x, int k, int4& to) {
        const int at = k * ctas + (k & 1 ? ctas - 1 - x : x);
        if (at >= total) return false;
        const int y = at / heads;
        int low = 0, high = most;
        while (high - low > 1) {
            const int mid = (low + high) >> 1;
            if (levels[mid] <= y) low = mid;
            else high = mid;
        }
        const int b = order[y - levels[low]];
        to = make_int4(q0[b], qn[b], most - 1 - low, at - y * heads);
        return true;
    };
    if (uneven) {
        int cost = 0;
        int4 it;
        for (int k = 0; tid < ctas && k < rounds; ++k)
            if (item(tid, k, it)) cost += work.item(AttnLengths{it.x, it.y, it.y}, it.z).tiles + kPromptSegmentCost;
        int all;
        short_sum<kWarps>(cost, all, (int32_t*)sums);  // kDealItems segments a CTA of up to kDealChunks * 2 tiles each
        if (__syncthreads_or(cost > all / ctas + kDealExcess)) return -1;
    }
    for (int k = tid; k < rounds; k += kThreads) {
        int4 it;
        if (item((int)blockIdx.x, k, it)) items[k] = it;
    }
    const int last = (rounds - 1) * ctas + (rounds - 1 & 1 ? ctas - 1 - (int)blockIdx.x : (int)blockIdx.x);
    return last < total ? rounds : rounds - 1;
}

__device__ __forceinline__ void tma_load(uint32_t dst, const CUtensorMap* map, int channel, int head, int token, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];"
        :
        : "r"(dst), "l"(map), "r"(channel), "r"(head), "r"(token), "r"(bar)
        : "memory");
}
// 16 lanes' rows: of 8 (x8: 64) columns a thread has columns 2 t, 2 t + 1 of row g, then of row g + 8 (t = lane % 4, g = lane / 4).
__device__ __forceinline__ void tc_ld_rows64(uint32_t a, uint32_t* v) {
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,"
        "%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
          "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15]), "=r"(v[16]),
          "=r"(v[17]), "=r"(v[18]), "=r"(v[19]), "=r"(v[20]), "=r"(v[21]), "=r"(v[22]), "=r"(v[23]), "=r"(v[24]),
          "=r"(v[25]), "=r"(v[26]), "=r"(v[27]), "=r"(v[28]), "=r"(v[29]), "=r"(v[30]), "=r"(v[31])
        : "r"(a));
}
__device__ __forceinline__ void tc_ld_rows32(uint32_t a, uint32_t* v) {
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
          "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
        : "r"(a));
}
__device__ __forceinline__ void tc_st_rows32(uint32_t a, const uint32_t* v) {
    asm volatile(
        "tcgen05.st.sync.aligned.16x256b.x4.b32 [%16], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15};"
        :
        : "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
          "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15]), "r"(a)
        : "memory");
}
// 32 columns, of each 4 a thread has column t of row g, then of row g + 8.
__device__ __forceinline__ void tc_st_weights(uint32_t a, const uint32_t* v) {
    asm volatile(
        "tcgen05.st.sync.aligned.16x128b.x8.b32 [%16], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15};"
        :
        : "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
          "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15]), "r"(a)
        : "memory");
}
__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}
// Word j of the four threads of a row goes to thread j: x[i] becomes thread i's word t.
__device__ __forceinline__ void quad_transpose(uint32_t* x) {
    const int t = threadIdx.x & 3;
#pragma unroll
    for (int o = 1; o <= 2; o <<= 1) {
        const bool up = t & o;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (i & o) continue;
            const uint32_t got = __shfl_xor_sync(0xffffffffu, up ? x[i] : x[i + o], o);
            if (up) x[i] = got;
            else x[i + o] = got;
        }
    }
}
template <typename T>
__device__ __forceinline__ uint32_t pack2(float a, float b);
template <>
__device__ __forceinline__ uint32_t pack2<__half>(float a, float b) { return pack_half2(a, b); }
template <>
__device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(float a, float b) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *(const uint32_t*)&h;
}
// Of each half of a word whether it is infinite or NaN: its top bit.
template <bool kHalf>
__device__ __forceinline__ uint32_t not_finite(uint32_t w) {
    return ((w & (kHalf ? 0x7c007c00u : 0x7f807f80u)) + (kHalf ? 0x04000400u : 0x00800080u)) & 0x80008000u;
}

// What tiles of a segment some row does not see whole: keys below `from` or from `to` on are in them.
struct PromptEdge {
    int from, to;
    __device__ __forceinline__ bool masks(int key0) const { return key0 < from || key0 + kPromptKeys > to; }
};

// A row's share of a segment: keys lo .. hi of the key tiles t0 .. t1, those of them that `edge` cuts.
struct PromptShare {
    PromptEdge edge;
    int64_t token0;
    int kv_head, t0, t1, lo, hi;
};
// Adds the row's values that are infinite or NaN to every fourth channel of its output, or of its part (the row's first
// thread's first word of it), from c on.  Rare, hence out of line and after the rest has been written.
template <typename T>
__device__ __noinline__ void add_lost(const PromptParams& p, const PromptShare& s, T* out, float* part, int c, int end) {
    for (; c < end; c += 4) {
        float sum = 0.f;
        for (int t = s.t0; t < s.t1; ++t) {
            const int key0 = t * kPromptKeys;
            if (!s.edge.masks(key0)) continue;
            for (int j = max(s.lo, key0); j < min(s.hi, key0 + kPromptKeys); ++j) {
                const float v = (float)*((const T*)p.a.v + (s.token0 + j) * p.a.v_token_stride + s.kv_head * p.a.v_head_stride + c);
                if (!(fabsf(v) < INFINITY)) sum += v;
            }
        }
        if (sum == 0.f) continue;
        if (out != nullptr) out[c] = (T)((float)out[c] + sum);
        else part[c / 8 * 128 + c % 8 / 2 * 4 + c % 2] += sum;
    }
}

template <typename T, int D, int TILES>
__global__ void __launch_bounds__(WholeShape<T, D, TILES>::kThreads, 1) prompt_attention_kernel(const __grid_constant__ PromptParams p) {
    using Sh = WholeShape<T, D, TILES>;
    extern __shared__ unsigned char raw_smem[];
    __shared__ __align__(8) uint64_t bar_mem[8 * TILES + 5 * Sh::kStages + 1];
    __shared__ int64_t part[Sh::kWarps];
    __shared__ uint32_t tmem_base;
    __shared__ volatile int32_t dirty[8];              // of every eighth segment: its number + 1 if values were taken out
    __shared__ volatile uint32_t arrived[2][TILES];    // of the run's first and last segment
    __shared__ volatile uint32_t added[2][TILES];      // whether this CTA has counted itself there
    __shared__ volatile int64_t of_run[3];
    __shared__ volatile int32_t of_deal;
    __shared__ PromptSegment start;
    __shared__ PromptSegment segments[Sh::kWarps];  // each warp's: registers are for scores
    __shared__ int4 items[kDealItems];
    const rra_prompt_attention_args_t& a = p.a;
    const int tid = (int)threadIdx.x, warp = tid >> 5;
    const uint32_t smem = (smem_u32(raw_smem) + 1023u) & ~1023u;
    int32_t* const chunk_sums = (int32_t*)(raw_smem + (smem - smem_u32(raw_smem)) + Sh::kSums);
    AttnWorkspace* const ws = (AttnWorkspace*)a.workspace;
    float* const parts = (float*)(ws + 1);

    const uint32_t bars = smem_u32(bar_mem);
    // q_full[i], pv_half[i]: what the next products of tile i wait for, with their turn; pv_full[i]: the second half of the
    // weights; s_full[i], half_done[i], o_full[i]: products that are done
    const uint32_t q_full = bars, q_empty = q_full + 8 * TILES, s_full = q_empty + 8 * TILES, pv_full = s_full + 8 * TILES,
                   o_full = pv_full + 8 * TILES, joined = o_full + 8 * TILES, k_full = joined + 8 * TILES, k_empty = k_full + 8 * Sh::kStages,
                   v_full = k_empty + 8 * Sh::kStages, v_empty = v_full + 8 * Sh::kStages, v_ready = v_empty + 8 * Sh::kStages, pv_half = v_ready + 8 * Sh::kStages, half_done = pv_half + 8 * TILES,
                   drained = half_done + 8 * TILES;
    constexpr uint32_t kTurn = TILES == 2 ? 1 : 0;
    pdl_release_early();
    if (tid == 32) {
        asm volatile("prefetch.tensormap [%0];" : : "l"(&p.q) : "memory");
        asm volatile("prefetch.tensormap [%0];" : : "l"(&p.k) : "memory");
        asm volatile("prefetch.tensormap [%0];" : : "l"(&p.v) : "memory");
    }
    if (tid == 0) {
        for (int i = 0; i < TILES; ++i) {
            added[0][i] = added[1][i] = 0u;
            mbar_init(q_full + 8 * i, 1 + kTurn);
            mbar_init(q_empty + 8 * i, 1);
            mbar_init(s_full + 8 * i, 1);
            mbar_init(pv_half + 8 * i, 2 * kPromptRows + kTurn);
            mbar_init(pv_full + 8 * i, 2 * kPromptRows);
            mbar_init(half_done + 8 * i, 1);
            mbar_init(o_full + 8 * i, 1);
            mbar_init(joined + 8 * i, 2 * kPromptRows);
        }
        for (int i = 0; i < Sh::kStages; ++i) {
            mbar_init(k_full + 8 * i, 1);
            mbar_init(k_empty + 8 * i, TILES);
            mbar_init(v_full + 8 * i, 1);
            mbar_init(v_empty + 8 * i, TILES);
            mbar_init(v_ready + 8 * i, 1);
        }
        for (int i = 0; i < 8; ++i) dirty[i] = 0;
        mbar_init(drained, TILES);
        if (kTurn) mbar_arrive(q_full);  // the first turn
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        fence_proxy_async_smem();
    }
    pdl_wait();
    // TMEM, while the work is dealt out.  Not before the wait: the grid before this one may still have to get its own on this SM,
    // and would wait for ours.
    if (warp == Sh::kIssue) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" : : "r"(smem_u32(&tmem_base)), "r"(Sh::kColumns) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }

    const WholeWork<TILES> work{p};
    // Its run, and all runs' length; or the segments that are dealt to it (-1: it has a run).  In shared memory, for registers.
    volatile const int64_t &r0 = of_run[0], &r1 = of_run[1], &run = of_run[2];
    volatile const int32_t& dealt = of_deal;
    bool idle;
    {
        int64_t from = 0, to = INT64_MAX, length = 1;
        const int given = prompt_deal<Sh::kWarps>(work, chunk_sums, part, items);
        __syncthreads();
        idle = given == 0 || (given < 0 && !prompt_run<Sh::kWarps>(work, chunk_sums, part, start, from, to, length));
        if (tid == 0) of_run[0] = from, of_run[1] = to, of_run[2] = length, of_deal = given;
    }
    fence_proxy_async_smem();  // the sums were where copies go next
    tc_before_sync();
    __syncthreads();
    tc_after_sync();
    const uint32_t tmem = tmem_base;
    if (idle) {
        if (warp == Sh::kIssue)
            asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" : : "r"(tmem), "r"(Sh::kColumns) : "memory");
        return;
    }
    // Segments: the first, and the next of one; those that are dealt out have a row of their own.
    auto given = [&](PromptSegment& s, int k) {
        const int4 it = items[k];
        s.n = AttnLengths{it.x, it.y, it.y};
        s.b = k, s.c = it.z, s.h = it.w, s.begin = 0;
    };
    auto next = [&](PromptSegment& at) {
        PromptSegment s = at;
        if (dealt >= 0 ? s.b + 1 == dealt : s.end >= r1) return false;
        if (dealt >= 0) given(s, s.b + 1);
        else prompt_step(work, s);
        prompt_place(work, s);
        __syncwarp();  // all lanes have read it; they write the same
        at = s;
        __syncwarp();
        return true;
    };
    PromptSegment& seg = segments[warp];
    {
        PromptSegment s = start;
        if (dealt >= 0) given(s, 0);
        else s.n = work.lengths(s.b);
        prompt_place(work, s);
        seg = s;
        __syncwarp();
    }
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

    auto edge_of = [&](const PromptSegment& s) {
        const int first = s.c * TILES * p.span, last = min(s.n.qn, first + TILES * p.span) - 1;
        return PromptEdge{p.window > 0 ? max(0, last - p.window + 1) : 0, a.causal ? first + 1 : s.n.qn};
    };

    uint32_t n = 0;   // key tiles of this run so far
    uint32_t sn = 0;  // segments so far that had tiles
    if (warp < Sh::kSoftmaxWarps) {
        // =============================== softmax: a thread has a quarter of two rows ====
        set_registers<Sh::kSoftmaxRegs, Sh::kLaunchRegs>();
        const int i = warp >> 3, lane = tid & 31, t = lane & 3, row0 = 32 * (warp & 3) + 16 * (warp >> 2 & 1) + (lane >> 2);
        const uint32_t lanes = tmem + ((uint32_t)(row0 & ~15) << 16);  // this warp's TMEM lanes
        const uint32_t s_at = lanes + 128 * i, o_at = lanes + 128 * (TILES + i);
        int tok[2], head_in[2];  // the rows' token and head in the tile
#pragma unroll
        for (int r = 0; r < 2; ++r) tok[r] = p.by_group(row0 + 8 * r), head_in[r] = row0 + 8 * r - tok[r] * p.group;
        const float factor = p.factor;
        const uint64_t factor2 = pair2(factor, factor);
        const bool flips = p.flip != 1.f;
        uint32_t joins = 0;
        bool ok = true;
        while (ok) {
            const int t0 = first_of(seg), t1 = end_of(seg);
            // Of row r: its token, whether it is one, and the keys that it sees.
            auto token_of = [&](int r) { return (seg.c * TILES + i) * p.span + (r ? tok[1] : tok[0]); };
            auto is_live = [&](int r) {
                return (r ? tok[1] : tok[0]) < p.span && token_of(r) < seg.n.qn &&
                       (seg.h - p.by_parts(seg.h) * p.parts) * p.group + (r ? head_in[1] : head_in[0]) < p.heads_of_kv;
            };
            auto lo_of = [&](int r) { return is_live(r) && p.window > 0 ? max(0, token_of(r) - p.window + 1) : 0; };
            auto hi_of = [&](int r) { return !is_live(r) ? INT32_MAX : a.causal ? token_of(r) + 1 : seg.n.qn; };
            const int edge_from = edge_of(seg).from, edge_to = edge_of(seg).to, first_tile = seg.first_tile;
            // What a row's weights are taken against, in units of log2 (kNone: it has seen no key yet), and their sum.
            // Rows that are no rows (behind the group's heads or the prompt's tokens: what memory or the next prompt has there) have
            // no say in the votes below, which change the others' roundings.  (28 heads over 4, one prompt of 2000: 39.6 us with,
            // 36.2 without their maxima.)
            constexpr float kNone = -FLT_MAX;
            const bool live[2] = {is_live(0), is_live(1)};
            float top[2] = {kNone, kNone}, less[2] = {0.f, 0.f}, l[2] = {0.f, 0.f};  // less: what is taken off scores
            bool fresh = true;  // some row has none
#pragma unroll 1
            for (int tl = t0; tl < t1; ++tl, ++n) {
                ok = wait(s_full + 8 * i, n);
                if (!ok) break;
                tc_after_sync();
                const int key0 = (first_tile + tl) * kPromptKeys;
                uint32_t v[64];  // v[4 j + 2 r + e]: row r, key 8 j + 2 t + e
                tc_ld_rows64(s_at, v);
                tc_ld_rows64(s_at + 64, v + 32);
                tc_wait_ld();
                const bool masks = PromptEdge{edge_from, edge_to}.masks(key0);
                if (masks || flips) {
                    if (flips)
#pragma unroll
                        for (int k = 0; k < 64; ++k) v[k] = __float_as_uint(__uint_as_float(v[k]) * p.flip);
                    // bit j of seen[2 r + e]: whether row r sees key 8 j + 2 t + e
                    const int lo[2] = {lo_of(0), lo_of(1)}, hi[2] = {hi_of(0), hi_of(1)};
                    uint32_t seen[4];
                    bool whole = true;
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        auto below = [&](int end) { return (1u << min(max((min(end - key0, 2 * kPromptKeys) - 2 * t - (k & 1) + 7) >> 3, 0), 16)) - 1u; };
                        seen[k] = below(hi[k >> 1]) & ~below(lo[k >> 1]);
                        whole = whole && seen[k] == 0xffffu;
                    }
                    if (!__all_sync(0xffffffffu, whole))
#pragma unroll
                        for (int k = 0; k < 64; ++k) v[k] = seen[k & 3] >> (k >> 2) & 1u ? v[k] : 0xff800000u;
                }
                // The halves of a tile's weights are given away one after the other: products begin with the first.
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    float all[2];
                    bool exact = fresh;
                    while (true) {
                        if (exact && (q == 0 || !fresh)) {  // against the maximum of what has not been given away
                            float by[2];
#pragma unroll
                            for (int r = 0; r < 2; ++r) {
                                float most[2] = {-INFINITY, -INFINITY};
#pragma unroll
                                for (int j = 8 * q; j < 16; ++j)
                                    most[j & 1] = max3(most[j & 1], __uint_as_float(v[4 * j + 2 * r]), __uint_as_float(v[4 * j + 2 * r + 1]));
                                float now = fmaxf(most[0], most[1]);
                                now = fmaxf(now, __shfl_xor_sync(0xffffffffu, now, 1));
                                now = fmaxf(now, __shfl_xor_sync(0xffffffffu, now, 2));
                                now = fmaxf(top[r], now * factor);  // no key: kNone
                                by[r] = exp2_fast(top[r] - now);
                                top[r] = now;
                                l[r] *= by[r];
                                less[r] = now == kNone ? 0.f : Sh::kLift - now;
                            }
                            if (q == 1) {  // products of the first half are under way
                                ok = wait(half_done + 8 * i, n);
                                tc_after_sync();
                            }
                            if (ok && (tl > t0 || q == 1) && __any_sync(0xffffffffu, by[0] != 1.f || by[1] != 1.f)) {
#pragma unroll 1
                                for (int x = 0; x < D / 32; ++x) {
                                    uint32_t o[16];
                                    tc_ld_rows32(o_at + 32 * x, o);
                                    tc_wait_ld();
#pragma unroll
                                    for (int k = 0; k < 16; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * by[k >> 1 & 1]);
                                    tc_st_rows32(o_at + 32 * x, o);
                                }
                            }
                        }
                        // ---- weights, where the scores were ----
                        const uint64_t less2[2] = {pair2(less[0], less[0]), pair2(less[1], less[1])};
                        uint64_t sum[2] = {pair2(0.f, 0.f), pair2(0.f, 0.f)};
                        uint32_t w[16];
#pragma unroll
                        for (int k = 0; k < 16; ++k) {
                            const int r = k & 1, at = 32 * q + 2 * k;
                            float e0, e1;
                            split2(fma2(pair2(__uint_as_float(v[at]), __uint_as_float(v[at + 1])), factor2, less2[r]), e0, e1);
                            e0 = exp2_fast(e0);
                            e1 = exp2_fast(e1);
                            sum[r] = add2(sum[r], pair2(e0, e1));
                            w[k] = pack2<T>(e0, e1);
                        }
                        tc_st_weights(s_at + 32 * q, w);
#pragma unroll
                        for (int r = 0; r < 2; ++r) {
                            float a0, a1;
                            split2(sum[r], a0, a1);
                            all[r] = a0 + a1;
                        }
                        if (exact || !__any_sync(0xffffffffu, (live[0] ? all[0] : 0.f) > Sh::kMost || (live[1] ? all[1] : 0.f) > Sh::kMost)) break;
                        exact = true;
                    }
                    l[0] += all[0];
                    l[1] += all[1];
                    tc_wait_st();
                    tc_before_sync();
                    mbar_arrive((q == 0 ? pv_half : pv_full) + 8 * i);
                }
                if (!ok) break;
                if (fresh) fresh = __any_sync(0xffffffffu, (live[0] && top[0] == kNone) || (live[1] && top[1] == kNone));
            }
            bool lost = false;
            if (ok && t0 < t1) {
                ok = wait(o_full + 8 * i, sn);
                tc_after_sync();
                lost = dirty[sn & 7] == (int32_t)sn + 1;
                ++sn;
            }
            if (!ok) break;
            // ---- the segment's end in this run ----
            const bool starts = seg.begin >= r0, ends = seg.end <= r1;
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                l[r] += __shfl_xor_sync(0xffffffffu, l[r], 1);
                l[r] += __shfl_xor_sync(0xffffffffu, l[r], 2);
                l[r] *= Sh::kUnlift;  // O stays lifted until it is divided by its sum
            }
            const int kv_head = p.by_parts(seg.h), head0 = (seg.h - kv_head * p.parts) * p.group;  // of the KV head's query heads
            const PromptEdge edge = {edge_from, edge_to};
            const int token[2] = {token_of(0), token_of(1)}, lo[2] = {lo_of(0), lo_of(1)}, hi[2] = {hi_of(0), hi_of(1)};
            T* out[2];
#pragma unroll
            for (int r = 0; r < 2; ++r)
                out[r] = (T*)a.out + (int64_t)(seg.n.q0 + token[r]) * a.out_token_stride + (kv_head * p.heads_of_kv + head0 + head_in[r]) * a.out_head_stride;
            // 32 channels of both rows, from c on, times inv: each thread writes 8 of them
            auto put = [&](const float* o, int c, const float* inv) {
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    uint32_t w[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) w[j] = pack2<T>(o[4 * j + 2 * r] * inv[r], o[4 * j + 2 * r + 1] * inv[r]);
                    quad_transpose(w);
                    if (live[r] && c + 8 * t < a.head_dim) *(uint4*)(out[r] + c + 8 * t) = make_uint4(w[0], w[1], w[2], w[3]);
                }
            };
            // what was taken out of the values comes back, into the output or a part
            auto add = [&](float* part) {
                if (!lost) return;
                __syncwarp();
#pragma unroll 1
                for (int r = 0; r < 2; ++r) {
                    const PromptShare share = {edge, seg.n.q0, kv_head, seg.first_tile + t0, seg.first_tile + t1, r ? lo[1] : lo[0], r ? hi[1] : hi[0]};
                    if (r ? live[1] : live[0])
                        add_lost<T>(p, share, part == nullptr ? (r ? out[1] : out[0]) : nullptr, part == nullptr ? nullptr : part + 2 * r, t, a.head_dim);
                }
                __syncwarp();
            };
            auto get = [&](int q, float* o) {  // 32 columns of O from its `q`th on
                tc_ld_rows32(o_at + 32 * q, (uint32_t*)o);
                tc_wait_ld();
            };
            auto statistics = [&](const float* best, const float* sum, float* inv) {
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    if (live[r] && t == 0 && a.lse != nullptr)
                        a.lse[(int64_t)(seg.n.q0 + token[r]) * a.q_heads + kv_head * p.heads_of_kv + head0 + head_in[r]] =
                            (best[r] + log2f(sum[r])) * 0.693147180559945309f;
                    inv[r] = sum[r] == 0.f ? 0.f : Sh::kUnlift / sum[r];
                }
            };
            if (starts && ends) {
                float inv[2];
                statistics(top, l, inv);
                float o[D / 2];
#pragma unroll
                for (int q = 0; q < D / 64; ++q) tc_ld_rows64(o_at + 64 * q, (uint32_t*)o + 32 * q);
                tc_wait_ld();
#pragma unroll
                for (int q = 0; q < D / 32; ++q) put(o + 16 * q, 32 * q, inv);
                add(nullptr);
            } else {
                // The last CTA to arrive adds the parts in order; its own, if it finds all others there, from where it is.
                const int i0 = (int)(seg.begin / run), i1 = (int)((seg.end - 1) / run), which = starts ? 1 : 0;
                uint32_t* const count = &ws->arrived[i0 * TILES + i];
                volatile uint32_t& others = arrived[which][i];
                const bool counts = (tid & 255) == 0;
                auto meet = [&]() {
                    mbar_arrive(joined + 8 * i);
                    return wait(joined + 8 * i, joins++);
                };
                // A part: of each warp, of every 8 channels, four values of each lane; then the rows' statistics.
                constexpr int kVectors = D / 4 * kPromptRows;
                auto part_of = [&](int x) {
                    return (float4*)(parts + (((int64_t)x * 2 + (x == i0 ? 1 : 0)) * TILES + i) * Sh::kPartFloats) + (warp & 7) * (D / 8) * 32 + lane;
                };
                auto stats_at = [&](int x, int r) {
                    return (float2*)((float4*)(parts + (((int64_t)x * 2 + (x == i0 ? 1 : 0)) * TILES + i) * Sh::kPartFloats) + kVectors) + row0 + 8 * r;
                };
                if (counts) others = ld_acquire_u32(count);
                ok = meet();
                if (!ok) break;
                int mine = (int)blockIdx.x;
                if (others != (uint32_t)(i1 - i0)) {
                    mine = -1;
                    if (t0 < t1) {
                        float4* const to = part_of((int)blockIdx.x);
#pragma unroll 1
                        for (int q = 0; q < D / 32; ++q) {
                            float o[16];
                            get(q, o);
#pragma unroll
                            for (int j = 0; j < 4; ++j) to[(4 * q + j) * 32] = make_float4(o[4 * j], o[4 * j + 1], o[4 * j + 2], o[4 * j + 3]);
                        }
                        add((float*)(to - t));
                    }
                    if (t == 0)
#pragma unroll
                        for (int r = 0; r < 2; ++r) *stats_at((int)blockIdx.x, r) = make_float2(top[r], l[r]);
                    __threadfence();
                    ok = meet();
                    if (ok && counts) {
                        others = atomicAdd(count, 1u);
                        added[which][i] = 1u;
                    }
                    ok = ok && meet();
                    if (!ok) break;
                }
                if (others == (uint32_t)(i1 - i0)) {
                    __threadfence();
                    auto stats_of = [&](int x, int r) { return x == mine ? make_float2(top[r], l[r]) : __ldcg(stats_at(x, r)); };
                    float best[2] = {-FLT_MAX, -FLT_MAX}, sum[2] = {0.f, 0.f}, inv[2];
#pragma unroll 4
                    for (int x = i0; x <= i1; ++x)
#pragma unroll
                        for (int r = 0; r < 2; ++r) best[r] = fmaxf(best[r], stats_of(x, r).x);
#pragma unroll 4
                    for (int x = i0; x <= i1; ++x)
#pragma unroll
                        for (int r = 0; r < 2; ++r) {
                            const float2 st = stats_of(x, r);
                            sum[r] += st.y * exp2_fast(st.x - best[r]);
                        }
                    statistics(best, sum, inv);
#pragma unroll 1
                    for (int q = 0; q < D / 32; ++q) {
                        float o[16];
#pragma unroll
                        for (int k = 0; k < 16; ++k) o[k] = 0.f;
#pragma unroll 1
                        for (int x = i0; x <= i1; ++x) {
                            float v[16];
                            if (x == mine) {
                                get(q, v);
                            } else {
#pragma unroll
                                for (int j = 0; j < 4; ++j) *(float4*)(v + 4 * j) = __ldcg(part_of(x) + (4 * q + j) * 32);
                            }
#pragma unroll
                            for (int r = 0; r < 2; ++r) {
                                const float2 st = stats_of(x, r);
                                if (st.y == 0.f) continue;  // nothing was seen there, and its channels may not have been written
                                const float by = exp2_fast(st.x - best[r]);
#pragma unroll
                                for (int j = 0; j < 4; ++j)
#pragma unroll
                                    for (int e = 0; e < 2; ++e) o[4 * j + 2 * r + e] = fmaf(v[4 * j + 2 * r + e], by, o[4 * j + 2 * r + e]);
                            }
                        }
                        put(o, 32 * q, inv);
                    }
                    if (mine >= 0) add(nullptr);
                    if (counts) *count = 0u;
                }
            }
            tc_before_sync();
            if (!next(seg)) break;
        }
        // A wait ran out: the results are lost, but the counters of the segments from here on have to be zero for the next
        // call.  So this CTA still counts itself, and whoever is last there clears them.
        if (!ok && (warp & 7) == 0)  // a whole warp, which goes from segment to segment together
#pragma unroll 1
            while (true) {
                const int which = seg.begin >= r0 ? 1 : 0;
                if (lane == 0 && (which == 0 || seg.end > r1)) {
                    const int i0 = (int)(seg.begin / run), i1 = (int)((seg.end - 1) / run);
                    uint32_t* const count = &ws->arrived[i0 * TILES + i];
                    const uint32_t before = added[which][i] != 0u ? arrived[which][i] : atomicAdd(count, 1u);
                    if (before == (uint32_t)(i1 - i0)) *count = 0u;
                }
                if (!next(seg)) break;
            }
    } else if (warp == Sh::kCopy) {
        // =============================== copies, ahead of the products by the stages ====
        set_registers<Sh::kIssueRegs, Sh::kLaunchRegs>();
        const uint32_t q_bytes = (uint32_t)(p.group * p.span) * 128u * (D / 64);
        bool ok = true;
        while (ok) {
            const int t0 = first_of(seg), t1 = end_of(seg);
            const int kv_head = p.by_parts(seg.h), head = kv_head * p.heads_of_kv + (seg.h - kv_head * p.parts) * p.group;
            if (t0 < t1) {
                for (int i = 0; i < TILES && ok; ++i) {
                    ok = sn == 0 || wait(q_empty + 8 * i, sn - 1);
                    if (ok && elected()) {
                        mbar_expect_tx(q_full + 8 * i, q_bytes);
#pragma unroll
                        for (int x = 0; x < D / 64; ++x)
                            tma_load(smem + i * Sh::kTile + x * Sh::kPanel, &p.q, 64 * x, head, seg.n.q0 + (seg.c * TILES + i) * p.span, q_full + 8 * i);
                    }
                    __syncwarp();
                }
                ++sn;
            }
#pragma unroll 1
            for (int tl = t0; tl < t1 && ok; ++tl, ++n) {
                const uint32_t stage = n % Sh::kStages, turn = n / Sh::kStages;
                const int token = seg.n.q0 + (seg.first_tile + tl) * kPromptKeys;
                ok = turn == 0 || wait(k_empty + 8 * stage, turn - 1);
                if (ok && elected()) {
                    mbar_expect_tx(k_full + 8 * stage, Sh::kTile);
#pragma unroll
                    for (int x = 0; x < D / 64; ++x)
                        tma_load(smem + Sh::kK + stage * Sh::kTile + x * Sh::kPanel, &p.k, 64 * x, kv_head, token, k_full + 8 * stage);
                }
                __syncwarp();
                if (!ok) break;
                ok = turn == 0 || wait(v_empty + 8 * stage, turn - 1);
                if (ok && elected()) {
                    mbar_expect_tx(v_full + 8 * stage, Sh::kTile);
#pragma unroll
                    for (int x = 0; x < D / 64; ++x)
                        tma_load(smem + Sh::kV + stage * Sh::kTile + x * Sh::kPanel, &p.v, 64 * x, kv_head, token, v_full + 8 * stage);
                }
                __syncwarp();
                if (!ok) {  // K of this tile is on its way
                    attn_wait_quiet(k_full + 8 * stage, turn & 1u);
                    break;
                }
            }
            if (!ok || !next(seg)) break;
        }
        // No copy is in flight when the CTA ends, also where nobody waited for it.
        for (int i = 0; i < TILES && sn > 0; ++i) attn_wait_quiet(q_full + 8 * i, (sn - 1) & 1u);
        for (uint32_t x = n > Sh::kStages ? n - Sh::kStages : 0; x < n; ++x) {
            attn_wait_quiet(k_full + 8 * (x % Sh::kStages), x / Sh::kStages & 1u);
            attn_wait_quiet(v_full + 8 * (x % Sh::kStages), x / Sh::kStages & 1u);
        }
    } else if (warp == Sh::kLook) {
        // =============================== values that some row does not see must be finite ====
        set_registers<Sh::kIssueRegs, Sh::kLaunchRegs>();
        for (bool ok = true; ok;) {
            const int t0 = first_of(seg), t1 = end_of(seg);
            const PromptEdge edge = edge_of(seg);
#pragma unroll 1
            for (int tl = t0; tl < t1; ++tl, ++n) {
                const uint32_t stage = n % Sh::kStages;
                ok = wait(v_full + 8 * stage, n / Sh::kStages);
                if (!ok) break;
                if (edge.masks((seg.first_tile + tl) * kPromptKeys)) {
#pragma unroll 1
                    for (uint32_t k = 0; k < Sh::kTile; k += 8 * 512) {
                        const uint32_t at = smem + Sh::kV + stage * Sh::kTile + k + 16 * (tid & 31);
                        uint32_t w[8][4], bad = 0;
#pragma unroll
                        for (int x = 0; x < 8; ++x)
                            asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(w[x][0]), "=r"(w[x][1]), "=r"(w[x][2]), "=r"(w[x][3]) : "r"(at + 512 * x));
#pragma unroll
                        for (int x = 0; x < 8; ++x)
#pragma unroll
                            for (int e = 0; e < 4; ++e) bad |= not_finite<Sh::kHalf>(w[x][e]);
                        if (bad == 0u) continue;
                        dirty[sn & 7] = (int32_t)sn + 1;
#pragma unroll
                        for (int x = 0; x < 8; ++x) {
#pragma unroll
                            for (int e = 0; e < 4; ++e) w[x][e] &= ~((not_finite<Sh::kHalf>(w[x][e]) >> 15) * 0xffffu);
                            sts_v4(at + 512 * x, w[x][0], w[x][1], w[x][2], w[x][3]);
                        }
                    }
                    fence_proxy_async_smem();
                }
                __syncwarp();
                if (elected()) mbar_arrive(v_ready + 8 * stage);
            }
            if (t0 < t1) ++sn;
            if (!ok || !next(seg)) break;
        }
    } else {
        // =============================== products of tile i: one thread issues ====
        set_registers<Sh::kIssueRegs, Sh::kLaunchRegs>();
        const int i = warp - Sh::kIssue;
        bool ok = i < TILES;
        constexpr uint32_t kQk = mma_desc(kPromptKeys, false, !Sh::kHalf), kPv = mma_desc(D, true, !Sh::kHalf);
        const uint32_t q_desc = tile_desc(smem + i * Sh::kTile, 16), k_desc = tile_desc(smem + Sh::kK, 16),
                       v_desc = tile_desc(smem + Sh::kV, Sh::kPanel);
        constexpr uint32_t kStep = Sh::kTile >> 4;  // from one tile to the next, in a descriptor
        const uint32_t s_at = tmem + 128 * i, o_at = tmem + 128 * (TILES + i);
        // The tiles' warps take turns, as in serve_prefill.cu.
        while (ok) {
            const int t0 = first_of(seg), t1 = end_of(seg);
            if (t0 < t1) {
#pragma unroll 1
                for (int tl = t0 - 1; tl < t1; ++tl) {  // products of tile tl, scores of the next
                    const bool values = tl >= t0, scores = tl + 1 < t1;
                    const uint32_t then = n + (values ? 1 : 0);  // the tile whose scores come next
                    // K and V are there long before: first their waits, so that nothing comes between the products
                    ok = (!scores || wait(k_full + 8 * (then % Sh::kStages), then / Sh::kStages)) &&
                         (!values || wait(v_ready + 8 * (n % Sh::kStages), n / Sh::kStages)) &&
                         (values ? wait(pv_half + 8 * i, n) : wait(q_full + 8 * i, sn));
                    if (!ok) break;
                    tc_after_sync();
                    const uint32_t k_at = k_desc + then % Sh::kStages * kStep, v_at = v_desc + n % Sh::kStages * kStep;
                    if (values) {  // O_i += P_i V
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            if (h == 1) {
                                ok = wait(pv_full + 8 * i, n);
                                tc_after_sync();
                            }
                            if (ok && elected()) {
#pragma unroll
                                for (int k = 4 * h; k < 4 * h + 4; ++k)
                                    tc_mma_ts(o_at, s_at + 8 * k, v_at + k * (2048 >> 4), kPv, tl > t0 || k > 0);
                                tc_commit(h == 0 ? half_done + 8 * i : v_empty + 8 * (n % Sh::kStages));
                            }
                            __syncwarp();
                        }
                        if (!ok) break;
                    }
                    if (elected()) {
                        if (scores) {  // S_i = Q_i K^T
#pragma unroll
                            for (int k = 0; k < D / 16; ++k) {
                                constexpr auto at = [](int x) { return (uint32_t)((x >> 2) * Sh::kPanel + (x & 3) * 32) >> 4; };
                                tc_mma(s_at, q_desc + at(k), k_at + at(k), kQk, k > 0);
                            }
                            tc_commit(s_full + 8 * i);
                            tc_commit(k_empty + 8 * (then % Sh::kStages));
                            if (tl + 2 == t1) tc_commit(q_empty + 8 * i);
                            if (kTurn) mbar_arrive(i == 1 ? pv_half : values ? pv_half + 8 : q_full + 8);
                        } else {
                            tc_commit(o_full + 8 * i);
                            if (kTurn) mbar_arrive(i == 0 ? pv_half + 8 : q_full);
                        }
                    }
                    __syncwarp();
                    n = then;
                }
                ++sn;
            }
            if (!ok || !next(seg)) break;
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

// ------------------------------------------------------------------ host ----
// The driver's function that describes a tensor to the copies; null where there is no driver.
using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                 const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
static EncodeTiled encode_tiled() {
    static const EncodeTiled fn = [] {
        void* f = nullptr;
        cudaDriverEntryPointQueryResult found = cudaDriverEntryPointSymbolNotFound;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &found) != cudaSuccess) cudaGetLastError();
        return found == cudaDriverEntryPointSuccess ? (EncodeTiled)f : nullptr;
    }();
    return fn;
}

// [tokens][heads][head_dim] of 16-bit values, in boxes of `span` tokens, `group` heads and 64 channels; what lies outside reads as 0.
static bool prompt_map(CUtensorMap* map, const void* at, bool half, int64_t tokens, int heads, int head_dim, int64_t token_stride,
                       int64_t head_stride, int group, int span) {
    const EncodeTiled encode = encode_tiled();
    if (encode == nullptr) return false;
    const cuuint64_t dims[3] = {(cuuint64_t)head_dim, (cuuint64_t)heads, (cuuint64_t)tokens};
    const cuuint64_t strides[2] = {(cuuint64_t)head_stride * 2, (cuuint64_t)token_stride * 2};
    const cuuint32_t box[3] = {64, (cuuint32_t)group, (cuuint32_t)span}, steps[3] = {1, 1, 1};
    return encode(map, half ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, (void*)at, dims, strides, box, steps,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename T, int D, int TILES>
static rra_status_t whole_launch(const PromptParams& p, int ctas, rra_stream_t stream) {
    using Sh = WholeShape<T, D, TILES>;
    const void* k = (const void*)prompt_attention_kernel<T, D, TILES>;
    static_assert(Sh::kSmem <= 227 * 1024 - 20480, "shared memory, with the list of segments");
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

template <typename T>
static rra_status_t whole_launch(const PromptParams& p, int tiles, int ctas, rra_stream_t stream) {
    if (p.a.head_dim > 64) return tiles == 2 ? whole_launch<T, 128, 2>(p, ctas, stream) : whole_launch<T, 128, 1>(p, ctas, stream);
    return tiles == 2 ? whole_launch<T, 64, 2>(p, ctas, stream) : whole_launch<T, 64, 1>(p, ctas, stream);
}

static bool prompt_args_ok(const rra_prompt_attention_args_t* a) {
    if (a == nullptr || a->requests < 0 || a->requests > RRA_SERVE_MAX_REQUESTS || a->tokens < 0 || a->tokens > INT32_MAX / 2 ||
        a->kv_heads < 1 || a->q_heads < 1 || a->q_heads % a->kv_heads != 0 || a->head_dim < 8 || a->head_dim > 128 || a->head_dim % 8 != 0 ||
        (a->half != 0 && a->half != 1) || a->max_len < 0 || a->window < 0 || !(fabs(a->scale) * 1.4426950408889634 <= FLT_MAX))
        return false;
    if (a->tokens * a->q_heads > INT32_MAX / 2) return false;  // rows are counted in 32 bits
    const int64_t far = (int64_t)1 << 39;  // the copies' strides are below 2^40 bytes
    auto fine = [&](const void* at, int64_t token, int64_t head, int heads) {
        return aligned16(at) && strides_ok(token, head, heads, a->head_dim, 2) && token < far && head < far;
    };
    if (!fine(a->q, a->q_token_stride, a->q_head_stride, a->q_heads) || !fine(a->k, a->k_token_stride, a->k_head_stride, a->kv_heads) ||
        !fine(a->v, a->v_token_stride, a->v_head_stride, a->kv_heads) || !fine(a->out, a->out_token_stride, a->out_head_stride, a->q_heads) ||
        ((uintptr_t)a->workspace & 255) != 0)
        return false;
    if (a->requests == 0 || a->tokens == 0) return true;
    return a->q != nullptr && a->k != nullptr && a->v != nullptr && a->out != nullptr && a->cu != nullptr && a->workspace != nullptr;
}

// Tiles of a CTA, by what was measured of either, for lengths as they are on average and at most (every choice is right for
// every call): a key tile takes 1.3 us for one tile and 1.7 for two (heads of 64: 1.15 and 1.35), a segment 2.8 and 5.8 (2.5
// and 5) more; 20 us to find that they are better cut into runs, and to join those.  (64 heads over 8 of 128: 16 tokens, 64
// requests, 21.9 and 31.6 us; 64 tokens 63.0 and 60.7; one request of 700 24.2 and 20.4, of 2000 94 and 68; 8192 and 3000
// 1320 and 850.  32 over 32: 64 of 300 214 and 257, 32 of 600 227 and 242, 16 of 1024 234 and 206.  8 over 1: 2000 27 and 34,
// 4000 48 and 55, 5000 67 and 66.)  Over 90 batches of 1 to 64 requests of up to 8192 tokens, 1 to 64 heads, with windows and
// without, the choice takes 1.0 % longer than the better one on average, 46 % at most; two tiles always 18 %.
static int prompt_tiles(const PromptParams& p) {
    const rra_prompt_attention_args_t& a = p.a;
    const bool big = a.head_dim > 64;
    const double sms = 152, most = std::max(a.max_len, 1), requests = std::max(a.requests, 1);
    const double length = std::min(std::max(a.tokens / requests, most / requests), most);
    const double usual = (length + most) / 2;  // of the prompt that a segment is from: long ones have more of them
    auto time = [&](int tiles) {
        const double step = tiles == 2 ? (big ? 1.7 : 1.35) : big ? 1.3 : 1.15, fixed = tiles == 2 ? (big ? 5.8 : 5) : big ? 2.8 : 2.5;
        const double chunk = tiles * p.span, chunks = std::ceil(length / chunk), segments = chunks * a.kv_heads * p.parts * requests;
        auto keys = [&](double n) {  // in tiles
            return std::max(1.0, (a.window > 0 ? std::min(n, (double)a.window + chunk) : n) / kPromptKeys);
        };
        const double mean = keys(a.causal ? std::min((std::ceil(usual / chunk) + 1) * chunk, usual + chunk) / 2 : usual), longest = std::ceil(keys(most));
        const bool alike = longest == 1 || !a.causal;  // CTAs have whole numbers of the same
        const double load = (alike ? std::ceil(segments / sms) : segments / sms + 0.25) * (mean * step + fixed);
        return std::min(std::max(load, longest * step + fixed), segments / sms * (mean * step + fixed) + 20);
    };
    return time(2) < time(1) ? 2 : 1;
}

// The rest of a call's parameters, but for the tensors' descriptions.
static void prompt_sizes(PromptParams& p, const rra_prompt_attention_args_t& a) {
    p.a = a;
    p.heads_of_kv = a.q_heads / a.kv_heads;
    p.parts = (p.heads_of_kv + kPromptRows - 1) / kPromptRows;
    p.group = (p.heads_of_kv + p.parts - 1) / p.parts;
    p.span = kPromptRows / p.group;
}

}  // namespace rra

extern "C" {

size_t rra_prompt_attention_workspace_bytes(void) { return sizeof(rra::AttnWorkspace) + rra::prefill_partial_bytes(128); }

rra_status_t rra_prompt_attention_plan(const rra_prompt_attention_args_t* args, const char** name) {
    if (name == nullptr || !rra::prompt_args_ok(args)) return RRA_ERR_INVALID_ARG;
    rra::PromptParams p;
    rra::prompt_sizes(p, *args);
    *name = rra::prompt_tiles(p) == 2 ? "prompt_attention_kernel<256 rows>" : "prompt_attention_kernel<128 rows>";
    return RRA_OK;
}

rra_status_t rra_prompt_attention(const rra_prompt_attention_args_t* args, rra_stream_t stream) {
    if (!rra::prompt_args_ok(args)) return RRA_ERR_INVALID_ARG;
    const rra_prompt_attention_args_t& a = *args;
    if (a.requests == 0 || a.tokens == 0) return RRA_OK;
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
        cudaGetLastError();
        return RRA_ERR_CUDA;
    }
    rra::PromptParams p;
    rra::prompt_sizes(p, a);
    const int tiles = rra::prompt_tiles(p);
    p.window = std::min(a.window, 1 << 30);
    p.by_group = rra::Divisor(p.group);
    p.by_parts = rra::Divisor(p.parts);
    p.by_chunk = rra::Divisor(tiles * p.span);
    p.factor = (float)(fabs(a.scale) * 1.4426950408889634);
    p.flip = a.scale > 0 ? 1.f : a.scale < 0 ? -1.f : 0.f;
    if (p.factor == 0.f) p.factor = 1.f, p.flip = 0.f;  // every score is 0
    if (!rra::prompt_map(&p.q, a.q, a.half != 0, a.tokens, a.q_heads, a.head_dim, a.q_token_stride, a.q_head_stride, p.group, p.span) ||
        !rra::prompt_map(&p.k, a.k, a.half != 0, a.tokens, a.kv_heads, a.head_dim, a.k_token_stride, a.k_head_stride, 1, rra::kPromptKeys) ||
        !rra::prompt_map(&p.v, a.v, a.half != 0, a.tokens, a.kv_heads, a.head_dim, a.v_token_stride, a.v_head_stride, 1, rra::kPromptKeys))
        return RRA_ERR_CUDA;
    const int ctas = std::min(sms, rra::kPromptMaxCtas);
    return a.half != 0 ? rra::whole_launch<__half>(p, tiles, ctas, stream) : rra::whole_launch<__nv_bfloat16>(p, tiles, ctas, stream);
}

}  // extern "C"
