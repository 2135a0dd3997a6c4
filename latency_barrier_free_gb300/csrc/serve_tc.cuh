// serve_tc.cuh -- what the prompts' kernels share (rra_serve.h): tcgen05 and its
// operands, and the cut of a batch into equal runs of key tiles.
#pragma once

#include "serve_attn.cuh"

namespace rra {

constexpr int kPromptKeys = 128;       // keys of a tile
constexpr int kPromptRows = 128;       // rows of a tile: the TMEM lanes
constexpr int kPromptMinRun = 4;       // key tiles a CTA takes at least
// What starting and ending a segment costs, in key tiles (3 requests of up to 1024 queries and 8192 keys, 64 heads over 8 of 128:
// 2, 3, 4, 5 and 6 take 304, 276, 259, 262 and 265 us: with less, a CTA that gets the shortest segments ends last).
constexpr int kPromptSegmentCost = 4;
constexpr int kPromptMaxCtas = 192;    // CTAs that the workspace has room for
static_assert(kPromptMaxCtas * 2 <= kAttnMaxCtas, "a counter for each tile of a CTA's last segment");

// ------------------------------------------------------------- tcgen05 ----
// A tile in shared memory as an operand.  Low word: start and, for the operand whose rows are keys, the distance of its
// panels of 64 columns, in 16 bytes; a step along the tile adds to the start.  High word: 8 rows apart by 1024 bytes,
// 128-byte swizzle.
__device__ __forceinline__ uint32_t tile_desc(uint32_t addr, uint32_t panels) { return addr >> 4 | panels >> 4 << 16; }
constexpr uint32_t kTileDescHigh = 1024u >> 4 | 1u << 14 | 2u << 29;
// binary32 sums of binary16 (or bfloat16) products, 128 rows, n columns; b_keys: B's rows are the summed index
constexpr uint32_t mma_desc(int n, bool b_keys, bool bfloat = false) {
    return 1u << 4 | (bfloat ? 1u << 7 | 1u << 10 : 0u) | (b_keys ? 1u << 16 : 0u) | (uint32_t)(n >> 3) << 17 | (uint32_t)(128 >> 4) << 24;
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
// A kernel's work W has requests() and heads(), and of a request lengths(b), chunks(lengths) and item(lengths, c): the key
// tiles of chunk c.  A segment is a chunk of one head; all segments stand in a row: first their cost, then their tiles.
struct PromptItem {
    int32_t first_tile, tiles;
};
__device__ __forceinline__ PromptItem prompt_item(int first_key, int end_key) {
    PromptItem t;
    t.first_tile = first_key / kPromptKeys;
    t.tiles = max(1, (end_key + kPromptKeys - 1) / kPromptKeys - t.first_tile);
    return t;
}

// A segment: chunk c of request b, head h, at begin..end of the row.
struct PromptSegment {
    AttnLengths n;
    int32_t b, c, h, chunks, first_tile;
    int64_t begin, end;
};
// Its place in the row, by its begin.
template <typename W>
__device__ __forceinline__ void prompt_place(const W& w, PromptSegment& s) {
    s.chunks = w.chunks(s.n);
    const PromptItem t = w.item(s.n, s.c);
    s.first_tile = t.first_tile;
    s.end = s.begin + t.tiles + kPromptSegmentCost;
}
template <typename W>
__device__ __forceinline__ void prompt_load(const W& w, PromptSegment& s) {
    s.n = w.lengths(s.b);
    prompt_place(w, s);
}
// To the next one, but for its place.
template <typename W>
__device__ __forceinline__ void prompt_step(const W& w, PromptSegment& s) {
    s.begin = s.end;
    if (++s.c >= s.chunks) {
        s.c = 0;
        do {
            if (++s.b == w.requests()) s.b = 0, ++s.h;
            s.n = w.lengths(s.b);
        } while (s.n.qn == 0 && s.h < w.heads());  // some request has queries: there is a segment
    }
}
template <typename W>
__device__ __forceinline__ void prompt_next(const W& w, PromptSegment& s) {
    prompt_step(w, s);
    prompt_load(w, s);
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

// This CTA's run r0 .. r1 of the row, the length of everybody's, and its first segment's b, c, h and begin (for prompt_load()).
// False if there is none.  chunk_sums: requests + 1 words of shared memory, sums: one for each warp; the whole block.
template <int kWarps, typename W>
__device__ __forceinline__ bool prompt_run(const W& work, int32_t* chunk_sums, int64_t* sums, PromptSegment& start, int64_t& r0, int64_t& r1,
                                           int64_t& run) {
    constexpr int kThreads = 32 * kWarps;
    const int tid = (int)threadIdx.x, requests = work.requests();
    // chunks of the requests, then the chunks' tiles, the same for every head
    int64_t total_chunks = 0;
    for (int b0 = 0; b0 < requests; b0 += kThreads) {
        const int b = b0 + tid;
        int64_t all;
        const int64_t at = block_sum<kWarps>(b < requests ? work.chunks(work.lengths(b)) : 0, all, sums);
        if (b < requests) chunk_sums[b] = (int32_t)(total_chunks + at);
        total_chunks += all;
    }
    // Chunks are counted in 32 bits, which the rows of any batch fit.  More of them are the same rows over and over: cu_q does
    // not ascend, and there is no result to give.
    if (total_chunks > INT32_MAX) return false;
    if (tid == 0) chunk_sums[requests] = (int32_t)total_chunks;
    __syncthreads();
    auto owner = [&](int n, int& b, int& c) {
        int low = 0, high = requests;
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
        return work.item(work.lengths(b), c).tiles + kPromptSegmentCost;
    };
    int64_t per_head = 0;
    for (int n0 = 0; n0 < total_chunks; n0 += kThreads) {
        int64_t all;
        block_sum<kWarps>(n0 + tid < total_chunks ? cost_of(n0 + tid) : 0, all, sums);
        per_head += all;
    }
    const int64_t total = per_head * work.heads();
    run = (total + gridDim.x - 1) / gridDim.x;
    run = run < kPromptMinRun + kPromptSegmentCost ? kPromptMinRun + kPromptSegmentCost : run;
    r0 = (int64_t)blockIdx.x * run, r1 = r0 + run < total ? r0 + run : total;
    if (r0 >= r1) return false;
    const int64_t h = r0 / per_head, w = r0 - h * per_head;
    int64_t before = 0;
    for (int n0 = 0; n0 < total_chunks && before <= w; n0 += kThreads) {
        int64_t all;
        const int n = n0 + tid, cost = n < total_chunks ? cost_of(n) : 0;
        const int64_t at = before + block_sum<kWarps>(cost, all, sums);
        if (at <= w && w < at + cost) {
            owner(n, start.b, start.c);
            start.h = (int)h;
            start.begin = h * per_head + at;
        }
        before += all;
    }
    return true;
}

}  // namespace rra
