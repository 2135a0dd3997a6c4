// serve_attn.cu -- attention over the 4-bit and the 8-bit cache for single tokens
// and a few drafted ones (rra_serve.h); the arithmetic is in serve_attn_rows.cuh and
// serve_attn_rows8.cuh.
//
// Work is split by keys.  A segment is the rows of one request and KV head
// that fit the instructions (8 NT); its tiles are 32 keys each.  All
// segments' tiles in a row are cut into equal runs, one per warp, so that
// ragged batches and single long requests load every scheduler alike.  A warp
// walks its run with its own ring of bulk copies in flight and no barrier: what
// it finds whole it writes out itself.  Of its first and last segment it may
// have a piece only; those are joined once, at the end of the CTA, and across
// CTAs by whichever finishes last, in the order of the runs.
//
// Bound by the pages' bytes in the middle and by latency at both ends.  64
// heads over 8 of 128, one query each: 131071 keys of one request, 151 MB, take
// 37.5 us (4.0 TB/s): 3.4 us to the first copy (lengths, page numbers, pages),
// 25 us of stream at 6 TB/s, then the joins.  64 ragged requests, 175 MB:
// 44.9 us (3.9 TB/s).  Half the instructions are the unpacking of codes, and the
// ALU pipe is half busy; four schedulers need the three warps each.
//
// Over the 8-bit cache 64 ragged requests, 312 MB, take 59.4 us (5.3 TB/s): 5 us to the
// first copy, 46 of stream at 6.8 TB/s, the copy's own rate, and 6 to 8 of joins.
#include <algorithm>
#include <cmath>

#include "serve_attn_rows8.cuh"

namespace rra {

constexpr double kLog2E = 1.4426950408889634;
constexpr int kAttnMinRun = 1;     // tiles a warp takes at least
constexpr int kAttnSegmentCost = 4;  // what starting and ending a segment costs, in tiles of 32 keys
constexpr int segment_cost(int blocks) { return kAttnSegmentCost * 2 / blocks; }  // in tiles of so many blocks of 16

// The queries and keys of request b, clamped to the buffers.
struct AttnRequest {
    int32_t q0, qn;       // first query token, how many
    int32_t kv;           // keys
    int32_t first_tile;   // tile of the first key that any query sees
    int32_t tiles;        // tiles of one segment, at least one
    int32_t chunks;       // segments of a KV head
};
template <int kRows, int NB>
__device__ __forceinline__ AttnRequest attn_request(const AttnParams& p, const AttnLengths& n) {
    constexpr int kKeys = NB * kKvBlockTokens;
    AttnRequest r;
    r.q0 = n.q0;
    r.qn = n.qn;
    r.kv = n.kv;
    r.first_tile = (p.window > 0 ? max(0, r.kv - r.qn - p.window + 1) : 0) / kKeys;
    r.tiles = max(1, (r.kv + kKeys - 1) / kKeys - r.first_tile);
    r.chunks = (r.qn * p.group + kRows - 1) / kRows;
    return r;
}

// A segment: rows of chunk c of KV head h of request b.  In the row of all
// segments it takes begin..end: first its cost, then its tiles.
struct AttnSegment {
    AttnRequest r;
    int32_t b, h, c;
    int64_t begin, end;
};
// `known`: the first requests' lengths, n of them, in shared memory.
template <int kRows, int NB>
__device__ __noinline__ void attn_next(const AttnParams& p, const AttnLengths* known, int n, AttnSegment& s) {  // out of line: once a segment, in two places
    if (++s.c >= s.r.chunks) {
        s.c = 0;
        if (++s.h == p.a.cache.kv_heads) {
            s.h = 0;
            do {
                if (++s.b >= p.a.requests) {
                    s.begin = s.end = INT64_MAX;
                    return;
                }
                s.r = attn_request<kRows, NB>(p, s.b < n ? known[s.b] : attn_lengths(p, s.b));
            } while (s.r.chunks == 0);
        }
    }
    s.begin = s.end;
    s.end += s.r.tiles + segment_cost(NB);
}

// x / y, which fits 32 bits; mostly x does too, and then the division is a short one.
__device__ __forceinline__ int quotient(int64_t x, int64_t y) {
    if (((uint64_t)x | (uint64_t)y) >> 32 == 0) return (int)((uint32_t)x / (uint32_t)y);
    return (int)(x / y);
}

// What a warp, or a CTA, has of a segment that others share.
struct AttnPiece {
    int32_t q0, rows, h, c;  // the request's first query token and number of rows
    int32_t flags;           // kHas, kStarts, kEnds
    int64_t begin, end;  // the whole segment
};
enum { kHas = 1, kStarts = 2, kEnds = 4 };

// NB: blocks of 16 keys that a warp takes at a time, a stage of its ring.
template <typename F, int D, int NT, int kWarps, int kStages, int NB>
struct AttnShape {
    using B = typename F::template Block<D>;
    static constexpr int kRows = 8 * NT;
    static constexpr int kThreads = 32 * kWarps;
    static constexpr int kStage = NB * B::kBytes;
    static constexpr int kPartial = kRows * (D + 2);           // floats of a piece: maximum and sum of each row, rows
    static constexpr int kRing = kWarps * kStages * kStage;    // a warp's last piece goes where its ring was
    static constexpr int kHeads = kWarps * kPartial * 4;       // a warp's first piece
    static constexpr int kBars = kWarps * kStages * 8;
    static constexpr int kFixed = kRing + kHeads + kBars;
    static_assert(kStages * kStage >= kPartial * 4, "a piece fits the ring");
    static size_t smem(int requests) { return (size_t)kFixed + 8 * ((size_t)requests + 1); }
};

// Adds a piece's row (maximum and sum st, four channels v) to sums whose maximum is top.
__device__ __forceinline__ void attn_add(float top, float& sum, float4& o, float2 st, float4 v) {
    const float by = exp2_fast(st.x - top);
    sum = fmaf(st.y, by, sum);
    o.x = fmaf(v.x, by, o.x);
    o.y = fmaf(v.y, by, o.y);
    o.z = fmaf(v.z, by, o.z);
    o.w = fmaf(v.w, by, o.w);
}

template <typename F, int D, int NT, int kWarps, int kStages, int NB>
__global__ void __launch_bounds__(32 * kWarps, 1) kv_attention_kernel(const __grid_constant__ AttnParams p) {
    using Sh = AttnShape<F, D, NT, kWarps, kStages, NB>;
    using B = typename F::template Block<D>;
    constexpr int J = D / 32, kRows = Sh::kRows;
    extern __shared__ __align__(128) unsigned char smem[];
    __shared__ int64_t warp_sum[kWarps];
    __shared__ AttnPiece pieces[2 * kWarps];
    __shared__ AttnLengths known[Sh::kThreads];
    __shared__ float2 joined[2 * kWarps][kRows];  // maximum and sum of a chain's rows
    __shared__ int2 chain[2 * kWarps];  // its lead, its pieces
    __shared__ int2 to_join[2];         // first CTA and number of CTAs of the first and last segment, 0 unless this one joins them
    const rra_kv_attention_args_t& a = p.a;
    const int tid = (int)threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int g = lane >> 2, t = lane & 3;
    int64_t* const sums = (int64_t*)(smem + Sh::kFixed);
    const uint32_t ring = smem_u32(smem) + (uint32_t)(warp * kStages * Sh::kStage);
    const uint32_t bars = smem_u32(smem) + (uint32_t)(Sh::kRing + Sh::kHeads + warp * kStages * 8);
    // piece i of warp w (0 its first, 1 its last segment): statistics of the rows, then the rows
    auto piece_at = [&](int w, int i) {
        return (float*)(i == 0 ? smem + Sh::kRing + w * Sh::kPartial * 4 : smem + w * kStages * Sh::kStage);
    };
    AttnWorkspace* const ws = (AttnWorkspace*)a.workspace;
    float* const partials = (float*)(ws + 1);

    pdl_release_early();
    if (lane == 0) {
#pragma unroll
        for (int i = 0; i < kStages; ++i) mbar_init(bars + 8 * i, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        fence_proxy_async_smem();
        pieces[2 * warp].flags = pieces[2 * warp + 1].flags = 0;
    }
    __syncwarp();
    pdl_wait();

    // running sums of the requests' segments
    int64_t total = 0;
    for (int b0 = 0; b0 < a.requests; b0 += Sh::kThreads) {
        const int b = b0 + tid;
        int64_t v = 0;
        if (b < a.requests) {
            const AttnLengths n = attn_lengths(p, b);
            if (b0 == 0) known[tid] = n;
            const AttnRequest r = attn_request<kRows, NB>(p, n);
            v = (int64_t)(r.tiles + segment_cost(NB)) * r.chunks * a.cache.kv_heads;
        }
        int64_t inc = v;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t up = __shfl_up_sync(0xffffffffu, inc, o);
            if (lane >= o) inc += up;
        }
        if (lane == 31) warp_sum[warp] = inc;
        __syncthreads();
        int64_t before = total, all = 0;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            if (w < warp) before += warp_sum[w];
            all += warp_sum[w];
        }
        if (b < a.requests) sums[b] = before + inc - v;
        total += all;
        __syncthreads();
    }
    if (tid == 0) sums[a.requests] = total;
    __syncthreads();
    // Little work is spread over the SMs first, four warps each: a warp that shares its scheduler takes longer for
    // a tile, and the smallest batches are all latency.
    int64_t run = kAttnMinRun;
    int warps = kWarps;
    if (total <= run * 4 * (int64_t)gridDim.x) {
        warps = 4;
    } else if (total > run * kWarps * (int64_t)gridDim.x) {
        run = (total + (int64_t)gridDim.x * kWarps - 1) / ((int64_t)gridDim.x * kWarps);
    }
    const int64_t cta_run = run * warps;
    if ((int64_t)blockIdx.x * cta_run >= total) return;
    const int64_t r0 = (int64_t)blockIdx.x * cta_run + warp * run;
    const int64_t r1 = r0 + run < total ? r0 + run : total;

    if (r0 < r1 && warp < warps) {
        // this warp's first segment
        AttnSegment seg;
        {
            int low = 0, high = a.requests;
            while (high - low > 1) {
                const int mid = (low + high) >> 1;
                if (sums[mid] <= r0) low = mid;
                else high = mid;
            }
            seg.b = low;
            seg.r = attn_request<kRows, NB>(p, low < Sh::kThreads ? known[low] : attn_lengths(p, low));
            const int each = seg.r.tiles + segment_cost(NB);
            const int i = quotient(r0 - sums[low], each);
            seg.h = i / seg.r.chunks;
            seg.c = i - seg.h * seg.r.chunks;
            seg.begin = sums[low] + (int64_t)i * each;
            seg.end = seg.begin + each;
        }
        auto first_tile = [&](const AttnSegment& s) {
            const int64_t from = (s.begin > r0 ? s.begin : r0) - s.begin - segment_cost(NB);
            return (int)(from > 0 ? from : 0);
        };
        auto end_tile = [&](const AttnSegment& s) {
            const int64_t to = (s.end < r1 ? s.end : r1) - s.begin - segment_cost(NB);
            return (int)(to > 0 ? to : 0);
        };

        // Queries of a segment, as they are; loaded ahead of the copies that the lanes set up meanwhile.
        typename F::template Rows<D, NT> att;
        auto load_queries = [&]() { att.load(p, seg.r.q0, seg.r.qn, seg.h, seg.c, first_tile(seg) < end_tile(seg)); };
        load_queries();

        // ---- copies, kStages tiles ahead.  Lane i holds the places of the run's next tiles but i. ----
        AttnSegment from = seg;             // segment of the next tile to copy
        int next = first_tile(seg), from_end = end_tile(seg);  // that tile, and the end of the run in its segment
        int held = 0, held_end = 0;         // lane that holds the next tile, lanes that hold one
        const char* src0 = nullptr;
        const char* src1 = nullptr;
        uint32_t ok0 = 0, ok1 = 0;          // which lanes' blocks exist
        int put = 0;                        // stage of the next copy
        uint32_t issued = 0;                // parity of the number of copies of each stage
        uint32_t valid = 0;                 // which blocks of each stage were copied, 2 bits a stage
        const int ps = a.cache.page_tokens, blocks = ps / kKvBlockTokens;
        auto copy_next = [&]() {
            if (held >= held_end) {
                while (next >= from_end) {
                    if (from.end >= r1) return;
                    attn_next<kRows, NB>(p, known, Sh::kThreads, from);
                    next = first_tile(from);
                    from_end = end_tile(from);
                }
                const int key = (from.r.first_tile + next + lane) * (NB * kKvBlockTokens);
                const int32_t* const row = a.block_table + from.b * a.table_stride;
                src0 = src1 = nullptr;
                auto place = [&](int k) -> const char* {
                    if (next + lane >= from_end || k >= from.r.kv) return nullptr;
                    const int i = p.by_page(k), page = row[i];
                    if (page < 0 || page >= a.cache.num_pages) return nullptr;
                    return (const char*)a.cache.pages +
                           (((int64_t)page * a.cache.kv_heads + from.h) * blocks + (k - i * ps) / kKvBlockTokens) * B::kBytes;
                };
                src0 = place(key);
                if (NB == 2) src1 = place(key + kKvBlockTokens);
                ok0 = __ballot_sync(0xffffffffu, src0 != nullptr);
                if (NB == 2) ok1 = __ballot_sync(0xffffffffu, src1 != nullptr);
                held = 0;
                held_end = min(32, from_end - next);
                next += held_end;
            }
            if (lane == held) {
                const uint32_t bar = bars + 8 * put, dst = ring + put * Sh::kStage;
                const bool h0 = src0 != nullptr, h1 = src1 != nullptr;
                mbar_expect_tx(bar, ((h0 ? 1u : 0u) + (h1 ? 1u : 0u)) * (uint32_t)B::kBytes);
                if (NB == 2 && h0 && src1 == src0 + B::kBytes) {
                    bulk_g2s(dst, src0, 2 * B::kBytes, bar);
                } else {
                    if (h0) bulk_g2s(dst, src0, B::kBytes, bar);
                    if (h1) bulk_g2s(dst + B::kBytes, src1, B::kBytes, bar);
                }
            }
            valid = (valid & ~(3u << (2 * put))) | ((ok0 >> held & 1u) | (ok1 >> held & 1u) << 1) << (2 * put);
            issued ^= 1u << put;
            ++held;
            put = put + 1 == kStages ? 0 : put + 1;
        };
#pragma unroll 1
        for (int i = 0; i < kStages; ++i) copy_next();

        auto drain = [&]() {  // waits for every copy
#pragma unroll 1
            for (int i = 0; i < kStages; ++i) attn_wait_quiet(bars + 8 * i, (issued >> i & 1u) ^ 1u);
        };
        int take = 0;
        uint32_t phase = 0;
        bool dead = false;  // a wait ran out: no more copies, no more sums

        while (true) {
            const int rows = seg.r.qn * p.group;
            const int tile0 = first_tile(seg), tile1 = end_tile(seg);
            att.start(p, seg.r.qn, seg.r.kv, seg.c);
            // ---- tiles ----
#pragma unroll 1
            for (int tl = tile0; tl < tile1; ++tl) {
                const uint32_t bar = bars + 8 * take, tile = ring + take * Sh::kStage;
                if (!dead)
                    dead = __any_sync(0xffffffffu, !attn_try(bar, phase >> take & 1u) && !attn_wait_slow(bar, phase >> take & 1u, ws));
                phase ^= 1u << take;
                const uint32_t have = dead ? 0u : (valid >> (2 * take)) & 3u;
#pragma unroll 1
                for (int i = 0; i < NB; ++i)
                    if (have >> i & 1u)
                        att.block(tile + i * B::kBytes, ((seg.r.first_tile + tl) * NB + i) * kKvBlockTokens);
                take = take + 1 == kStages ? 0 : take + 1;
                __syncwarp();  // every lane has read the stage
                if (!dead) copy_next();
            }

            // ---- the segment's end in this run: written out if whole, else kept as a piece ----
            const bool starts = seg.begin >= r0, ends = seg.end <= r1;
            const int which = starts ? 1 : 0;
            float* const piece = piece_at(warp, which);
            if (!(starts && ends)) {
                if (which == 1 && dead) drain();  // the ring must be quiet before it is written
                __syncwarp();
                if (lane == 0)
                    pieces[2 * warp + which] =
                        AttnPiece{seg.r.q0, rows, seg.h, seg.c, kHas | (starts ? kStarts : 0) | (ends ? kEnds : 0), seg.begin, seg.end};
            }
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    float sum = att.l[n][k];
                    sum += __shfl_xor_sync(0xffffffffu, sum, 4);
                    sum += __shfl_xor_sync(0xffffffffu, sum, 8);
                    sum += __shfl_xor_sync(0xffffffffu, sum, 16);
                    const int r = 8 * n + 2 * t + k, row = seg.c * kRows + r;
                    const float top = att.top(n, k);
                    if (!(starts && ends)) {
                        if (g == 0) *(float2*)(piece + 2 * r) = make_float2(top, sum);
#pragma unroll
                        for (int j = 0; j < J; ++j)
                            *(float4*)(piece + 2 * kRows + r * D + att.channel(j, g)) = att.output(j, n, k);
                    } else if (row < rows) {
                        float inv;
                        __nv_bfloat16* const to = attn_row(p, seg.r.q0, seg.h, row, top, sum, g == 0, inv);
#pragma unroll
                        for (int j = 0; j < J; ++j)
                            attn_store(to + att.channel(j, g), att.output(j, n, k), inv);
                    }
                }
            if (seg.end >= r1) break;
            attn_next<kRows, NB>(p, known, Sh::kThreads, seg);
            load_queries();
        }
        if (dead) drain();  // copies in flight at this point: none, or those that a wait gave up on
    }
    __syncthreads();

    // ---- join the CTA's pieces.  A chain is the pieces of one segment, in order; its first piece leads. ----
    constexpr int kItems = kRows * D / 4;  // four channels of a row each
    static_assert(2 * kWarps <= 32 && kItems % 32 == 0, "a lane for each piece, a warp in one chain");
    const int my_flags = lane < 2 * kWarps ? pieces[lane].flags : 0;
    const uint32_t has = __ballot_sync(0xffffffffu, (my_flags & kHas) != 0);
    if (has == 0u) return;
    const uint32_t leads = __ballot_sync(0xffffffffu, (my_flags & kStarts) != 0) | (has & -has);
    const int chains = __popc(leads);
    {
        // the lanes of this lane's chain, from its lead to the one before the next lead
        const uint32_t until = (2u << lane) - 1u, later = leads & ~until;
        const int lead = 31 - __clz((int)(leads & until | 1u)), last = later != 0u ? __ffs((int)later) - 2 : 31;
        if (warp == kWarps - 1 && leads >> lane & 1u)
            chain[__popc(leads & until) - 1] = make_int2(lane, (int)(has & ~((1u << lane) - 1u) & ((2u << last) - 1u)));
        // A warp takes a row, a lane a piece: a piece's maximum becomes its weight.
        for (int r = warp; r < kRows; r += kWarps) {
            const bool mine = has >> lane & 1u;
            float* const at = piece_at(lane >> 1, lane & 1) + 2 * r;
            const float2 st = mine ? *(const float2*)at : make_float2(-FLT_MAX, 0.f);
            float top = st.x;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const float up = __shfl_up_sync(0xffffffffu, top, o);
                if (lane - o >= lead) top = fmaxf(top, up);
            }
            top = __shfl_sync(0xffffffffu, top, last);
            const float by = exp2_fast(st.x - top);
            float sum = mine ? st.y * by : 0.f;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const float up = __shfl_up_sync(0xffffffffu, sum, o);
                if (lane - o >= lead) sum += up;
            }
            sum = __shfl_sync(0xffffffffu, sum, last);
            if (mine) *at = by;
            if (leads >> lane & 1u) joined[lane][r] = make_float2(top, sum);
        }
    }
    __syncthreads();
    for (int item = tid; item < chains * kItems; item += Sh::kThreads) {
        const int i = item % kItems, lead = chain[item / kItems].x;
        const uint32_t members = (uint32_t)chain[item / kItems].y;
        const int r = i / (D / 4), d = i % (D / 4) * 4;
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
        constexpr int kAhead = 2;  // most chains are two pieces (4: 1 % more for 64 ragged requests)
#pragma unroll 1
        for (uint32_t x = members; x != 0u;) {
            float by[kAhead];
            float4 v[kAhead];
#pragma unroll
            for (int k = 0; k < kAhead; ++k) {
                by[k] = 0.f;
                v[k] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (x != 0u) {
                    const int at = __ffs((int)x) - 1;
                    const float* const src = piece_at(at >> 1, at & 1);
                    by[k] = src[2 * r];
                    v[k] = *(const float4*)(src + 2 * kRows + r * D + d);
                }
                x &= x - 1u;
            }
#pragma unroll
            for (int k = 0; k < kAhead; ++k) {
                o.x = fmaf(v[k].x, by[k], o.x);
                o.y = fmaf(v[k].y, by[k], o.y);
                o.z = fmaf(v[k].z, by[k], o.z);
                o.w = fmaf(v[k].w, by[k], o.w);
            }
        }
        const float2 st = joined[lead][r];
        const AttnPiece& pc = pieces[lead];
        const int starts = pc.flags & kStarts, ends = pieces[31 - __clz((int)members)].flags & kEnds;
        if (starts && ends) {
            const int row = pc.c * kRows + r;
            if (row < pc.rows) {
                float inv;
                __nv_bfloat16* const to = attn_row(p, pc.q0, pc.h, row, st.x, st.y, d == 0, inv);
                attn_store(to + d, o, inv);
            }
        } else {
            float* const dst = partials + ((int64_t)blockIdx.x * 2 + (starts ? 1 : 0)) * Sh::kPartial;
            *(float4*)(dst + 2 * kRows + r * D + d) = o;
            if (d == 0) *(float2*)(dst + 2 * r) = st;
        }
    }

    // ---- join the CTAs that share a segment, the CTA's first chain's or its last's: the last to arrive adds them in order ----
    const int64_t cta0 = (int64_t)blockIdx.x * cta_run, cta1 = cta0 + cta_run;
    const int ends_at[2] = {__ffs((int)leads) - 1, 31 - __clz((int)leads)};
    bool shared[2];
#pragma unroll
    for (int k = 0; k < 2; ++k)
        shared[k] = (k == 0 || chains > 1) && (pieces[ends_at[k]].begin < cta0 || pieces[ends_at[k]].end > cta1);
    if (!shared[0] && !shared[1]) return;
    __syncthreads();
    if (tid < 2) {
        int i0 = 0, parts = 0;
        if (shared[tid]) {
            const AttnPiece& pc = pieces[ends_at[tid]];
            i0 = quotient(pc.begin, cta_run);
            parts = quotient(pc.end - 1, cta_run) - i0 + 1;
            __threadfence();  // of the whole CTA's part: the barrier comes before it
            if (atomicAdd(&ws->arrived[i0], 1u) != (uint32_t)(parts - 1)) parts = 0;
            else ws->arrived[i0] = 0u;
            __threadfence();
        }
        to_join[tid] = make_int2(i0, parts);
    }
    __syncthreads();
    for (int item = tid; item < 2 * kItems; item += Sh::kThreads) {
        const int i = item % kItems, parts = to_join[item / kItems].y;
        const AttnPiece& pc = pieces[item < kItems ? ends_at[0] : ends_at[1]];
        const int r = i / (D / 4), d = i % (D / 4) * 4;
        const int row = pc.c * kRows + r;
        if (parts == 0 || row >= pc.rows) continue;
        constexpr int64_t kStep = 2 * Sh::kPartial;
        const float* const base = partials + (int64_t)to_join[item / kItems].x * kStep;
        float top = -FLT_MAX, sum = 0.f;
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
        constexpr int kAhead = 20;  // parts in flight: a round trip to L2 each otherwise
#pragma unroll 1
        for (int x0 = 0; x0 < parts; x0 += kAhead) {
            float2 st[kAhead];
            float4 v[kAhead];
            const float* src = base + x0 * kStep + (x0 == 0 ? Sh::kPartial : 0);
#pragma unroll
            for (int x = 0; x < kAhead; ++x) {
                st[x] = make_float2(-FLT_MAX, 0.f);
                v[x] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (x0 + x < parts) {
                    st[x] = __ldcg((const float2*)(src + 2 * r));
                    v[x] = __ldcg((const float4*)(src + 2 * kRows + r * D + d));
                }
                src += x0 + x == 0 ? kStep - Sh::kPartial : kStep;
            }
            float now = top;
#pragma unroll
            for (int x = 0; x < kAhead; ++x) now = fmaxf(now, st[x].x);
            const float keep = exp2_fast(top - now);
            top = now;
            sum *= keep;
            o = make_float4(o.x * keep, o.y * keep, o.z * keep, o.w * keep);
#pragma unroll
            for (int x = 0; x < kAhead; ++x) attn_add(top, sum, o, st[x], v[x]);
        }
        float inv;
        __nv_bfloat16* const to = attn_row(p, pc.q0, pc.h, row, top, sum, d == 0, inv);
        attn_store(to + d, o, inv);
    }
}

template <typename F, int D, int NT, int kWarps, int kStages, int NB = 2>
static rra_status_t attn_launch(const AttnParams& p, int ctas, rra_stream_t stream) {
    using Sh = AttnShape<F, D, NT, kWarps, kStages, NB>;
    const void* k = (const void*)kv_attention_kernel<F, D, NT, kWarps, kStages, NB>;
    static_assert(Sh::kFixed + 8 * (RRA_SERVE_MAX_REQUESTS + 1) <= 227 * 1024 - 10240, "shared memory");
    if (configure_cluster_kernel(k, (int)Sh::smem(RRA_SERVE_MAX_REQUESTS)) != cudaSuccess) {
        cudaGetLastError();
        return RRA_ERR_CUDA;
    }
    void* args[] = {(void*)&p};
    return serve_launch(k, dim3((unsigned)ctas), Sh::kThreads, Sh::smem(p.a.requests), 1, stream, args);
}

static bool attn_args_ok(const rra_kv_attention_args_t* a) {
    if (a == nullptr || !kv_cache_ok(a->cache) || a->reserved != 0) return false;
    const int hk = a->cache.kv_heads;
    if (a->requests < 0 || a->requests > RRA_SERVE_MAX_REQUESTS || a->tokens < 0 || a->tokens > INT32_MAX / 2 ||
        a->q_heads < 1 || a->q_heads % hk != 0 || a->table_pages < 0 || a->table_stride < a->table_pages ||
        a->max_q < 0 || a->max_kv < 0 || a->window < 0 || !(fabs(a->scale) * kLog2E <= FLT_MAX))
        return false;
    // rows, and the keys of one request, are counted in 32 bits
    if (a->tokens * a->q_heads > INT32_MAX / 2 || (int64_t)a->table_pages * a->cache.page_tokens > INT32_MAX / 2)
        return false;
    if (!strides_ok(a->q_token_stride, a->q_head_stride, a->q_heads, a->cache.head_dim, 2) ||
        !strides_ok(a->out_token_stride, a->out_head_stride, a->q_heads, a->cache.head_dim, 2) || !aligned16(a->q) ||
        !aligned16(a->out) || ((uintptr_t)a->workspace & 255) != 0)
        return false;
    if (a->requests == 0 || a->tokens == 0) return true;
    return a->q != nullptr && a->out != nullptr && a->cu_q != nullptr && a->kv_len != nullptr &&
           (a->block_table != nullptr || a->table_pages == 0) && a->workspace != nullptr;
}

// Which kernel: the one with the shortest time by what was measured of each, for the sizes that the caller expects (every
// kernel is right for every call).  Times in microseconds, for heads of 128 (64); work on the busiest of 152 SMs:
//   8 or 16 rows     11.5 or 14 (9.5 or 12) + a chunk's tiles of 32 keys at 0.125 or 0.2 (0.085 or 0.135)
//   128 or 256 rows  8 or 11 + tiles of 128 keys at 2.7 or 3.2 (1.9 or 2.0), + joining a segment's parts, 2 (1.1) each
//                    (short segments included: in long ones a tile of 256 rows takes 2.1)
//   8 rows, a cluster of 1, 2, 4, 8 CTAs   3.5 to 4.4 + a warp's tiles of 32 keys at 0.83 (0.64), times 1.1 (0.7) for each
//                    CTA on an SM
// (64 heads over 8 of 128, 8 requests, 4096 keys: 4 queries 37.1, 32.7, 51.5, 56.1 us; 8: 64, 53, 52, 57; 32: 217, 172, 80,
// 58; 32768 keys, 64 queries: 3207, 2376, 932, 525.  1 request and query, 500 keys: 8.1 us against 6.7, 5.6, 4.8, 5.0 in
// clusters; 8000 keys: 13.8 against 57, 31, 17.8, 11.0; 32000: 19.6 against 31.5 in clusters of 8.)
// Over the 8-bit cache, whose codes take fewer instructions and have no second product: 11.2 or 13.8 (10.2 or 12.1) + 0.138 or
// 0.252 (0.078 or 0.133); 10.6 or 17.4 (8.8 or 12.7) + 2.2 or 2.6 (1.65 or 1.95), joins 1.9 (1.1) each; clusters 4.6 to 5.3
// (4.2 to 5.3) + 0.76 (0.62), times 1.03 (0.78).  (Same heads and requests: 1 query, 8192 keys, 31.5, 40.0, 81.0, 97.8 us, in
// clusters 59, 33, 25, 30; 4, 2048: 25.3, 28.5, 40, 48, and 22, 26, 35, 52; 2 requests, 32 queries, 512 keys, 20.0, 23.5, 15.0,
// 20.6, and 17.5, 27.8.  Over 756 sizes of 1 to 32 requests, 1 to 256 queries, 512 to 32768 keys the choice takes 0.8 %
// longer than the best on average, 27 % at most; by the 4-bit cache's numbers 3.2 %, 57 %.)
struct AttnCosts {
    double rows8[2], rows16[2], prompt128[2], prompt256[2], join, team[4], team_tile, team_share;  // what it starts with, and a tile
};
constexpr AttnCosts kAttnCosts[2][2] = {  // 4 bits, 8 bits; heads of 64, of 128
    {{{9.5, 0.085}, {12, 0.135}, {8, 1.9}, {11, 2.0}, 1.1, {3.5, 4.0, 4.1, 4.4}, 0.64, 0.7},
     {{11.5, 0.125}, {14, 0.2}, {8, 2.7}, {11, 3.2}, 2, {3.5, 4.0, 4.1, 4.4}, 0.83, 1.1}},
    {{{10.2, 0.078}, {12.1, 0.133}, {8.76, 1.65}, {12.7, 1.96}, 1.1, {4.2, 5.2, 5.17, 5.29}, 0.62, 0.78},
     {{11.18, 0.138}, {13.8, 0.252}, {10.6, 2.166}, {17.35, 2.573}, 1.87, {4.59, 4.87, 5.01, 5.27}, 0.762, 1.033}}};
enum AttnKernel { kRows8, kRows16, kPrompt128, kPrompt256, kTeam1, kTeam2, kTeam4, kTeam8 };
static AttnKernel attn_kernel_of(const rra_kv_attention_args_t& a, int bits) {
    const AttnCosts& cost = kAttnCosts[bits == 8][a.cache.head_dim == 128];
    const double sms = 152;
    const double rows = (double)std::max(a.max_q, 1) * (a.q_heads / a.cache.kv_heads);
    const double seen = a.window > 0 ? std::min((double)a.max_kv, (double)a.window + a.max_q) : (double)a.max_kv;
    const double heads = (double)std::max(a.requests, 1) * a.cache.kv_heads, tiles = std::max(1.0, std::ceil(seen / kAttnTile));
    auto segments = [&](double n) { return heads * std::ceil(rows / n); };
    auto few = [&](double n, const double* by) { return by[0] + segments(n) * (tiles + kAttnSegmentCost) / sms * by[1]; };
    auto many = [&](double n, const double* by) {
        const double of = std::ceil(seen / 128), run = std::max(6.0, segments(n) * (of + 2) / sms);
        return by[0] + (segments(n) <= sms ? std::min(of, run) : run) * by[1] + (of > run ? of / run * cost.join : 0);
    };
    auto team = [&](double size, double fixed) {
        const double ctas = segments(8) * size;
        if (ctas > 16 * sms) return 1e30;
        return fixed + std::ceil(tiles / (kTeamWarps * size)) * cost.team_tile * std::max(1.0, cost.team_share * ctas / sms);
    };
    const double t[8] = {few(8, cost.rows8),     few(16, cost.rows16),  many(128, cost.prompt128), many(256, cost.prompt256),
                         team(1, cost.team[0]), team(2, cost.team[1]), team(4, cost.team[2]),     team(8, cost.team[3])};
    return (AttnKernel)(std::min_element(t, t + 8) - t);
}

}  // namespace rra

extern "C" {

size_t rra_kv_attention_workspace_bytes(int head_dim) {
    if (head_dim != 64 && head_dim != 128) return 0;
    const size_t decode = (size_t)rra::kAttnMaxCtas * 2 * rra::kAttnMaxRows * ((size_t)head_dim + 2) * sizeof(float);
    return sizeof(rra::AttnWorkspace) + std::max(decode, rra::prefill_partial_bytes(head_dim));
}

static rra_status_t kv_attention_plan(const rra_kv_attention_args_t* args, int bits, const char** name) {
    if (name == nullptr || !rra::attn_args_ok(args)) return RRA_ERR_INVALID_ARG;
    static const char* const names[] = {"kv_attention_kernel<8 rows>", "kv_attention_kernel<16 rows>",
                                        "kv_attention_prompt_kernel<128 rows>", "kv_attention_prompt_kernel<256 rows>",
                                        "kv_attention_team_kernel<1 CTA>", "kv_attention_team_kernel<2 CTAs>",
                                        "kv_attention_team_kernel<4 CTAs>", "kv_attention_team_kernel<8 CTAs>"};
    *name = names[rra::attn_kernel_of(*args, bits)];
    return RRA_OK;
}

rra_status_t rra_kv_attention_plan(const rra_kv_attention_args_t* args, const char** name) { return kv_attention_plan(args, 4, name); }

rra_status_t rra_kv8_attention_plan(const rra_kv_attention_args_t* args, const char** name) { return kv_attention_plan(args, 8, name); }

static rra_status_t kv_attention(const rra_kv_attention_args_t* args, int bits, rra_stream_t stream) {
    if (!rra::attn_args_ok(args)) return RRA_ERR_INVALID_ARG;
    if (args->requests == 0 || args->tokens == 0) return RRA_OK;
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
        cudaGetLastError();
        return RRA_ERR_CUDA;
    }
    rra::AttnParams p;
    p.a = *args;
    p.scale_log2 = (float)(args->scale * rra::kLog2E);
    p.group = args->q_heads / args->cache.kv_heads;
    p.by_group = rra::Divisor(p.group);
    p.by_page = rra::Divisor(args->cache.page_tokens);
    p.room = args->table_pages * args->cache.page_tokens;
    p.window = std::min(args->window, 1 << 30);
    const rra::AttnKernel kernel = rra::attn_kernel_of(*args, bits);
    if (kernel >= rra::kTeam1)
        return rra::launch_team(p, bits, (int)(((int64_t)std::max(args->max_q, 1) * p.group + 7) / 8), 1 << (kernel - rra::kTeam1), stream);
    if (kernel == rra::kPrompt128 || kernel == rra::kPrompt256)
        return rra::launch_prefill(p, bits, kernel == rra::kPrompt256 ? 2 : 1, sms, stream);
    const int ctas = std::min(sms, rra::kAttnMaxCtas);
    using rra::Cache4;
    using rra::Cache8;
    const bool eight = kernel == rra::kRows8;
    if (bits == 8) {
        // pages are twice as large: one block a stage where two take the room of warps (64 ragged requests: 60.3 us, with two 61.8)
        if (args->cache.head_dim == 128)
            return eight ? rra::attn_launch<Cache8, 128, 1, 12, 2, 1>(p, ctas, stream) : rra::attn_launch<Cache8, 128, 2, 6, 2>(p, ctas, stream);
        return eight ? rra::attn_launch<Cache8, 64, 1, 12, 3>(p, ctas, stream) : rra::attn_launch<Cache8, 64, 2, 8, 3>(p, ctas, stream);
    }
    if (args->cache.head_dim == 128)
        return eight ? rra::attn_launch<Cache4, 128, 1, 12, 2>(p, ctas, stream) : rra::attn_launch<Cache4, 128, 2, 8, 2>(p, ctas, stream);
    return eight ? rra::attn_launch<Cache4, 64, 1, 12, 3>(p, ctas, stream) : rra::attn_launch<Cache4, 64, 2, 8, 4>(p, ctas, stream);
}

rra_status_t rra_kv_attention(const rra_kv_attention_args_t* args, rra_stream_t stream) { return kv_attention(args, 4, stream); }

rra_status_t rra_kv8_attention(const rra_kv_attention_args_t* args, rra_stream_t stream) { return kv_attention(args, 8, stream); }

}  // extern "C"
