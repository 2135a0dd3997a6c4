// serve_attn_team.cu -- attention over the 4-bit cache for few requests, where
// latency is all (rra_serve.h).
//
// A thread-block cluster takes eight rows of one request and KV head; its warps
// share the keys in equal runs of tiles (32 keys).  The warps' results meet in
// shared memory, the CTAs' through distributed shared memory between two cluster
// barriers: against serve_attn.cu there is no scan of the batch before the first
// copy, and no fence, counter and round trip to L2 after the last key.  What
// remains is lengths, page numbers, pages: three round trips, one after another.
// 8 heads over 1 of 128: 2000 keys in 5.6 us (the other kernel: 9.7).  24
// requests of up to 5 queries, 14 heads over 2 of 64, a window of 1000: 10.8 us.
#include "serve_attn_rows.cuh"

namespace rra {

constexpr int kTeamStages = 2;

template <int D>
struct TeamShape {
    using B = KvBlock<D>;
    static constexpr int kThreads = 32 * kTeamWarps;
    static constexpr int kStage = 2 * B::kBytes;
    static constexpr int kRing = kTeamWarps * kTeamStages * kStage;
    static constexpr int kPart = 8 * (D + 2) * 4;            // maximum and sum of each row, rows
    static constexpr int kParts = kRing;                     // of the warps, then of the CTA
    static constexpr int kBars = kParts + (kTeamWarps + 1) * kPart;
    static constexpr int kSmem = kBars + kTeamWarps * kTeamStages * 8;
};

__device__ __forceinline__ float2 ld_peer_v2(uint32_t addr) {
    float2 v;
    asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ float4 ld_peer_v4(uint32_t addr) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr) : "memory");
    return v;
}

// Sums of parts: `get(x)` the maximum and sum, and four channels, of part x < n.
template <int kMost, typename F>
__device__ __forceinline__ void team_add(int n, F&& get, float& top, float& sum, float4& o) {
    float2 st[kMost];
    float4 v[kMost];
#pragma unroll
    for (int x = 0; x < kMost; ++x) {
        st[x] = make_float2(-FLT_MAX, 0.f);
        v[x] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (x < n) get(x, st[x], v[x]);
    }
    top = -FLT_MAX;
#pragma unroll
    for (int x = 0; x < kMost; ++x) top = fmaxf(top, st[x].x);
    sum = 0.f;
    o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int x = 0; x < kMost; ++x) {
        const float by = exp2_fast(st[x].x - top);
        sum = fmaf(st[x].y, by, sum);
        o.x = fmaf(v[x].x, by, o.x);
        o.y = fmaf(v[x].y, by, o.y);
        o.z = fmaf(v[x].z, by, o.z);
        o.w = fmaf(v[x].w, by, o.w);
    }
}

// Cluster i: KV head and request of segment i, rows 8 c .. of chunk c, and of chunk c + chunks and so on.
template <int D>
__global__ void __launch_bounds__(32 * kTeamWarps, 3) kv_attention_team_kernel(const __grid_constant__ AttnParams p, int chunks) {
    using Sh = TeamShape<D>;
    using B = KvBlock<D>;
    constexpr int kItems = 8 * D / 4;  // four channels of a row each
    extern __shared__ __align__(128) unsigned char smem[];
    const rra_kv_attention_args_t& a = p.a;
    const int tid = (int)threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
    const int rank = (int)cluster_ctarank(), team = kTeamWarps * (int)(gridDim.x / (unsigned)(a.requests * a.cache.kv_heads * chunks));
    const int size = team / kTeamWarps, mine = rank * kTeamWarps + warp;
    int segment = (int)cluster_id();
    const int b = segment / (a.cache.kv_heads * chunks);
    segment -= b * a.cache.kv_heads * chunks;
    const int h = segment / chunks, c0 = segment - h * chunks;
    const uint32_t ring = smem_u32(smem) + warp * kTeamStages * Sh::kStage, bars = smem_u32(smem) + Sh::kBars + warp * kTeamStages * 8;
    float* const whole = (float*)(smem + Sh::kParts + kTeamWarps * Sh::kPart);  // the CTA's part
    auto part_of = [&](int w) { return (float*)(smem + Sh::kParts + w * Sh::kPart); };
    AttnWorkspace* const ws = (AttnWorkspace*)a.workspace;

    pdl_release_early();
    if (lane == 0) {
#pragma unroll
        for (int i = 0; i < kTeamStages; ++i) mbar_init(bars + 8 * i, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        fence_proxy_async_smem();
    }
    __syncwarp();
    pdl_wait();
    const AttnLengths n = attn_lengths(p, b);
    const int rows = n.qn * p.group;
    const int first = (p.window > 0 ? max(0, n.kv - n.qn - p.window + 1) : 0) / kAttnTile;
    const int tiles = max(1, (n.kv + kAttnTile - 1) / kAttnTile - first);
    const int run = (tiles + team - 1) / team;
    const int t0 = min(tiles, mine * run), t1 = min(tiles, t0 + run);
    const int ps = a.cache.page_tokens, blocks = ps / kKvBlockTokens;
    const int32_t* const table = a.block_table + b * a.table_stride;
    int put = 0, take = 0;                    // stages of the next copy and of the next tile
    uint32_t valid = 0, issued = 0, phase = 0;
    bool dead = false;  // a wait ran out: no more copies, no more sums

    for (int c = c0; c * 8 < rows; c += chunks) {  // the same for every CTA of the cluster
        AttnRows<D, 1> att;
        att.load(p, n.q0, n.qn, h, c, t0 < t1);
        // copies, kTeamStages tiles ahead; lane i holds the places of tile `from` + i
        int next = t0, from = t0 - 32;
        const char* src0 = nullptr;
        const char* src1 = nullptr;
        uint32_t ok0 = 0, ok1 = 0;
        auto copy_next = [&]() {
            if (next >= t1) return;
            if (next >= from + 32) {
                from = next;
                auto place = [&](int k) -> const char* {
                    if (from + lane >= t1 || k >= n.kv) return nullptr;
                    const int i = p.by_page(k), page = table[i];
                    if (page < 0 || page >= a.cache.num_pages) return nullptr;
                    return (const char*)a.cache.pages +
                           (((int64_t)page * a.cache.kv_heads + h) * blocks + (k - i * ps) / kKvBlockTokens) * B::kBytes;
                };
                src0 = place((first + from + lane) * kAttnTile);
                src1 = place((first + from + lane) * kAttnTile + kKvBlockTokens);
                ok0 = __ballot_sync(0xffffffffu, src0 != nullptr);
                ok1 = __ballot_sync(0xffffffffu, src1 != nullptr);
            }
            const int held = next - from;
            if (lane == held) {
                const uint32_t bar = bars + 8 * put, dst = ring + put * Sh::kStage;
                const bool h0 = src0 != nullptr, h1 = src1 != nullptr;
                mbar_expect_tx(bar, ((h0 ? 1u : 0u) + (h1 ? 1u : 0u)) * (uint32_t)B::kBytes);
                if (h0) bulk_g2s(dst, src0, B::kBytes, bar);
                if (h1) bulk_g2s(dst + B::kBytes, src1, B::kBytes, bar);
            }
            valid = (valid & ~(3u << (2 * put))) | ((ok0 >> held & 1u) | (ok1 >> held & 1u) << 1) << (2 * put);
            issued ^= 1u << put;
            put = put + 1 == kTeamStages ? 0 : put + 1;
            ++next;
        };
        if (!dead) {
#pragma unroll 1
            for (int i = 0; i < kTeamStages; ++i) copy_next();
        }
        att.start(p, n.qn, n.kv, c);
#pragma unroll 1
        for (int tl = t0; tl < t1 && !dead; ++tl) {
            const uint32_t bar = bars + 8 * take;
            dead = __any_sync(0xffffffffu, !attn_try(bar, phase >> take & 1u) && !attn_wait_slow(bar, phase >> take & 1u, ws));
            if (dead) break;
            phase ^= 1u << take;
            const uint32_t have = valid >> (2 * take) & 3u;
#pragma unroll 1
            for (int i = 0; i < 2; ++i)
                if (have >> i & 1u)
                    att.block(ring + take * Sh::kStage + i * B::kBytes, (first + tl) * kAttnTile + kKvBlockTokens * i);
            take = take + 1 == kTeamStages ? 0 : take + 1;
            __syncwarp();  // every lane has read the stage
            copy_next();
        }

        // ---- the warp's part, the CTA's, the cluster's ----
        float* const part = part_of(warp);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            float sum = att.l[0][k];
            sum += __shfl_xor_sync(0xffffffffu, sum, 4);
            sum += __shfl_xor_sync(0xffffffffu, sum, 8);
            sum += __shfl_xor_sync(0xffffffffu, sum, 16);
            const int r = 2 * t + k;
            if (g == 0) *(float2*)(part + 2 * r) = make_float2(att.top(0, k), sum);
#pragma unroll
            for (int j = 0; j < B::kGroups; ++j) *(float4*)(part + 16 + r * D + 32 * j + 4 * g) = att.output(j, 0, k);
        }
        __syncthreads();
        for (int i = tid; i < kItems; i += Sh::kThreads) {
            const int r = i / (D / 4), d = i % (D / 4) * 4;
            float top, sum;
            float4 o;
            team_add<kTeamWarps>(kTeamWarps, [&](int x, float2& st, float4& v) {
                st = *(const float2*)(part_of(x) + 2 * r);
                v = *(const float4*)(part_of(x) + 16 + r * D + d);
            }, top, sum, o);
            if (d == 0) *(float2*)(whole + 2 * r) = make_float2(top, sum);
            *(float4*)(whole + 16 + r * D + d) = o;
        }
        if (size > 1) cluster_sync();
        else __syncthreads();
        for (int i = rank * Sh::kThreads + tid; i < kItems; i += size * Sh::kThreads) {
            const int r = i / (D / 4), d = i % (D / 4) * 4, row = c * 8 + r;
            if (row >= rows) continue;
            float top, sum;
            float4 o;
            team_add<8>(size, [&](int x, float2& st, float4& v) {
                st = ld_peer_v2(map_to_rank(smem_u32(whole + 2 * r), (uint32_t)x));
                v = ld_peer_v4(map_to_rank(smem_u32(whole + 16 + r * D + d), (uint32_t)x));
            }, top, sum, o);
            float inv;
            __nv_bfloat16* const to = attn_row(p, n.q0, h, row, top, sum, d == 0, inv);
            attn_store(to + d, o, inv);
        }
        if (size > 1) cluster_sync();  // the parts have been read
        else __syncthreads();
    }
    if (dead)  // copies that a wait gave up on
        for (int i = 0; i < kTeamStages; ++i) attn_wait_quiet(bars + 8 * i, (issued >> i & 1u) ^ 1u);
}

rra_status_t launch_team(const AttnParams& p, int chunks, int size, rra_stream_t stream) {
    const bool big = p.a.cache.head_dim == 128;
    const void* const k = big ? (const void*)kv_attention_team_kernel<128> : (const void*)kv_attention_team_kernel<64>;
    const int smem = big ? TeamShape<128>::kSmem : TeamShape<64>::kSmem;
    if (configure_cluster_kernel(k, smem) != cudaSuccess) {
        cudaGetLastError();
        return RRA_ERR_CUDA;
    }
    void* args[] = {(void*)&p, &chunks};
    return serve_launch(k, dim3((unsigned)(p.a.requests * p.a.cache.kv_heads * chunks * size)), 32 * kTeamWarps, (size_t)smem, size, stream, args);
}

}  // namespace rra
