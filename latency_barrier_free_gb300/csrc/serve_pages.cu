// serve_pages.cu -- pages that requests share (rra_serve.h): fork, release,
// compact, and the copies that go with them.
//
// The first three are bookkeeping, bound by latency like the slot map: one
// cluster, whose barriers separate what is read from what is written to the same
// buffers, and whose CTAs share rows and pages.  The copies are bound by HBM.
//
// One prompt into 8 samples 4.8 us with its copies, 32 into 8 each 12.3 (63 MB).  After 500 requests over 22773 pages
// release takes 12.0 us, compaction 13.0, the copies of 5620 pages of 33 KB 58 (6.4 TB/s); after 9 requests 3.8, 5.3 and 1.5.
#include <algorithm>

#include "cluster_prims.cuh"
#include "kernel_attrs.h"
#include "serve_common.cuh"

namespace rra {

constexpr int kPagesThreads = 1024;
constexpr int kPagesMaxCluster = 16;
constexpr int kPagesMost = (1 << 30) - 1;  // tokens of a request
constexpr int kPagesPool = 1 << 24;        // pages of a pool: a bit each in the cluster's shared memory

__device__ __forceinline__ void pages_sync() {
    if (gridDim.x > 1) cluster_sync();
    else __syncthreads();
}

// Sum over the block, and this thread's exclusive part of it; part: a word for each warp.
__device__ __forceinline__ int pages_scan(int v, int& total, int* part) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int inc = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int up = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += up;
    }
    if (lane == 31) part[warp] = inc;
    __syncthreads();
    int w = lane < (int)(blockDim.x >> 5) ? part[lane] : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int up = __shfl_up_sync(0xffffffffu, w, o);
        if (lane >= o) w += up;
    }
    total = __shfl_sync(0xffffffffu, w, 31);
    const int before = warp > 0 ? __shfl_sync(0xffffffffu, w, warp - 1) : 0;
    __syncthreads();
    return before + inc - v;
}

__device__ __forceinline__ int ld_peer_int(uint32_t addr) {
    int v;
    asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
    return v;
}
// Sums over the cluster of a word of each CTA's shared memory, of those before this CTA and of all; between two cluster
// barriers after it was written, before it is written again.
__device__ __forceinline__ void pages_meet(const int* mine, int& before, int& all) {
    before = 0, all = 0;
    if (gridDim.x == 1) {
        all = *mine;
        return;
    }
    for (uint32_t x = 0; x < gridDim.x; ++x) {
        const int v = ld_peer_int(map_to_rank(smem_u32(mine), x));
        if (x < blockIdx.x) before += v;
        all += v;
    }
}

// Pages as bits in the shared memory of the cluster: CTA x has the words of pages x * run .. (x + 1) * run.
struct PageBits {
    uint32_t* words;
    int run, begin, end, count;  // pages of a CTA, this one's, its words
    __device__ __forceinline__ PageBits(uint32_t* at, int n) : words(at) {
        run = (int)(((int64_t)n + gridDim.x - 1) / gridDim.x + 31) & ~31;
        begin = (int)min((int64_t)n, (int64_t)run * blockIdx.x);
        end = min(n, begin + run);
        count = (end - begin + 31) >> 5;
        for (int i = (int)threadIdx.x; i < run >> 5; i += (int)blockDim.x) words[i] = 0u;
    }
    __device__ __forceinline__ void set(int page) const {
        const uint32_t cta = (uint32_t)page / (uint32_t)run, in = (uint32_t)page - cta * (uint32_t)run;
        const uint32_t at = smem_u32(words + (in >> 5)), bit = 1u << (in & 31);
        if (gridDim.x == 1) atomicOr(words + (in >> 5), bit);
        else asm volatile("red.relaxed.cluster.shared::cluster.or.b32 [%0], %1;" : : "r"(map_to_rank(at, cta)), "r"(bit) : "memory");
    }
};

// ================================================================= fork ====
struct ForkParams {
    rra_pages_fork_args_t a;
    Divisor by_page;
};

__global__ void __launch_bounds__(kPagesThreads, 1) pages_fork_kernel(const __grid_constant__ ForkParams p) {
    __shared__ int part[32];
    const rra_pages_fork_args_t& a = p.a;
    const int tid = (int)threadIdx.x, nt = (int)blockDim.x, lane = tid & 31;
    const int me = (int)blockIdx.x * nt + tid, all = (int)gridDim.x * nt;
    extern __shared__ int32_t fork_mem[];  // of every fork: its rank among the pages popped, -1: none
    pdl_release_early();
    pdl_wait();
    const int count = min(max(a.free_count[0], 0), a.num_pages);
    // What is not in place is copied; the forks' own lengths and counts come after the barrier.
    if (a.kv_len != a.seq_len)
        for (int b = me; b < a.requests; b += all) a.kv_len[b] = a.seq_len[b];
    if (a.shared_out != a.shared)
        for (int i = me; i < a.num_pages; i += all) a.shared_out[i] = a.shared[i];
    auto good = [&](int i, int& from, int& to) {
        from = a.source[i], to = a.target[i];
        return from >= 0 && from < a.requests && to >= 0 && to < a.requests;
    };
    auto whole = [&](int from, int& length) {  // full pages of a request
        length = min(max(a.seq_len[from], 0), kPagesMost);
        return min(p.by_page(length), a.table_pages);
    };
    int wanted = 0;
    for (int i0 = 0; i0 < a.forks; i0 += nt) {
        const int i = i0 + tid;
        int from, to, length, needs = 0, total;
        if (i < a.forks && good(i, from, to)) {
            const int full = whole(from, length);
            if (full < a.table_pages && length > full * a.page_tokens) {
                const int page = a.block_table[from * a.table_stride + full];
                needs = page >= 0 && page < a.num_pages;
            }
        }
        const int rank = wanted + pages_scan(needs, total, part);
        if (i < a.forks) fork_mem[i] = needs ? rank : -1;
        wanted += total;
    }
    pages_sync();  // lengths and counts that were copied, and the ranks
    // a warp a fork
    for (int i = me >> 5; i < a.forks; i += all >> 5) {
        int from, to, length;
        int source = -1, fresh = -1;
        if (good(i, from, to)) {
            const int full = whole(from, length), rank = fork_mem[i];
            const int32_t* const src = a.block_table + from * a.table_stride;
            int32_t* const dst = a.block_table + to * a.table_stride;
            constexpr int kAhead = 4;
            for (int j0 = 0; j0 < full; j0 += 32 * kAhead) {
                int page[kAhead];
#pragma unroll
                for (int k = 0; k < kAhead; ++k) page[k] = j0 + 32 * k + lane < full ? src[j0 + 32 * k + lane] : -1;
#pragma unroll
                for (int k = 0; k < kAhead; ++k) {
                    if (j0 + 32 * k + lane >= full) continue;
                    dst[j0 + 32 * k + lane] = page[k];
                    if (page[k] >= 0 && page[k] < a.num_pages) atomicAdd(a.shared_out + page[k], 1);
                }
            }
            if (full < a.table_pages && length > full * a.page_tokens && lane == 0) {
                const int page = src[full];
                if (rank >= 0 && rank < count) fresh = a.free_pages[count - 1 - rank];
                if (fresh < 0 || fresh >= a.num_pages) fresh = -1;
                else source = page;
                dst[full] = rank >= 0 ? fresh : page;
            }
            if (lane == 0) a.kv_len[to] = max(a.seq_len[from], 0);
        }
        if (lane == 0) {
            a.copy_from[i] = source;
            a.copy_to[i] = fresh;
        }
    }
    pages_sync();  // everybody has read the count that free_left may be
    if (me == 0) {
        a.free_left[0] = max(0, count - wanted);
        a.pages_short[0] = max(0, wanted - count);
    }
}

// ============================================================== release ====
struct ReleaseParams {
    rra_pages_release_args_t a;
    Divisor by_page;
};

__global__ void __launch_bounds__(kPagesThreads, 1) pages_release_kernel(const __grid_constant__ ReleaseParams p) {
    extern __shared__ uint32_t bits_mem[];
    __shared__ int part[32], gone;
    const rra_pages_release_args_t& a = p.a;
    const int tid = (int)threadIdx.x, nt = (int)blockDim.x, lane = tid & 31;
    const int me = (int)blockIdx.x * nt + tid, all = (int)gridDim.x * nt;
    pdl_release_early();
    const PageBits bits(bits_mem, a.num_pages);  // pages that lose their last holder
    pdl_wait();
    const int count = min(max(a.free_count[0], 0), a.num_pages);
    if (a.shared_out != a.shared)
        for (int i = me; i < a.num_pages; i += all) a.shared_out[i] = a.shared[i];
    pages_sync();
    // A holder less for every page of a request that ends.  Whoever takes the last one away marks the page, and a page that is
    // listed more often than held has its count put right at the end.
    for (int b = me >> 5; b < a.requests; b += all >> 5) {
        const int length = min(max(a.seq_len[b], 0), kPagesMost);
        const bool ends = a.new_len[b] < 0;
        __syncwarp();
        if (lane == 0) a.kv_len[b] = ends ? 0 : a.seq_len[b];
        if (!ends) continue;
        const int held = min(length > 0 ? p.by_page(length - 1) + 1 : 0, a.table_pages);
        const int32_t* const row = a.block_table + b * a.table_stride;
        constexpr int kAhead = 4;
        for (int j0 = 0; j0 < held; j0 += 32 * kAhead) {
            int page[kAhead];
#pragma unroll
            for (int k = 0; k < kAhead; ++k) page[k] = j0 + 32 * k + lane < held ? row[j0 + 32 * k + lane] : -1;
#pragma unroll
            for (int k = 0; k < kAhead; ++k)
                if (page[k] >= 0 && page[k] < a.num_pages && atomicSub(a.shared_out + page[k], 1) <= 0) bits.set(page[k]);
        }
    }
    pages_sync();
    // Marked pages go back, in their order: a word a thread.
    int mine = 0;
    for (int i = tid; i < bits.count; i += nt) mine += __popc(bits.words[i]);
    int total, before, whole;
    pages_scan(mine, total, part);
    if (tid == 0) gone = total;
    pages_sync();
    pages_meet(&gone, before, whole);
    int at = count + before;
    if (total > 0)
        for (int i0 = 0; i0 < bits.count; i0 += nt) {
            uint32_t who = i0 + tid < bits.count ? bits.words[i0 + tid] : 0u;
            int some, rank = at + pages_scan(__popc(who), some, part);
            for (; who != 0u; who &= who - 1u, ++rank) {
                const int page = bits.begin + 32 * (i0 + tid) + __ffs((int)who) - 1;
                if (rank < a.num_pages) a.free_pages[rank] = page;
                a.shared_out[page] = 0;
            }
            at += some;
        }
    pages_sync();  // `gone` has been read, and the count that free_left may be
    if (me == 0) a.free_left[0] = min(count + whole, a.num_pages);
}

// ============================================================== compact ====
struct CompactParams {
    rra_pages_compact_args_t a;
    Divisor by_page;
};

__global__ void __launch_bounds__(kPagesThreads, 1) pages_compact_kernel(const __grid_constant__ CompactParams p) {
    extern __shared__ uint32_t bits_mem[];
    __shared__ int part[32], holes;
    const rra_pages_compact_args_t& a = p.a;
    const int tid = (int)threadIdx.x, nt = (int)blockDim.x, lane = tid & 31;
    const int me = (int)blockIdx.x * nt + tid, all = (int)gridDim.x * nt;
    pdl_release_early();
    const int n = a.num_pages;
    const PageBits bits(bits_mem, n);  // pages that are free
    pages_sync();
    pdl_wait();
    const int count = min(max(a.free_count[0], 0), n);
    for (int i = me; i < count; i += all) {
        const int page = a.free_pages[i];
        if (page >= 0 && page < n) bits.set(page);
    }
    if (a.shared_out != a.shared)
        for (int i = me; i < n; i += all) a.shared_out[i] = a.shared[i];
    for (int i = me; i < a.max_moves; i += all) a.move_from[i] = a.move_to[i] = -1;
    pages_sync();
    // ---- how many are free, and how many of those lie below the number in use ----
    int mine = 0, total, before, free_all;
    for (int i = tid; i < bits.count; i += nt) mine += __popc(bits.words[i]);
    pages_scan(mine, total, part);
    if (tid == 0) holes = total;
    pages_sync();
    pages_meet(&holes, before, free_all);
    const int used = n - free_all;
    int moves;
    {
        // those of the CTAs before the one that has page `used`, and of its words up to there
        const int cta = used < n ? used / bits.run : (int)gridDim.x, in = used - cta * bits.run;
        int low = 0;
        if (gridDim.x == 1) {
            for (int i = tid; i < in >> 5; i += nt) low += __popc(bits.words[i]);
            if (cta == 0 && tid == 0 && (in & 31) != 0) low += __popc(bits.words[in >> 5] & ((1u << (in & 31)) - 1u));
            if (cta == 1 && tid == 0) low = free_all;
        } else {
            if (tid < (int)gridDim.x && tid < cta) low += ld_peer_int(map_to_rank(smem_u32(&holes), (uint32_t)tid));
            if (cta < (int)gridDim.x)
                for (int i = tid; 32 * i < in; i += nt) {
                    const uint32_t w = (uint32_t)ld_peer_int(map_to_rank(smem_u32(bits.words + i), (uint32_t)cta));
                    low += __popc(in - 32 * i >= 32 ? w : w & ((1u << (in - 32 * i)) - 1u));
                }
        }
        int low_all;
        pages_scan(low, low_all, part);
        moves = min(low_all, a.max_moves);
    }
    // ---- the lists.  Of page i: `lower` free pages and i - lower used ones lie below it.  moved[] of a page that leaves: the
    // complement of 1 + the number of its move, until the move's other end is known ----
    int at = before;
    for (int i0 = 0; i0 < bits.count; i0 += nt >> 3) {  // eight threads a word, four pages each
        const int word = i0 + (tid >> 3);
        const uint32_t whole_word = word < bits.count ? bits.words[word] : 0u, who = whole_word >> (4 * (tid & 7)) & 15u;
        int some, lower = at + pages_scan(__popc(who), some, part);
        const int first = bits.begin + 32 * word + 4 * (tid & 7);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int i = first + k;
            if (word >= bits.count || i >= bits.end) continue;
            const int used_below = i - lower;
            bool now;  // free afterwards
            int to = -1;
            if (who >> k & 1u) {
                now = lower >= moves;  // its rank among the holes
                if (!now) a.move_to[lower] = i;
            } else {
                const int above = used - 1 - used_below;
                now = above < moves;
                if (now) a.move_from[above] = i;
                to = now ? ~(1 + above) : i;
            }
            a.moved[i] = to;
            if (now) {
                const int rank = lower - min(lower, moves) + max(0, used_below - (used - moves));  // free afterwards and lower
                a.free_out[free_all - 1 - rank] = i;
            }
            lower += who >> k & 1u;
        }
        at += some;
    }
    pages_sync();
    for (int i = me; i < moves; i += all) {
        const int from = __ldcg(a.move_from + i), to = __ldcg(a.move_to + i);
        a.moved[from] = to;
        a.shared_out[to] = __ldcg(a.shared_out + from);
        a.shared_out[from] = 0;
    }
    if (me == 0) {
        a.free_left[0] = free_all;
        a.move_count[0] = moves;
    }
    // ---- the tables: a warp a row.  What moved[] says may be either, the move's number or its end ----
    for (int b = me >> 5; b < a.requests; b += all >> 5) {
        const int length = min(max(a.seq_len[b], 0), kPagesMost);
        const int held = min(length > 0 ? p.by_page(length - 1) + 1 : 0, a.table_pages);
        const int32_t* const row = a.block_table + b * a.table_stride;
        int32_t* const to = a.table_out + b * a.table_out_stride;
        const int entries = a.table_out == a.block_table ? held : a.table_pages;
        constexpr int kAhead = 4;
        for (int j0 = 0; j0 < entries; j0 += 32 * kAhead) {
            int page[kAhead];
#pragma unroll
            for (int k = 0; k < kAhead; ++k) page[k] = j0 + 32 * k + lane < entries ? row[j0 + 32 * k + lane] : -1;
            int now[kAhead];
#pragma unroll
            for (int k = 0; k < kAhead; ++k) {
                now[k] = page[k];
                if (j0 + 32 * k + lane < held && page[k] >= 0 && page[k] < n) now[k] = __ldcg(a.moved + page[k]);
            }
#pragma unroll
            for (int k = 0; k < kAhead; ++k) {
                const int j = j0 + 32 * k + lane;
                if (j >= entries) continue;
                if (j < held && page[k] >= 0 && page[k] < n && now[k] < -1) now[k] = __ldcg(a.move_to + (~now[k] - 1));
                to[j] = now[k];
            }
        }
    }
}

// ================================================================= copy ====
constexpr int kCopyThreads = 256;
constexpr int kCopyAhead = 8;  // 16-byte loads of a thread in flight
constexpr int kCopyCtas = 152 * 16;  // (5620 pages of 33 KB: 8 an SM 60.8 us, 16 59.1, 32 58.0, but of 8192 listed moves 626 9.1, 8.4 and 10.5)

struct CopyParams {
    rra_pages_copy_args_t a;
    Divisor by_pieces; // pieces of a page
    int32_t total;     // pieces of all pages
    int32_t vectors;   // of a piece, the last one's may be fewer
    int64_t page;      // vectors of a page
};

// A CTA takes every gridDim'th piece; it looks at kCopyThreads pairs at once, so that lists that are mostly empty (the
// moves of a pool that needs few) cost a round trip, not one a pair.
__global__ void __launch_bounds__(kCopyThreads) pages_copy_kernel(const __grid_constant__ CopyParams p) {
    const rra_pages_copy_args_t& a = p.a;
    __shared__ const uint4* srcs[kCopyThreads];
    __shared__ uint4* dsts[kCopyThreads];
    __shared__ int32_t lengths[kCopyThreads];
    pdl_release_early();
    pdl_wait();
    for (int64_t w0 = blockIdx.x; w0 < p.total; w0 += (int64_t)gridDim.x * kCopyThreads) {
        const int64_t w = w0 + (int64_t)threadIdx.x * gridDim.x;
        int length = 0;
        if (w < p.total) {
            const int i = p.by_pieces((int)w);
            const int64_t piece = w - (int64_t)i * p.by_pieces.d;
            const int from = a.from[i], to = a.to[i];
            if (from >= 0 && to >= 0 && from < a.from_num && to < a.to_num) {
                srcs[threadIdx.x] = (const uint4*)((const char*)a.from_pages + (int64_t)from * a.page_bytes) + piece * p.vectors;
                dsts[threadIdx.x] = (uint4*)((char*)a.to_pages + (int64_t)to * a.page_bytes) + piece * p.vectors;
                length = (int)min((int64_t)p.vectors, p.page - piece * p.vectors);
            }
        }
        lengths[threadIdx.x] = length;
        const int some = __syncthreads_or(length > 0);
        if (some)
            for (int k = 0; k < kCopyThreads && w0 + (int64_t)k * gridDim.x < p.total; ++k) {
                const int n = lengths[k];
                if (n == 0) continue;
                const uint4* const src = srcs[k] + threadIdx.x;
                uint4* const dst = dsts[k] + threadIdx.x;
                uint4 x[kCopyAhead];
#pragma unroll
                for (int v = 0; v < kCopyAhead; ++v)
                    if ((int)threadIdx.x + v * kCopyThreads < n) x[v] = __ldcs(src + v * kCopyThreads);
#pragma unroll
                for (int v = 0; v < kCopyAhead; ++v)
                    if ((int)threadIdx.x + v * kCopyThreads < n) __stcs(dst + v * kCopyThreads, x[v]);
            }
        __syncthreads();
    }
}

// CTAs for so many items of a thread's work.
static int pages_ctas(int64_t items) {
    int ctas = 1;
    while (ctas < kPagesMaxCluster && (int64_t)ctas * kPagesThreads < items) ctas *= 2;
    return ctas;
}

// Threads of a CTA: fewer warps meet sooner.  (256, 512 and 1024: release, compaction and copies after 9 requests 11.0, 10.7 and
// 11.4 us, after 30 14.2, 12.5 and 11.9.)
static int pages_threads(int64_t items) { return items <= 768 ? 512 : kPagesThreads; }

// Bytes of shared memory that so many pages take in each CTA.
static size_t pages_bits(int pages, int ctas) { return ((size_t)pages / (size_t)ctas + 32) / 32 * 4 + 4; }

static bool pages_ok(int requests, int table_pages, int64_t stride, int page_tokens, int num_pages, const void* table, const void* lengths) {
    if (requests < 0 || requests > RRA_SERVE_MAX_REQUESTS || table_pages < 0 || stride < table_pages || page_tokens < 1 ||
        num_pages < 0 || num_pages > kPagesPool)
        return false;
    return requests == 0 || (lengths != nullptr && (table_pages == 0 || table != nullptr));
}

}  // namespace rra

extern "C" {

rra_status_t rra_pages_fork(const rra_pages_fork_args_t* args, rra_stream_t stream) {
    if (args == nullptr) return RRA_ERR_INVALID_ARG;
    const rra_pages_fork_args_t& a = *args;
    if (!rra::pages_ok(a.requests, a.table_pages, a.table_stride, a.page_tokens, a.num_pages, a.block_table, a.seq_len) ||
        a.reserved != 0 || a.forks < 0 || a.forks > RRA_SERVE_MAX_REQUESTS || a.free_count == nullptr || a.free_left == nullptr ||
        a.pages_short == nullptr || (a.requests > 0 && a.kv_len == nullptr) ||
        (a.num_pages > 0 && (a.free_pages == nullptr || a.shared == nullptr || a.shared_out == nullptr)) ||
        (a.forks > 0 && (a.source == nullptr || a.target == nullptr || a.copy_from == nullptr || a.copy_to == nullptr)))
        return RRA_ERR_INVALID_ARG;
    rra::ForkParams p;
    p.a = a;
    p.by_page = rra::Divisor(a.page_tokens);
    const void* k = (const void*)rra::pages_fork_kernel;
    if (rra::configure_cluster_kernel(k, RRA_SERVE_MAX_REQUESTS * 4) != cudaSuccess) {
        cudaGetLastError();
        return RRA_ERR_CUDA;
    }
    const int64_t items = std::max<int64_t>((int64_t)a.forks * 64, a.shared == a.shared_out ? 0 : a.num_pages / 4);
    const int ctas = rra::pages_ctas(items);
    void* kargs[] = {(void*)&p};
    return rra::serve_launch(k, dim3((unsigned)ctas), rra::pages_threads(items), (size_t)a.forks * 4, ctas, stream, kargs);
}

rra_status_t rra_pages_release(const rra_pages_release_args_t* args, rra_stream_t stream) {
    if (args == nullptr) return RRA_ERR_INVALID_ARG;
    const rra_pages_release_args_t& a = *args;
    if (!rra::pages_ok(a.requests, a.table_pages, a.table_stride, a.page_tokens, a.num_pages, a.block_table, a.seq_len) ||
        a.free_count == nullptr || a.free_left == nullptr || (a.requests > 0 && (a.kv_len == nullptr || a.new_len == nullptr)) ||
        (a.num_pages > 0 && (a.free_pages == nullptr || a.shared == nullptr || a.shared_out == nullptr)))
        return RRA_ERR_INVALID_ARG;
    rra::ReleaseParams p;
    p.a = a;
    p.by_page = rra::Divisor(a.page_tokens);
    const void* k = (const void*)rra::pages_release_kernel;
    if (rra::configure_cluster_kernel(k, (int)rra::pages_bits(rra::kPagesPool, rra::kPagesMaxCluster)) != cudaSuccess) {
        cudaGetLastError();
        return RRA_ERR_CUDA;
    }
    const int64_t items = std::max<int64_t>((int64_t)a.requests * 32, a.num_pages / 4);
    const int ctas = rra::pages_ctas(items);
    void* kargs[] = {(void*)&p};
    return rra::serve_launch(k, dim3((unsigned)ctas), rra::pages_threads(items), rra::pages_bits(a.num_pages, ctas), ctas, stream, kargs);
}

rra_status_t rra_pages_compact(const rra_pages_compact_args_t* args, rra_stream_t stream) {
    if (args == nullptr) return RRA_ERR_INVALID_ARG;
    const rra_pages_compact_args_t& a = *args;
    if (!rra::pages_ok(a.requests, a.table_pages, a.table_stride, a.page_tokens, a.num_pages, a.block_table, a.seq_len) ||
        !rra::pages_ok(a.requests, a.table_pages, a.table_out_stride, a.page_tokens, a.num_pages, a.table_out, a.seq_len) ||
        (a.table_out == a.block_table && a.table_out_stride != a.table_stride) || a.reserved != 0 || a.max_moves < 0 ||
        a.free_count == nullptr || a.free_left == nullptr || a.move_count == nullptr ||
        (a.max_moves > 0 && (a.move_from == nullptr || a.move_to == nullptr)) ||
        (a.num_pages > 0 && (a.free_pages == nullptr || a.free_out == nullptr || a.shared == nullptr || a.shared_out == nullptr ||
                             a.moved == nullptr)))
        return RRA_ERR_INVALID_ARG;
    rra::CompactParams p;
    p.a = a;
    p.by_page = rra::Divisor(a.page_tokens);
    const void* k = (const void*)rra::pages_compact_kernel;
    if (rra::configure_cluster_kernel(k, (int)rra::pages_bits(rra::kPagesPool, rra::kPagesMaxCluster)) != cudaSuccess) {
        cudaGetLastError();
        return RRA_ERR_CUDA;
    }
    const int64_t items = std::max<int64_t>((int64_t)a.requests * 64, a.num_pages / 4);
    const int ctas = rra::pages_ctas(items);
    void* kargs[] = {(void*)&p};
    return rra::serve_launch(k, dim3((unsigned)ctas), rra::pages_threads(items), rra::pages_bits(a.num_pages, ctas), ctas, stream, kargs);
}

rra_status_t rra_pages_copy(const rra_pages_copy_args_t* args, rra_stream_t stream) {
    if (args == nullptr) return RRA_ERR_INVALID_ARG;
    const rra_pages_copy_args_t& a = *args;
    if (a.count < 0 || a.from_num < 0 || a.to_num < 0 || a.page_bytes < 16 || a.page_bytes % 16 != 0 || a.page_bytes > (int64_t)1 << 40 ||
        a.reserved != 0 || !rra::aligned16(a.from_pages) || !rra::aligned16(a.to_pages))
        return RRA_ERR_INVALID_ARG;
    if (a.count == 0 || a.from_num == 0 || a.to_num == 0) return RRA_OK;
    if (a.from_pages == nullptr || a.to_pages == nullptr || a.from == nullptr || a.to == nullptr) return RRA_ERR_INVALID_ARG;
    rra::CopyParams p;
    p.a = a;
    p.page = a.page_bytes / 16;
    constexpr int kMost = rra::kCopyThreads * rra::kCopyAhead;
    const int64_t pieces = (p.page + kMost - 1) / kMost;
    if (pieces > INT32_MAX / 2 / a.count) return RRA_ERR_INVALID_ARG;  // pieces are counted in 32 bits
    p.by_pieces = rra::Divisor((int32_t)pieces);
    p.total = (int32_t)(pieces * a.count);
    p.vectors = (int32_t)((p.page + pieces - 1) / pieces);
    void* kargs[] = {(void*)&p};
    return rra::serve_launch((const void*)rra::pages_copy_kernel, dim3((unsigned)std::min<int64_t>(p.total, rra::kCopyCtas)), rra::kCopyThreads, 0, 1, stream, kargs);
}

}  // extern "C"
