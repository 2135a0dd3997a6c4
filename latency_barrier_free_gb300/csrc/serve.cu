// serve.cu -- page bookkeeping, head norms with position rotation, and the
// writes and reads of the 4-bit cache (rra_serve.h).
#include <algorithm>

#include "cluster_prims.cuh"
#include "kernel_attrs.h"
#include "serve_common.cuh"

namespace rra {

// =========================================================== slot map ====
// One cluster.  Every CTA scans all requests (a few kilobytes, from L2) into
// running sums in shared memory; then the cluster shares the pages to push,
// the pages to pop and the tokens to place, each found by binary search in the
// sums.  The cluster barrier between the pushes and the pops is the only
// synchronisation between CTAs, and also separates all reads of the lengths
// from the writes that may go to the same buffers.  It is all latency: lengths,
// then pages, then the stack, a round trip to L2 each (64 requests that decode:
// 2 KB in 4.4 us; 1000 requests with 65536 new tokens, one in 16 ending: 0.9 MB
// in 12.0 us, of which scan and counting take a third, the push and the barrier
// a quarter).
constexpr int kSlotThreads = 1024;
constexpr int kSlotMaxCluster = 16;
constexpr int kSlotAhead = 8;   // loads of a row in flight
constexpr int kSlotRun = 4;     // neighbouring tokens of a thread

// Index of the last entry of sums[0..n] (ascending, sums[0] = 0) that is <= x, below n.
__device__ __forceinline__ int owner_of(const int32_t* sums, int n, int x) {
    int low = 0, high = n;  // sums[low] <= x < sums[high]
    while (high - low > 1) {
        const int mid = (low + high) >> 1;
        if (sums[mid] <= x) low = mid;
        else high = mid;
    }
    return low;
}

// Exclusive sums of three values over the block; the totals in tot[3].
__device__ __forceinline__ void block_sums3(int v[3], int tot[3], int32_t (*part)[32]) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int inc[3];
#pragma unroll
    for (int k = 0; k < 3; ++k) {
        inc[k] = v[k];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int up = __shfl_up_sync(0xffffffffu, inc[k], o);
            if (lane >= o) inc[k] += up;
        }
        if (lane == 31) part[k][warp] = inc[k];
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < 3; ++k) {
        int w = lane < (int)(blockDim.x >> 5) ? part[k][lane] : 0;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int up = __shfl_up_sync(0xffffffffu, w, o);
            if (lane >= o) w += up;
        }
        tot[k] = __shfl_sync(0xffffffffu, w, 31);
        const int before = __shfl_sync(0xffffffffu, w, warp > 0 ? warp - 1 : 0);
        v[k] = inc[k] - v[k] + (warp > 0 ? before : 0);
    }
    __syncthreads();  // part is free again
}

// Lengths as used: none below 0, and no sum of the new ones past 32 bits.
constexpr int kSlotMost = (1 << 30) - 1;

struct SlotParams {
    rra_slot_map_args_t a;
    Divisor by_page;
    int32_t most_new;  // of one request
    bool wide;         // slots and positions take 16-byte stores
};

__device__ __forceinline__ int pages_for(const SlotParams& p, int tokens) {
    return tokens > 0 ? p.by_page(tokens - 1) + 1 : 0;
}

// Calls f(page, lane's rank in order) for a row's first `held` valid entries, 32 * kSlotAhead at a time; whole warps.
template <typename F>
__device__ __forceinline__ int valid_pages(const rra_slot_map_args_t& a, int b, int held, F&& f) {
    const int lane = threadIdx.x & 31;
    const int32_t* const row = a.block_table + b * a.table_stride;
    int count = 0;
    for (int i0 = 0; i0 < held; i0 += 32 * kSlotAhead) {
        int page[kSlotAhead];
#pragma unroll
        for (int k = 0; k < kSlotAhead; ++k) page[k] = i0 + 32 * k + lane < held ? row[i0 + 32 * k + lane] : -1;
#pragma unroll
        for (int k = 0; k < kSlotAhead; ++k) {
            const bool good = page[k] >= 0 && page[k] < a.num_pages;
            const uint32_t who = __ballot_sync(0xffffffffu, good);
            if (good) f(page[k], count + __popc(who & ((1u << lane) - 1u)));
            count += __popc(who);
        }
    }
    return count;
}

__global__ void __launch_bounds__(kSlotThreads, 1) slot_map_kernel(const __grid_constant__ SlotParams p) {
    extern __shared__ int32_t sums_mem[];
    __shared__ int32_t part[3][32];
    __shared__ int32_t over_total, endings;
    pdl_release_early();
    const rra_slot_map_args_t& a = p.a;
    const int n = a.requests;
    // before request b: pages pushed, pages popped, new tokens; and the tokens that it holds
    int32_t* const back = sums_mem;
    int32_t* const fresh = back + (n + 1);
    int32_t* const tokens = fresh + (n + 1);
    int32_t* const holds = tokens + (n + 1);
    uint16_t* const ending = (uint16_t*)(holds + (n + 1));  // the requests that end, in any order
    const int tid = (int)threadIdx.x, nt = (int)blockDim.x, lane = tid & 31;
    const int me = (int)blockIdx.x * nt + tid, all = (int)gridDim.x * nt;
    if (tid == 0) over_total = endings = 0;
    __syncthreads();
    pdl_wait();
    const int count = min(max(a.free_count[0], 0), a.num_pages);

    // Lengths, once; holds[b] is the complement for a request that ends.
    for (int b = tid; b < n; b += nt) {
        const int add = min(a.new_len[b], p.most_new), held = min(max(a.seq_len[b], 0), kSlotMost);
        holds[b] = add < 0 ? ~held : held;
        tokens[b] = max(add, 0);
        back[b] = 0;
        if (add < 0) ending[atomicAdd(&endings, 1)] = (uint16_t)b;
    }
    __syncthreads();
    // pages that come back: valid entries of the rows of requests that end, a warp each
    for (int e = tid >> 5; e < endings; e += nt >> 5) {
        const int b = ending[e];
        const int c = valid_pages(a, b, min(pages_for(p, ~holds[b]), a.table_pages), [](int, int) {});
        if (lane == 0) back[b] = c;
    }
    if (endings > 0) __syncthreads();

    // running sums over the requests
    int base[3] = {0, 0, 0};
    for (int b0 = 0; b0 < n; b0 += nt) {
        const int b = b0 + tid;
        int v[3] = {0, 0, 0}, tot[3];
        if (b < n) {
            const int held = holds[b], add = tokens[b];
            v[0] = back[b];
            if (held >= 0) {
                const int first = pages_for(p, held), last = add > 0 ? pages_for(p, held + add) : first;
                v[1] = max(0, min(last, a.table_pages) - first);
                v[2] = add;
                const int over = last - max(first, a.table_pages);
                if (over > 0) atomicAdd(&over_total, over);
            }
        }
        block_sums3(v, tot, part);
        if (b < n) {
            back[b] = base[0] + v[0];
            fresh[b] = base[1] + v[1];
            tokens[b] = base[2] + v[2];
        }
#pragma unroll
        for (int k = 0; k < 3; ++k) base[k] += tot[k];
    }
    if (tid == 0) {
        back[n] = base[0];
        fresh[n] = base[1];
        tokens[n] = base[2];
    }
    __syncthreads();

    // push: a warp of the cluster per request that ends (by number where there are several CTAs: their lists' orders differ)
    const bool one = gridDim.x == 1;
    for (int i = me >> 5; i < (one || endings == 0 ? endings : n); i += all >> 5) {
        const int b = one ? ending[i] : i;
        if (holds[b] >= 0) continue;
        const int at = count + back[b];
        valid_pages(a, b, min(pages_for(p, ~holds[b]), a.table_pages), [&](int page, int rank) {
            if (at + rank < a.num_pages) a.free_pages[at + rank] = page;
        });
    }
    const int top = min(count + base[0], a.num_pages);

    if (gridDim.x > 1) cluster_sync();
    else __syncthreads();
    for (int b = me; b <= n; b += all) {
        a.cu_new[b] = tokens[b];
        if (b < n) a.kv_len[b] = holds[b] < 0 ? 0 : holds[b] + tokens[b + 1] - tokens[b];
    }

    // pop: new entries of the tables
    for (int i = me; i < base[1]; i += all) {
        const int page = i < top ? a.free_pages[top - 1 - i] : -1;
        const int b = owner_of(fresh, n, i);
        a.block_table[b * a.table_stride + pages_for(p, holds[b]) + i - fresh[b]] = page;
    }
    // place: slots and positions of kSlotRun new tokens
    for (int64_t t0 = (int64_t)me * kSlotRun; t0 < a.tokens; t0 += (int64_t)all * kSlotRun) {
        int64_t slot[kSlotRun];
        int pos[kSlotRun], page[kSlotRun];
        int b = t0 < base[2] ? owner_of(tokens, n, (int)t0) : 0;
#pragma unroll
        for (int k = 0; k < kSlotRun; ++k) {
            const int64_t t = t0 + k;
            pos[k] = 0;
            page[k] = -1;
            if (t < base[2] && t < a.tokens) {
                while (tokens[b + 1] <= (int)t) ++b;
                const int held = holds[b];
                pos[k] = held + ((int)t - tokens[b]);
                const int at = p.by_page(pos[k]), first = pages_for(p, held);
                if (at < a.table_pages) {
                    const int i = fresh[b] + at - first;
                    if (at < first) page[k] = a.block_table[b * a.table_stride + at];
                    else if (i < top) page[k] = a.free_pages[top - 1 - i];
                }
            }
        }
#pragma unroll
        for (int k = 0; k < kSlotRun; ++k)
            slot[k] = page[k] >= 0 ? (int64_t)page[k] * a.page_tokens + (pos[k] - p.by_page(pos[k]) * a.page_tokens) : -1;
        if (p.wide && t0 + kSlotRun <= a.tokens) {
            *(longlong2*)(a.slots + t0) = make_longlong2(slot[0], slot[1]);
            *(longlong2*)(a.slots + t0 + 2) = make_longlong2(slot[2], slot[3]);
            *(int4*)(a.positions + t0) = make_int4(pos[0], pos[1], pos[2], pos[3]);
        } else {
#pragma unroll
            for (int k = 0; k < kSlotRun; ++k)
                if (t0 + k < a.tokens) {
                    a.slots[t0 + k] = slot[k];
                    a.positions[t0 + k] = pos[k];
                }
        }
    }
    if (me == 0) {
        a.free_left[0] = max(0, top - base[1]);
        a.pages_short[0] = max(0, base[1] - top) + over_total;
    }
}

// ============================================== head norms and rotation ====
// Eight channels a chunk.  A thread owns the two chunks that rotate with each
// other (channels j.. and j + rot/2.., or a chunk and its neighbour), so the
// rotation needs no exchange; head_dim / 16 threads, padded to a power of two,
// share a row and add its squares by shuffles.  A thread has several heads of
// one token in flight and keeps its cosines and sines for them.
template <typename T>
__device__ __forceinline__ void load8(const T* p, float* x);
template <>
__device__ __forceinline__ void load8<float>(const float* p, float* x) {
    const float4 a = *(const float4*)p, b = *(const float4*)(p + 4);
    x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
    x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
}
template <>
__device__ __forceinline__ void load8<__nv_bfloat16>(const __nv_bfloat16* p, float* x) {
    const uint4 v = *(const uint4*)p;
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}
// Streaming stores: at sizes that pass L2 a result is not read before it has left (8192 tokens rotated: 57 -> 50 us).
template <typename T>
__device__ __forceinline__ void store8(T* p, const float* x);
template <>
__device__ __forceinline__ void store8<float>(float* p, const float* x) {
    __stcs((float4*)p, make_float4(x[0], x[1], x[2], x[3]));
    __stcs((float4*)(p + 4), make_float4(x[4], x[5], x[6], x[7]));
}
template <>
__device__ __forceinline__ void store8<__nv_bfloat16>(__nv_bfloat16* p, const float* x) {
    uint4 v;
    uint32_t* w = (uint32_t*)&v;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
        w[i] = *(const uint32_t*)&h;
    }
    __stcs((uint4*)p, v);
}

template <typename T>
struct Raw8;  // eight channels as they are in memory
template <>
struct Raw8<float> {
    float4 a, b;
    __device__ __forceinline__ void get(const float* p) { a = __ldcs((const float4*)p), b = __ldcs((const float4*)p + 1); }
    __device__ __forceinline__ void to(float* x) const {
        x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
        x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
    }
};
template <>
struct Raw8<__nv_bfloat16> {
    uint4 v;
    __device__ __forceinline__ void get(const __nv_bfloat16* p) { v = __ldcs((const uint4*)p); }
    __device__ __forceinline__ void to(float* x) const {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[2 * i] = __uint_as_float(w[i] << 16);
            x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
};

// 128 bytes of a thread in flight (8192 tokens of 72 heads of 128, bfloat16: 4 heads in blocks of 256 took 66 us, 8 heads
// 57 us, and in blocks of 128, whose starts hide each other better, 56 us; with streaming stores 50 us, 6.1 TB/s).
constexpr int kRopeThreads = 128;
template <typename T>
constexpr int kRopeHeads = 16 / (int)sizeof(T);  // heads of a thread, where there are enough

struct RopeParams {
    rra_qk_norm_rope_args_t a;
    Divisor by_units;  // units of a token: kHeads heads of q, or of k
    int32_t q_units;
    int32_t lanes_log2;
    int32_t items;     // tokens * units
};

// With weights w, cosine c and sine s of the pair (x, y), and inv = 1 / sqrt(mean of squares + eps), the result is
// inv * (x (w_x c) - y (w_y s)) and inv * (y (w_y c) + x (w_x s)): the four products are the same for all of a thread's heads.
template <typename T, int kHeads, bool kInterleaved>
__global__ void __launch_bounds__(kRopeThreads, kHeads > 1 ? 4 : 8) qk_norm_rope_kernel(const __grid_constant__ RopeParams r) {
    const rra_qk_norm_rope_args_t& a = r.a;
    pdl_release_early();
    const int lanes = 1 << r.lanes_log2;
    const int pair = (int)threadIdx.x & (lanes - 1);       // this thread's pair of chunks
    const int64_t at = ((int64_t)blockIdx.x * kRopeThreads + threadIdx.x) >> r.lanes_log2;
    const int item = (int)(at < r.items ? at : r.items - 1);
    const int t = r.by_units(item);
    const int unit = item - t * r.by_units.d;
    const bool is_q = unit < r.q_units;
    const int h0 = (is_q ? unit : unit - r.q_units) * kHeads;
    const int pairs = a.head_dim / 16, turning = a.rot / 16;
    const bool mine = pair < pairs && at < r.items;
    const int live = mine ? min(kHeads, (is_q ? a.q_heads : a.k_heads) - h0) : 0;  // heads of this thread
    const bool turns = mine && pair < turning;
    int c0, c1;  // first channels of the two chunks
    if (!kInterleaved && pair < turning) {
        c0 = pair * 8;
        c1 = c0 + a.rot / 2;
    } else {
        c0 = pair * 16;
        c1 = c0 + 8;
    }
    const int64_t head_stride = is_q ? a.q_head_stride : a.k_head_stride;
    const T* x = (is_q ? (const T*)a.q + t * a.q_token_stride : (const T*)a.k + t * a.k_token_stride) + h0 * head_stride;
    const T* const w = (const T*)(is_q ? a.q_weight : a.k_weight);
    pdl_wait();
    const int64_t position = turns ? a.positions[t] : 0;
    Raw8<T> raw[kHeads][2];
#pragma unroll
    for (int e = 0; e < kHeads; ++e)
        if (e < live) {
            raw[e][0].get(x + c0);
            raw[e][1].get(x + c1);
            x += head_stride;
        }
    // channel i of a chunk pairs with channel i of the other, or with its neighbour in its own
    constexpr auto first = [](int i) { return kInterleaved ? 2 * i : i; };
    constexpr auto second = [](int i) { return kInterleaved ? 2 * i + 1 : i + 8; };
    float by[16], cross[16];  // what a channel is multiplied with, and what its partner is
#pragma unroll
    for (int i = 0; i < 16; ++i) by[i] = 1.f, cross[i] = 0.f;
    if (mine && w != nullptr) {
        load8(w + c0, by);
        load8(w + c1, by + 8);
    }
    if (turns) {
        float cs[8], sn[8];
        if (position >= 0 && position < a.max_position) {
            load8(a.cos + position * (a.rot / 2) + pair * 8, cs);
            load8(a.sin + position * (a.rot / 2) + pair * 8, sn);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) cs[i] = sn[i] = __int_as_float(0x7fffffff);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            cross[first(i)] = -by[second(i)] * sn[i];
            cross[second(i)] = by[first(i)] * sn[i];
            by[first(i)] *= cs[i];
            by[second(i)] *= cs[i];
        }
    }
    const float eps = (float)a.eps, each = 1.f / (float)a.head_dim;
    const int64_t out_stride = is_q ? a.q_out_head_stride : a.k_out_head_stride;
    T* y = (is_q ? (T*)a.q_out + t * a.q_out_token_stride : (T*)a.k_out + t * a.k_out_token_stride) + h0 * out_stride;
#pragma unroll
    for (int e = 0; e < kHeads; ++e) {
        float u[16];
        if (e < live) {
            raw[e][0].to(u);
            raw[e][1].to(u + 8);
        } else {
#pragma unroll
            for (int i = 0; i < 16; ++i) u[i] = 0.f;
        }
        float sq = 0.f;  // exchanged by every thread, whether its heads are normed or not
#pragma unroll
        for (int i = 0; i < 16; ++i) sq = fmaf(u[i], u[i], sq);
        for (int o = lanes >> 1; o > 0; o >>= 1) sq += __shfl_xor_sync(0xffffffffu, sq, o);
        const float inv = w != nullptr ? rsqrtf(fmaf(sq, each, eps)) : 1.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float p = u[first(i)], q = u[second(i)];
            float to_p = p * by[first(i)], to_q = q * by[second(i)];
            if (turns) {  // not with zeros: an infinity beside a channel that does not turn is none of its business
                to_p = fmaf(q, cross[first(i)], to_p);
                to_q = fmaf(p, cross[second(i)], to_q);
            }
            u[first(i)] = to_p * inv;
            u[second(i)] = to_q * inv;
        }
        if (e < live) {
            store8(y + c0, u);
            store8(y + c1, u + 8);
            y += out_stride;
        }
    }
}

template <typename T>
static const void* rope_kernel(bool many, bool interleaved) {
    if (many) return interleaved ? (const void*)qk_norm_rope_kernel<T, kRopeHeads<T>, true> : (const void*)qk_norm_rope_kernel<T, kRopeHeads<T>, false>;
    return interleaved ? (const void*)qk_norm_rope_kernel<T, 1, true> : (const void*)qk_norm_rope_kernel<T, 1, false>;
}

// ======================================= the 4-bit cache: write and read ====
// The K and V rows of a token and head are head_dim / 8 threads of eight
// neighbouring channels, so values move in 16-byte vectors and a group's
// maximum is taken over four threads.  In a row's codes those eight channels
// are two half words (four channels each) that belong to different words;
// thread 4 j + u (group j) swaps one of them with its neighbour in group j ^ 1,
// after which each holds a whole word and the row's codes leave as one
// coalesced run.  Bound by the values' traffic and, in the write, by nearly as
// much arithmetic; a thread has up to kKvPairs pairs of rows in flight.  16384
// tokens of 8 heads of 128, nothing of it in L2: bfloat16 written in 18.5 us, read
// in 17.7 us (4.6, 4.9 TB/s), binary32 in 30.0 and 30.9 us (5.1, 5.0 TB/s); the one
// after the other, bfloat16, with codes still in L2, 31.0 us.
constexpr int kKvThreads = 128;
// Where there are enough; one otherwise (16384 tokens of 8 heads of 128, written and read: 31.0 us, with one pair 36.3; 16 tokens:
// 3.9 us, with one pair 2.9).
constexpr int kKvPairs = 2;

struct KvTokensParams {
    rra_kv_tokens_args_t a;
    Divisor by_heads;
    Divisor by_page;   // blocks of a page
    int64_t room;      // slots of the cache
    int32_t pairs;     // tokens * kv_heads
    int32_t stride;    // pairs between those of a thread
};

// The codes of eight values over their scale, the first in the low nibble: nearest e2m1, ties to even, saturating.
__device__ __forceinline__ uint32_t to_e2m1x8(const float* y) {
    uint32_t r;
    asm("{\n\t.reg .b8 a, b, c, d;\n\tcvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\tcvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\tcvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\tmov.b32 %0, {a, b, c, d};\n\t}"
        : "=r"(r)
        : "f"(y[0]), "f"(y[1]), "f"(y[2]), "f"(y[3]), "f"(y[4]), "f"(y[5]), "f"(y[6]), "f"(y[7]));
    return r;
}
// (x, y) * by + 24 - 24 of two values in one instruction each, every step rounded to nearest.
__device__ __forceinline__ void on_grid(float& x, float& y, float by) {
    asm("{\n\t.reg .b64 v, b, c;\n\tmov.b64 v, {%0, %1};\n\tmov.b64 b, {%2, %2};\n\tmov.b64 c, {%3, %3};\n\t"
        "fma.rn.f32x2 v, v, b, c;\n\tmov.b64 c, {%4, %4};\n\tadd.rn.f32x2 v, v, c;\n\tmov.b64 {%0, %1}, v;\n\t}"
        : "+f"(x), "+f"(y) : "f"(by), "f"(24.f), "f"(-24.f));
}

// Eight channels of a row being written: the group's part of the maximum, and the codes.
template <typename T>
struct KvWrite;
template <>
struct KvWrite<float> {
    Raw8<float> raw;
    __device__ __forceinline__ void clean() {  // NaN is stored as 0
        float* const x = (float*)&raw;
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = x[i] == x[i] ? x[i] : 0.f;
    }
    __device__ __forceinline__ float most() const {
        float x[8], m = 0.f;
        raw.to(x);
#pragma unroll
        for (int i = 0; i < 8; ++i) m = fmaxf(m, fabsf(x[i]));
        return m;
    }
    __device__ __forceinline__ uint32_t codes(float d) const {
        float x[8];
        raw.to(x);
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = __fdiv_rn(x[i], d);
        return to_e2m1x8(x);
    }
};
// bfloat16 values (8 bits) over a scale of 11 bits are a midpoint of two codes (a multiple of 1/4 of at most 3 bits) or at
// least 2^-14 of it away.  x / d enters the rounding as x * (1 / d), within 2^-23 of it, put on a grid of 2^-19 by adding
// and taking off 24 (so that sums of what does not saturate lie in [16, 32)): what was a midpoint, 5 at most, is one
// again, and nothing else becomes one.  The
// rounded division took more instructions than all the rest (16384 tokens, 8 heads of 128: 40 us against 21 us; with two values an instruction 17.6).
template <>
struct KvWrite<__nv_bfloat16> {
    Raw8<__nv_bfloat16> raw;
    __device__ __forceinline__ void clean() {
        // a sum of the eight that is NaN shows that one is (or that infinities cancelled): rare, then look at each
        const __nv_bfloat162* w = (const __nv_bfloat162*)&raw;
        const __nv_bfloat162 sum = __hadd2(__hadd2(w[0], w[1]), __hadd2(w[2], w[3]));
        if (__low2float(sum) + __high2float(sum) == __low2float(sum) + __high2float(sum)) return;
        uint16_t* const x = (uint16_t*)&raw;
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if ((x[i] & 0x7fff) > 0x7f80) x[i] = 0;
    }
    __device__ __forceinline__ float most() const {
        const __nv_bfloat162* w = (const __nv_bfloat162*)&raw;
        const __nv_bfloat162 m = __hmax2(__hmax2(__habs2(w[0]), __habs2(w[1])), __hmax2(__habs2(w[2]), __habs2(w[3])));
        return fmaxf(__low2float(m), __high2float(m));
    }
    __device__ __forceinline__ uint32_t codes(float d) const {
        float x[8], by;
        raw.to(x);
        asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(by) : "f"(d));
#pragma unroll
        for (int i = 0; i < 8; i += 2) on_grid(x[i], x[i + 1], by);
        // a zero has its value's sign
        const uint32_t low = __byte_perm(raw.v.x, raw.v.y, 0x7351), high = __byte_perm(raw.v.z, raw.v.w, 0x7351);
        return to_e2m1x8(x) | (__byte_perm(low, high, 0x5410) >> 4 & 0x08080808u) | (__byte_perm(low, high, 0x7632) & 0x80808080u);
    }
};

// Pair i of a call: its token and head, and where its block and row are; block < 0 if the slot is outside.
struct KvPair {
    int32_t token, head, row;
    int64_t block;
};
__device__ __forceinline__ KvPair kv_pair(const KvTokensParams& p, int i) {
    KvPair r;
    const rra_kv_cache_t& c = p.a.cache;
    r.token = p.by_heads(i);
    r.head = i - r.token * p.by_heads.d;
    const int64_t slot = p.a.slots[r.token];  // not through the non-coherent path: written while this grid is resident already
    r.row = (int)slot & (kKvBlockTokens - 1);
    r.block = -1;
    if ((uint64_t)slot < (uint64_t)p.room) {
        const int at = (int)((uint64_t)slot / kKvBlockTokens), page = p.by_page(at);
        r.block = (page * c.kv_heads + r.head) * p.by_page.d + (at - page * p.by_page.d);
    }
    return r;
}

template <typename T, int D, int kPairs>
__global__ void __launch_bounds__(kKvThreads) kv_append_kernel(const __grid_constant__ KvTokensParams p) {
    using B = KvBlock<D>;
    constexpr int kLanes = D / 8;
    const rra_kv_tokens_args_t& a = p.a;
    pdl_release_early();
    const int m = (int)threadIdx.x % kLanes, j = m >> 2, u = m & 3;
    const int first = ((int)blockIdx.x * kKvThreads + (int)threadIdx.x) / kLanes;
    pdl_wait();
    KvPair pair[kPairs];
    KvWrite<T> in[kPairs][2];
#pragma unroll
    for (int k = 0; k < kPairs; ++k) {
        const int i = first + k * p.stride;
        pair[k].block = -1;
        if (first < p.stride && i < p.pairs) pair[k] = kv_pair(p, i);
        if (pair[k].block >= 0) {
            const KvPair& r = pair[k];
            in[k][0].raw.get((const T*)a.k + r.token * a.k_token_stride + r.head * a.k_head_stride + 8 * m);
            in[k][1].raw.get((const T*)a.v + r.token * a.v_token_stride + r.head * a.v_head_stride + 8 * m);
        } else {
            in[k][0] = in[k][1] = KvWrite<T>{};
        }
    }
    const bool odd = j & 1;
    const int word_at = ((2 * u + (odd ? 1 : 0)) * B::kGroups + (j & ~1)) * 2;
#pragma unroll
    for (int k = 0; k < kPairs; ++k) {
        char* const block = (char*)a.cache.pages + pair[k].block * B::kBytes;
#pragma unroll
        for (int v = 0; v < 2; ++v) {
            KvWrite<T>& x = in[k][v];
            x.clean();
            float most = x.most();
            most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, 1));
            most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, 2));
            const __half s = __float2half_rn(fminf(fmaxf(most * (1.f / 6.f), 6.103515625e-05f), 2048.f));
            const float d = __half2float(s);
            const uint32_t codes = x.codes(d);
            // even groups keep their first half and get their neighbour's, odd ones the second
            const uint32_t got = __shfl_xor_sync(0xffffffffu, odd ? codes : codes >> 16, 4);
            const uint32_t word = __byte_perm(codes, got, odd ? 0x3254 : 0x5410);
            if (pair[k].block >= 0) {
                *(uint32_t*)(block + v * B::kV + pair[k].row * B::kRow + word_at) = word;
                if (u == 0) *(__half*)(block + (v ? B::kScaleV : B::kScaleK) + pair[k].row * B::kScaleRow + 2 * j) = s;
            }
        }
    }
}

template <typename T, int D, int kPairs>
__global__ void __launch_bounds__(kKvThreads) kv_read_kernel(const __grid_constant__ KvTokensParams p) {
    using B = KvBlock<D>;
    constexpr int kLanes = D / 8;
    const rra_kv_tokens_args_t& a = p.a;
    pdl_release_early();
    const int m = (int)threadIdx.x % kLanes, j = m >> 2, u = m & 3;
    const int first = ((int)blockIdx.x * kKvThreads + (int)threadIdx.x) / kLanes;
    const bool odd = j & 1;
    const int word_at = ((2 * u + (odd ? 1 : 0)) * B::kGroups + (j & ~1)) * 2;
    pdl_wait();
    KvPair pair[kPairs];
    uint32_t word[kPairs][2];
    __half scale[kPairs][2];
#pragma unroll
    for (int k = 0; k < kPairs; ++k) {
        const int i = first + k * p.stride;
        pair[k].block = pair[k].token = -1;
        if (first < p.stride && i < p.pairs) pair[k] = kv_pair(p, i);
#pragma unroll
        for (int v = 0; v < 2; ++v) {
            word[k][v] = 0u;
            scale[k][v] = __ushort_as_half(0);
            if (pair[k].block >= 0) {
                const char* const block = (const char*)a.cache.pages + pair[k].block * B::kBytes;
                word[k][v] = *(const uint32_t*)(block + v * B::kV + pair[k].row * B::kRow + word_at);
                scale[k][v] = *(const __half*)(block + (v ? B::kScaleV : B::kScaleK) + pair[k].row * B::kScaleRow + 2 * j);
            }
        }
    }
#pragma unroll
    for (int k = 0; k < kPairs; ++k)
#pragma unroll
        for (int v = 0; v < 2; ++v) {
            const uint32_t mine = word[k][v];
            const uint32_t got = __shfl_xor_sync(0xffffffffu, odd ? mine & 0xffffu : mine >> 16, 4);
            uint32_t f[4];
            from_e2m1x8(odd ? got | (mine & 0xffff0000u) : (mine & 0xffffu) | got << 16, f);
            const float d = __half2float(scale[k][v]);
            float x[8];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 y = __half22float2(*(const __half2*)&f[i]);
                x[2 * i] = y.x * d;
                x[2 * i + 1] = y.y * d;
            }
            if (pair[k].token >= 0)
                store8(v ? (T*)a.v + pair[k].token * a.v_token_stride + pair[k].head * a.v_head_stride + 8 * m
                         : (T*)a.k + pair[k].token * a.k_token_stride + pair[k].head * a.k_head_stride + 8 * m, x);
        }
}

template <typename T, int D>
static const void* kv_tokens_kernel(bool append, bool many) {
    if (append) return many ? (const void*)kv_append_kernel<T, D, kKvPairs> : (const void*)kv_append_kernel<T, D, 1>;
    return many ? (const void*)kv_read_kernel<T, D, kKvPairs> : (const void*)kv_read_kernel<T, D, 1>;
}

static rra_status_t kv_tokens(const rra_kv_tokens_args_t* a, rra_stream_t stream, bool append) {
    if (a == nullptr || !kv_cache_ok(a->cache) || a->tokens < 0 || a->reserved != 0) return RRA_ERR_INVALID_ARG;
    if (a->dtype != RRA_FP32 && a->dtype != RRA_BF16) return RRA_ERR_INVALID_ARG;
    const int elem = a->dtype == RRA_FP32 ? 4 : 2;
    const rra_kv_cache_t& c = a->cache;
    if (!strides_ok(a->k_token_stride, a->k_head_stride, c.kv_heads, c.head_dim, elem) ||
        !strides_ok(a->v_token_stride, a->v_head_stride, c.kv_heads, c.head_dim, elem) || !aligned16(a->k) ||
        !aligned16(a->v))
        return RRA_ERR_INVALID_ARG;
    if (a->tokens == 0) return RRA_OK;
    if (a->k == nullptr || a->v == nullptr || a->slots == nullptr) return RRA_ERR_INVALID_ARG;
    if (a->tokens > INT32_MAX / 32 / c.kv_heads) return RRA_ERR_INVALID_ARG;  // threads are counted in 32 bits
    KvTokensParams p;
    p.a = *a;
    p.by_heads = Divisor(c.kv_heads);
    p.by_page = Divisor(c.page_tokens / kKvBlockTokens);
    p.room = c.num_pages * c.page_tokens;
    p.pairs = (int)(a->tokens * c.kv_heads);
    const int per_cta = kKvThreads / (c.head_dim / 8);
    const bool many = p.pairs >= 8192;
    p.stride = many ? (p.pairs + kKvPairs - 1) / kKvPairs : p.pairs;
    const int blocks = (p.stride + per_cta - 1) / per_cta;
    const void* k = elem == 4 ? (c.head_dim == 64 ? kv_tokens_kernel<float, 64>(append, many) : kv_tokens_kernel<float, 128>(append, many))
                              : (c.head_dim == 64 ? kv_tokens_kernel<__nv_bfloat16, 64>(append, many)
                                                  : kv_tokens_kernel<__nv_bfloat16, 128>(append, many));
    void* args[] = {(void*)&p};
    return serve_launch(k, dim3((unsigned)blocks), kKvThreads, 0, 1, stream, args);
}

}  // namespace rra

// ==================================================================== C ABI ==
extern "C" {

rra_status_t rra_slot_map(const rra_slot_map_args_t* args, rra_stream_t stream) {
    if (args == nullptr) return RRA_ERR_INVALID_ARG;
    const rra_slot_map_args_t& a = *args;
    if (a.requests < 0 || a.requests > RRA_SERVE_MAX_REQUESTS || a.tokens < 0 || a.tokens > INT32_MAX / 2 ||
        a.page_tokens < 1 || a.num_pages < 0 || a.table_pages < 0 || a.table_stride < a.table_pages)
        return RRA_ERR_INVALID_ARG;
    if (a.free_count == nullptr || a.free_left == nullptr || a.pages_short == nullptr || a.cu_new == nullptr)
        return RRA_ERR_INVALID_ARG;
    if (a.requests > 0 && (a.seq_len == nullptr || a.new_len == nullptr || a.kv_len == nullptr ||
                           (a.table_pages > 0 && a.block_table == nullptr)))
        return RRA_ERR_INVALID_ARG;
    if ((a.num_pages > 0 && a.free_pages == nullptr) || (a.tokens > 0 && (a.slots == nullptr || a.positions == nullptr)))
        return RRA_ERR_INVALID_ARG;
    const void* k = (const void*)rra::slot_map_kernel;
    const size_t smem = 18 * ((size_t)a.requests + 1);
    if (rra::configure_cluster_kernel(k, 18 * (RRA_SERVE_MAX_REQUESTS + 1)) != cudaSuccess) {
        cudaGetLastError();
        return RRA_ERR_CUDA;
    }
    rra::SlotParams p;
    p.a = a;
    p.by_page = rra::Divisor(a.page_tokens);
    p.most_new = rra::kSlotMost / (a.requests > 0 ? a.requests : 1);
    p.wide = rra::aligned16(a.slots) && rra::aligned16(a.positions);
    // as many CTAs as have two runs of tokens a thread (1000 requests, 65536 tokens: 43 us with one CTA, 23, 16 and 12 us with
    // 4, 8 and 16); fewer warps meet sooner (64 requests, 64 tokens: 4.4 us with 256 threads, 5.1 with 1024)
    const int64_t items = a.tokens / rra::kSlotRun + a.requests;
    int ctas = 1;
    while (ctas < rra::kSlotMaxCluster && (int64_t)ctas * rra::kSlotThreads * 2 < items) ctas *= 2;
    const int threads = items <= 512 ? 256 : rra::kSlotThreads;
    void* kargs[] = {(void*)&p};
    return rra::serve_launch(k, dim3((unsigned)ctas), threads, smem, ctas, stream, kargs);
}

rra_status_t rra_qk_norm_rope(const rra_qk_norm_rope_args_t* args, rra_stream_t stream) {
    if (args == nullptr) return RRA_ERR_INVALID_ARG;
    const rra_qk_norm_rope_args_t& a = *args;
    if (a.dtype != RRA_FP32 && a.dtype != RRA_BF16) return RRA_ERR_INVALID_ARG;
    const int elem = a.dtype == RRA_FP32 ? 4 : 2;
    if (a.tokens < 0 || a.q_heads < 0 || a.k_heads < 0 || a.head_dim < 16 || a.head_dim > 256 || a.head_dim % 16 != 0 ||
        a.rot < 0 || a.rot > a.head_dim || a.rot % 16 != 0 || !(a.eps >= 0.0) || a.max_position < 0)
        return RRA_ERR_INVALID_ARG;
    if (a.tokens == 0 || a.q_heads + (int64_t)a.k_heads == 0) return RRA_OK;
    if (a.q_heads > 0 &&
        (a.q == nullptr || a.q_out == nullptr || !rra::aligned16(a.q) || !rra::aligned16(a.q_out) ||
         !rra::aligned16(a.q_weight) || !rra::strides_ok(a.q_token_stride, a.q_head_stride, a.q_heads, a.head_dim, elem) ||
         !rra::strides_ok(a.q_out_token_stride, a.q_out_head_stride, a.q_heads, a.head_dim, elem)))
        return RRA_ERR_INVALID_ARG;
    if (a.k_heads > 0 &&
        (a.k == nullptr || a.k_out == nullptr || !rra::aligned16(a.k) || !rra::aligned16(a.k_out) ||
         !rra::aligned16(a.k_weight) || !rra::strides_ok(a.k_token_stride, a.k_head_stride, a.k_heads, a.head_dim, elem) ||
         !rra::strides_ok(a.k_out_token_stride, a.k_out_head_stride, a.k_heads, a.head_dim, elem)))
        return RRA_ERR_INVALID_ARG;
    if (a.rot > 0 && (a.cos == nullptr || a.sin == nullptr || a.positions == nullptr || !rra::aligned16(a.cos) ||
                      !rra::aligned16(a.sin)))
        return RRA_ERR_INVALID_ARG;
    const int heads = a.q_heads + a.k_heads;
    if (a.q_heads > INT32_MAX / 4 || a.k_heads > INT32_MAX / 4 || a.tokens > INT32_MAX / 2 / heads) return RRA_ERR_INVALID_ARG;
    rra::RopeParams r;
    r.a = a;
    r.lanes_log2 = 0;
    while (1 << r.lanes_log2 < a.head_dim / 16) ++r.lanes_log2;
    // heads of a thread, where the SMs stay full (4 tokens of 72 heads: 1.5 us with one a thread, 3.1 with eight; 1021 of 12: the
    // same; 8192 of 72: 66 us and 50)
    const bool many = a.tokens * heads >= 16384;
    const int each = !many ? 1 : elem == 4 ? rra::kRopeHeads<float> : rra::kRopeHeads<__nv_bfloat16>;
    r.q_units = (a.q_heads + each - 1) / each;
    const int units = r.q_units + (a.k_heads + each - 1) / each;
    r.by_units = rra::Divisor(units);
    r.items = (int)(a.tokens * units);
    const int64_t blocks = (((int64_t)r.items << r.lanes_log2) + rra::kRopeThreads - 1) / rra::kRopeThreads;
    void* kargs[] = {(void*)&r};
    const void* k = elem == 4 ? rra::rope_kernel<float>(many, a.interleaved != 0) : rra::rope_kernel<__nv_bfloat16>(many, a.interleaved != 0);
    return rra::serve_launch(k, dim3((unsigned)blocks), rra::kRopeThreads, 0, 1, stream, kargs);
}

size_t rra_kv_page_bytes(int page_tokens, int kv_heads, int head_dim) {
    if (page_tokens < 16 || page_tokens > 4096 || page_tokens % 16 != 0 || kv_heads < 1 || kv_heads > 65536 ||
        (head_dim != 64 && head_dim != 128))
        return 0;
    return (size_t)kv_heads * (size_t)(page_tokens / 16) * 18u * (size_t)head_dim;
}

rra_status_t rra_kv_append(const rra_kv_tokens_args_t* args, rra_stream_t stream) {
    return rra::kv_tokens(args, stream, true);
}

rra_status_t rra_kv_read(const rra_kv_tokens_args_t* args, rra_stream_t stream) {
    return rra::kv_tokens(args, stream, false);
}

}  // extern "C"
