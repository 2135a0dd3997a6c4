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
// synchronisation, and also separates all reads of the lengths from the writes
// that may go to the same buffers.
constexpr int kSlotThreads = 1024;
constexpr int kSlotMaxCluster = 16;

struct SlotSums {  // running sums before request b, [requests + 1]
    int32_t* back;    // pages pushed
    int32_t* fresh;   // pages popped
    int32_t* tokens;  // new tokens
};

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
__device__ __forceinline__ int held_of(const rra_slot_map_args_t& a, int b) {
    return min(max(a.seq_len[b], 0), kSlotMost);
}
__device__ __forceinline__ int added_to(const rra_slot_map_args_t& a, int b) {
    return min(a.new_len[b], kSlotMost / a.requests);
}
__device__ __forceinline__ int pages_for(int tokens, int page_tokens) {
    return tokens > 0 ? (tokens - 1) / page_tokens + 1 : 0;
}

__global__ void __launch_bounds__(kSlotThreads) slot_map_kernel(const __grid_constant__ rra_slot_map_args_t a) {
    extern __shared__ int32_t sums_mem[];
    __shared__ int32_t part[3][32];
    __shared__ int32_t over_total;
    pdl_release_early();
    const int n = a.requests;
    const SlotSums s{sums_mem, sums_mem + (n + 1), sums_mem + 2 * (n + 1)};
    const int tid = (int)threadIdx.x, nt = (int)blockDim.x;
    const int lane = tid & 31;
    const int me = (int)blockIdx.x * nt + tid, all = (int)gridDim.x * nt;
    if (tid == 0) over_total = 0;
    pdl_wait();

    // pages that come back, for each request that ends: valid entries of its row
    for (int b = tid; b < n; b += nt) s.back[b] = 0;
    __syncthreads();
    for (int b0 = (tid >> 5) * 32; b0 < n; b0 += nt) {
        const int b = b0 + lane;
        const bool ends = b < n && a.new_len[b] < 0;
        uint32_t todo = __ballot_sync(0xffffffffu, ends);
        while (todo != 0u) {
            const int e = b0 + __ffs((int)todo) - 1;
            todo &= todo - 1;
            const int held = min(pages_for(held_of(a, e), a.page_tokens), a.table_pages);
            int count = 0;
            for (int i = lane; i - lane < held; i += 32) {
                const int page = i < held ? a.block_table[e * a.table_stride + i] : -1;
                count += __popc(__ballot_sync(0xffffffffu, page >= 0 && page < a.num_pages));
            }
            if (lane == 0) s.back[e] = count;
        }
    }
    __syncthreads();

    // running sums over the requests
    int base[3] = {0, 0, 0};
    for (int b0 = 0; b0 < n; b0 += nt) {
        const int b = b0 + tid;
        int v[3] = {0, 0, 0}, tot[3];
        if (b < n) {
            const int add = added_to(a, b);
            const int held = add < 0 ? 0 : held_of(a, b);
            const int first = pages_for(held, a.page_tokens);
            const int last = add > 0 ? pages_for(held + add, a.page_tokens) : first;
            v[0] = s.back[b];
            v[1] = max(0, min(last, a.table_pages) - first);
            v[2] = max(add, 0);
            const int over = last - max(first, a.table_pages);
            if (over > 0) atomicAdd(&over_total, over);
        }
        block_sums3(v, tot, part);
        if (b < n) {
            s.back[b] = base[0] + v[0];
            s.fresh[b] = base[1] + v[1];
            s.tokens[b] = base[2] + v[2];
        }
#pragma unroll
        for (int k = 0; k < 3; ++k) base[k] += tot[k];
    }
    if (tid == 0) {
        s.back[n] = base[0];
        s.fresh[n] = base[1];
        s.tokens[n] = base[2];
    }
    const int count = min(max(a.free_count[0], 0), a.num_pages);
    __syncthreads();

    // push: a warp per request that ends
    if (base[0] > 0) {
        for (int b = me >> 5; b < n; b += all >> 5) {
            if (s.back[b + 1] == s.back[b]) continue;
            const int held = min(pages_for(held_of(a, b), a.page_tokens), a.table_pages);
            int at = count + s.back[b];
            for (int i = lane; i - lane < held; i += 32) {
                const int page = i < held ? a.block_table[b * a.table_stride + i] : -1;
                const bool good = page >= 0 && page < a.num_pages;
                const uint32_t who = __ballot_sync(0xffffffffu, good);
                const int to = at + __popc(who & ((1u << lane) - 1u));
                if (good && to < a.num_pages) a.free_pages[to] = page;
                at += __popc(who);
            }
        }
    }
    const int top = min(count + base[0], a.num_pages);

    if (gridDim.x > 1) cluster_sync();
    else __syncthreads();

    // pop: new entries of the tables
    for (int i = me; i < base[1]; i += all) {
        const int b = owner_of(s.fresh, n, i);
        const int at = pages_for(held_of(a, b), a.page_tokens) + i - s.fresh[b];
        a.block_table[b * a.table_stride + at] = i < top ? a.free_pages[top - 1 - i] : -1;
    }
    // place: slots and positions of the new tokens
    for (int64_t t = me; t < a.tokens; t += all) {
        int64_t slot = -1;
        int pos = 0;
        if (t < base[2]) {
            const int b = owner_of(s.tokens, n, (int)t);
            const int held = held_of(a, b);
            pos = held + ((int)t - s.tokens[b]);
            const int at = pos / a.page_tokens, first = pages_for(held, a.page_tokens);
            if (at < a.table_pages) {
                int page;
                if (at < first) {
                    page = a.block_table[b * a.table_stride + at];
                } else {
                    const int i = s.fresh[b] + at - first;
                    page = i < top ? a.free_pages[top - 1 - i] : -1;
                }
                if (page >= 0) slot = (int64_t)page * a.page_tokens + pos % a.page_tokens;
            }
        }
        a.slots[t] = slot;
        a.positions[t] = pos;
    }
    for (int b = me; b <= n; b += all) a.cu_new[b] = s.tokens[b];
    if (me == 0) {
        a.free_left[0] = max(0, top - base[1]);
        a.pages_short[0] = max(0, base[1] - top) + over_total;
    }
    // kv_len last: it may be seq_len, which the other CTAs read above
    if (gridDim.x > 1) cluster_sync();
    else __syncthreads();
    for (int b = me; b < n; b += all) {
        const int add = added_to(a, b);
        a.kv_len[b] = add < 0 ? 0 : held_of(a, b) + add;
    }
}

// ============================================== head norms and rotation ====
// Eight channels a chunk.  A thread owns the two chunks that rotate with each
// other (channels j.. and j + rot/2.., or a chunk and its neighbour), so the
// rotation needs no exchange; head_dim / 16 threads, padded to a power of two,
// share a row and add its squares by shuffles.  A thread keeps its cosines and
// sines for kRopeHeads heads of one token.
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
template <typename T>
__device__ __forceinline__ void store8(T* p, const float* x);
template <>
__device__ __forceinline__ void store8<float>(float* p, const float* x) {
    *(float4*)p = make_float4(x[0], x[1], x[2], x[3]);
    *(float4*)(p + 4) = make_float4(x[4], x[5], x[6], x[7]);
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
    *(uint4*)p = v;
}

constexpr int kRopeThreads = 256;

template <typename T>
__global__ void __launch_bounds__(kRopeThreads) qk_norm_rope_kernel(const __grid_constant__ rra_qk_norm_rope_args_t a,
                                                                    int lanes, int heads_each, int units) {
    pdl_release_early();
    const int pair = (int)threadIdx.x % lanes;             // this thread's pair of chunks
    const int64_t item = ((int64_t)blockIdx.x * kRopeThreads + threadIdx.x) / lanes;
    const int64_t t = item / units;
    const int h0 = (int)(item % units) * heads_each;
    const int pairs = a.head_dim / 16, turning = a.rot / 16;
    const bool mine = pair < pairs && t < a.tokens;
    int c0, c1;  // first channels of the two chunks
    if (!a.interleaved && pair < turning) {
        c0 = pair * 8;
        c1 = c0 + a.rot / 2;
    } else {
        c0 = pair * 16;
        c1 = c0 + 8;
    }
    pdl_wait();
    float cs[8], sn[8];
    const bool turns = mine && pair < turning;
    if (turns) {
        const int64_t p = a.positions[t];
        if (p >= 0 && p < a.max_position) {
            load8(a.cos + p * (a.rot / 2) + pair * 8, cs);
            load8(a.sin + p * (a.rot / 2) + pair * 8, sn);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) cs[i] = sn[i] = __int_as_float(0x7fffffff);
        }
    }
    const int heads = a.q_heads + a.k_heads;
    const bool normed = a.q_weight != nullptr || a.k_weight != nullptr;
    for (int e = 0; e < heads_each; ++e) {  // the same count in every thread: they exchange sums
        const int h = min(h0 + e, heads - 1);  // past the end the last head again, not stored
        const bool live = mine && h0 + e < heads;
        const bool is_q = h < a.q_heads;
        const int hh = is_q ? h : h - a.q_heads;
        const T* x = is_q ? (const T*)a.q + t * a.q_token_stride + hh * a.q_head_stride
                          : (const T*)a.k + t * a.k_token_stride + hh * a.k_head_stride;
        T* y = is_q ? (T*)a.q_out + t * a.q_out_token_stride + hh * a.q_out_head_stride
                    : (T*)a.k_out + t * a.k_out_token_stride + hh * a.k_out_head_stride;
        const T* w = (const T*)(is_q ? a.q_weight : a.k_weight);
        float u[8], v[8];
        if (mine) {
            load8(x + c0, u);
            load8(x + c1, v);
        }
        if (normed) {
            float sq = 0.f;
            if (mine) {
#pragma unroll
                for (int i = 0; i < 8; ++i) sq = fmaf(u[i], u[i], fmaf(v[i], v[i], sq));
            }
            for (int o = lanes >> 1; o > 0; o >>= 1) sq += __shfl_xor_sync(0xffffffffu, sq, o);
            const float inv = rsqrtf(sq / (float)a.head_dim + (float)a.eps);
            if (mine && w != nullptr) {
                float wu[8], wv[8];
                load8(w + c0, wu);
                load8(w + c1, wv);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    u[i] = u[i] * inv * wu[i];
                    v[i] = v[i] * inv * wv[i];
                }
            }
        }
        if (turns) {
            if (!a.interleaved) {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float p = u[i], q = v[i];
                    u[i] = p * cs[i] - q * sn[i];
                    v[i] = q * cs[i] + p * sn[i];
                }
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float p = u[2 * i], q = u[2 * i + 1], r = v[2 * i], z = v[2 * i + 1];
                    u[2 * i] = p * cs[i] - q * sn[i];
                    u[2 * i + 1] = q * cs[i] + p * sn[i];
                    v[2 * i] = r * cs[4 + i] - z * sn[4 + i];
                    v[2 * i + 1] = z * cs[4 + i] + r * sn[4 + i];
                }
            }
        }
        if (live) {
            store8(y + c0, u);
            store8(y + c1, v);
        }
    }
}

// ================================================ the 4-bit cache: write ====
// A row (one token, head, K or V) is head_dim / 8 threads: thread m holds the
// channels of one 4-byte word of the row's codes, that is four channels of two
// neighbouring groups, so a row's codes leave as one coalesced run.  A group's
// maximum is taken over its eight threads.
constexpr int kKvThreads = 256;

template <typename T>
__device__ __forceinline__ void load4(const T* p, float* x);
template <>
__device__ __forceinline__ void load4<float>(const float* p, float* x) {
    const float4 v = *(const float4*)p;
    x[0] = v.x; x[1] = v.y; x[2] = v.z; x[3] = v.w;
}
template <>
__device__ __forceinline__ void load4<__nv_bfloat16>(const __nv_bfloat16* p, float* x) {
    const uint2 v = *(const uint2*)p;
    x[0] = __uint_as_float(v.x << 16);
    x[1] = __uint_as_float(v.x & 0xffff0000u);
    x[2] = __uint_as_float(v.y << 16);
    x[3] = __uint_as_float(v.y & 0xffff0000u);
}
__device__ __forceinline__ void store4(float* p, const float* x) { *(float4*)p = make_float4(x[0], x[1], x[2], x[3]); }
__device__ __forceinline__ void store4(__nv_bfloat16* p, const float* x) {
    const __nv_bfloat162 a = __floats2bfloat162_rn(x[0], x[1]), b = __floats2bfloat162_rn(x[2], x[3]);
    *(uint2*)p = make_uint2(*(const uint32_t*)&a, *(const uint32_t*)&b);
}

// Two values as e2m1, `lo` in the low nibble: nearest, ties to even, saturating.
__device__ __forceinline__ uint32_t to_e2m1x2(float lo, float hi) {
    uint32_t r;
    asm("{\n\t.reg .b8 b;\n\tcvt.rn.satfinite.e2m1x2.f32 b, %1, %2;\n\tcvt.u32.u8 %0, b;\n\t}" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
// Address of the head's block and token row of a slot; null if the slot is outside the cache.
template <int D>
__device__ __forceinline__ char* kv_block(const rra_kv_cache_t& c, int64_t slot, int head, int& row) {
    if (slot < 0 || slot >= c.num_pages * c.page_tokens) return nullptr;
    const int64_t page = slot / c.page_tokens;
    const int in = (int)(slot - page * c.page_tokens);
    row = in % kKvBlockTokens;
    const int blocks = c.page_tokens / kKvBlockTokens;
    return (char*)c.pages + ((page * c.kv_heads + head) * blocks + in / kKvBlockTokens) * KvBlock<D>::kBytes;
}

template <typename T, int D>
__global__ void __launch_bounds__(kKvThreads) kv_append_kernel(const __grid_constant__ rra_kv_tokens_args_t a) {
    using B = KvBlock<D>;
    constexpr int kLanes = D / 8, kHalf = B::kGroups / 2;
    pdl_release_early();
    const int m = (int)threadIdx.x % kLanes;
    const int c = m / kHalf, j = m % kHalf * 2;
    const int64_t row_id = ((int64_t)blockIdx.x * kKvThreads + threadIdx.x) / kLanes;
    const int64_t th = row_id >> 1;  // K and V of one token and head sit side by side
    const bool is_v = row_id & 1;
    const int64_t t = th / a.cache.kv_heads;
    const int h = (int)(th - t * a.cache.kv_heads);
    pdl_wait();
    int row = 0;
    char* const block = t < a.tokens ? kv_block<D>(a.cache, a.slots[t], h, row) : nullptr;
    float x[2][4] = {};
    if (block != nullptr) {
        const T* p = is_v ? (const T*)a.v + t * a.v_token_stride + h * a.v_head_stride
                          : (const T*)a.k + t * a.k_token_stride + h * a.k_head_stride;
        load4(p + kKvGroup * j + 4 * c, x[0]);
        load4(p + kKvGroup * (j + 1) + 4 * c, x[1]);
    }
    float s[2];
#pragma unroll
    for (int g = 0; g < 2; ++g) {
        float most = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[g][i] = x[g][i] == x[g][i] ? x[g][i] : 0.f;  // NaN is stored as 0
            most = fmaxf(most, fabsf(x[g][i]));
        }
#pragma unroll
        for (int o = kHalf; o < kLanes; o <<= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, o));
        s[g] = fminf(fmaxf(most * (1.f / 6.f), 6.103515625e-05f), 2048.f);
    }
    if (block == nullptr) return;
    const __half2 sh = __floats2half2_rn(s[0], s[1]);
    const float2 sf = __half22float2(sh);
    uint32_t word = 0;
#pragma unroll
    for (int g = 0; g < 2; ++g) {
        const float d = g ? sf.y : sf.x;
#pragma unroll
        for (int i = 0; i < 2; ++i)  // the division decides ties as written down, so it is the rounded one
            word |= to_e2m1x2(__fdiv_rn(x[g][2 * i], d), __fdiv_rn(x[g][2 * i + 1], d)) << (16 * g + 8 * i);
    }
    *(uint32_t*)(block + (is_v ? B::kV : 0) + row * B::kRow + 4 * m) = word;
    if (c == 0) *(__half2*)(block + (is_v ? B::kScaleV : B::kScaleK) + row * B::kScaleRow + 2 * j) = sh;
}

template <typename T, int D>
__global__ void __launch_bounds__(kKvThreads) kv_read_kernel(const __grid_constant__ rra_kv_tokens_args_t a) {
    using B = KvBlock<D>;
    constexpr int kLanes = D / 8, kHalf = B::kGroups / 2;
    pdl_release_early();
    const int m = (int)threadIdx.x % kLanes;
    const int c = m / kHalf, j = m % kHalf * 2;
    const int64_t row_id = ((int64_t)blockIdx.x * kKvThreads + threadIdx.x) / kLanes;
    const int64_t th = row_id >> 1;
    const bool is_v = row_id & 1;
    const int64_t t = th / a.cache.kv_heads;
    const int h = (int)(th - t * a.cache.kv_heads);
    pdl_wait();
    if (t >= a.tokens) return;
    int row = 0;
    const char* const block = kv_block<D>(a.cache, a.slots[t], h, row);
    float x[2][4] = {};
    if (block != nullptr) {
        const uint32_t word = *(const uint32_t*)(block + (is_v ? B::kV : 0) + row * B::kRow + 4 * m);
        const __half2 sh = *(const __half2*)(block + (is_v ? B::kScaleV : B::kScaleK) + row * B::kScaleRow + 2 * j);
        uint32_t v[4];
        from_e2m1x8(word, v);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = __half22float2(*(const __half2*)&v[i]);
            const float d = i < 2 ? __low2float(sh) : __high2float(sh);
            x[i >> 1][(i & 1) * 2] = f.x * d;
            x[i >> 1][(i & 1) * 2 + 1] = f.y * d;
        }
    }
    T* p = is_v ? (T*)a.v + t * a.v_token_stride + h * a.v_head_stride
                : (T*)a.k + t * a.k_token_stride + h * a.k_head_stride;
    store4(p + kKvGroup * j + 4 * c, x[0]);
    store4(p + kKvGroup * (j + 1) + 4 * c, x[1]);
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
    const int64_t threads = a->tokens * c.kv_heads * 2 * (c.head_dim / 8);
    const int64_t blocks = (threads + kKvThreads - 1) / kKvThreads;
    if (a->tokens > (INT64_MAX >> 24) || blocks > INT32_MAX) return RRA_ERR_INVALID_ARG;
    const void* k;
    if (append)
        k = elem == 4 ? (c.head_dim == 64 ? (const void*)kv_append_kernel<float, 64> : (const void*)kv_append_kernel<float, 128>)
                      : (c.head_dim == 64 ? (const void*)kv_append_kernel<__nv_bfloat16, 64>
                                          : (const void*)kv_append_kernel<__nv_bfloat16, 128>);
    else
        k = elem == 4 ? (c.head_dim == 64 ? (const void*)kv_read_kernel<float, 64> : (const void*)kv_read_kernel<float, 128>)
                      : (c.head_dim == 64 ? (const void*)kv_read_kernel<__nv_bfloat16, 64>
                                          : (const void*)kv_read_kernel<__nv_bfloat16, 128>);
    void* args[] = {(void*)a};
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
    const size_t smem = 3 * sizeof(int32_t) * ((size_t)a.requests + 1);
    if (rra::configure_cluster_kernel(k, 3 * (int)sizeof(int32_t) * (RRA_SERVE_MAX_REQUESTS + 1)) != cudaSuccess) {
        cudaGetLastError();
        return RRA_ERR_CUDA;
    }
    const int64_t items = a.tokens + a.requests;
    int ctas = 1;
    while (ctas < rra::kSlotMaxCluster && (int64_t)ctas * rra::kSlotThreads * 2 < items) ctas *= 2;
    void* kargs[] = {(void*)args};
    return rra::serve_launch(k, dim3((unsigned)ctas), rra::kSlotThreads, smem, ctas, stream, kargs);
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
    int lanes = 1;
    while (lanes < a.head_dim / 16) lanes *= 2;
    const int heads = a.q_heads + a.k_heads;
    const int heads_each = a.tokens * heads >= 16384 ? 4 : 1;
    int units = (heads + heads_each - 1) / heads_each;
    const int64_t threads = a.tokens * units * lanes;
    const int64_t blocks = (threads + rra::kRopeThreads - 1) / rra::kRopeThreads;
    if (blocks > INT32_MAX) return RRA_ERR_INVALID_ARG;
    int each = heads_each;
    void* kargs[] = {(void*)args, &lanes, &each, &units};
    const void* k = elem == 4 ? (const void*)rra::qk_norm_rope_kernel<float> : (const void*)rra::qk_norm_rope_kernel<__nv_bfloat16>;
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
