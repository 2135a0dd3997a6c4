// serve_kv8.cu -- the writes and reads of the 8-bit cache (rra_serve.h).
//
// Write.  A block of 16 tokens and a head shares an exponent, so its tokens have
// to be looked at together: a warp takes one run of neighbouring tokens of one
// block, one head, K or V.  A CTA finds the runs that begin among its tokens (a
// prompt: one in 16; a decode step: each), then its warps share runs x heads x 2.
// A run's values stay in registers from their maximum to their codes.
//
// Read.  A thread takes 8 channels of a row of K, and of V (16: 11.0 us against 7.9 for 8754 tokens of 8 heads of 128).
//
// Four prompts, 8754 tokens of 8 heads of 128, bfloat16, 108 MB: 23.1 us for both, 4.7 TB/s, over three sets of buffers in
// turn; the write 13.9 and the read 11.1 us alone (7.8 where it finds the pages in L2).  The read waits for memory.  The write is
// bound by the chain list of tokens, slots, values, maximum, codes: a third of the warps wait for memory, a fifth for the list.
// One token for each request, 16: 4.5 us, launches and round trips.
// Of a step of 8192 slots 16 that are not padding: the write takes 25 us, two CTAs having them all (of 16 slots: 3.1).
#include <algorithm>

#include "serve_common.cuh"

namespace rra {

constexpr int kKv8Threads = 256;
constexpr int kKv8Span = 16;      // tokens of a CTA, at most

struct Kv8Params {
    rra_kv_tokens_args_t a;
    Divisor by_heads;
    Divisor by_page;   // blocks of a page
    int64_t room;      // slots of the cache
    int32_t span;      // tokens of a CTA
    int32_t heads;     // heads of a CTA
};

// The block of head h that slot is in.
template <typename B>
__device__ __forceinline__ char* kv8_block(const Kv8Params& p, int64_t slot, int h) {
    const rra_kv_cache_t& c = p.a.cache;
    const int at = (int)((uint64_t)slot / kKvBlockTokens), page = p.by_page(at);
    return (char*)c.pages + ((int64_t)(page * c.kv_heads + h) * p.by_page.d + (at - page * p.by_page.d)) * B::kBytes;
}

// Eight channels as they are in memory.
template <typename T>
struct Kv8Raw;
template <>
struct Kv8Raw<float> {
    float x[8];
    __device__ __forceinline__ void load(const float* from) {
        const float4 a = __ldcs((const float4*)from), b = __ldcs((const float4*)from + 1);
        x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
    }
    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = 0.f;
    }
    __device__ __forceinline__ float get(int i) const { return x[i]; }
    __device__ __forceinline__ float most() const {  // NaN counts for nothing
        float m = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) m = fmaxf(m, fabsf(x[i]));
        return m;
    }
    __device__ __forceinline__ bool odd() const {  // whether some may be NaN
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) sum += x[i] * 0.f;
        return sum != 0.f;  // NaN or infinity: 0 times it is NaN
    }
};
template <>
struct Kv8Raw<__nv_bfloat16> {
    uint32_t w[4];
    __device__ __forceinline__ void load(const __nv_bfloat16* from) {
        const uint4 v = __ldcs((const uint4*)from);
        w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
    }
    __device__ __forceinline__ void clear() { w[0] = w[1] = w[2] = w[3] = 0u; }
    __device__ __forceinline__ float get(int i) const { return __uint_as_float(i & 1 ? w[i >> 1] & 0xffff0000u : w[i >> 1] << 16); }
    __device__ __forceinline__ float most() const {
        const __nv_bfloat162* const h = (const __nv_bfloat162*)w;
        const __nv_bfloat162 m = __hmax2(__hmax2(__habs2(h[0]), __habs2(h[1])), __hmax2(__habs2(h[2]), __habs2(h[3])));
        return fmaxf(__low2float(m), __high2float(m));  // NaN counts for nothing
    }
    __device__ __forceinline__ bool odd() const {
        uint32_t any = 0u;
#pragma unroll
        for (int i = 0; i < 4; ++i) any |= ((w[i] & 0x7f807f80u) + 0x00800080u) & 0x80008000u;
        return any != 0u;
    }
};
__device__ __forceinline__ void kv8_store(float* to, const float* x) {
    __stcs((float4*)to, make_float4(x[0], x[1], x[2], x[3]));
    __stcs((float4*)to + 1, make_float4(x[4], x[5], x[6], x[7]));
}
__device__ __forceinline__ void kv8_store(__nv_bfloat16* to, const float* x) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
        w[i] = *(const uint32_t*)&h;
    }
    __stcs((uint4*)to, make_uint4(w[0], w[1], w[2], w[3]));
}

// The codes of four values, the first in the low byte: nearest e4m3, ties to even, saturating.
__device__ __forceinline__ uint32_t to_e4m3x4(float a, float b, float c, float d) {
    uint32_t r;
    asm("{\n\t.reg .b16 x, y;\n\tcvt.rn.satfinite.e4m3x2.f32 x, %2, %1;\n\tcvt.rn.satfinite.e4m3x2.f32 y, %4, %3;\n\tmov.b32 %0, {x, y};\n\t}"
        : "=r"(r) : "f"(a), "f"(b), "f"(c), "f"(d));
    return r;
}

// The smallest e with most <= 448 * 2^e = 1.75 * 2^(8 + e), within the limits.
__device__ __forceinline__ int kv8_exponent_of(float most) {
    const uint32_t bits = __float_as_uint(most);
    const int e = (int)(bits >> 23) - 127 - 8 + ((bits & 0x7fffffu) > 0x600000u ? 1 : 0);
    return min(max(e, kKv8Low), kKv8High);  // most = 0 and its neighbours end up at the lower one
}

// The place of the nearest slot inside the cache from `from` on, forwards (1) or backwards (-1); -1: there is none.  The whole CTA:
// steps of fixed shape may be padding for the most part, which a warp would pass a round trip to memory for every 32.
template <int kWay>
__device__ __forceinline__ int64_t kv8_find(const Kv8Params& p, int64_t from, int* nearest) {
    constexpr int kLook = 8;  // of a thread at once
    for (; kWay > 0 ? from < p.a.tokens : from >= 0; from += kWay * kLook * kKv8Threads) {
        if (threadIdx.x == 0) *nearest = INT32_MAX;
        int64_t s[kLook];
#pragma unroll
        for (int i = 0; i < kLook; ++i) {
            const int64_t t = from + kWay * (i * kKv8Threads + (int)threadIdx.x);
            s[i] = t >= 0 && t < p.a.tokens ? p.a.slots[t] : -1;
        }
        int mine = INT32_MAX;
#pragma unroll
        for (int i = kLook - 1; i >= 0; --i) mine = (uint64_t)s[i] < (uint64_t)p.room ? i * kKv8Threads + (int)threadIdx.x : mine;
        __syncthreads();
        if (mine != INT32_MAX) atomicMin(nearest, mine);
        __syncthreads();
        const int n = *nearest;
        __syncthreads();
        if (n != INT32_MAX) return from + kWay * n;
    }
    return -1;
}

// The next tokens of a run from `at` on, after the n that picks has, up to 16, as token * 16 + row; skipped slots between them do
// not end it.  Where there are more (the same slots over and over), `at` becomes the next one's place; with kPause also where 32
// skipped slots come next, the place behind them.  A whole warp.
enum Kv8Left { kNothing, kMore, kPadding };
template <bool kPause>
__device__ __forceinline__ Kv8Left kv8_gather(const Kv8Params& p, int64_t& at, int& n, int32_t* picks, const int64_t* slots, int64_t t0) {
    const int lane = (int)threadIdx.x & 31;
    int64_t block = -1;
    Kv8Left left = kNothing;
    for (;; at += 32) {
        const int64_t t = at + lane, s = t - t0 < kKv8Span + kKvBlockTokens ? slots[t - t0] : t < p.a.tokens ? p.a.slots[t] : -1;
        if (block < 0) block = __shfl_sync(0xffffffffu, s, 0) >> 4;  // the first is inside the cache
        const bool valid = (uint64_t)s < (uint64_t)p.room, same = valid && s >> 4 == block;
        const uint32_t ends = __ballot_sync(0xffffffffu, (valid && !same) || t >= p.a.tokens);
        const uint32_t in = __ballot_sync(0xffffffffu, same) & ((ends & (0u - ends)) - 1u);
        const int place = n + __popc(in & ((1u << lane) - 1u));
        const bool mine = in >> lane & 1u;
        if (mine && place < kKvBlockTokens) picks[place] = (int32_t)t * kKvBlockTokens + ((int32_t)s & (kKvBlockTokens - 1));
        const uint32_t over = __ballot_sync(0xffffffffu, mine && place == kKvBlockTokens);
        n += __popc(in);
        if (over != 0u) {
            at += __ffs((int)over) - 1;
            left = kMore;
            break;
        }
        if (ends != 0u) break;
        if (kPause && in == 0u) {
            at += 32;
            left = kPadding;
            break;
        }
    }
    __syncwarp();
    n = min(n, kKvBlockTokens);
    return left;
}

// A run of a CTA: its slot, its first tokens, and where it goes on (-1: it does not).
struct Kv8Run {
    int64_t slot, more;
    int32_t length;
    uint32_t rows;  // which rows it writes
    int32_t picks[kKvBlockTokens];
};

// The codes that are there, in a unit 2^k as large.
__device__ __forceinline__ void kv8_round_again(char* codes, int vectors, int k) {
    const float down = two_to(-k);
    for (int i = (int)threadIdx.x & 31; i < vectors; i += 32) {
        uint4 c = *((uint4*)codes + i);
        uint32_t* const w = (uint32_t*)&c;
#pragma unroll
        for (int x = 0; x < 4; ++x) {
            uint32_t low, high;
            from_e4m3x4(w[x], low, high);
            const float2 y = __half22float2(*(const __half2*)&low), z = __half22float2(*(const __half2*)&high);
            w[x] = to_e4m3x4(y.x * down, y.y * down, z.x * down, z.y * down);
        }
        *((uint4*)codes + i) = c;
    }
    __syncwarp();
}

template <typename T, int D>
__global__ void __launch_bounds__(kKv8Threads, sizeof(T) == 2 ? 4 : 2) kv8_append_kernel(const __grid_constant__ Kv8Params p) {
    using B = Kv8Block<D>;
    constexpr int kLanes = D / 8, kRows = 32 / kLanes;  // lanes of a row, rows that a warp takes at once
    constexpr int kHeld = kKvBlockTokens / kRows;       // rows of a lane
    __shared__ int64_t slots[kKv8Span + kKvBlockTokens];
    __shared__ Kv8Run runs[kKv8Span];
    __shared__ int firsts[kKv8Span], count, nearest;
    __shared__ int64_t before, behind;  // where the whole CTA looks for the slot before its own, and for more of its last run; -1: nowhere
    __shared__ int32_t again[kKv8Threads / 32][kKvBlockTokens];  // tokens behind a run's first 16
    const rra_kv_tokens_args_t& a = p.a;
    const int tid = (int)threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int64_t t0 = (int64_t)blockIdx.x * p.span;
    const int h0 = (int)blockIdx.y * p.heads, heads = min(p.heads, a.cache.kv_heads - h0);
    pdl_release_early();
    pdl_wait();
    // ---- the runs that begin among this CTA's tokens ----
    auto begin = [&](int64_t earlier) {  // warp 0; earlier: the slot before them, not counting those that are skipped; -1: none
        const int64_t slot = slots[lane];
        const bool inside = (uint64_t)slot < (uint64_t)p.room;
        const uint32_t lower = __ballot_sync(0xffffffffu, inside) & ((1u << lane) - 1u);
        int64_t left = __shfl_sync(0xffffffffu, slot, 31 - __clz((int)(lower | 1u)));
        if (lower == 0u) left = earlier;
        const bool begins = lane < p.span && inside && (left < 0 || left >> 4 != slot >> 4);
        const uint32_t who = __ballot_sync(0xffffffffu, begins);
        if (begins) firsts[__popc(who & ((1u << lane) - 1u))] = lane;
        if (lane == 0) count = __popc(who);
    };
    if (warp == 0) {
        const int64_t slot = t0 + lane < a.tokens ? a.slots[t0 + lane] : -1;
        const int64_t s = t0 - 32 + lane >= 0 ? a.slots[t0 - 32 + lane] : -1;
        slots[lane] = slot;
        __syncwarp();
        const bool inside = (uint64_t)slot < (uint64_t)p.room;
        const uint32_t there = __ballot_sync(0xffffffffu, (uint64_t)s < (uint64_t)p.room);
        const bool open = __any_sync(0xffffffffu, inside) && there == 0u && t0 > 32;  // what comes before is further back
        if (!open) begin(there != 0u ? __shfl_sync(0xffffffffu, s, 31 - __clz((int)there)) : -1);
        if (lane == 0) before = open ? t0 - 33 : -1, behind = -1;
    }
    __syncthreads();
    if (before >= 0) {
        const int64_t at = kv8_find<-1>(p, before, &nearest);
        if (warp == 0) begin(at >= 0 ? a.slots[at] : -1);
        __syncthreads();
    }
    // Of run r, its tokens: those that it has, and those from `at` on.
    auto gather = [&](int r, int64_t at) {
        Kv8Run& run = runs[r];
        int n = run.length;
        const Kv8Left left = kv8_gather<true>(p, at, n, run.picks, slots, t0);
        const uint32_t row = lane < n ? 1u << (run.picks[lane] & (kKvBlockTokens - 1)) : 0u, rows = __reduce_or_sync(0xffffffffu, row);
        if (lane == 0) {
            run.more = left == kMore ? at : -1, run.length = n, run.rows = rows;
            if (r == count - 1) behind = left == kPadding ? at : -1;  // others have ended
        }
    };
    for (int r = warp; r < count; r += kKv8Threads / 32) {
        if (lane == 0) runs[r].slot = slots[firsts[r]], runs[r].length = 0;
        __syncwarp();
        gather(r, t0 + firsts[r]);
    }
    __syncthreads();
    while (behind >= 0) {
        const int64_t at = kv8_find<1>(p, behind, &nearest);
        __syncthreads();
        if (warp == 0) {
            if (at >= 0 && a.slots[at] >> 4 == runs[count - 1].slot >> 4) gather(count - 1, at);
            else if (lane == 0) behind = -1;
        }
        __syncthreads();
    }
    const int sub = lane / kLanes, m = lane % kLanes;  // this lane's row of those that the warp takes at once, and its eight channels
    const int items = count * heads * 2;
    for (int item = warp; item < items; item += kKv8Threads / 32) {
        const int v = item & 1, r = (item >> 1) / heads, h = h0 + (item >> 1) - r * heads;
        const Kv8Run& run = runs[r];
        char* const block = kv8_block<B>(p, run.slot, h);
        char* const codes = block + v * B::kV;
        const T* const from = (v ? (const T*)a.v + h * a.v_head_stride : (const T*)a.k + h * a.k_head_stride) + 8 * m;
        const int64_t stride = v ? a.v_token_stride : a.k_token_stride;
        Kv8Raw<T> x[kHeld];
        auto take = [&](const int32_t* picks, int n) {
#pragma unroll
            for (int i = 0; i < kHeld; ++i) {
                if (i * kRows + sub < n) x[i].load(from + (picks[i * kRows + sub] >> 4) * stride);
                else x[i].clear();
            }
        };
        bool odd = false;  // NaN or infinity: rare
        auto most_of = [&]() {
            odd = false;
#pragma unroll
            for (int i = 0; i < kHeld; ++i) odd |= x[i].odd();
            float most = 0.f;
            if (!odd) {
#pragma unroll
                for (int i = 0; i < kHeld; ++i) most = fmaxf(most, x[i].most());
            } else {
#pragma unroll
                for (int i = 0; i < kHeld; ++i)
#pragma unroll
                    for (int c = 0; c < 8; ++c) {
                        const float size = fabsf(x[i].get(c));
                        if (size < INFINITY) most = fmaxf(most, size);
                    }
            }
            return most;
        };
        take(run.picks, run.length);
        const int old = kv8_exponent(*(const uint32_t*)(block + B::kExponents), v);
        float most = most_of();
        bool anew = (run.rows & 1u) != 0u;
        if (run.more >= 0) {  // all others are looked at before any is written
            int64_t at = run.more;
            for (bool more = true; more;) {
                int n = 0;
                more = kv8_gather<false>(p, at, n, again[warp], slots, t0) == kMore;
                anew |= __any_sync(0xffffffffu, lane < n && (again[warp][lane & 15] & 15) == 0);
                take(again[warp], n);
                most = fmaxf(most, most_of());
                __syncwarp();
            }
            take(run.picks, run.length);
            most = fmaxf(most, most_of());
        }
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, o));
        int e = kv8_exponent_of(most);
        if (!anew) e = max(e, old);
        if (!anew && e > old) kv8_round_again(codes, D, e - old);
        const float by = two_to(-e);
        auto put = [&](const int32_t* picks, int n) {
#pragma unroll
            for (int i = 0; i < kHeld; ++i) {
                if (i * kRows + sub >= n) continue;
                float y[8];
#pragma unroll
                for (int c = 0; c < 8; ++c) y[c] = x[i].get(c) * by;
                if (odd)
#pragma unroll
                    for (int c = 0; c < 8; ++c) y[c] = y[c] == y[c] ? y[c] : 0.f;  // NaN is stored as 0
                *(uint2*)(codes + B::at(picks[i * kRows + sub] & (kKvBlockTokens - 1), m >> 1) + 8 * (m & 1)) =
                    make_uint2(to_e4m3x4(y[0], y[1], y[2], y[3]), to_e4m3x4(y[4], y[5], y[6], y[7]));
            }
        };
        put(run.picks, run.length);
        if (run.more >= 0) {
            int64_t at = run.more;
            for (bool more = true; more;) {
                int n = 0;
                more = kv8_gather<false>(p, at, n, again[warp], slots, t0) == kMore;
                take(again[warp], n);
                most_of();
                put(again[warp], n);
                __syncwarp();
            }
        }
        if (lane == 0) *(int8_t*)(block + B::kExponents + v) = (int8_t)e;
    }
}

template <typename T, int D>
__global__ void __launch_bounds__(kKv8Threads) kv8_read_kernel(const __grid_constant__ Kv8Params p) {
    using B = Kv8Block<D>;
    constexpr int kLanes = D / 8;
    const rra_kv_tokens_args_t& a = p.a;
    pdl_release_early();
    const int m = (int)threadIdx.x % kLanes, pair = (int)((blockIdx.x * (uint32_t)kKv8Threads + threadIdx.x) / kLanes);
    const int t = p.by_heads(pair), h = pair - t * p.by_heads.d;
    pdl_wait();
    if (t >= a.tokens) return;
    const int64_t slot = a.slots[t];
    float x[2][8];
#pragma unroll
    for (int v = 0; v < 2; ++v)
#pragma unroll
        for (int c = 0; c < 8; ++c) x[v][c] = 0.f;
    if ((uint64_t)slot < (uint64_t)p.room) {
        const char* const block = kv8_block<B>(p, slot, h);
        const int row = (int)slot & (kKvBlockTokens - 1);
        const uint32_t e = *(const uint32_t*)(block + B::kExponents);
        uint2 w[2];
#pragma unroll
        for (int v = 0; v < 2; ++v) w[v] = *(const uint2*)(block + v * B::kV + B::at(row, m >> 1) + 8 * (m & 1));
#pragma unroll
        for (int v = 0; v < 2; ++v) {
            const float by = two_to(kv8_exponent(e, v));
            uint32_t f[4];
            from_e4m3x4(w[v].x, f[0], f[1]);
            from_e4m3x4(w[v].y, f[2], f[3]);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 y = __half22float2(*(const __half2*)&f[i]);
                x[v][2 * i] = y.x * by, x[v][2 * i + 1] = y.y * by;
            }
        }
    }
    kv8_store((T*)a.k + t * a.k_token_stride + h * a.k_head_stride + 8 * m, x[0]);
    kv8_store((T*)a.v + t * a.v_token_stride + h * a.v_head_stride + 8 * m, x[1]);
}

static rra_status_t kv8_tokens(const rra_kv_tokens_args_t* a, rra_stream_t stream, bool append) {
    if (a == nullptr || !kv_cache_ok(a->cache) || a->tokens < 0 || a->reserved != 0) return RRA_ERR_INVALID_ARG;
    if (a->dtype != RRA_FP32 && a->dtype != RRA_BF16) return RRA_ERR_INVALID_ARG;
    const int elem = a->dtype == RRA_FP32 ? 4 : 2;
    const rra_kv_cache_t& c = a->cache;
    if (!strides_ok(a->k_token_stride, a->k_head_stride, c.kv_heads, c.head_dim, elem) ||
        !strides_ok(a->v_token_stride, a->v_head_stride, c.kv_heads, c.head_dim, elem) || !aligned16(a->k) || !aligned16(a->v))
        return RRA_ERR_INVALID_ARG;
    if (a->tokens == 0) return RRA_OK;
    if (a->k == nullptr || a->v == nullptr || a->slots == nullptr) return RRA_ERR_INVALID_ARG;
    if (a->tokens > INT32_MAX / 32 / c.kv_heads) return RRA_ERR_INVALID_ARG;  // threads are counted in 32 bits
    Kv8Params p;
    p.a = *a;
    p.by_heads = Divisor(c.kv_heads);
    p.by_page = Divisor(c.page_tokens / kKvBlockTokens);
    p.room = c.num_pages * c.page_tokens;
    const bool big = c.head_dim == 128;
    dim3 grid;
    const void* k;
    if (append) {
        // A CTA takes four heads of a token, of more tokens only where there are more CTAs than run at once: a decode step's
        // tokens are blocks of their own, which its warps take one after the other.  (8 heads of 128, single tokens of 1, 2, 4, 8
        // and 16 a CTA: 256 tokens 5.0, 5.5, 7.6, 12.7, 23.7 us; 1024 13.2, 12.2, 13.0, 15.1, 23.6; 4096 47, 42, 40, 40, 47.  A
        // prompt's: 256 4.3, 4.2, 4.0, 3.7, 3.8; 1024 6.7, 5.7, 5.2, 5.1, 3.9; 8192 29.4, 19.7, 14.9, 12.3, 10.3.)
        p.heads = std::min(4, c.kv_heads);
        const int64_t ctas = a->tokens * ((c.kv_heads + p.heads - 1) / p.heads);
        for (p.span = 1; p.span < kKv8Span && ctas > 4 * 152 * p.span;) p.span *= 2;
        grid = dim3((unsigned)((a->tokens + p.span - 1) / p.span), (unsigned)((c.kv_heads + p.heads - 1) / p.heads));
        k = elem == 4 ? (big ? (const void*)kv8_append_kernel<float, 128> : (const void*)kv8_append_kernel<float, 64>)
                      : (big ? (const void*)kv8_append_kernel<__nv_bfloat16, 128> : (const void*)kv8_append_kernel<__nv_bfloat16, 64>);
    } else {
        const int per_cta = kKv8Threads / (c.head_dim / 8);
        p.span = p.heads = 1;
        grid = dim3((unsigned)((a->tokens * c.kv_heads + per_cta - 1) / per_cta));
        k = elem == 4 ? (big ? (const void*)kv8_read_kernel<float, 128> : (const void*)kv8_read_kernel<float, 64>)
                      : (big ? (const void*)kv8_read_kernel<__nv_bfloat16, 128> : (const void*)kv8_read_kernel<__nv_bfloat16, 64>);
    }
    void* args[] = {(void*)&p};
    return serve_launch(k, grid, kKv8Threads, 0, 1, stream, args);
}

}  // namespace rra

extern "C" {

size_t rra_kv8_page_bytes(int page_tokens, int kv_heads, int head_dim) {
    if (rra_kv_page_bytes(page_tokens, kv_heads, head_dim) == 0) return 0;
    return (size_t)kv_heads * (size_t)(page_tokens / rra::kKvBlockTokens) * (32u * (size_t)head_dim + 16u);
}

rra_status_t rra_kv8_append(const rra_kv_tokens_args_t* args, rra_stream_t stream) { return rra::kv8_tokens(args, stream, true); }

rra_status_t rra_kv8_read(const rra_kv_tokens_args_t* args, rra_stream_t stream) { return rra::kv8_tokens(args, stream, false); }

}  // extern "C"
