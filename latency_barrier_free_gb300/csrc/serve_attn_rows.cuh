// serve_attn_rows.cuh -- eight rows (or 8 NT) of a request and KV head against
// blocks of the 4-bit cache in shared memory, by one warp: scores, softmax,
// output, on the m16n8k16 matrix instructions.
//
// A row is one query of one head.  With K' the codes (exact in binary16) and a
// scale per 32 channels,
//     s = sum_g scale_g (q_g . K'_g),   out = sum_keys (p scale_g) V'_g,
// so the matrix instructions take codes as they are, and a scale costs one
// multiply-add per score and group (K) or one multiply per weight and group (V).
// Keys are the instruction's 16 rows, query rows its 8 columns; scores leave in
// the layout of an accumulator and enter the second product, whose columns are
// the query rows again, by one 8 x 8 transpose.
#pragma once

#include "serve_attn.cuh"

namespace rra {

constexpr float kAttnSlack = 4.f;  // log2 of how far weights may pass 1 before the maximum moves
// A weight, and a weight times a value's scale, is rounded to binary16, which has few bits left below 2^-14 and none below
// 2^-25.  So weights are taken 2^kAttnLift times as large, and scales are brought below 2 by a power of two, which the sums
// get back at the segment's end: 2^(4 + 10) * 2 fits.  Scales below 2 (values below 12) need no such power; one bit of a scale
// tells, and the rest is done where a maximum moves.  (60000 keys, values of 2e-4, queries of 4: the result's error 0.2 %, with
// no lift 1 %; 64 ragged requests take 2 % longer; over values of 12 and more 8 % longer again.)
constexpr float kAttnLift = 10.f;
constexpr uint32_t kAttnLarge = 0x40004000u;  // a bit of two scales each that are 2 or more

__device__ __forceinline__ void mma_f16(float* c, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// The same, from zero.
__device__ __forceinline__ void mma_f16_first(float* c, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                              uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
        : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}
__device__ __forceinline__ uint32_t mul_half2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("mul.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ void bulk_g2s(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
                 :
                 : "r"(dst), "l"(src), "r"(bytes), "r"(bar)
                 : "memory");
}
template <int N>
__device__ __forceinline__ void lds_words(uint32_t addr, uint32_t* w) {
    if constexpr (N == 4)
        asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "r"(addr));
    else if constexpr (N == 2)
        asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(addr));
    else
        asm volatile("ld.shared.u32 %0, [%1];" : "=r"(w[0]) : "r"(addr));
}

// The keys that the rows of 2 t, 2 t + 1 of every n-tile see, and those that all, or any, of the rows do.
template <int NT>
struct AttnRange {
    int first_key[NT][2], end_key[NT][2];
    int all_first, all_end, any_first, any_end;

    __device__ __forceinline__ void clear() { all_first = 0, all_end = INT32_MAX, any_first = INT32_MAX, any_end = 0; }
    // Row r of the request's `rows`, column 2 t + k of n-tile n.
    __device__ __forceinline__ void add(const AttnParams& p, int n, int k, int r, int rows, int qn, int kv) {
        int lo = 0, hi = 0;
        if (r < rows) {
            const int pos = kv - qn + p.by_group(r);
            hi = p.a.causal ? max(0, min(kv, pos + 1)) : kv;
            lo = p.window > 0 ? max(0, pos - p.window + 1) : 0;
            all_first = max(all_first, lo);
            all_end = min(all_end, hi);
            any_first = min(any_first, lo);
            any_end = max(any_end, hi);
        }
        first_key[n][k] = lo;
        end_key[n][k] = hi;
    }
    __device__ __forceinline__ void meet() {
#pragma unroll
        for (int o = 1; o <= 2; o <<= 1) {
            all_first = max(all_first, __shfl_xor_sync(0xffffffffu, all_first, o));
            all_end = min(all_end, __shfl_xor_sync(0xffffffffu, all_end, o));
            any_first = min(any_first, __shfl_xor_sync(0xffffffffu, any_first, o));
            any_end = max(any_end, __shfl_xor_sync(0xffffffffu, any_end, o));
        }
    }
    __device__ __forceinline__ bool sees(int n, int k, int key) const { return key >= first_key[n][k] && key < end_key[n][k]; }
};

template <int D, int NT>
struct AttnRows : AttnRange<NT> {
    using B = KvBlock<D>;
    using AttnRange<NT>::all_first;
    using AttnRange<NT>::all_end;
    using AttnRange<NT>::any_first;
    using AttnRange<NT>::any_end;
    static constexpr int J = B::kGroups, kRows = 8 * NT;
    static __device__ __forceinline__ int channel(int j, int g) { return 32 * j + 4 * g; }  // first of output(j)'s, lanes g, t
    uint2 raw[NT][J][2];            // queries as they are: loaded some time before start()
    uint32_t q[NT][J][2][2];        // as B operands, each row scaled to [1, 2) by a power of two
    float factor[NT][2];            // of columns 2 t, 2 t + 1: |softmax scale| times that power, above 0
    // Maximum m, the score that moves it, sum l; -FLT_MAX stands for no key yet.  m is one of the scores, and
    // weights are 2^((s - m) factor): with s factor - m factor, rounded apart, huge scores would overflow.
    float m[NT][2], limit[NT][2], l[NT][2];
    float acc[J][2][NT][4];
    float grown;                    // what scales are divided by, and so the sums too short by: 1, or 2^k with all scales below 2^(k + 1)
    uint32_t shrink;                // 1 / grown, twice
    uint32_t large;                 // bits of scales that need a look: kAttnLarge, or all once they are divided

    // Of column 2 t + k of n-tile n: the maximum that sum and channels go with, in units of log2.  Of a row that saw
    // nothing the factor must not make it infinite.
    __device__ __forceinline__ float top(int n, int k) const { return fmaxf(m[n][k] * factor[n][k], -FLT_MAX) - kAttnLift; }
    // Of column 2 t + k of n-tile n: channels 32 j + 4 g .. + 3 (not divided by the sum)
    __device__ __forceinline__ float4 output(int j, int n, int k) const {
        return make_float4(acc[j][0][n][k] * grown, acc[j][0][n][k + 2] * grown, acc[j][1][n][k] * grown, acc[j][1][n][k + 2] * grown);
    }

    // Rows c * kRows .. of the queries q0 .. q0 + qn and KV head h (none unless `live`).
    __device__ __forceinline__ void load(const AttnParams& p, int q0, int qn, int h, int c, bool live) {
        const int g = (threadIdx.x & 31) >> 2, t = threadIdx.x & 3;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const int row = c * kRows + 8 * n + g;
            const bool mine = live && row < qn * p.group;
            const int i = p.by_group(row);
            const __nv_bfloat16* x = (const __nv_bfloat16*)p.a.q + (q0 + i) * p.a.q_token_stride +
                                     (h * p.group + row - i * p.group) * p.a.q_head_stride;
#pragma unroll
            for (int j = 0; j < J; ++j)
#pragma unroll
                for (int s = 0; s < 2; ++s) raw[n][j][s] = mine ? *(const uint2*)(x + 32 * j + 4 * (2 * t + s)) : make_uint2(0u, 0u);
        }
    }

    // After load(): the rows over kv keys, nothing seen yet.
    __device__ __forceinline__ void start(const AttnParams& p, int qn, int kv, int c) {
        const int t = threadIdx.x & 3, rows = qn * p.group;
        this->clear();
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            float most = 0.f;
#pragma unroll
            for (int j = 0; j < J; ++j)
#pragma unroll
                for (int s = 0; s < 2; ++s) {
                    const uint32_t v[2] = {raw[n][j][s].x, raw[n][j][s].y};
#pragma unroll
                    for (int k = 0; k < 2; ++k)
                        most = fmaxf(most, fmaxf(fabsf(__uint_as_float(v[k] << 16)),
                                                 fabsf(__uint_as_float(v[k] & 0xffff0000u))));
                }
            most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, 1));
            most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, 2));
            float f, down;
            attn_row_scale(p, most, down, f);
#pragma unroll
            for (int j = 0; j < J; ++j)
#pragma unroll
                for (int s = 0; s < 2; ++s) {
                    const uint32_t v[2] = {raw[n][j][s].x, raw[n][j][s].y};
#pragma unroll
                    for (int k = 0; k < 2; ++k)
                        q[n][j][s][k] = pack_half2(__uint_as_float(v[k] << 16) * down,
                                                   __uint_as_float(v[k] & 0xffff0000u) * down);
                }
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                factor[n][k] = __shfl_sync(0xffffffffu, f, (2 * t + k) * 4);
                this->add(p, n, k, c * kRows + 8 * n + 2 * t + k, rows, qn, kv);
            }
        }
        this->meet();

#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int k = 0; k < 2; ++k) m[n][k] = limit[n][k] = -FLT_MAX, l[n][k] = 0.f;
        grown = 1.f;
        shrink = 0x3c003c00u;
        large = kAttnLarge;
#pragma unroll
        for (int j = 0; j < J; ++j)
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int k = 0; k < 4; ++k) acc[j][i][n][k] = 0.f;
    }

    // The keys key0 .. key0 + 15 of a block at shared address `base`.
    __device__ __forceinline__ void block(uint32_t base, int key0) {
        const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
        // keys of this lane's score rows: block row (g >> 1) + 4 (g & 1), and 8 above
        const int krow = (g >> 1) + 4 * (g & 1);
        float s[NT][4];
        uint32_t sv[4][J / 2];
        auto load_scales = [&]() {  // of values, well before they are looked at
#pragma unroll
            for (int r = 0; r < 4; ++r) lds_words<J / 2>(base + t * B::kScaleRow + B::kScaleV + 4 * r * B::kScaleRow, sv[r]);
        };
        load_scales();
        {
            uint32_t k0[J], k1[J], s0[J / 2], s1[J / 2];
            lds_words<J>(base + krow * B::kRow + t * 4 * J, k0);
            lds_words<J>(base + krow * B::kRow + t * 4 * J + 8 * B::kRow, k1);
            lds_words<J / 2>(base + krow * B::kScaleRow + B::kScaleK, s0);
            lds_words<J / 2>(base + krow * B::kScaleRow + B::kScaleK + 8 * B::kScaleRow, s1);
            // word s * J/2 + j/2 holds, for group j (bytes 2 (j & 1), + 1), channels 32 j + 4 (2 t + s) + 0..3
#pragma unroll
            for (int jj = 0; jj < J / 2; ++jj) {
                uint32_t x[2][4], y[2][4];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    from_e2m1x8(k0[h * (J / 2) + jj], x[h]);
                    from_e2m1x8(k1[h * (J / 2) + jj], y[h]);
                }
                const float2 f0 = __half22float2(*(const __half2*)&s0[jj]), f1 = __half22float2(*(const __half2*)&s1[jj]);
#pragma unroll
                for (int e = 0; e < 2; ++e)
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        float c[4];
                        const uint32_t(*qj)[2] = q[n][2 * jj + e];
                        mma_f16_first(c, x[0][2 * e], y[0][2 * e], x[0][2 * e + 1], y[0][2 * e + 1], qj[0][0], qj[0][1]);
                        mma_f16(c, x[1][2 * e], y[1][2 * e], x[1][2 * e + 1], y[1][2 * e + 1], qj[1][0], qj[1][1]);
                        const float u = e ? f0.y : f0.x, v = e ? f1.y : f1.x;
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const float w = k < 2 ? u : v;
                            s[n][k] = jj + e == 0 ? w * c[k] : fmaf(w, c[k], s[n][k]);
                        }
                    }
            }
        }
        if (!(key0 >= all_first && key0 + kKvBlockTokens <= all_end)) {
            // Scores of keys that a row does not see, and the scales of keys that no row sees: their
            // memory may never have been written.  The store goes where a copy comes next, hence the fence.
            if (lane < kKvBlockTokens && (key0 + lane < any_first || key0 + lane >= any_end))
#pragma unroll
                for (int jj = 0; jj < J / 2; ++jj)
                    asm volatile("st.shared.u32 [%0], %1;" : : "r"(base + B::kScaleV + lane * B::kScaleRow + 4 * jj), "r"(0u) : "memory");
            fence_proxy_async_smem();
            __syncwarp();
            load_scales();
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int key = key0 + krow + 8 * (k >> 1);
                    s[n][k] = this->sees(n, k & 1, key) ? s[n][k] : -INFINITY;
                }
        }
        // ---- does a score pass the running maximum, or a scale what the sums allow? ----
        uint32_t any = 0;
#pragma unroll
        for (int r = 0; r < 4; ++r)
#pragma unroll
            for (int jj = 0; jj < J / 2; ++jj) any |= sv[r][jj];
        bool moves = false;
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int k = 0; k < 2; ++k) moves |= fmaxf(s[n][k], s[n][k + 2]) > limit[n][k];
        if (__any_sync(0xffffffffu, moves || (any & large) != 0u)) {
            float down = 1.f;
            if (large != kAttnLarge) {
                any = 0;
#pragma unroll
                for (int r = 0; r < 4; ++r)
#pragma unroll
                    for (int jj = 0; jj < J / 2; ++jj) any |= sv[r][jj] = mul_half2(sv[r][jj], shrink);
            }
            if (__any_sync(0xffffffffu, (any & kAttnLarge) != 0u)) {
                uint32_t most = 0;
#pragma unroll
                for (int r = 0; r < 4; ++r)
#pragma unroll
                    for (int jj = 0; jj < J / 2; ++jj) most = max(most, max(sv[r][jj] >> 16, sv[r][jj] & 0xffffu));
                // by the power of two at or below the largest scale, these and all that follow
                const float up = __half2float(__ushort_as_half((uint16_t)(__reduce_max_sync(0xffffffffu, most) & 0x7c00u)));
                down = __fdividef(1.f, up);
                const uint32_t by = pack_half2(down, down);
#pragma unroll
                for (int r = 0; r < 4; ++r)
#pragma unroll
                    for (int jj = 0; jj < J / 2; ++jj) sv[r][jj] = mul_half2(sv[r][jj], by);
                grown *= up;
                shrink = mul_half2(shrink, by);
                large = 0xffffffffu;
            }
            if (__any_sync(0xffffffffu, moves) || down != 1.f) {
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        float top = fmaxf(s[n][k], s[n][k + 2]);
                        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 4));
                        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 8));
                        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 16));
                        top = fmaxf(top, m[n][k]);
                        const float by = exp2_fast((m[n][k] - top) * factor[n][k]);
                        m[n][k] = top;
                        limit[n][k] = top + __fdividef(kAttnSlack, factor[n][k]);
                        l[n][k] *= by;
#pragma unroll
                        for (int j = 0; j < J; ++j)
#pragma unroll
                            for (int d = 0; d < 2; ++d) {
                                acc[j][d][n][k] *= by * down;
                                acc[j][d][n][k + 2] *= by * down;
                            }
                    }
            }
        }
        // ---- weights, and their products with the values ----
        uint32_t b0[NT], b1[NT];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            float e[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                e[k] = exp2_fast(fmaf(s[n][k] - m[n][k & 1], factor[n][k & 1], kAttnLift));
                l[n][k & 1] += e[k];
            }
            b0[n] = transpose8(pack_half2(e[0], e[1]));  // head g, keys t and t + 4
            b1[n] = transpose8(pack_half2(e[2], e[3]));  // head g, keys t + 8 and t + 12
        }
        uint32_t v[4][J / 2];
#pragma unroll
        for (int r = 0; r < 4; ++r) lds_words<J / 2>(base + t * B::kRow + g * 2 * J + B::kV + 4 * r * B::kRow, v[r]);
#pragma unroll
        for (int jj = 0; jj < J / 2; ++jj) {
            // nibbles of two keys side by side: even channels in x, odd ones in y
            uint32_t x[2][4], y[2][4];
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const uint32_t u = v[2 * r][jj], z = v[2 * r + 1][jj];
                from_e2m1x8((u & 0x0f0f0f0fu) | ((z << 4) & 0xf0f0f0f0u), x[r]);
                from_e2m1x8(((u >> 4) & 0x0f0f0f0fu) | (z & 0xf0f0f0f0u), y[r]);
            }
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const uint32_t sel = e ? 0x7632u : 0x5410u;
                const uint32_t w0s = __byte_perm(sv[0][jj], sv[1][jj], sel), w1s = __byte_perm(sv[2][jj], sv[3][jj], sel);
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    const uint32_t p0 = mul_half2(b0[n], w0s), p1 = mul_half2(b1[n], w1s);
#pragma unroll
                    for (int d = 0; d < 2; ++d)
                        mma_f16(acc[2 * jj + e][d][n], x[0][2 * e + d], y[0][2 * e + d], x[1][2 * e + d],
                                y[1][2 * e + d], p0, p1);
                }
            }
        }
    }
};

// The 4-bit cache, to the kernels that take either.
struct Cache4 {
    static constexpr int kBits = 4;
    template <int D>
    using Block = KvBlock<D>;
    template <int D, int NT>
    using Rows = AttnRows<D, NT>;
};

}  // namespace rra
