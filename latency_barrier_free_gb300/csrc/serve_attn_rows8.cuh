// serve_attn_rows8.cuh -- the same as serve_attn_rows.cuh for blocks of the
// 8-bit cache: eight rows (or 8 NT) of a request and KV head against 16 keys in
// shared memory, by one warp, on the m16n8k16 matrix instructions.
//
// A block has one exponent for its keys and one for its values: with codes K', V'
// (exact in binary16), x the exponents,
//     s = 2^xk (q . K'),   out = sum_blocks 2^xv (sum_keys p V').
// The first is a multiply of the finished score.  The second is not worth one for
// every output and block; instead 2^xv goes into the weight's exponent,
//     w = 2^((s - m) factor + xv - x),
// with m the maximum and x an exponent for the sums; the softmax's own sum gets
// 2^(x - xv) of a block's weights, in binary32.  For w to be in binary16's range x
// becomes xv where that is larger, and also where it is smaller by more than kKv8Apart:
// a block's exponent may be that of values which a row does not see, or of other
// channels, and must not cost what the row does see its bits.  The sums, in binary32,
// have room for all exponents at once.
//
// A lane takes D / 4 channels in a row of a key (operands of the first product:
// the sum's order is free) and D / 8 of four keys (the second's rows are channels,
// in any order), so both are 16-byte loads of plain rows.
#pragma once

#include "serve_attn_rows.cuh"

namespace rra {

// How far a block's exponent may be below that of the sums.  A weight, near 2^lift where it counts most, is rounded by 2^-25 at
// least: 2^(kKv8Apart - lift - 25) of what its key would count for alone, for prompts (lift 7) 2^-24.
constexpr int kKv8Apart = 8;

template <int D, int NT>
struct AttnRows8 : AttnRange<NT> {
    using B = Kv8Block<D>;
    using AttnRange<NT>::all_first;
    using AttnRange<NT>::all_end;
    using AttnRange<NT>::any_first;
    using AttnRange<NT>::any_end;
    static constexpr int kRows = 8 * NT, kSteps = D / 16, kWide = D / 32;
    static __device__ __forceinline__ int channel(int j, int g) { return D / 8 * g + 4 * j; }  // first of output(j)'s, lanes g, t
    uint4 raw[NT][kWide];           // queries as they are, channels D / 4 t ..: loaded some time before start()
    uint32_t q[NT][kSteps][2];      // as B operands, each row scaled to [1, 2) by a power of two
    float factor[NT][2];            // of columns 2 t, 2 t + 1: |softmax scale| times that power, above 0
    // Maximum m (-FLT_MAX: no key yet), exponent x of the sums; sum l, of 2^((s - m) factor + lift).
    float m[NT][2], l[NT][2];
    int x;                          // the same for all rows of the warp
    float acc[kSteps][NT][4];       // of 2^((s - m) factor + xv - x + lift) times codes; channels D / 8 g + 2 i, + 1

    __device__ __forceinline__ float top(int n, int k) const { return fmaxf(m[n][k] * factor[n][k], -FLT_MAX) - kAttnLift; }
    // Of column 2 t + k of n-tile n: channels channel(j, g) .. + 3 (not divided by the sum)
    __device__ __forceinline__ float4 output(int j, int n, int k) const {
        const float up = two_to(x);
        return make_float4(acc[2 * j][n][k] * up, acc[2 * j][n][k + 2] * up, acc[2 * j + 1][n][k] * up, acc[2 * j + 1][n][k + 2] * up);
    }

    // Rows c * kRows .. of the queries q0 .. q0 + qn and KV head h (none unless `live`).
    __device__ __forceinline__ void load(const AttnParams& p, int q0, int qn, int h, int c, bool live) {
        const int g = (threadIdx.x & 31) >> 2, t = threadIdx.x & 3;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const int row = c * kRows + 8 * n + g;
            const bool mine = live && row < qn * p.group;
            const int i = p.by_group(row);
            const __nv_bfloat16* from = (const __nv_bfloat16*)p.a.q + (q0 + i) * p.a.q_token_stride +
                                        (h * p.group + row - i * p.group) * p.a.q_head_stride + D / 4 * t;
#pragma unroll
            for (int j = 0; j < kWide; ++j) raw[n][j] = mine ? *((const uint4*)from + j) : make_uint4(0u, 0u, 0u, 0u);
        }
    }

    // After load(): the rows over kv keys, nothing seen yet.
    __device__ __forceinline__ void start(const AttnParams& p, int qn, int kv, int c) {
        const int t = threadIdx.x & 3, rows = qn * p.group;
        this->clear();
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const uint32_t* const w = (const uint32_t*)raw[n];
            float most = 0.f;
#pragma unroll
            for (int i = 0; i < 4 * kWide; ++i)
                most = fmaxf(most, fmaxf(fabsf(__uint_as_float(w[i] << 16)), fabsf(__uint_as_float(w[i] & 0xffff0000u))));
            most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, 1));
            most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, 2));
            float f, down;
            attn_row_scale(p, most, down, f);
#pragma unroll
            for (int i = 0; i < 4 * kWide; ++i)
                q[n][i >> 1][i & 1] = pack_half2(__uint_as_float(w[i] << 16) * down, __uint_as_float(w[i] & 0xffff0000u) * down);
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                factor[n][k] = __shfl_sync(0xffffffffu, f, (2 * t + k) * 4);
                this->add(p, n, k, c * kRows + 8 * n + 2 * t + k, rows, qn, kv);
                m[n][k] = -FLT_MAX, l[n][k] = 0.f;
            }
        }
        x = kKv8Low;
        this->meet();
#pragma unroll
        for (int i = 0; i < kSteps; ++i)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int k = 0; k < 4; ++k) acc[i][n][k] = 0.f;
    }

    // The keys key0 .. key0 + 15 of a block at shared address `base`.
    __device__ __forceinline__ void block(uint32_t base, int key0) {
        const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
        uint32_t exponents;
        lds_words<1>(base + B::kExponents, &exponents);
        float s[NT][4];
        {
            uint32_t k0[kSteps], k1[kSteps];  // keys g and g + 8
#pragma unroll
            for (int i = 0; i < D / 64; ++i) {
                const uint32_t at = base + B::at(g, D / 64 * t + i);
                lds_words<4>(at, k0 + 4 * i);
                lds_words<4>(at + 8 * D, k1 + 4 * i);
            }
            float c[2][NT][4];  // two sums, so that no product waits for the one before
#pragma unroll
            for (int i = 0; i < kSteps; ++i) {
                uint32_t a0, a1, a2, a3;
                from_e4m3x4(k0[i], a0, a2);
                from_e4m3x4(k1[i], a1, a3);
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    if (i < 2) mma_f16_first(c[i][n], a0, a1, a2, a3, q[n][i][0], q[n][i][1]);
                    else mma_f16(c[i & 1][n], a0, a1, a2, a3, q[n][i][0], q[n][i][1]);
                }
            }
            const float unit = two_to(kv8_exponent(exponents, 0));
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int k = 0; k < 4; ++k) s[n][k] = (c[0][n][k] + c[1][n][k]) * unit;
        }
        if (!(key0 >= all_first && key0 + kKvBlockTokens <= all_end)) {
            // Scores of keys that a row does not see, and the values of keys that no row sees: their memory may never
            // have been written, and 0 times NaN is none.  The store goes where a copy comes next, hence the fence.
#pragma unroll 1
            for (int r = 0; r < kKvBlockTokens; ++r)
                if ((key0 + r < any_first || key0 + r >= any_end) && lane < D / 4)
                    asm volatile("st.shared.u32 [%0], %1;" : : "r"(base + B::kV + B::at(r, lane >> 2) + 4 * (lane & 3)), "r"(0u) : "memory");
            fence_proxy_async_smem();
            __syncwarp();
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int k = 0; k < 4; ++k) s[n][k] = this->sees(n, k & 1, key0 + g + 8 * (k >> 1)) ? s[n][k] : -INFINITY;
        }
        // ---- does a weight get large, or are all far from it? ----
        const int xv = kv8_exponent(exponents, 1);
        bool moves = xv < x - kKv8Apart;
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int k = 0; k < 2; ++k)
                moves |= fmaf(fmaxf(s[n][k], s[n][k + 2]) - m[n][k], factor[n][k], (float)(xv - x)) > kAttnSlack;
        if (__any_sync(0xffffffffu, moves)) {
            const int to = xv > x || xv < x - kKv8Apart ? xv : x;
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    float now = fmaxf(s[n][k], s[n][k + 2]);
                    now = fmaxf(now, __shfl_xor_sync(0xffffffffu, now, 4));
                    now = fmaxf(now, __shfl_xor_sync(0xffffffffu, now, 8));
                    now = fmaxf(now, __shfl_xor_sync(0xffffffffu, now, 16));
                    now = fmaxf(now, m[n][k]);
                    const float up = (m[n][k] - now) * factor[n][k], by = exp2_fast(up + (float)(x - to));
                    l[n][k] *= exp2_fast(up);
                    m[n][k] = now;
#pragma unroll
                    for (int i = 0; i < kSteps; ++i) {
                        acc[i][n][k] *= by;
                        acc[i][n][k + 2] *= by;
                    }
                }
            x = to;
        }
        // ---- weights, and their products with the values ----
        uint32_t b0[NT], b1[NT];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            float e[4];
#pragma unroll
            for (int k = 0; k < 4; ++k)
                e[k] = exp2_fast(fmaf(s[n][k] - m[n][k & 1], factor[n][k & 1], kAttnLift + (float)(xv - x)));
#pragma unroll
            for (int k = 0; k < 2; ++k) l[n][k] = fmaf(e[k] + e[k + 2], two_to(x - xv), l[n][k]);
            b0[n] = transpose8(pack_half2(e[0], e[1]));  // row g, keys 2 t and 2 t + 1
            b1[n] = transpose8(pack_half2(e[2], e[3]));  // row g, keys 2 t + 8 and + 9
        }
        uint32_t v[4][kWide];  // keys 2 t, 2 t + 1, 2 t + 8, 2 t + 9
#pragma unroll
        for (int r = 0; r < 4; ++r)
            lds_words<kWide>(base + B::kV + B::at(2 * t + (r & 1), g * (D / 8) / 16) + g * (D / 8) % 16 + 8 * D * (r >> 1), v[r]);
#pragma unroll
        for (int j = 0; j < kWide; ++j)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                // codes of two keys side by side, of channels 2 h and 2 h + 1 of the word
                uint32_t a0, a1, a2, a3;
                from_e4m3x4(__byte_perm(v[0][j], v[1][j], h ? 0x7362 : 0x5140), a0, a1);
                from_e4m3x4(__byte_perm(v[2][j], v[3][j], h ? 0x7362 : 0x5140), a2, a3);
#pragma unroll
                for (int n = 0; n < NT; ++n) mma_f16(acc[2 * j + h][n], a0, a1, a2, a3, b0[n], b1[n]);
            }
    }
};

// The 8-bit cache, to the kernels that take either.
struct Cache8 {
    static constexpr int kBits = 8;
    template <int D>
    using Block = Kv8Block<D>;
    template <int D, int NT>
    using Rows = AttnRows8<D, NT>;
};

}  // namespace rra
