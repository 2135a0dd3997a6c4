// serve_common.cuh -- what the operators of rra_serve.h share: the layout of
// the 4-bit cache, checks of arguments, launches.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "prims.cuh"
#include "rra_serve.h"

namespace rra {

constexpr int kKvBlockTokens = 16;   // tokens of one block of a page
constexpr int kKvGroup = 32;         // channels that share a scale

// Byte offsets inside one head's block of 16 tokens.
template <int D>
struct KvBlock {
    static constexpr int kRow = D / 2;                    // codes of one token
    static constexpr int kGroups = D / kKvGroup;
    static constexpr int kScaleRow = kGroups * 2;         // scales of one token
    static constexpr int kV = kKvBlockTokens * kRow;      // V codes
    static constexpr int kScaleK = 2 * kV;
    static constexpr int kScaleV = kScaleK + kKvBlockTokens * kScaleRow;
    static constexpr int kBytes = kScaleV + kKvBlockTokens * kScaleRow;  // 18 D
};
static_assert(KvBlock<64>::kBytes == 18 * 64 && KvBlock<128>::kBytes == 18 * 128, "18 bytes a channel");

// The same of the 8-bit cache.
template <int D>
struct Kv8Block {
    static constexpr int kV = kKvBlockTokens * D;        // V codes
    static constexpr int kExponents = 2 * kV;            // of K, of V: a signed byte each
    static constexpr int kBytes = kExponents + 16;       // 32 D + 16
    // Offset of 16-byte piece `piece` of row `row` in its codes.  Pieces of a 128-byte line change places so that neither the
    // lanes that read eight rows (K) nor those that read four rows two apart (V) meet in a bank.
    static __host__ __device__ constexpr int at(int row, int piece) {
        const int x = row * (D / 16) + piece;
        return ((x & ~7) | ((x ^ (D == 128 ? row : row & 6)) & 7)) * 16;
    }
};
static_assert(Kv8Block<64>::kBytes % 16 == 0 && Kv8Block<128>::kBytes == 4112, "blocks of whole bulk copies");
constexpr int kKv8Low = -32, kKv8High = 32;  // exponents

// 2^e, -126 <= e <= 127.
__device__ __forceinline__ float two_to(int e) { return __uint_as_float((uint32_t)(127 + e) << 23); }
// The exponents of K and of V from a block's last word but three.
__device__ __forceinline__ int kv8_exponent(uint32_t w, int v) {
    return min(max((int)(int8_t)(w >> (8 * v)), kKv8Low), kKv8High);  // clamped: memory that was never written may hold anything
}
// Two e4m3 codes, the lower byte in the lower half.
__device__ __forceinline__ uint32_t from_e4m3x2(uint32_t w) {
    uint32_t r;
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\t}" : "=r"(r) : "r"(w));
    return r;
}
// Four e4m3 codes as two pairs.
__device__ __forceinline__ void from_e4m3x4(uint32_t w, uint32_t& low, uint32_t& high) {
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
        : "=r"(low), "=r"(high) : "r"(w));
}

// The four pairs of values of a word of codes, byte i in out[i].
__device__ __forceinline__ void from_e2m1x8(uint32_t w, uint32_t* out) {
    asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %4;\n\tcvt.rn.f16x2.e2m1x2 %0, a;\n\t"
        "cvt.rn.f16x2.e2m1x2 %1, b;\n\tcvt.rn.f16x2.e2m1x2 %2, c;\n\tcvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
        : "=r"(out[0]), "=r"(out[1]), "=r"(out[2]), "=r"(out[3])
        : "r"(w));
}

// Blocks of all pages and heads are counted in 32 bits (2^31 of them would be terabytes).
inline bool kv_cache_ok(const rra_kv_cache_t& c) {
    return c.pages != nullptr && ((uintptr_t)c.pages & 15) == 0 && c.num_pages >= 0 && c.num_pages <= INT32_MAX &&
           c.reserved == 0 && rra_kv_page_bytes(c.page_tokens, c.kv_heads, c.head_dim) != 0 &&
           c.num_pages * (c.page_tokens / kKvBlockTokens) <= INT32_MAX / c.kv_heads;
}

// Division of 0 <= x < 2^31 by a divisor the host knows: x * ceil(2^(31 + s) / d) >> (31 + s) with 2^s >= d is exact,
// since the factor's excess is below d <= 2^s, so the product's is below x / 2^31 < 1 part in d.
struct Divisor {
    uint32_t factor, shift;
    int32_t d;
    Divisor() = default;
    explicit Divisor(int32_t by) : factor(0), shift(31), d(by) {
        while (shift < 62 && (int64_t)1 << (shift - 31) < by) ++shift;
        factor = (uint32_t)((((uint64_t)1 << shift) + (uint64_t)by - 1) / (uint64_t)by);
    }
    __device__ __forceinline__ int operator()(int x) const { return (int)(((uint64_t)(uint32_t)x * factor) >> shift); }
};

// Rows of `heads` heads: both strides hold whole 16-byte vectors, and one
// head's channels do not run into the next.
inline bool strides_ok(int64_t token, int64_t head, int64_t heads, int64_t head_dim, int64_t elem) {
    return token > 0 && head >= head_dim && token * elem % 16 == 0 && head * elem % 16 == 0 && heads >= 0;
}

inline bool aligned16(const void* p) { return ((uintptr_t)p & 15) == 0; }

// One launch: with programmatic stream serialisation (the kernel waits for its
// predecessor itself) and, if cluster > 1, in clusters of that many CTAs.
inline rra_status_t serve_launch(const void* kernel, dim3 grid, int threads, size_t smem, int cluster,
                                 rra_stream_t stream, void** args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = (cudaStream_t)stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.numAttrs = 1;
    if (cluster > 1) {
        attr[1].id = cudaLaunchAttributeClusterDimension;
        attr[1].val.clusterDim.x = (unsigned)cluster;
        attr[1].val.clusterDim.y = 1;
        attr[1].val.clusterDim.z = 1;
        cfg.numAttrs = 2;
    }
    cfg.attrs = attr;
    if (cudaLaunchKernelExC(&cfg, kernel, args) != cudaSuccess) {
        cudaGetLastError();
        return RRA_ERR_CUDA;
    }
    return RRA_OK;
}

}  // namespace rra
