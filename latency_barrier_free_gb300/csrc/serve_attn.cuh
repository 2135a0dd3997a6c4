// serve_attn.cuh -- what the two attention kernels of rra_serve.h share: the
// workspace, a request's clamped lengths, queries as binary16, stored rows.
#pragma once

#include <float.h>
#include <math.h>

#include "cluster_prims.cuh"
#include "kernel_attrs.h"
#include "serve_common.cuh"

namespace rra {

constexpr int kAttnTile = 32;      // keys of one step of a warp
constexpr int kTeamWarps = 4;      // warps of a CTA of serve_attn_team.cu: one for each scheduler, a tile is a chain of latencies
constexpr int kAttnMaxCtas = 512;  // CTAs a workspace has room for
// A wait gives up after kAttnWaitNs, one try of it after about kAttnTryNs.  Both are 0 in a build that a test makes, so that
// waits do run out: what is not done when it is first looked at is given up.
#ifndef RRA_ATTN_WAIT_NS
#define RRA_ATTN_WAIT_NS 1000000000
#define RRA_ATTN_TRY_NS 20000
#endif
constexpr uint32_t kAttnWaitNs = RRA_ATTN_WAIT_NS, kAttnTryNs = RRA_ATTN_TRY_NS;
constexpr uint32_t kAttnQuietNs = 1000000000;  // the same for what must not be in flight any more
constexpr int kAttnMaxRows = 16;

// Start of the workspace: status word, then a counter for each CTA, then two
// partial results for each CTA: maximum and sum of every row, then the rows.
struct AttnWorkspace {
    uint32_t status;
    uint32_t pad[63];
    uint32_t arrived[kAttnMaxCtas];
    uint32_t pad_end[1024 - 64 - kAttnMaxCtas];
};
static_assert(sizeof(AttnWorkspace) == 4096, "the part of the workspace that starts as zero");
// One try of a wait on a barrier of this CTA: returns when its phase is done, or after about kAttnTryNs.  Acquire in the
// CTA only: at cluster scope every try also drops the L1 cache.
__device__ __forceinline__ bool attn_try(uint32_t bar, uint32_t parity) {
    uint32_t done;
#if RRA_ATTN_TRY_NS == 0
    asm volatile(
        "{\n\t.reg .pred p;\n\tmbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(done)
        : "r"(bar), "r"(parity)
        : "memory");
#else
    asm volatile(
        "{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\tselp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(done)
        : "r"(bar), "r"(parity), "r"(kAttnTryNs)
        : "memory");
#endif
    return done != 0;
}
// The rest of a wait whose first try did not see the phase done.  Gives up after kAttnWaitNs, or soon after another wait
// did, and says so in the status word.
__device__ __forceinline__ bool attn_wait_slow(uint32_t bar, uint32_t parity, AttnWorkspace* ws) {
    const uint64_t start = globaltimer_ns();
    while (!attn_try(bar, parity)) {
        const uint64_t waited = globaltimer_ns() - start;
        if (waited >= kAttnWaitNs) {
            atomicCAS(&ws->status, 0u, (uint32_t)RRA_ERR_TIMEOUT);
            return false;
        }
        if (waited > kStatusAfterNs && ld_relaxed_u32(&ws->status) != 0u) return false;
    }
    return true;
}

// Waits for what must not be in flight any more: copies and products that a wait gave up on.
__device__ __forceinline__ void attn_wait_quiet(uint32_t bar, uint32_t parity) {
    const uint64_t start = globaltimer_ns();
    while (!attn_try(bar, parity))
        if (globaltimer_ns() - start > kAttnQuietNs) break;
}

struct AttnParams {
    rra_kv_attention_args_t a;
    float scale_log2;
    int32_t group;   // query heads of a KV head
    Divisor by_group, by_page;
    int32_t room;    // keys that a row of the table has pages for
    int32_t window;  // a.window, at most 2^30
};

__device__ __forceinline__ float exp2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *(const uint32_t*)&h;
}
// Where row's channels go, and its sum's reciprocal; writes its lse (maximum top in units of log2).
__device__ __forceinline__ __nv_bfloat16* attn_row(const AttnParams& p, int q0, int h, int row, float top, float sum,
                                                   bool with_lse, float& inv) {
    const rra_kv_attention_args_t& a = p.a;
    const int i = p.by_group(row), head = h * p.group + row - i * p.group;
    const int64_t token = q0 + i;
    inv = sum == 0.f ? 0.f : 1.f / sum;  // no key seen: 0
    if (with_lse && a.lse != nullptr) a.lse[token * a.q_heads + head] = (top + log2f(sum)) * 0.693147180559945309f;
    return (__nv_bfloat16*)a.out + token * a.out_token_stride + head * a.out_head_stride;
}
__device__ __forceinline__ void attn_store(__nv_bfloat16* to, float4 o, float inv) {
    const __nv_bfloat162 x = __floats2bfloat162_rn(o.x * inv, o.y * inv), y = __floats2bfloat162_rn(o.z * inv, o.w * inv);
    *(uint2*)to = make_uint2(*(const uint32_t*)&x, *(const uint32_t*)&y);
}

// A request's queries and keys, clamped to the buffers.
struct AttnLengths {
    int32_t q0, qn, kv;  // first query token, how many, keys
};
__device__ __forceinline__ AttnLengths attn_lengths(const AttnParams& p, int b) {
    const int most_q = (int)p.a.tokens;
    AttnLengths r;
    r.q0 = min(max(p.a.cu_q[b], 0), most_q);
    r.qn = max(0, min(p.a.cu_q[b + 1], most_q) - r.q0);
    r.kv = min(max(p.a.kv_len[b], 0), p.room);
    return r;
}

// Queries enter the matrix instructions as binary16, each row scaled to [1, 2) by a power of two (exact but for
// elements below 2^-17 of the row's largest: the last of a bfloat16's 8 bits is then below 2^-24): `down` is that factor, with the softmax scale's sign, and `factor`, above 0,
// what scores are multiplied with to be in units of log2.
__device__ __forceinline__ void attn_row_scale(const AttnParams& p, float most, float& down, float& factor) {
    int e = most > 0.f ? (int)(__float_as_uint(most) >> 23) - 127 : 0;
    e = min(max(e, -120), 120);
    factor = fabsf(p.scale_log2) * __uint_as_float((uint32_t)(127 + e) << 23);
    down = __uint_as_float((uint32_t)(127 - e) << 23);
    if (p.scale_log2 < 0.f) down = -down;
    if (factor == 0.f) factor = 1.f, down = 0.f;  // every score is 0
}

// Few requests (serve_attn_team.cu): clusters of `size` CTAs (at most 8), `chunks` of them for a request and KV head.
rra_status_t launch_team(const AttnParams& p, int chunks, int size, rra_stream_t stream);
// Prompts (serve_prefill.cu): `tiles` (1 or 2) of 128 rows a CTA.
rra_status_t launch_prefill(const AttnParams& p, int tiles, int sms, rra_stream_t stream);
size_t prefill_partial_bytes(int head_dim);

}  // namespace rra
