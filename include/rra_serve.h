/*
 * rra_serve.h -- operators of a decode step around the AllReduce (C ABI).
 *
 * A tensor-parallel decode step alternates AllReduces (rra.h) with attention
 * over the keys and values of the tokens so far.  These operators are what a
 * rank runs between two AllReduces, and once per step before them:
 *
 *   rra_slot_map      page tables and slots of the step's tokens, from request
 *                     lengths, on the GPU (no host round trip per step)
 *   rra_qk_norm_rope  norms of queries and keys for each head, with the
 *                     position rotation, in one pass
 *   rra_kv_append     keys and values of the new tokens into a paged cache
 *                     held in 4 bits
 *   rra_kv_read       what the cache holds for given tokens, as values
 *   rra_kv_attention  attention over that cache: single tokens, a few drafted
 *                     tokens, chunks of a prompt
 *
 * Rules common to all.  Every call only enqueues work on `stream` (one
 * kernel), never synchronises and allocates nothing, so it can be captured
 * into a CUDA graph.  Arguments travel in a structure of plain values and
 * device pointers that is read before the call returns.  Buffers belong to
 * the caller, are device memory of the current GPU, and stay alive until the
 * work on `stream` completes.  Argument errors return RRA_ERR_INVALID_ARG and
 * enqueue nothing; a failed launch returns RRA_ERR_CUDA.  Indices that only
 * the device can see (slots, page numbers, positions, lengths) are checked
 * by the kernels, which never touch memory outside the buffers for them;
 * what happens instead stands at each operator.
 */
#ifndef RRA_SERVE_H
#define RRA_SERVE_H

#include <stddef.h>
#include <stdint.h>

#include "rra.h"

#ifdef __cplusplus
extern "C" {
#endif

#define RRA_SERVE_MAX_REQUESTS 4096   /* requests of one call */

/* ------------------------------------------------------- page bookkeeping --
 * rra_slot_map: one step of the paged cache's bookkeeping.  A page holds
 * page_tokens tokens; request b's token i lives in page block_table[b][i /
 * page_tokens], and its slot is page * page_tokens + i % page_tokens.  Pages
 * that no request holds are a stack, free_pages[0 .. *free_count).
 *
 *   new_len[b] >= 0: request b gets new_len[b] tokens after its seq_len[b].
 *   new_len[b] <  0: request b ends; its pages go back, its length is 0.
 *
 * In this order: (1) the pages of the requests that end are pushed, request
 * by request, each in the order of its row (entries outside
 * [0, num_pages) are skipped, and so is what would not fit num_pages);
 * (2) the pages that the new tokens need beyond those held are popped from
 * the top, request by request.  Then
 *   kv_len[b]       seq_len[b] + new_len[b] (0 if it ended)
 *   cu_new[0..B]    running sum of the new tokens
 *   block_table     the entries of the new pages
 *   slots[t], positions[t]   slot and position in its request of new token t,
 *                   t < tokens, in the order of the requests; beyond the last
 *                   new token -1 and 0 (padding of a step of fixed shape)
 *   *free_left      pages left on the stack
 *   *pages_short    pages wanted but not given: the stack was empty (their
 *                   entries become -1) or the row too short.  Tokens without a
 *                   page get slot -1, which rra_kv_append skips.
 * A request whose pages ran short keeps its length: the caller ends or
 * resubmits it.  New tokens beyond `tokens` get pages but no slot.  Rows of
 * ended requests are left as they are.  Lengths below 0 count as
 * 0, seq_len above 2^30 - 1 and new_len above (2^30 - 1) / requests as that.
 * kv_len may be seq_len, free_left may be free_count; nothing else overlaps.
 * requests 0..RRA_SERVE_MAX_REQUESTS; table_pages <= table_stride. */
typedef struct {
    const int32_t* seq_len;     /* [requests] */
    const int32_t* new_len;     /* [requests] */
    int32_t* block_table;       /* [requests][table_stride], table_pages used */
    int32_t* free_pages;        /* [num_pages] */
    const int32_t* free_count;  /* [1] */
    int32_t* kv_len;            /* [requests] */
    int32_t* cu_new;            /* [requests + 1] */
    int64_t* slots;             /* [tokens] */
    int32_t* positions;         /* [tokens] */
    int32_t* free_left;         /* [1] */
    int32_t* pages_short;       /* [1] */
    int64_t table_stride;
    int64_t tokens;
    int32_t requests;
    int32_t table_pages;
    int32_t page_tokens;
    int32_t num_pages;
} rra_slot_map_args_t;

rra_status_t rra_slot_map(const rra_slot_map_args_t* args, rra_stream_t stream);

/* ------------------------------------------------- head norms and rotation --
 * rra_qk_norm_rope: for every token t and every head x of q and of k
 *     y[i] = x[i] / sqrt(mean(x^2) + eps) * weight[i]
 *     out  = y with its first `rot` channels rotated by the token's position p:
 *            (a, b) -> (a cos[p][j] - b sin[p][j], b cos[p][j] + a sin[p][j])
 * for the pairs (a, b) = (y[j], y[j + rot/2]), or (y[2j], y[2j + 1]) with
 * `interleaved`, j < rot/2.  All in binary32, rounded once.  A NULL weight
 * leaves out that tensor's norm (rotation only).
 *   dtype RRA_FP32 or RRA_BF16, of q, k, the weights and the outputs;
 *   cos, sin binary32 [max_position][rot/2].
 *   Strides are in elements, between tokens and between heads; a head's
 *   channels are adjacent.  Pointers are 16-byte aligned, strides multiples of
 *   16 bytes.  q_out may be q, k_out may be k (same strides), other overlaps
 *   are not allowed.  q_heads or k_heads may be 0 (that tensor is not touched).
 *   head_dim a multiple of 16 up to 256; rot <= head_dim a multiple of 16 (0: no
 *   rotation; cos, sin and positions are then not read).
 * A position outside [0, max_position) makes the rotated channels NaN. */
typedef struct {
    const void* q;
    const void* k;
    void* q_out;
    void* k_out;
    const void* q_weight;       /* [head_dim] or NULL */
    const void* k_weight;
    const float* cos;
    const float* sin;
    const int32_t* positions;   /* [tokens] */
    int64_t q_token_stride, q_head_stride;
    int64_t k_token_stride, k_head_stride;
    int64_t q_out_token_stride, q_out_head_stride;
    int64_t k_out_token_stride, k_out_head_stride;
    int64_t tokens;
    int64_t max_position;
    double eps;
    int32_t q_heads, k_heads;
    int32_t head_dim, rot;
    int32_t interleaved;
    int32_t dtype;              /* rra_dtype_t */
} rra_qk_norm_rope_args_t;

rra_status_t rra_qk_norm_rope(const rra_qk_norm_rope_args_t* args, rra_stream_t stream);

/* ------------------------------------------------------- the 4-bit cache ---
 * A page: for each KV head, for each 16 of its page_tokens tokens, a block of
 * 18 * head_dim bytes:
 *     K codes [16][head_dim / 2]   V codes [16][head_dim / 2]
 *     K scales [16][head_dim / 32] V scales [16][head_dim / 32]   (binary16)
 * A value is code * scale.  A code is e2m1, sign in bit 3: 0, .5, 1, 1.5, 2,
 * 3, 4, 6.  Channels 32 j .. 32 j + 31 share scale j.  Channel 32 j + 4 c + e
 * (e < 4) is in byte (c * head_dim/32 + j) * 2 + e/2 of its row, the low
 * nibble for even e: so that a warp's lanes find the operands of its matrix
 * instructions in whole words.  4.5 bits a value.
 *
 * Writing: scale = max |x| over the group, times 1/6 (binary32 multiply),
 * clamped to [2^-14, 2048], rounded to binary16; code = x / scale (binary32
 * division) rounded to the nearest e2m1, ties to even, magnitudes above 6 to
 * 6.  So the cache resolves values from 3e-5 to 12288; NaN is stored as 0,
 * infinities as the largest code.
 *
 * page_tokens: a multiple of 16, 16..4096.  head_dim: 64 or 128.  The cache has
 * up to 2^31 - 1 blocks (num_pages * page_tokens / 16 * kv_heads). */
typedef struct {
    void* pages;                /* [num_pages][rra_kv_page_bytes()], 16-byte aligned */
    int64_t num_pages;
    int32_t page_tokens;
    int32_t kv_heads;
    int32_t head_dim;
    int32_t reserved;           /* 0 */
} rra_kv_cache_t;

/* Bytes of a page; 0 if the arguments are not supported. */
size_t rra_kv_page_bytes(int page_tokens, int kv_heads, int head_dim);

/* rra_kv_append writes k[t][h], v[t][h] to slot slots[t] (page * page_tokens
 * + token in the page); slots outside the cache are skipped.  A slot that
 * occurs twice in one call gets either token's values, K and V of a head not
 * necessarily the same token's.
 * rra_kv_read does the reverse: k[t][h], v[t][h] become what slot slots[t]
 * holds, rounded to dtype (exact in binary32); slots outside the cache read as 0.
 * dtype RRA_BF16 or RRA_FP32; strides in elements, channels adjacent; pointers
 * 16-byte aligned, strides multiples of 16 bytes. */
typedef struct {
    rra_kv_cache_t cache;
    void* k;                    /* read by append, written by read */
    void* v;
    const int64_t* slots;       /* [tokens] */
    int64_t k_token_stride, k_head_stride;
    int64_t v_token_stride, v_head_stride;
    int64_t tokens;
    int32_t dtype;              /* rra_dtype_t */
    int32_t reserved;           /* 0 */
} rra_kv_tokens_args_t;

rra_status_t rra_kv_append(const rra_kv_tokens_args_t* args, rra_stream_t stream);
rra_status_t rra_kv_read(const rra_kv_tokens_args_t* args, rra_stream_t stream);

/* ------------------------------------------------------------- attention ---
 * rra_kv_attention: request b has the query tokens cu_q[b] .. cu_q[b + 1) and
 * the first kv_len[b] tokens of its row of block_table in the cache, its own
 * included (append first).  Query i of its n has position p = kv_len[b] - n +
 * i and sees key j if
 *     j < kv_len[b],  j <= p (if causal),  j > p - window (if window > 0).
 * Query head h uses KV head h / (q_heads / kv_heads):
 *     s_j = scale * q . k_j,  out = sum_j exp(s_j) v_j / sum_j exp(s_j),
 *     lse = log sum_j exp(s_j).
 * A query that sees no key gets out = 0 and lse = -inf.  Products accumulate
 * in binary32; the softmax's maximum, sum and weights are binary32; out is
 * rounded to bfloat16 once.  A query is scaled by a power of two to [1, 2) and
 * then binary16: its elements keep their 8 bits down to 2^-17 of its largest, and
 * those below 2^-25 of it count as 0.  Scores take every key exactly: code times
 * scale, 13 bits, as two products.  For the sum over values binary16 (11 bits)
 * holds: for few queries, the weight (times 2^10, against its underflow) and the
 * weight times scale, the codes being exact; in the kernel for prompts, the
 * weight (times 2^7), and code times scale apart.  The
 * result does not depend on timing: partial results of a split request are
 * joined in a fixed order.
 *   q, out bfloat16 [tokens][q_heads][head_dim], strides in elements, channels
 *   adjacent, pointers 16-byte aligned, strides multiples of 8; out may not
 *   overlap q.  lse NULL or binary32 [tokens][q_heads], contiguous.
 *   Rows of out and lse that no request has (a step's padding after cu_q[B]) stay
 *   as they are: fill them before, if anything reads them.
 *   cu_q ascends; where it does not, rows may be computed several times or not at
 *   all.  Its values are clamped to [0, tokens], kv_len to [0, table_pages *
 *   page_tokens]; keys in pages outside [0, num_pages) are not seen.
 *   max_q, max_kv: the longest query and key counts expected.  They steer the
 *   choice of kernel and its split only: longer requests are still right.
 *   workspace: rra_kv_attention_workspace_bytes() bytes, 256-byte aligned, its
 *   first 4096 zero before its first use; every call leaves it ready for the
 *   next.  Calls that share a workspace are ordered on one stream.
 *   Its first 32-bit word is a status: RRA_OK, or RRA_ERR_TIMEOUT if a wait for
 *   the kernel's own copies or products ran out.  The results of that call are
 *   then not valid, nor are later ones until the caller has set the word to 0,
 *   in the order of the stream; the rest of the workspace is ready all the same.
 * requests 0..RRA_SERVE_MAX_REQUESTS; q_heads a multiple of kv_heads; tokens *
 * q_heads and table_pages * page_tokens up to 2^30 - 1. */
typedef struct {
    rra_kv_cache_t cache;
    const void* q;
    void* out;
    float* lse;
    const int32_t* cu_q;        /* [requests + 1] */
    const int32_t* kv_len;      /* [requests] */
    const int32_t* block_table; /* [requests][table_stride], table_pages used */
    void* workspace;
    int64_t q_token_stride, q_head_stride;
    int64_t out_token_stride, out_head_stride;
    int64_t table_stride;
    int64_t tokens;             /* rows of q and out */
    double scale;               /* usually 1 / sqrt(head_dim); times log2(e) finite in binary32, as scores are */
    int32_t requests;
    int32_t table_pages;
    int32_t q_heads;
    int32_t max_q, max_kv;
    int32_t causal;
    int32_t window;             /* 0: no window */
    int32_t reserved;           /* 0 */
} rra_kv_attention_args_t;

rra_status_t rra_kv_attention(const rra_kv_attention_args_t* args, rra_stream_t stream);

/* Bytes of the workspace of rra_kv_attention for heads of head_dim channels
 * (0 if not supported); independent of the batch. */
size_t rra_kv_attention_workspace_bytes(int head_dim);

/* The kernel that rra_kv_attention launches for these arguments (host
 * arithmetic only): its name in a profiler's launch list, then the form in
 * angle brackets, "kv_attention_kernel<8 rows>" or <16 rows> (few queries, the
 * batch's keys in equal runs), "kv_attention_team_kernel<1 CTA>", <2 CTAs>,
 * <4 CTAs>, <8 CTAs> (few requests, a cluster for each 8 rows) or
 * "kv_attention_prompt_kernel<128 rows>", <256 rows>. */
rra_status_t rra_kv_attention_plan(const rra_kv_attention_args_t* args, const char** name);

#ifdef __cplusplus
}
#endif

#endif /* RRA_SERVE_H */
