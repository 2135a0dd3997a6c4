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
 *   rra_kv8_append, rra_kv8_read, rra_kv8_attention   the same over a cache of 8 bits
 *   rra_prompt_attention  attention of whole prompts over their own keys and values
 *   rra_pages_fork, rra_pages_release, rra_pages_compact, rra_pages_copy
 *                     pages that several requests share: samples of a prompt,
 *                     their end, holes in the pool closed
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

/* ------------------------------------------------------- the 8-bit cache ---
 * The same calls over a cache of 8 bits (8 + 8 / head_dim with its exponents),
 * for those to whom 4 bits are too few: the structures above, with pages of
 * rra_kv8_page_bytes() bytes.  A page: for each KV head, for each 16 of its
 * page_tokens tokens, a block of 32 * head_dim + 16 bytes:
 *     K codes [16][head_dim]   V codes [16][head_dim]
 *     exponent of K, of V (a signed byte each)   14 bytes that nothing uses
 * A value is code * 2^exponent.  A code is e4m3: sign, 4 bits of exponent, 3 of
 * mantissa, up to 448, down to 2^-9.  The 16-byte piece i of row r's codes is in
 * the 128-byte line that row order gives, at i ^ (r & 7) within it for heads of
 * 128, at i ^ (r & 6) for heads of 64 (two rows a line).
 *
 * Writing: a block's exponent, for each head, K and V apart, is the smallest whole
 * number with max |x| <= 448 * 2^e over its values, within [-32, 32]; code = x *
 * 2^-e rounded to the nearest e4m3, ties to even, saturating.  Writing the token
 * at a block's start begins it anew: what it held before goes.  Writing others
 * keeps what is there and can only raise the exponent; the codes that are there
 * are then rounded again, to the new unit (a power of two: only those that get
 * below 2^-6 of it lose bits, at most 2^-10 of it each time).  So a value x, up to
 * 448 * 2^32, is off by at most 2^-4 |x| + 2^-9 * 2^e, with the e that its block has
 * now: half a step of its code, and 2^-10 of each unit that the block has had.  NaN
 * is stored as 0; infinities as the largest code, and do not count for the exponent.
 *
 * rra_kv8_append: slots of one block are neighbours in the list, in any order, as
 * rra_slot_map gives them (slots outside the cache are skipped and do not come
 * between neighbours).  Where one block's slots come in several places of one
 * call, its codes and exponents may not belong together.  A slot that occurs
 * twice gets either token's values, channel by channel.
 * rra_kv8_read, rra_kv8_attention: as rra_kv_read, rra_kv_attention; every code
 * and exponent enters exactly.  Codes are binary16 in the products, weights too:
 * off by 2^-11 of themselves, or where they are small by 2^-24 of the largest; so
 * a key adds an error of 2^-24 of its value at most, whatever the exponents of other
 * blocks, and of values that a row does not see.  Scores are below 2^26, as in
 * rra_prompt_attention.  The workspace is the same. */
size_t rra_kv8_page_bytes(int page_tokens, int kv_heads, int head_dim);
rra_status_t rra_kv8_append(const rra_kv_tokens_args_t* args, rra_stream_t stream);
rra_status_t rra_kv8_read(const rra_kv_tokens_args_t* args, rra_stream_t stream);
rra_status_t rra_kv8_attention(const rra_kv_attention_args_t* args, rra_stream_t stream);
rra_status_t rra_kv8_attention_plan(const rra_kv_attention_args_t* args, const char** name);

/* ------------------------------------------------- attention of prompts ---
 * rra_prompt_attention: attention of whole prompts over their own keys and
 * values, as the projection gives them, before or beside their way into a cache.
 * Request b has the tokens cu[b] .. cu[b + 1) of q, k, v and out.  Its token i sees
 * its token j if
 *     j <= i (if causal),  j > i - window (if window > 0).
 * Query head h uses KV head h / (q_heads / kv_heads); formulas, lse and scale as in
 * rra_kv_attention.  Queries, keys and values enter their products as they are;
 * products, the softmax's maximum, sum and weights are binary32; for the sum over
 * values a weight is rounded to the values' type (bfloat16, 8 bits; binary16, 11 bits,
 * times 2^7 against its underflow), out to it once.  Results do not depend on timing.
 * Scores, times log2(e), are below 2^26: where binary32 has no bits left for their
 * differences, above that, rows may become NaN.
 *   A NaN, or an infinite value, makes the rows that see its token NaN or infinite, no
 *   others.  Infinite queries and keys make infinite scores: +inf makes its row NaN or
 *   infinite; -inf has weight 0, and a row with no other scores sees no key.
 *   q, out [tokens][q_heads][head_dim], k, v [tokens][kv_heads][head_dim], all
 *   bfloat16, or binary16 (`half`); strides in elements, multiples of 8, below 2^39;
 *   channels adjacent; pointers 16-byte aligned; out overlaps nothing.  They may be
 *   parts of a packed projection.  lse NULL or binary32 [tokens][q_heads], contiguous.
 *   Rows after cu[B] stay as they are.  head_dim a multiple of 8 up to 128.
 *   cu ascends; where it does not, rows may be computed several times or not at all.
 *   Its values are clamped to [0, tokens].
 *   max_len: the longest prompt expected; it steers the choice of kernel only.
 *   workspace: rra_prompt_attention_workspace_bytes() bytes, with the rules of
 *   rra_kv_attention's.
 * requests 0..RRA_SERVE_MAX_REQUESTS; tokens * q_heads up to 2^30 - 1. */
typedef struct {
    const void* q;
    const void* k;
    const void* v;
    void* out;
    float* lse;
    const int32_t* cu;          /* [requests + 1] */
    void* workspace;
    int64_t q_token_stride, q_head_stride;
    int64_t k_token_stride, k_head_stride;
    int64_t v_token_stride, v_head_stride;
    int64_t out_token_stride, out_head_stride;
    int64_t tokens;             /* rows of q, k, v and out */
    double scale;               /* usually 1 / sqrt(head_dim); times log2(e) finite in binary32 */
    int32_t requests;
    int32_t q_heads, kv_heads;
    int32_t head_dim;
    int32_t half;               /* 0: bfloat16, 1: binary16 */
    int32_t max_len;
    int32_t causal;
    int32_t window;             /* 0: no window */
} rra_prompt_attention_args_t;

rra_status_t rra_prompt_attention(const rra_prompt_attention_args_t* args, rra_stream_t stream);
size_t rra_prompt_attention_workspace_bytes(void);

/* The kernel that rra_prompt_attention launches for these arguments:
 * "prompt_attention_kernel<128 rows>" or <256 rows>, a CTA's. */
rra_status_t rra_prompt_attention_plan(const rra_prompt_attention_args_t* args, const char** name);

/* ---------------------------------------------------------- shared pages ---
 * Requests that share pages: samples of one prompt, prompts with a common start.
 * shared[p] counts the holders of page p beyond the first: 0 for pages that one
 * request holds or none, never below.  rra_slot_map knows nothing of it: it pops
 * pages, whose count is 0, and a request's new tokens go behind those it has, so
 * it needs only that no request shares a page that is not full.  rra_pages_fork
 * sees to that.  Requests that end are given to rra_pages_release first; it sets
 * their length to 0, so that rra_slot_map returns nothing for them again.
 *
 * Common to the three.  A request of length n holds the first ceil(n /
 * page_tokens) entries of its row of block_table (at most table_pages).  Lengths
 * below 0 count as 0.  Entries outside [0, num_pages) are no pages: they are
 * copied as they are and counted nowhere.  free_pages[0 .. *free_count) is the
 * stack of rra_slot_map.  Outputs that are named "may be" an input may be the
 * same buffer; nothing else overlaps.  Each call is one kernel and moves no page:
 * fork and compact write lists for rra_pages_copy, which is called for the pages
 * of every layer.
 * requests 0..RRA_SERVE_MAX_REQUESTS; num_pages up to 2^24.
 *
 * rra_pages_fork: for i < forks, row target[i] becomes a copy of row source[i]:
 *   its whole pages are shared (shared + 1 for each), and a page of its own is
 *   popped, fork by fork, for one that is not full:
 *     copy_from[i], copy_to[i]   that page and the new one; -1 and -1 if there is
 *                                nothing to copy
 *     kv_len                     seq_len, and for the targets their sources'
 *     *free_left, *pages_short   as in rra_slot_map (entries without a page: -1)
 *   What a target's row held before is not given back.  Forks whose source or
 *   target is outside [0, requests) do nothing but write -1.  No row is target of two
 *   forks, or target and source: what such rows then hold is not defined.
 *   shared_out may be shared, kv_len may be seq_len, free_left may be free_count. */
typedef struct {
    const int32_t* seq_len;     /* [requests] */
    const int32_t* source;      /* [forks] */
    const int32_t* target;      /* [forks] */
    int32_t* block_table;       /* [requests][table_stride], table_pages used */
    const int32_t* free_pages;  /* [num_pages] */
    const int32_t* free_count;  /* [1] */
    const int32_t* shared;      /* [num_pages] */
    int32_t* kv_len;            /* [requests] */
    int32_t* shared_out;        /* [num_pages] */
    int32_t* copy_from;         /* [forks] */
    int32_t* copy_to;           /* [forks] */
    int32_t* free_left;         /* [1] */
    int32_t* pages_short;       /* [1] */
    int64_t table_stride;
    int32_t requests;
    int32_t forks;              /* 0..RRA_SERVE_MAX_REQUESTS */
    int32_t table_pages;
    int32_t page_tokens;
    int32_t num_pages;
    int32_t reserved;           /* 0 */
} rra_pages_fork_args_t;

rra_status_t rra_pages_fork(const rra_pages_fork_args_t* args, rra_stream_t stream);

/* rra_pages_release: requests with new_len[b] < 0 end.  Each page that such a
 *   request holds has one holder less; pages without any are pushed on the stack,
 *   in ascending order of their numbers (those that would not fit num_pages are
 *   dropped).  kv_len[b] is 0 for the requests that end, seq_len[b] for the others;
 *   block_table is not changed.  A page that is listed more often than it has
 *   holders is pushed once.
 *   shared_out may be shared, kv_len may be seq_len, free_left may be free_count. */
typedef struct {
    const int32_t* seq_len;     /* [requests] */
    const int32_t* new_len;     /* [requests] */
    const int32_t* block_table; /* [requests][table_stride], table_pages used */
    int32_t* free_pages;        /* [num_pages] */
    const int32_t* free_count;  /* [1] */
    const int32_t* shared;      /* [num_pages] */
    int32_t* kv_len;            /* [requests] */
    int32_t* shared_out;        /* [num_pages] */
    int32_t* free_left;         /* [1] */
    int64_t table_stride;
    int32_t requests;
    int32_t table_pages;
    int32_t page_tokens;
    int32_t num_pages;
} rra_pages_release_args_t;

rra_status_t rra_pages_release(const rra_pages_release_args_t* args, rra_stream_t stream);

/* rra_pages_compact: moves pages in use to the pool's low end.  Every page that is
 *   not on the stack is in use, whoever holds it.  The highest page in use goes
 *   to the lowest free page, the next highest to the next lowest, while that is
 *   lower and up to max_moves:
 *     move_from[i], move_to[i]   the moves (i < max_moves; -1 behind the last);
 *     *move_count                how many
 *     moved[p]                   page p's new number; -1 for pages that were free
 *     table_out                  block_table with the new numbers in the entries that requests hold
 *     free_out, *free_left       the pages that are free now, the lowest on top
 *     shared_out                 counts, moved along
 *   With max_moves >= num_pages / 2 the pages in use end up as 0 .. n - 1.  Nothing
 *   may use the pages between this call and rra_pages_copy's.
 *   table_out may be block_table (then with the same stride, and other entries are
 *   not touched; else they are copied), free_out may be free_pages, free_left may
 *   be free_count, shared_out may be shared. */
typedef struct {
    const int32_t* seq_len;     /* [requests] */
    const int32_t* block_table; /* [requests][table_stride], table_pages used */
    const int32_t* free_pages;  /* [num_pages] */
    const int32_t* free_count;  /* [1] */
    const int32_t* shared;      /* [num_pages] */
    int32_t* table_out;         /* [requests][table_out_stride] */
    int32_t* free_out;          /* [num_pages] */
    int32_t* free_left;         /* [1] */
    int32_t* shared_out;        /* [num_pages] */
    int32_t* moved;             /* [num_pages] */
    int32_t* move_from;         /* [max_moves] */
    int32_t* move_to;           /* [max_moves] */
    int32_t* move_count;        /* [1] */
    int64_t table_stride, table_out_stride;
    int32_t requests;
    int32_t table_pages;
    int32_t page_tokens;
    int32_t num_pages;
    int32_t max_moves;
    int32_t reserved;           /* 0 */
} rra_pages_compact_args_t;

rra_status_t rra_pages_compact(const rra_pages_compact_args_t* args, rra_stream_t stream);

/* rra_pages_copy: page to[i] of the pool `to_pages` becomes page from[i] of
 * `from_pages` (which may be the same pool), i < count.  Pairs with either outside
 * its pool are skipped.  A page that is both read and written, or written twice,
 * in one call may get a mixture.  page_bytes is a multiple of 16; pages are 16-byte
 * aligned. */
typedef struct {
    const void* from_pages;     /* [from_num][page_bytes] */
    void* to_pages;             /* [to_num][page_bytes] */
    const int32_t* from;        /* [count] */
    const int32_t* to;          /* [count] */
    int64_t from_num, to_num;
    int64_t page_bytes;
    int32_t count;
    int32_t reserved;           /* 0 */
} rra_pages_copy_args_t;

rra_status_t rra_pages_copy(const rra_pages_copy_args_t* args, rra_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* RRA_SERVE_H */
