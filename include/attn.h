/*
 * The attention step of serving on one GB300 GPU (sm_103a), part of libmoe: grouped-query
 * attention over a paged key/value cache held in 4 bits, with what a step needs around it.
 * In the order in which a step runs them:
 *
 *   attn_plan           block tables and slot maps from the requests' lengths, on the GPU
 *   attn_qk_norm_rope   norm of every query and key head and the position rotation, one pass
 *   attn_kv4_append     keys and values quantised into their cached rows
 *   attn_kv4_forward    causal attention of the new tokens over the cached rows
 *   attn_kv4_read       cached rows back as bf16 (to move, share or inspect a prefix)
 *
 * and, for steps that verify drafted trees and for layers that see a window of their context,
 *
 *   attn_tree_plan             depths and ancestor masks of drafted trees, behind attn_plan
 *   attn_qk_norm_rope_append   norm, rotation and quantisation of a step's rows, one pass
 *   attn_kv4_forward_masked    attention through a window with first tokens, or of a tree
 *   attn_kv4_accept            the accepted tokens' cached rows moved to where they belong
 *   attn_kv4_accept_pages      the same, and the rejected ones' pages put back on the free list
 *
 * Source: "Optimizing on-device inference for Apple Silicon", § "Read attention cache
 * efficiently" (16 query heads over 2 key/value heads of 256 channels; the query heads of a
 * key/value head share one pass over its cached rows) and § "Reduce intermediate and state
 * traffic" (query and key preparation before attention in one kernel).  The page's cache is
 * not in 4 bits and not paged; the 4-bit form here is that of the page's weights (§ "Dequantize
 * weights during matrix multiplication": groups of 64 with a scale and a bias).
 *
 * Definitions.  Hq query heads, Hkv key/value heads, G = Hq / Hkv, D channels a head, pages of P
 * tokens; request b has n_b new tokens this step after c_b cached ones.
 *
 *   plan: request b needs ceil((c_b + n_b) / P) - ceil(c_b / P) new pages, taken in order from
 *     the free list; token i of request b is at position c_b + i, in slot
 *     block_table[b][pos / P] * P + pos % P.
 *   norm and rotation: y = x * rsqrt(mean(x^2) + eps) * w over a head's D channels; then, of the
 *     first r channels, the pairs (i, i + r/2) (or, interleaved, (2i, 2i + 1)) turn by the angle
 *     whose cosine and sine the table holds for the token's position:
 *     (a, b) -> (a cos - b sin, b cos + a sin).  In fp32, rounded once to bf16.
 *   cached row: per group of 64 channels lo = min, step = bf16((max - lo) / 15), code =
 *     clamp(rint((x - lo) / step), 0, 15) (ties to even; 0 where step is 0), read back as
 *     step * code + lo; every operation in fp32, so the codes are the same everywhere.  If a
 *     channel of a token's key or value row of a head is not finite, or 2^116 or larger, the key
 *     row's scales become 0 and biases NaN and the value row's 0: every query that sees the token
 *     reads NaN and no other query does.
 *   attention: o_i = sum_t softmax_t(scale q_i . k_t) v_t over the cached tokens t <= kv_b - n_b +
 *     i of request b (kv_b = its cached tokens with the new ones); a query that sees no token
 *     gives 0.  Scores, softmax sums and outputs are held in fp32 and rounded once to bf16.
 *     Scores are in range below 2^23 (in units of log 2): a row with larger ones may read NaN, and
 *     from 2^28 on it does.
 *     A value loses bits beside another one, 2^20 times as large, of a weight that counts (with more
 *     than 32 query rows a key/value head, where tokens have the largest weight of the 16 that share a
 *     record, and channels 2^18 below its largest lose bits too).  Tokens that a query does not see cost
 *     it nothing, whatever they hold.
 *   window and first tokens: a query at position p sees the cached tokens t <= p with t < S or t > p -
 *     W (a window of W tokens, the query's own among them, and S first tokens).
 *   tree: the n_b new tokens of request b are drafted, token i behind token parent_i < i, or
 *     (parent_i = -1) behind the context.  All are appended, token i in row kv_b - n_b + i as by the
 *     plan; its position is kv_b - n_b plus its depth, the number of its ancestors.  Token i sees all
 *     cached tokens before the drafted ones, its ancestors and itself.  Once some are accepted,
 *     their rows move to rows kv_b - n_b, kv_b - n_b + 1, ...; the cache is as if no other had been.
 *
 * Cache of one layer: one caller-owned device array of n_pages * Hkv * P * (D + D / 8) bytes (0.5625
 * bytes a channel), 128-byte aligned, written by attn_kv4_append only: records [n_pages][Hkv][P / 16]
 * of 16 tokens of one head each, so that an attention kernel takes 16 tokens in one copy.  A record:
 *   key codes     uint8 [16][D/2]
 *   key params    uint32 [16][D/64]: group g's scale (bf16, lower half) and bias (upper half)
 *   value params  uint32 [16][D/64]
 *   value codes   uint8 [16][D/2]
 * Slot s = page * P + offset is row offset % 16 of record offset / 16 of its page.  Inside a row of
 * codes, 32-bit word j (0..7) of group g holds the codes of channels 64g + 8j .. 64g + 8j + 7, the
 * lowest nibble first, and lies at word (j ^ f(s)) * (D/64) + g, f(s) = 2 (s & 3) ^ (s & 4): the
 * order in which the attention kernels read rows without shared-memory bank conflicts.
 *
 * Ownership and threading: every tensor is a caller-owned device pointer; calls only enqueue
 * work on `stream` (a cudaStream_t as void*, NULL = the legacy default stream) and never
 * synchronise the host or allocate.  The handle owns a device workspace (partial results of
 * contexts that several blocks share; contexts in the form that prompts read, 4 bytes for each
 * channel that the cache's pages hold, 512 MB at most: longer ones are read as they are, more
 * slowly) and an error word; use a handle on one stream at a time, and every call with the device
 * current on which it was created.
 * Rows are strided: a stride is the distance between tokens in elements, a multiple of 8 and at
 * least the width of a token's heads; heads are adjacent, their channels contiguous.  Row
 * pointers are 16-byte aligned, index arrays 4-byte aligned.  Outputs must not overlap inputs,
 * except where stated.
 *
 * Errors (status values of moe.h): invalid host arguments are rejected before anything is
 * enqueued.  What only the device sees goes to the handle's error word (attn_get_device_error):
 * MOE_ERR_NO_MEMORY (the plan ran out of pages), MOE_ERR_INVALID_ARG (the plan found lengths that
 * do not fit), MOE_ERR_DEVICE (a position, slot, page or length out of range: the access is left
 * out or moved into range and the output is undefined), MOE_ERR_TIMEOUT (a bounded wait expired).
 * Of several the largest value stays.
 */
#ifndef ATTN_H
#define ATTN_H

#include <stddef.h>
#include <stdint.h>

#include "moe.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct attn_handle_s* attn_handle;

typedef struct {
  int n_q_heads;    /* Hq: a multiple of n_kv_heads, at most 16 n_kv_heads */
  int n_kv_heads;   /* Hkv: 1..128 */
  int head_dim;     /* D: 64, 128 or 256 */
  int page_size;    /* P: 16, 32, 64, 128 or 256 */
  int n_pages;      /* pages of a layer's cache; n_pages * page_size < 2^31 */
  int max_requests; /* largest B accepted later: 1..1024 */
  float scale;      /* softmax scale, > 0; 0 means D^-1/2 */
} attn_config;

/* Validates cfg, allocates the workspace on the current CUDA device and returns a handle in *out.
 * May synchronise the device.  On failure *out is NULL and nothing stays allocated.  One handle
 * serves every layer of the same shape. */
int attn_create(const attn_config* cfg, attn_handle* out);

/* Frees the workspace and the handle (synchronises the device).  NULL is accepted. */
int attn_destroy(attn_handle h);

/* Synchronises `stream`, then returns and clears the handle's device error word. */
int attn_get_device_error(attn_handle h, void* stream);

/* Block tables and slot maps of one step from the requests' lengths; one launch.
 *   block_table [B][table_width] int32, in and out: page ids of the cached tokens; the new pages'
 *                 ids are written behind them, nothing else is changed
 *   ctx_lens, new_lens [B] int32   cached and new tokens of each request (c_b, n_b >= 0)
 *   free_pages [n_free] int32      the free list; *cursor (int32) entries of it are taken
 *   T                              capacity of positions and slots
 *   q_offsets [B+1] int32, out     first new token of each request, clamped to T
 *   kv_lens [B] int32, out         c_b + n_b, 0 for a refused request
 *   positions, slots [T] int32, out: of each new token; slot -1 for a refused request's tokens,
 *                 position 0 and slot -1 behind the last request's tokens
 *   cursor_out int32, out          *cursor plus the pages taken; may be `cursor` itself
 * Request b is refused for lack of pages if it needs any and the needs of requests 0..b together
 * exceed n_free - *cursor (MOE_ERR_NO_MEMORY); for its lengths if one is negative or above 2^30,
 * its pages exceed table_width, or its tokens end behind T (MOE_ERR_INVALID_ARG; it then needs no
 * pages).  A refused request's table row is left as it is, so it can be planned again later. */
int attn_plan(attn_handle h, int32_t* block_table, int table_width, const int32_t* ctx_lens,
              const int32_t* new_lens, int B, const int32_t* free_pages, int n_free,
              const int32_t* cursor, int T, int32_t* q_offsets, int32_t* kv_lens,
              int32_t* positions, int32_t* slots, int32_t* cursor_out, void* stream);

/* Norm and rotation of T tokens' queries [T][Hq][D] and keys [T][Hkv][D] (bf16); one launch.
 *   positions [T] int32; q_weight, k_weight [D] bf16, 16-byte aligned
 *   cos_sin [n_positions][rotary_dim] fp32, 16-byte aligned: the cosines of a position's
 *     rotary_dim / 2 angles, then their sines
 *   rotary_dim: 0 (no rotation; positions and cos_sin are not read) or a multiple of 16 up to D
 * q_out and k_out may be q and k themselves (same pointer and stride).  A position out of range
 * turns by position 0's angles (MOE_ERR_DEVICE). */
int attn_qk_norm_rope(attn_handle h, const void* q, int64_t q_stride, const void* k,
                      int64_t k_stride, const int32_t* positions, const void* q_weight,
                      const void* k_weight, float eps, const float* cos_sin, int n_positions,
                      int rotary_dim, int interleaved, int T, void* q_out, int64_t q_out_stride,
                      void* k_out, int64_t k_out_stride, void* stream);

/* Quantises T tokens' keys and values [T][Hkv][D] (bf16) into the cached rows of their slots
 * [T] (int32); one launch.  A negative slot is skipped; one beyond the cache is skipped and
 * recorded (MOE_ERR_DEVICE).  The slots of a call are distinct. */
int attn_kv4_append(attn_handle h, const void* k, int64_t k_stride, const void* v,
                    int64_t v_stride, const int32_t* slots, int T, void* cache, void* stream);

/* Cached rows of T slots as bf16 [T][Hkv][D], step * code + lo in fp32 rounded once; a slot
 * outside the cache gives zeros (recorded unless negative). */
int attn_kv4_read(attn_handle h, const void* cache, const int32_t* slots, int T, void* k,
                  int64_t k_stride, void* v, int64_t v_stride, void* stream);

/* Causal attention of B requests' new tokens over the cache (their own rows are appended
 * already).  q, out [T][Hq][D] bf16: request b's tokens are rows q_offsets[b] .. q_offsets[b+1] - 1;
 * kv_lens [B] counts its cached tokens with the new ones; block_table [B][table_width].
 * max_q_len >= 1 and max_kv_len >= 0 bound n_b and kv_b (from above; they choose kernels and
 * grids, a capacity will do): a request beyond max_q_len is cut to it (MOE_ERR_DEVICE).  Rows of
 * out that belong to no request are left as they are.  The same inputs give the same bits. */
int attn_kv4_forward(attn_handle h, const void* q, int64_t q_stride, const void* cache,
                     const int32_t* block_table, int table_width, const int32_t* q_offsets,
                     const int32_t* kv_lens, int B, int T, int max_q_len, int max_kv_len,
                     void* out, int64_t out_stride, void* stream);

/* Depths and ancestor masks of B requests' drafted trees; one launch.
 *   parents [T] int32     index in its request of each new token's parent, below its own; -1 where it
 *                         follows the context.  Others are recorded (MOE_ERR_INVALID_ARG) and count
 *                         as -1.
 *   q_offsets, kv_lens    as for attn_kv4_forward
 *   max_q_len             1..256 and at most 32 mask_words: bounds n_b; a request beyond it is
 *                         cut to it (MOE_ERR_DEVICE)
 *   positions [T] int32, out: kv_b - n_b (0 where that is negative) plus the token's depth
 *   masks [T][mask_words] uint32, out: bit j % 32 of word j / 32 for each token j of its request that
 *                         it sees: its ancestors and itself
 * Rows of the outputs behind the last request's tokens become 0. */
int attn_tree_plan(attn_handle h, const int32_t* parents, const int32_t* q_offsets,
                   const int32_t* kv_lens, int B, int T, int max_q_len, int32_t* positions,
                   uint32_t* masks, int mask_words, void* stream);

/* attn_qk_norm_rope of T tokens' queries and keys and attn_kv4_append of the turned keys and the
 * values v [T][Hkv][D], in one launch: the keys are not written as bf16.  Arguments as there, but
 * q_weight and k_weight may both be NULL: no norm then, the rotation alone.  q_out may be q itself.
 * The turned key rows are rounded to bf16 and quantised.  Every operation on them before is a single
 * one in fp32, so the codes are the same everywhere: the sum of a row's squares, rounded once, times
 * 1 / D, plus eps; 1 / sqrt of it, two operations; x times that, times the weight; a cos - b sin and
 * b cos + a sin, three operations each.  (attn_qk_norm_rope rounds in other places, so its rows may
 * differ in the last bit.)  Queries of tokens whose slot is negative are formed all the same. */
int attn_qk_norm_rope_append(attn_handle h, const void* q, int64_t q_stride, const void* k,
                             int64_t k_stride, const void* v, int64_t v_stride,
                             const int32_t* positions, const int32_t* slots, const void* q_weight,
                             const void* k_weight, float eps, const float* cos_sin,
                             int n_positions, int rotary_dim, int interleaved, int T, void* q_out,
                             int64_t q_out_stride, void* cache, void* stream);

/* attn_kv4_forward with a narrower view:
 *   window      W >= 1, or 0: no window; at most 2^30
 *   sinks       S >= 0 first tokens that stay visible behind the window (without one they mean
 *               nothing); at most 2^30
 *   masks       [T][mask_words] uint32, or NULL: causal.  Bit j of its row tells whether a query sees
 *               drafted token j of its request (bits from n_b on mean nothing); the cached tokens
 *               before the drafted ones it sees all, as far as a window lets it.  Its position is
 *               kv_b - n_b plus the number of drafted tokens that it sees besides one (itself).
 *               max_q_len is at most 256 and 32 mask_words, and at most W if there is a window (so a
 *               window never hides drafted tokens).
 * A query that sees no token gives 0.  Pages that lie between the first tokens and every window of
 * their request are not read: their entries of block_table may be anything, such as those of pages
 * given back. */
int attn_kv4_forward_masked(attn_handle h, const void* q, int64_t q_stride, const void* cache,
                            const int32_t* block_table, int table_width, const int32_t* q_offsets,
                            const int32_t* kv_lens, int B, int T, int max_q_len, int max_kv_len,
                            int window, int sinks, const uint32_t* masks, int mask_words,
                            void* out, int64_t out_stride, void* stream);

/* Moves the cached rows (codes and parameters, bit for bit) of accepted tokens: of request b, row
 * ctx_lens[b] + paths[b][i] to row ctx_lens[b] + i, for i = 0 .. path_lens[b] - 1; one launch.
 *   ctx_lens [B] int32       cached tokens before the drafted ones
 *   paths [B][path_width] int32   accepted tokens by their index in their request, ascending; the
 *                            entries behind path_lens[b] are not read
 *   path_lens [B] int32      0 .. path_width
 * Rows behind the accepted ones keep what they hold.  attn_plan counts a request's pages from its
 * ctx_lens: pages taken for rejected tokens alone are put back by attn_kv4_accept_pages, or else by the
 * caller; the next plan replaces them in the table, and what is not put back is lost.  Requests share
 * none of the pages that they move rows in.  A length out of range moves nothing; an entry that is negative
 * or not above the one before it, or a row outside the table or the cache, is left out
 * (MOE_ERR_DEVICE; the request's moved rows are then undefined). */
int attn_kv4_accept(attn_handle h, void* cache, const int32_t* block_table, int table_width,
                    const int32_t* ctx_lens, const int32_t* paths, int path_width,
                    const int32_t* path_lens, int B, void* stream);

/* The same, and the pages that the step's plan took for rejected tokens alone go back on the free list:
 * of request b the table's entries from page (ctx_lens[b] + path_lens[b] + P - 1) / P up to the last one of
 * kv_lens[b] tokens, to free_pages [n_free] in front of *cursor, requests in order; the cursor moves
 * back by as many.  One launch as well.
 *   kv_lens [B] int32   lengths with the drafted tokens, as attn_plan wrote them (a refused request's 0
 *                       puts nothing back, nor does one below ctx_lens[b])
 *   free_pages, n_free, cursor   of the plan; read and written
 * The table keeps its entries; the next plan replaces them.  A request whose path_lens or ctx_lens is out of
 * range puts nothing back; a page id that the cache does not have is left out, and a cursor that is not
 * in 0 .. n_free, or with fewer entries before it, leaves list and cursor alone (MOE_ERR_DEVICE). */
int attn_kv4_accept_pages(attn_handle h, void* cache, const int32_t* block_table, int table_width,
                          const int32_t* ctx_lens, const int32_t* paths, int path_width,
                          const int32_t* path_lens, int B, const int32_t* kv_lens,
                          int32_t* free_pages, int n_free, int32_t* cursor, void* stream);

#ifdef __cplusplus
}
#endif

#endif
