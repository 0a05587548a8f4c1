/* gdn_serve.h — the serving side of libgdn on MI355X (gfx950): what a stack
 * that interleaves delta-rule layers with exact attention needs at every step
 * next to gdn_prefill and gdn_decode (gdn.h).
 *
 *   gdn_batch_tables     packed offsets, block tables, slot map and positions of
 *                        a step, built on the device from the requests' lengths
 *   gdn_cache_write      new keys and values into a paged 8-bit cache
 *   gdn_cache_attention  causal attention of the new tokens over that cache
 *   gdn_decode_pool      the delta rule's recurrent form on a pool of states
 *
 * The conventions of gdn.h hold: device pointers of the current HIP device,
 * work enqueued on `stream` without waiting, status codes, argument errors
 * reported before any memory is touched, no allocation, no state kept between
 * calls, calls on different streams independent of each other, every call
 * capturable into a graph (GDN_VALIDATE=1 aside, which waits for the stream).
 * Contents of index arrays are checked in the kernels where a bad value could
 * address memory outside the arrays given, as stated at each call.  Floating
 * inputs with NaN or Inf are not masked: they propagate, and only where the
 * definition lets them.
 *
 * The paged cache.  A page holds page_size consecutive tokens of one request
 * for every key/value head:
 *   k_cache  [num_pages, H_kv, page_size, d_k]  e4m3 codes
 *   v_cache  [num_pages, H_kv, page_size / 16, d_v, 16]  e4m3 codes, 16 tokens
 *            of a channel side by side
 *   k_scale  [num_pages, H_kv] fp32             one scale per page and head,
 *   v_scale  [num_pages, H_kv] fp32             a power of two
 * A key is code * scale.  e4m3 is the 8-bit format with 4 exponent and 3
 * mantissa bits, largest value 448, no infinities (code 0x7f and 0xff: NaN).
 * page_size is 64, 128 or 256.  Token t of a request lies in the page that
 * entry t / page_size of its row of the block table names, at place
 * t % page_size; its slot is page * page_size + t % page_size.  A matrix-core
 * operand takes consecutive tokens of one value channel, so 16 tokens of each
 * channel lie side by side and the attention kernels load them as they are
 * stored; a new token then touches 16 * d_v neighbouring bytes.
 */
#ifndef GDN_SERVE_H
#define GDN_SERVE_H

#include "gdn.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Tables of one step of a server, from the requests' lengths on the device.
 *
 *   context_lens  device int32 [num_seqs]: tokens request n already holds
 *   new_lens      device int32 [num_seqs]: tokens it adds in this step (0 is
 *                 fine); negative: the request has ended and gives its pages back
 *   rows          device int32 [num_seqs]: its row of block_table and
 *                 page_counts, or NULL for row n.  Rows of one call are distinct.
 *   num_seqs, T_total  the sum of the new lengths is at most T_total; tokens
 *                 past T_total are cut off the last requests
 *   block_table   device int32 [num_rows, max_blocks], updated: the page of each
 *                 block of each row; a new page is written where it is needed,
 *                 a page given back is replaced by -1
 *   page_counts   device int32 [num_rows], updated: pages each row owns (its
 *                 first page_counts entries).  They may be more than
 *                 context_lens needs (say after drafted tokens were dropped):
 *                 pages that are there are used first.
 *   free_pages    device int32 [num_pages], updated: a ring of the free pages
 *   free_state    device int32 [3], updated: place of the first free page in the
 *                 ring, number of free pages, and (written) the number of
 *                 requests that this call refused
 *   cu_seqlens    device int32 [num_seqs + 1], written: packed offsets of the
 *                 new tokens, as every packed call of this library takes them
 *   kv_lens       device int32 [num_seqs], written: tokens held after the step
 *   slots         device int32 [T_total], written: slot of each new token, -1
 *                 for tokens without one (behind the last request, or of a
 *                 refused one)
 *   positions     device int32 [T_total], written: position of each new token
 *                 in its request (0 behind the last request)
 *   workspace     gdn_batch_tables_workspace_bytes(num_seqs, T_total) bytes
 *
 * Pages are taken from the ring's start in the order of the requests and pages
 * that come back go to its end, so the result does not depend on timing.  A
 * request needs the pages behind those it owns up to the block of its last new
 * token; it is refused, and gets nothing, when its need and the need of the
 * requests before it do not fit in the free pages, when its row has no room
 * (max_blocks), when it owns fewer pages than context_lens needs, or when
 * rows[n] is outside [0, num_rows).  A refused request keeps its pages and its
 * kv_lens entry is context_lens[n]; its tokens stay in cu_seqlens, without slots.
 * What the step's layers then compute for them is not the request's: its outputs
 * are to be dropped and its state kept.  kv_lens[n] - context_lens[n], the tokens
 * that were taken, is 0 for it: as `commit` of gdn_decode_pool that difference
 * leaves the states of refused requests (and of ended ones) as they are, and
 * behind gdn_prefill it says which final states to store.  Pages given
 * back in a call are free for the next call.  Calling again with the same
 * lengths changes nothing, unless a request was refused (free_state[2]): the call
 * after it may find pages for it, those that the first one got back among them.
 * A call reads and updates the tables and the ring:
 * calls on the same ones are ordered by the caller, as on one stream.
 * GDN_VALIDATE=1 copies the lengths, the rows, the counts and the ring to the
 * host and returns GDN_ERR_DOMAIN for negative context_lens, new lengths whose sum
 * passes T_total, rows that repeat or lie outside, and a ring that does not fit its
 * array. */
int32_t gdn_batch_tables(const int32_t* context_lens, const int32_t* new_lens, const int32_t* rows, int32_t num_seqs,
                         int64_t T_total, int32_t page_size, int32_t* block_table, int32_t num_rows,
                         int32_t max_blocks, int32_t* page_counts, int32_t* free_pages, int32_t num_pages,
                         int32_t* free_state, int32_t* cu_seqlens, int32_t* kv_lens, int32_t* slots,
                         int32_t* positions, void* workspace, size_t workspace_bytes, void* stream);

/* Device scratch bytes of gdn_batch_tables (0 for invalid arguments). */
size_t gdn_batch_tables_workspace_bytes(int32_t num_seqs, int64_t T_total);

/* New keys and values into the paged cache.
 *
 *   k      device [T_total, H_kv, d_k], dtype     v  device [T_total, H_kv, d_v], dtype
 *   slots  device int32 [T_total]: slot of each token; tokens with a slot
 *          outside [0, num_pages * page_size) are skipped
 *   k_cache, v_cache, k_scale, v_scale   updated
 *
 * The tokens of one page are neighbours in the call, at consecutive slots (as
 * gdn_batch_tables gives them).  For the tokens of a call in one page, at
 * places a .. b-1, and one head, with amax their largest finite magnitude and
 *     need = max(2^-100, 2^ceil(log2(amax / 448)))
 * the page's scale becomes need when a = 0 (the page begins anew, and places
 * behind b - 1 are cleared to code 0), else max(its scale, need); when that
 * raises it, the codes of the page's other places are rounded to the new scale
 * (exact but for codes that become subnormal: scales are powers of two).  A new
 * code is the value over the scale rounded to nearest even.  Inf and NaN are
 * stored as NaN.  Pages and heads without a new token are left as they are.
 * Alignment: k, v and the caches 16 bytes, slots and scales 4.
 * GDN_VALIDATE=1 copies the slots to the host and returns GDN_ERR_DOMAIN when
 * a page's tokens are not one run of consecutive slots. */
int32_t gdn_cache_write(const void* k, const void* v, const int32_t* slots, int64_t T_total, void* k_cache,
                        void* v_cache, float* k_scale, float* v_scale, int64_t num_pages, int32_t page_size,
                        int32_t H_kv, int32_t d_k, int32_t d_v, int32_t dtype, void* stream);

/* Causal attention of the new tokens over the paged cache, which holds them
 * already (gdn_cache_write comes first).
 *
 *   q            device [T_total, H, d_k], dtype; H a multiple of H_kv, query
 *                head h reads key/value head h / (H / H_kv)
 *   block_table  device int32 [num_rows, max_blocks]
 *   rows         device int32 [num_seqs]: request n's row, or NULL for row n
 *   kv_lens      device int32 [num_seqs]: tokens request n holds, its new ones
 *                included (more than max_blocks * page_size: cut to that)
 *   cu_seqlens   device int32 [num_seqs + 1]: its new tokens are rows
 *                cu_seqlens[n] .. cu_seqlens[n+1]-1 of q and o, and are the last
 *                of its kv_lens[n] tokens
 *   scale        factor of q . k (finite)
 *   max_new, max_kv  bounds on the new tokens of a request and on kv_lens, for
 *                planning only (0: unknown); a wrong bound never changes the
 *                result beyond rounding
 *   o            device [T_total, H, d_v], dtype.  Rows behind
 *                cu_seqlens[num_seqs] are left as they were.
 *   workspace    gdn_cache_attention_workspace_bytes(...) bytes, 16-byte aligned
 *
 * o = sum_j p_j v_j, p the softmax over j of scale * q . k_j, j from 0 to the
 * token's own position.  Tokens whose block table entry is outside
 * [0, num_pages) or whose row is outside [0, num_rows) are left out; a row that
 * sees no token (kv_lens 0, or more new tokens than kv_lens) is 0.  A NaN in a
 * key or value reaches only the rows that see its token; Inf in a query makes
 * its row NaN, also where it makes all its scores -Inf.  Scales that are not
 * powers of two are not supported (they are exact factors of bf16 operands).
 * Two calls in flight at once need two workspaces.
 * GDN_VALIDATE=1 returns GDN_ERR_DOMAIN for offsets that decrease or end behind
 * T_total, lengths below 0 or past the table, and scales of held pages that are
 * not positive powers of two.
 *
 * GDN_BF16: products on bf16 matrix cores (e4m3 codes are exact in bf16) with
 * fp32 accumulation, softmax in fp32, p rounded to bf16 for the second
 * product.  GDN_F32: q and p are split into three bf16 parts, whose products
 * with the codes are exact, so that the arithmetic is fp32's.
 * The cache of few rows, or of the last of many, may be cut into parts computed
 * side by side and joined by another launch.  Pages left out cost many rows up to
 * 16% of the time (bf16, 128 channels): tiles behind the first of them run on a
 * slower path. */
int32_t gdn_cache_attention(const void* q, const void* k_cache, const void* v_cache, const float* k_scale,
                            const float* v_scale, const int32_t* block_table, const int32_t* rows,
                            const int32_t* kv_lens, const int32_t* cu_seqlens, int32_t num_seqs, int64_t T_total,
                            int64_t max_new, int64_t max_kv, int64_t num_pages, int32_t page_size, int32_t num_rows,
                            int32_t max_blocks, float scale, void* o, int32_t H, int32_t H_kv, int32_t d_k,
                            int32_t d_v, int32_t dtype, void* workspace, size_t workspace_bytes, void* stream);

/* Device scratch bytes of gdn_cache_attention; a function of the arguments
 * only (0 for invalid ones). */
size_t gdn_cache_attention_workspace_bytes(int32_t num_seqs, int64_t T_total, int64_t max_new, int64_t max_kv,
                                           int32_t page_size, int32_t max_blocks, int32_t H, int32_t H_kv,
                                           int32_t d_k, int32_t d_v);

/* The delta rule's recurrent form on a pool of states: gdn_decode for a server
 * whose requests come and go, with one or a few tokens for each.
 *
 *   q, k    device [T_total, H_k, d_k], dtype;  v  device [T_total, H, d_v], dtype;
 *           H a multiple of H_k, state head h reads key head h / (H / H_k)
 *   g       device fp32 log-decay, [T_total, H, d_k], or [T_total, H] when
 *           head_gate is not 0; any value <= 0 (the recurrence has no exponent
 *           budget, so the unbounded gate is fine too)
 *   beta    device fp32 [T_total, H]
 *   states  device fp32 [num_slots, H, d_k, d_v], updated in place
 *   slots   device int32 [num_seqs]: request n's state; a request whose slot is
 *           outside [0, num_slots) is skipped and its rows of o are left as they
 *           were.  Slots inside are distinct.
 *   cu_seqlens  device int32 [num_seqs + 1], or NULL: one token per request
 *           (then T_total = num_seqs).  Offsets are cut to [0, T_total].
 *   commit  device int32 [num_seqs], or NULL for all: the state that is stored
 *           is the one after the first commit[n] tokens (cut to the request's
 *           tokens; 0 or less: the state stays).  o is written for every token,
 *           so drafted tokens can be tried without being kept.  Behind
 *           gdn_batch_tables it is kv_lens - context_lens, so that a refused
 *           request's state stays.
 *   q_scale factor of q
 *   l2_eps  > 0: q and k are first divided by sqrt(sum of squares + l2_eps)
 *           over d_k, per token and head; 0: they are taken as they are
 *   o       device [T_total, H, d_v], dtype
 *
 * Per token: S' = diag(e^g) S, u = beta (v - S'^T k), S = S' + k u^T,
 * o = S^T (q_scale q), all in fp32.  The state is read and written once per call
 * whatever the number of tokens; a request with many tokens is better served by
 * gdn_prefill, which is parallel over them.
 * Alignment: q, k, v, o, states and a per-channel g 16 bytes, the rest 4.
 * GDN_VALIDATE=1 returns GDN_ERR_DOMAIN for offsets that decrease or do not end
 * at T_total, slots that repeat and g above 0. */
int32_t gdn_decode_pool(const void* q, const void* k, const void* v, const float* g, int32_t head_gate,
                        const float* beta, float* states, const int32_t* slots, const int32_t* cu_seqlens,
                        const int32_t* commit, int32_t num_seqs, int64_t T_total, int32_t num_slots, float q_scale,
                        float l2_eps, void* o, int32_t H, int32_t H_k, int32_t d_k, int32_t d_v, int32_t dtype,
                        void* stream);

#ifdef __cplusplus
}
#endif

#endif /* GDN_SERVE_H */
