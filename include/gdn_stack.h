/* gdn_stack.h — what a stack of delta-rule layers on MI355X (gfx950) has around
 * the calls of gdn.h and gdn_serve.h, trained and served:
 *
 *   gdn_qk_norm                 queries and keys normalised for each head, scaled
 *                               and rotated by their positions, as gdn_prefill,
 *                               gdn_cache_write and gdn_cache_attention take them
 *   gdn_qk_norm_backward        its gradients, behind gdn_prefill_backward
 *   gdn_scan, gdn_scan_backward the gated linear recurrence with a vector state,
 *                               over packed sequences, and its gradients
 *   gdn_scan_pool               that recurrence on a pool of states, one or a few
 *                               tokens for each request
 *   gdn_cache_attention_prefix  gdn_cache_attention for requests that share the
 *                               pages of a long beginning
 *
 * The conventions of gdn.h and gdn_serve.h hold: device pointers of the current
 * HIP device, work enqueued on `stream` without waiting, status codes, argument
 * errors reported before any memory is touched, no allocation, no state kept
 * between calls, calls on different streams independent of each other, every
 * call capturable into a graph (GDN_VALIDATE=1 aside, which waits for the
 * stream).  Two calls in flight at once need two workspaces.  Contents of index
 * arrays never make a kernel address memory outside the arrays given.  NaN and
 * Inf are not masked: they propagate as far as the definitions let them, and
 * never from one sequence into another.  The passages of the pages that gdn.h
 * cites name neither of the first two; the batch that shares a beginning is the
 * serving of long contexts of section 5.3 of "Trillion-Parameter MoE Multimodal
 * LLMs: How to Evaluate the New Generation".
 */
#ifndef GDN_STACK_H
#define GDN_STACK_H

#include "gdn.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Norm of gdn_qk_norm, over the d channels of a head:
 *   GDN_NORM_NONE  r = 1
 *   GDN_NORM_L2    r = 1 / sqrt(sum of squares + eps), what the delta rule wants
 *                  of its keys (l2_eps of gdn_decode_pool)
 *   GDN_NORM_RMS   r = 1 / sqrt(mean of squares + eps) */
typedef enum gdn_norm { GDN_NORM_NONE = 0, GDN_NORM_L2 = 1, GDN_NORM_RMS = 2 } gdn_norm;

/* Queries and keys, normalised and rotated:
 *     z = w * (r x),   y = scale * R(position) z
 * for every token and head, w one weight per channel shared by the heads, scale
 * q_scale for queries and 1 for keys.  R turns `rotary` channels in pairs,
 *     (u, v) -> (u cos a - v sin a, u sin a + v cos a),  a = position * inv_freq[i],
 * pair i being channels i and i + rotary / 2, or with `interleaved` channels 2 i
 * and 2 i + 1; channels from `rotary` on stay.
 *
 *   q, k        device [T_total, H, d] and [T_total, H_k, d], dtype: the heads of
 *               a token side by side, tokens q_stride and k_stride elements apart
 *               (slices of one projection's output need no copy).  H or H_k 0:
 *               none of that kind, its pointers may be NULL.
 *   q_weight, k_weight  device fp32 [d], or NULL for 1
 *   positions   device int32 [T_total] (any value; gdn_batch_tables writes them);
 *               NULL with rotary 0
 *   inv_freq    device fp32 [rotary / 2]; NULL with rotary 0
 *   rotary      a multiple of 8 from 0 to d
 *   eps         a normal number > 0 (of any value with GDN_NORM_NONE)
 *   q_out, k_out  device [T_total, H, d] and [T_total, H_k, d], dtype, contiguous.
 *               q_out may be q where q_stride is H * d, k_out k likewise; else
 *               outputs and inputs do not overlap.
 *
 * d is 64 or 128.  Alignment: q, k, outputs and weights 16 bytes, inv_freq 16,
 * strides a multiple of 16 bytes and at least H * d, positions 4.
 * All arithmetic is fp32, the angles' is 64 bits (a position of a million is
 * turned as exactly as position 1); one rounding to bf16 at the end.  Squares are
 * fp32's: a head whose sum of squares is above fp32's numbers (3.4e38) normalises
 * to 0, as the formula in fp32 does, and its gradient is 0. */
int32_t gdn_qk_norm(const void* q, int64_t q_stride, const void* k, int64_t k_stride, int64_t T_total, int32_t H,
                    int32_t H_k, int32_t d, int32_t norm, float eps, const float* q_weight, const float* k_weight,
                    const int32_t* positions, const float* inv_freq, int32_t rotary, int32_t interleaved, float q_scale,
                    void* q_out, void* k_out, int32_t dtype, void* stream);

/* Gradients of gdn_qk_norm.  q, k and the arguments they share are those of the
 * forward call (its inputs, not its outputs).
 *
 *   d_q_out, d_k_out  device [T_total, H, d] and [T_total, H_k, d], dtype,
 *               contiguous: gradients of the outputs
 *   dq, dk      device, dtype, tokens dq_stride and dk_stride elements apart (they
 *               may be slices of one tensor), written; not overlapping the inputs,
 *               but for dq being d_q_out where dq_stride is H * d, dk d_k_out likewise
 *   d_q_weight, d_k_weight  device fp32 [d], written; NULL: not wanted
 *   workspace   gdn_qk_norm_backward_workspace_bytes(...) bytes, 16-byte aligned;
 *               needed for the weights' gradients only
 *
 * With n = r x and dz = scale * R^T dy: dw = sum over tokens and heads of dz n,
 * dx = r (w dz - n <w dz, n>) for L2, with <,> / d for RMS, w dz without a norm.
 * The weights' gradients are summed in fp32 in an order that sizes alone decide.
 * T_total 0 writes zeros to them. */
int32_t gdn_qk_norm_backward(const void* q, int64_t q_stride, const void* k, int64_t k_stride, const void* d_q_out,
                             const void* d_k_out, int64_t T_total, int32_t H, int32_t H_k, int32_t d, int32_t norm,
                             float eps, const float* q_weight, const float* k_weight, const int32_t* positions,
                             const float* inv_freq, int32_t rotary, int32_t interleaved, float q_scale, void* dq,
                             int64_t dq_stride, void* dk, int64_t dk_stride, float* d_q_weight, float* d_k_weight,
                             int32_t dtype, void* workspace, size_t workspace_bytes, void* stream);

/* Device scratch bytes of gdn_qk_norm_backward when a weight's gradient is wanted
 * (0 for invalid sizes). */
size_t gdn_qk_norm_backward_workspace_bytes(int64_t T_total, int32_t H, int32_t H_k, int32_t d);

/* The gated linear recurrence of every channel, over packed sequences:
 *     h_t = e^g_t h_{t-1} + b_t,   b_t = x_t, or with `mix` (1 - e^g_t) x_t
 *
 *   x           device [T_total, C], dtype; C a multiple of 4
 *   g           device fp32 [T_total, C], log-decay, any value <= 0
 *   cu_seqlens  device int32 [num_seqs + 1], as in gdn_prefill
 *   initial_state  device fp32 [num_seqs, C], or NULL for 0
 *   final_state    device fp32 [num_seqs, C], written (a sequence without a token
 *               keeps its initial state), or NULL.  It must not overlap
 *               initial_state.
 *   h           device [T_total, C], dtype; it may be x, and else overlaps no
 *               input.  Rows behind cu_seqlens[num_seqs] are left as they were.
 *   checkpoints device, gdn_scan_checkpoint_bytes(T_total, C) bytes, written, or
 *               NULL: states along the sequences, for gdn_scan_backward
 *   workspace   gdn_scan_workspace_bytes(T_total, C) bytes, 16-byte aligned.  The
 *               call's workgroups wait for each other's entries in it, each for about
 *               0.8 s at most: where something else writes to it before the call has
 *               ended (a second call, say), the outputs behind a lost entry are NaN,
 *               and the status is GDN_OK all the same
 *
 * States are fp32; h is rounded once.  e^g is fp32's, and 0 below its normal numbers
 * (g under -87.3).  An infinite state stays infinite however small the product of
 * decays above 0, and a decay of 0 makes it NaN; a finite one it ends, to the last
 * bit.  gdn_scan_backward's l is as the state is.  Alignment: 16 bytes, cu_seqlens 4.  The
 * result's bits do not depend on timing (but for a workspace that is written to).
 * Below 2^23 tiles of 64 tokens and 256 channels.
 * GDN_VALIDATE=1 returns GDN_ERR_DOMAIN for offsets that decrease, do not begin
 * at 0 or end behind T_total, and for g of a sequence above 0 or NaN. */
int32_t gdn_scan(const void* x, const float* g, const int32_t* cu_seqlens, int32_t num_seqs, int64_t T_total, int32_t C,
                 int32_t mix, const float* initial_state, float* final_state, void* h, float* checkpoints,
                 int32_t dtype, void* workspace, size_t workspace_bytes, void* stream);

/* Device bytes of the states that gdn_scan keeps for gdn_scan_backward, and
 * scratch bytes of gdn_scan and of gdn_scan_backward (0 for invalid sizes). */
size_t gdn_scan_checkpoint_bytes(int64_t T_total, int32_t C);
size_t gdn_scan_workspace_bytes(int64_t T_total, int32_t C);
size_t gdn_scan_backward_workspace_bytes(int64_t T_total, int32_t C);

/* Gradients of gdn_scan.  x, g and the arguments they share are those of the
 * forward call.
 *
 *   d_h            device [T_total, C], dtype
 *   d_final_state  device fp32 [num_seqs, C], or NULL for 0
 *   checkpoints    what gdn_scan wrote for the same inputs, or NULL: the states
 *                  are computed again, for one more reading of x and g
 *   dx             device [T_total, C], dtype, written; it may be d_h, and else
 *                  overlaps no input
 *   dg             device fp32 [T_total, C], written.  Rows of dx and dg behind
 *                  cu_seqlens[num_seqs] are left as they were.
 *   d_initial_state  device fp32 [num_seqs, C], written (the final state's
 *                  gradient for a sequence without a token), or NULL.  It must not
 *                  overlap d_final_state.
 *   workspace      gdn_scan_backward_workspace_bytes(T_total, C) bytes, as gdn_scan's
 *
 * With l_t = d_h_t + e^g_{t+1} l_{t+1} (the last token of a sequence: + its
 * d_final_state): dx = l, with `mix` (1 - e^g) l;  dg = e^g l h_{t-1}, with `mix`
 * e^g l (h_{t-1} - x);  d_initial_state = e^g l of the first token.  States and
 * l are fp32, from x and not from the rounded h. */
int32_t gdn_scan_backward(const void* x, const float* g, const int32_t* cu_seqlens, int32_t num_seqs, int64_t T_total,
                          int32_t C, int32_t mix, const float* initial_state, const float* checkpoints,
                          const void* d_h, const float* d_final_state, void* dx, float* dg, float* d_initial_state,
                          int32_t dtype, void* workspace, size_t workspace_bytes, void* stream);

/* The recurrence of gdn_scan on a pool of states, as gdn_decode_pool has the
 * delta rule's: one or a few tokens for each request.
 *
 *   x, g, mix   as in gdn_scan
 *   states      device fp32 [num_slots, C], updated in place
 *   slots       device int32 [num_seqs]: request n's state; a request whose slot is
 *               outside [0, num_slots) is skipped and its rows of h are left as
 *               they were.  Slots inside are distinct.
 *   cu_seqlens  device int32 [num_seqs + 1], or NULL: one token per request (then
 *               T_total = num_seqs).  Offsets are cut to [0, T_total].
 *   commit      device int32 [num_seqs], or NULL for all: the state that is stored
 *               is the one after the first commit[n] tokens (cut to the request's
 *               tokens; 0 or less: the state stays).  h is written for every token.
 *   h           device [T_total, C], dtype; it may be x, and else overlaps no input
 *
 * Alignment: 16 bytes, index arrays 4.
 * GDN_VALIDATE=1 returns GDN_ERR_DOMAIN for offsets that decrease or do not end
 * at T_total, slots that repeat and g above 0 or NaN. */
int32_t gdn_scan_pool(const void* x, const float* g, float* states, const int32_t* slots, const int32_t* cu_seqlens,
                      const int32_t* commit, int32_t num_seqs, int64_t T_total, int32_t num_slots, int32_t C,
                      int32_t mix, void* h, int32_t dtype, void* stream);

/* gdn_cache_attention (gdn_serve.h) for requests of which groups share the pages
 * of a long beginning (a common prompt): a group's queries read it once.
 *
 *   group_offsets  device int32 [num_groups + 1]: group i is requests
 *                  group_offsets[i] .. group_offsets[i+1]-1, which are neighbours;
 *                  a request that shares with no other is a group of its own, or
 *                  in none
 *   prefix_lens    device int32 [num_groups]: tokens at the beginning of each
 *                  request of the group that lie in the same pages; what is
 *                  behind the last whole page of them is read by each request
 *   max_prefix     bound on prefix_lens, for planning only (0: unknown)
 *   workspace      gdn_cache_attention_prefix_workspace_bytes(...) bytes, 16-byte
 *                  aligned
 *
 * The other arguments and the result are gdn_cache_attention's: the rows of the
 * block table that a group's requests have agree in the blocks of the beginning,
 * and these are read through one of them.  A request that holds fewer than
 * prefix_lens tokens before its new ones (a refused one, say), or whose row is
 * outside the table, takes no part and reads all of its own.  Where the bounds say
 * that reading the beginnings apart would cost more than it saves (short beginnings,
 * few requests, requests of more than 128 rows by max_new and on average) the call is
 * gdn_cache_attention itself.  Sums of parts are joined
 * in an order that sizes, lengths and groups decide; outputs differ from
 * gdn_cache_attention's by rounding.
 * GDN_VALIDATE=1 returns GDN_ERR_DOMAIN for what gdn_cache_attention does, for
 * group offsets that decrease, do not begin at 0 or end behind num_seqs, negative
 * prefix_lens, and requests of a group whose blocks of the beginning differ. */
int32_t gdn_cache_attention_prefix(const void* q, const void* k_cache, const void* v_cache, const float* k_scale,
                                   const float* v_scale, const int32_t* block_table, const int32_t* rows,
                                   const int32_t* kv_lens, const int32_t* cu_seqlens, const int32_t* group_offsets,
                                   const int32_t* prefix_lens, int32_t num_seqs, int32_t num_groups, int64_t T_total,
                                   int64_t max_new, int64_t max_kv, int64_t max_prefix, int64_t num_pages,
                                   int32_t page_size, int32_t num_rows, int32_t max_blocks, float scale, void* o,
                                   int32_t H, int32_t H_kv, int32_t d_k, int32_t d_v, int32_t dtype, void* workspace,
                                   size_t workspace_bytes, void* stream);

/* Device scratch bytes of gdn_cache_attention_prefix; a function of the arguments
 * only (0 for invalid ones). */
size_t gdn_cache_attention_prefix_workspace_bytes(int32_t num_seqs, int32_t num_groups, int64_t T_total,
                                                  int64_t max_new, int64_t max_kv, int64_t max_prefix,
                                                  int32_t page_size, int32_t max_blocks, int32_t H, int32_t H_kv,
                                                  int32_t d_k, int32_t d_v);

#ifdef __cplusplus
}
#endif

#endif /* GDN_STACK_H */
