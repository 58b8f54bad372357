/*
 * dilution_attn.h -- C ABI of the GB300 (sm_103a) dilution-attention library.
 *
 * The operator ("DilutionAttention v0.1.0 · results", section "The operator"):
 * for every (batch b, head h) independently, with queries i and keys k,
 *
 *     s_ik      = tau * (q_i . k_k) / sqrt(d)                    (k <= i only)
 *     p_ik      = exp(s_ik) / sum_{k' <= i} exp(s_ik')           causal softmax: the bids
 *     committed = sum_{j < i} p_jk                               demand from earlier queries
 *     share_ik  = p_ik / (committed_ik + p_ik + eps)
 *     out_i     = sum_k share_ik v_k / sum_k share_ik             A = share / rowsum(share)
 *
 * tau is a logit multiplier (1 by default).  A focal temperature t
 * ("Focal Attention", arXiv 2511.06818, section "Transformer with Constant
 * Temperature", eq. focal-const) is tau = 1/t; YaRN's sharpening
 * ("YaRN › Attention Temperature Scaling", temperature formula) is
 * tau = sqrt(0.1 ln s + 1).
 *
 * Conventions shared by every entry point
 *   - Layout: q, k, v, out are contiguous [B, H, T, d] (d fastest); per-row
 *     vectors (lse2, rowsum, demand) are contiguous [B, H, T].
 *   - Pointers are DEVICE pointers unless stated otherwise, 16-byte aligned.
 *     The caller owns every buffer; the library allocates nothing and keeps
 *     no state between calls.  Scratch memory is the caller's workspace.
 *   - stream is a cudaStream_t (NULL = legacy default stream).  Compute
 *     calls are asynchronous: argument errors are returned synchronously
 *     before anything is enqueued; kernel-side errors (a bounded wait that
 *     timed out) are written to a status word at the start of the workspace
 *     and read back with dilution_attn_get_error().
 *   - Supported: d == 64 or d == 128 (other head sizes return
 *     DA_ERR_UNSUPPORTED and a workspace size of 0); dtype DA_F32 (fp32
 *     in/out, fp32 SIMT arithmetic) or DA_BF16 (bf16 in/out, bf16
 *     tensor-core products, fp32 accumulation and fp32 softmax/demand
 *     arithmetic).  tau >= 0 and finite; eps > 0 and
 *     finite (eps = 0 would make masked and underflowed entries 0/0).
 *     B, H, T >= 0; a call with B*H*T == 0 does nothing and returns DA_OK.
 *     T <= DA_MAX_T.  The DA_BF16 forward needs eps >= 1e-18 (it forms one
 *     reciprocal for each pair of denominators, each >= eps); smaller eps
 *     returns DA_ERR_UNSUPPORTED.
 */
#ifndef DILUTION_ATTN_H
#define DILUTION_ATTN_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Status codes returned by every call. */
#define DA_OK              0
#define DA_ERR_INVALID     1   /* bad argument: null/misaligned pointer, negative size, eps <= 0, ... */
#define DA_ERR_UNSUPPORTED 2   /* valid but not implemented: d not 64 or 128, T > DA_MAX_T, ...   */
#define DA_ERR_CUDA        3   /* a CUDA runtime call failed (launch, tensor-map encode, copy)   */
#define DA_ERR_TIMEOUT     4   /* a kernel's bounded wait expired; results are not valid         */
#define DA_ERR_WORKSPACE   5   /* workspace pointer null or smaller than the *_workspace_size    */

/* Element types. */
#define DA_F32  0
#define DA_BF16 1

#define DA_MAX_T (1 << 24)

/* Flags of the *_ex entry points (bitwise or; other bits are DA_ERR_INVALID). */
#define DA_FLAG_EARLIER_DEMAND_ONLY 1   /* share = p / (committed + eps): see below */
#define DA_FLAG_KEEP_FOR_BACKWARD   2   /* forward leaves its state for the backward: see below */

/* Human-readable name of a status code (static string, never NULL). */
const char *dilution_attn_status_string(int status);

/* Library ABI version (major*100 + minor). */
int dilution_attn_version(void);

/* ------------------------------------------------------------------------
 * Prefill forward.
 *
 * Computes out for all T queries of each (b, h) (the operator above), plus
 * optional per-row side outputs:
 *   lse2_out   [B,H,T] fp32, nullable: log2 of the softmax normaliser of the
 *              scaled logits, log2(sum_{k<=i} 2^(s_ik * log2 e)); the bid is
 *              p_ik = 2^(s_ik*log2 e - lse2_i).
 *   rowsum_out [B,H,T] fp32, nullable: R_i = sum_k share_ik, the normaliser
 *              of row i of A = share / R (whose rows therefore sum to 1 by
 *              construction); out_i = sum_k share_ik v_k / R_i.
 *   demand_out [B,H,T] fp32, nullable: column totals sum_i p_ik over all T
 *              queries -- the decode demand cache after prefill
 *              ("DilutionAttention v0.1.0 · results", section "The operator",
 *              cached decoding).
 * workspace: device scratch of at least dilution_attn_fwd_workspace_size()
 * bytes; its first 256 bytes hold the status word.  For bf16 inputs, int32
 * word 4 of that block counts the rows whose softmax normaliser the
 * tensor-core pass handed to an exact per-row recomputation (its running sum
 * overflowed: a logit more than ~106 log2 units above the maximum of the
 * row's first 32 keys); diagnostic only.  Every call overwrites the
 * workspace, so concurrent calls on different streams need distinct
 * workspaces.  Errors: DA_ERR_INVALID, DA_ERR_UNSUPPORTED, DA_ERR_WORKSPACE,
 * DA_ERR_CUDA (launch failure).
 * ---------------------------------------------------------------------- */
size_t dilution_attn_fwd_workspace_size(int B, int H, int T, int d, int dtype);

int dilution_attn_fwd(const void *q, const void *k, const void *v, void *out,
                      float *lse2_out, float *rowsum_out, float *demand_out,
                      int B, int H, int T, int d, float tau, float eps, int dtype,
                      void *workspace, size_t workspace_bytes, void *stream);

/* Same computation as dilution_attn_fwd; additionally records events[0..3]
 * (cudaEvent_t handles created by the caller, each may be NULL) on `stream`:
 * [0] before the row-statistics kernel, [1] before the demand sweep, [2]
 * before the finalize kernel, [3] after it.  Used to time each kernel on the
 * stream it runs on.  events == NULL is the same as dilution_attn_fwd. */
int dilution_attn_fwd_with_events(const void *q, const void *k, const void *v, void *out,
                                  float *lse2_out, float *rowsum_out, float *demand_out,
                                  int B, int H, int T, int d, float tau, float eps, int dtype,
                                  void *workspace, size_t workspace_bytes, void *stream,
                                  void *const *events);

/* ------------------------------------------------------------------------
 * Extended forward: dilution_attn_fwd_with_events plus two options.
 *
 *   tau_bh  nullable DEVICE pointer to B*H fp32 logit multipliers, index
 *           b*H + h: head (b, h) uses tau_bh[b*H + h] instead of `tau` (a
 *           per-head temperature, "Learning to Focus: Focal Attention for
 *           Selective and Scalable Transformers", section "Transformer with
 *           Learned Temperature": learned there, an input here).  4-byte
 *           aligned.  `tau` is still validated but unused when tau_bh is
 *           given.  Entries must be finite and >= 0; the kernels cannot
 *           return a synchronous error for device data, so a negative, NaN or
 *           infinite entry sets DA_ERR_INVALID in the status word
 *           (dilution_attn_get_error) and that head's results are unspecified.
 *           The backward and decode calls of the same model must receive the
 *           same array.
 *   flags   DA_FLAG_EARLIER_DEMAND_ONLY: the ablation of "DilutionAttention
 *           v0.1.0 · results" (paragraph after "The operator") that divides
 *           each bid by the demand of earlier queries alone,
 *               share_ik = p_ik / (committed_ik + eps),
 *           so every key's first query (the key itself) gets share p_ii / eps
 *           and, as eps -> 0, the layer tends to the identity map.  For
 *           DA_BF16, shares up to 1/eps are fed to the value product in bf16;
 *           eps >= 1e-18 as for the default operator.
 *           DA_FLAG_KEEP_FOR_BACKWARD (DA_BF16 only, else DA_ERR_UNSUPPORTED):
 *           the workspace must be at least dilution_attn_bwd_workspace_size()
 *           (else DA_ERR_WORKSPACE); the forward also leaves there what the
 *           backward would otherwise recompute (the demand of every key at
 *           every 32-query chunk and the unnormalised outputs), so that a
 *           dilution_attn_bwd_ex with the same flag, the same inputs,
 *           options and workspace skips that pass.  The caller must not
 *           touch the workspace in between.
 *   events  as for dilution_attn_fwd_with_events (nullable).
 * Other arguments, outputs and errors as for dilution_attn_fwd; unknown flag
 * bits or a misaligned tau_bh return DA_ERR_INVALID.
 * ---------------------------------------------------------------------- */
int dilution_attn_fwd_ex(const void *q, const void *k, const void *v, void *out,
                         float *lse2_out, float *rowsum_out, float *demand_out,
                         int B, int H, int T, int d, float tau, const float *tau_bh, float eps,
                         int flags, int dtype, void *workspace, size_t workspace_bytes, void *stream,
                         void *const *events);

/* ------------------------------------------------------------------------
 * Backward: gradients dq, dk, dv [B,H,T,d] of sum(dout * out) for the
 * forward above (the page states only that exact gradients exist; they are
 * the chain rule through the causal softmax, the exclusive column cumsum, the
 * share and the renormalisation).
 *   lse2 [B,H,T] fp32: the forward's lse2_out for the same q, k, tau.
 *   dtype applies to q, k, v, dout, dq, dk, dv.  DA_BF16 runs on tcgen05
 *   tensor cores (bf16 products, fp32 accumulation and fp32 demand
 *   arithmetic, the demand recomputed from checkpoints every 32 queries; the
 *   products' operands are rounded to bf16: the shares, u = p dp, p rho, ds
 *   and dout divided by each row's sum of shares);
 *   DA_F32 runs on CUDA cores in fp32 (column sums of the demand in fp64).
 * workspace: at least dilution_attn_bwd_workspace_size(); errors as for
 * dilution_attn_fwd.
 * ---------------------------------------------------------------------- */
size_t dilution_attn_bwd_workspace_size(int B, int H, int T, int d, int dtype);

int dilution_attn_bwd(const void *q, const void *k, const void *v, const void *dout,
                      const float *lse2, void *dq, void *dk, void *dv,
                      int B, int H, int T, int d, float tau, float eps, int dtype,
                      void *workspace, size_t workspace_bytes, void *stream);

/* Backward with the options of dilution_attn_fwd_ex: tau_bh (nullable device
 * [B*H]) and flags (DA_FLAG_EARLIER_DEMAND_ONLY), which must match the
 * forward that produced lse2.  DA_FLAG_KEEP_FOR_BACKWARD (DA_BF16 only):
 * workspace is the one the forward ran with under the same flag and still
 * holds its state; lse2 is then not read (but must still be a valid pointer).
 * With DA_FLAG_EARLIER_DEMAND_ONLY, D_jk = committed_jk + eps and the direct
 * term of dp_jk is dr_jk / D_jk.  Errors as for dilution_attn_bwd
 * plus those of dilution_attn_fwd_ex for tau_bh and flags. */
int dilution_attn_bwd_ex(const void *q, const void *k, const void *v, const void *dout,
                         const float *lse2, void *dq, void *dk, void *dv,
                         int B, int H, int T, int d, float tau, const float *tau_bh, float eps,
                         int flags, int dtype, void *workspace, size_t workspace_bytes, void *stream);

/* ------------------------------------------------------------------------
 * Cached decode step ("DilutionAttention v0.1.0 · results", section "The
 * operator": the ordinary key/value cache plus one running demand total per
 * key and head).
 *
 * For each (b, h): the cache holds keys/values 0 .. n_ctx-1 in
 * k_cache/v_cache [B,H,T_cap,d] and their demand totals in demand
 * [B,H,T_cap] (fp32; sum of every bid each key has received so far).  The
 * step
 *   1. writes k_new/v_new [B,H,d] to position n_ctx of the caches,
 *   2. forms the bids p_k of q_new [B,H,d] over keys 0 .. n_ctx (causal
 *      softmax of the scaled logits),
 *   3. share_k = p_k / (demand_k + p_k + eps), with demand_{n_ctx} = 0,
 *   4. out [B,H,d] = sum_k share_k v_k / sum_k share_k,
 *   5. demand_k += p_k for k <= n_ctx (in place; demand_{n_ctx} = p_{n_ctx}).
 * Requires 0 <= n_ctx < T_cap.  After the call the cache holds n_ctx + 1
 * tokens.  dtype applies to q/k/v/out and the caches (DA_BF16 only).
 * workspace: at least dilution_attn_decode_workspace_size(B,H,T_cap,d).
 * ---------------------------------------------------------------------- */
size_t dilution_attn_decode_workspace_size(int B, int H, int T_cap, int d);

int dilution_attn_decode_step(const void *q_new, const void *k_new, const void *v_new,
                              void *k_cache, void *v_cache, float *demand,
                              int n_ctx, int T_cap, void *out,
                              int B, int H, int d, float tau, float eps, int dtype,
                              void *workspace, size_t workspace_bytes, void *stream);

/* Decode step with the options of dilution_attn_fwd_ex: tau_bh (nullable
 * device [B*H]) and flags.  With DA_FLAG_EARLIER_DEMAND_ONLY step 3 becomes
 * share_k = p_k / (demand_k + eps); the demand update is unchanged, so a
 * cache built by a flagged prefill continues the flagged operator.  Errors as
 * for dilution_attn_decode_step plus those of dilution_attn_fwd_ex for tau_bh
 * and flags (DA_FLAG_KEEP_FOR_BACKWARD is DA_ERR_INVALID here). */
int dilution_attn_decode_step_ex(const void *q_new, const void *k_new, const void *v_new,
                                 void *k_cache, void *v_cache, float *demand,
                                 int n_ctx, int T_cap, void *out,
                                 int B, int H, int d, float tau, const float *tau_bh, float eps,
                                 int flags, int dtype, void *workspace, size_t workspace_bytes, void *stream);

/* ------------------------------------------------------------------------
 * Cached decode step that allocates nothing (no counterpart on the pages: an
 * interface convenience, not part of the method).
 *
 * Same arguments, semantics and errors as dilution_attn_decode_step, without
 * the workspace: scratch comes from a fixed 16 MiB array built into the
 * library (dilution_attn_decode_noalloc_scratch_bytes()).  It is for callers
 * that cannot allocate device memory while decoding -- a runtime whose memory
 * pool is fixed for the duration of a request, or a host that can pass only
 * the tensors it already owns.  Every GPU that loads the library keeps the
 * array until the process exits.
 *   - Returns DA_ERR_WORKSPACE when dilution_attn_decode_workspace_size(B, H,
 *     T_cap, d) exceeds the array (e.g. 8 x 12 heads fit T_cap up to ~42K).
 *   - Calls no cudaMalloc/cudaFree; the first call on a device looks up the
 *     array's device address (cudaGetSymbolAddress), so make that first call
 *     before any stream capture.
 *   - All calls share the array and it keeps the last call's contents (the
 *     status word is cleared at the start of each call): calls that overlap on
 *     the GPU race with each other, so issue them on one stream or order them.
 *   - Errors found on the device (a bounded wait that ran out, an invalid
 *     per-head scale) land in the array's status word: read and clear it with
 *     dilution_attn_decode_noalloc_get_error.
 * ---------------------------------------------------------------------- */
int dilution_attn_decode_step_noalloc(const void *q_new, const void *k_new, const void *v_new,
                                      void *k_cache, void *v_cache, float *demand,
                                      int n_ctx, int T_cap, void *out,
                                      int B, int H, int d, float tau, float eps, int dtype,
                                      void *stream);

/* Size in bytes of the fixed scratch array of dilution_attn_decode_step_noalloc. */
size_t dilution_attn_decode_noalloc_scratch_bytes(void);

/* Synchronises `stream` and returns the status word of the fixed array on the
 * current device (DA_OK, or the first error a kernel of an earlier no-alloc
 * call recorded, e.g. DA_ERR_TIMEOUT), clearing it; DA_ERR_CUDA if the array
 * cannot be reached.  Same semantics as dilution_attn_get_error on a
 * workspace. */
int dilution_attn_decode_noalloc_get_error(void *stream);

/* ------------------------------------------------------------------------
 * Rotary positions of queries and keys, with one to four position axes.
 *
 * A token at position n_a on axis a turns pair j of a head's elements by the
 * angle theta_j = n_{axis(j)} * inv_freq_j (radians):
 *     (x, y) -> (x cos theta_j - y sin theta_j,  y cos theta_j + x sin theta_j).
 * Pair j is the elements (j, n_pairs + j), or (2j, 2j + 1) if `adjacent` is
 * set; elements from 2 n_pairs on pass unchanged.  Text has one axis; images
 * and video give each pair the axis (time, height, width) that pair_axis
 * names.  The angle is taken modulo one turn in 64-bit fixed point, so far
 * positions lose nothing; the products run in fp32 and are rounded once.
 * ---------------------------------------------------------------------- */
#define DA_MAX_ROPE_PAIRS 64
#define DA_MAX_ROPE_AXES  4

typedef struct dilution_attn_rope_spec {
  const float *inv_freq;                 /* DEVICE [n_pairs] fp32, |inv_freq| < 2^24 (others give NaN) */
  int32_t n_pairs;                       /* 0 .. d/2 (0: every element passes unchanged) */
  int32_t n_axes;                        /* 1 .. DA_MAX_ROPE_AXES */
  int32_t adjacent;                      /* 0: pairs (j, n_pairs + j), 1: pairs (2j, 2j + 1) */
  uint8_t pair_axis[DA_MAX_ROPE_PAIRS];  /* axis of each pair, < n_axes */
} dilution_attn_rope_spec;

/* q_out, k_out [B,H,T,d] = q, k turned by +theta (k and k_out may both be NULL
 * with Hk = 0).  The four *_strides are HOST arrays of three element strides
 * (b, h, t), or NULL for contiguous [B,H,T,d]; d is always contiguous, so the
 * inputs may be views of a fused projection [B,T,(Hq + 2 Hk) d].  Input
 * strides may be 0 (a head or batch entry read several times).  Outputs must
 * not address an element twice (their strides, sorted, must each step over
 * the extent below; else DA_ERR_INVALID).  An output may be its own input
 * (same pointer and strides); other overlaps are not allowed (an output at an
 * input's pointer with other strides, or at another operand's pointer, is
 * DA_ERR_INVALID; the rest is not checked).
 * positions: DEVICE int32 [n_axes][pos_batch][T], pos_batch 1 (every batch
 * entry alike) or B; negative positions are valid.
 * spec is a HOST struct, read during the call.  No workspace.  Errors as for
 * dilution_attn_fwd, without a workspace; any 2-byte (bf16) or 4-byte (fp32)
 * aligned pointer is accepted, rows whose pointers and strides are all
 * multiples of 16 bytes take the fast path. */
int dilution_attn_rope(const void *q, const int64_t *q_strides, const void *k, const int64_t *k_strides,
                       void *q_out, const int64_t *q_out_strides, void *k_out, const int64_t *k_out_strides,
                       const int32_t *positions, int pos_batch, const dilution_attn_rope_spec *spec,
                       int B, int Hq, int Hk, int T, int d, int dtype, void *stream);

/* Backward of dilution_attn_rope: dq, dk = the upstream gradients dq_out,
 * dk_out turned by -theta (positions and frequencies take no gradient).  Same
 * arguments and errors; the gradients' strides let them be written straight
 * into a fused projection's gradient. */
int dilution_attn_rope_bwd(const void *dq_out, const int64_t *dq_out_strides, const void *dk_out,
                           const int64_t *dk_out_strides, void *dq, const int64_t *dq_strides, void *dk,
                           const int64_t *dk_strides, const int32_t *positions, int pos_batch,
                           const dilution_attn_rope_spec *spec, int B, int Hq, int Hk, int T, int d, int dtype,
                           void *stream);

/* ------------------------------------------------------------------------
 * Paged cache of S sequences of different lengths.
 *
 * Keys and values live in pages of page_size tokens, the demand totals (one
 * per key and QUERY head) in pages of their own:
 *   k_pages, v_pages [num_pages, Hkv, page_size, d],
 *   demand_pages     [num_demand_pages, Hq, page_size] fp32.
 * Token t of sequence s has its key and value in row t % page_size of page
 * page_table[s][t / page_size], its demand in that row of page
 * demand_table[s][t / page_size].  Sequences that share a prefix may name the
 * same key/value pages; the demand differs between them, so a demand page
 * belongs to one place of one table row (two places naming one demand page, or
 * two sequences appending to one key/value page, race with each other).  Query head h reads key head
 * h / (Hq / Hkv).  Rows past a sequence's length are never used, whatever
 * they hold, nor are table entries past its last page.
 *
 * The tables and seq_lens are device data that the kernels check: a length
 * that is negative or longer than the table (or max_len), or a page id outside
 * the pool, records DA_ERR_INVALID in the workspace's status word; nothing
 * outside the pools is read or written, an append skips that token, and a
 * decode step's results for that sequence are unspecified.  page_size is 16, 32,
 * 64, 128 or 256; Hq is a multiple of Hkv; d 64 or 128; pools and out 16-byte
 * aligned.
 *
 * Unlike the calls above, the paged calls leave the status word alone unless
 * they record an error: the caller zeroes the first 256 bytes of a workspace
 * once before its first use (and again after DA_ERR_TIMEOUT), and
 * dilution_attn_get_error reads and clears the first error recorded since.  A
 * decode step overwrites the rest of its workspace: calls that may overlap on
 * the GPU need workspaces of their own.  At most 2^14 heads and 2^24 sequences x
 * query heads, and for a decode step 2^31 - 1 pages x key heads and 2^32 - 1 runs
 * of 16 rows in the demand pool (DA_ERR_UNSUPPORTED beyond).
 * ---------------------------------------------------------------------- */
typedef struct dilution_attn_paged_cache {
  void *k_pages, *v_pages;               /* DEVICE, dtype */
  float *demand_pages;                   /* DEVICE */
  const int32_t *page_table;             /* DEVICE [S][max_pages] */
  const int32_t *demand_table;           /* DEVICE [S][max_pages] */
  const int32_t *seq_lens;               /* DEVICE [S] */
  int32_t S, Hq, Hkv, d, page_size, num_pages, num_demand_pages, max_pages, dtype;
} dilution_attn_paged_cache;

/* Appends new tokens: sequence s receives tokens cu_tokens[s] ..
 * cu_tokens[s+1] - 1 of the N given, as its LAST tokens; cache->seq_lens
 * already counts them.  For each token
 *   - its key, turned by its position, goes to its row of k_pages, its value
 *     unchanged to v_pages;
 *   - its demand becomes demand[n][h] (a prompt's demand_out after prefill),
 *     or 0 where demand is NULL (a token about to be decoded);
 *   - q (nullable), turned likewise, goes to q_out [N,Hq,d] contiguous.
 * q [N,Hq,d], k, v [N,Hkv,d]: *_strides are HOST arrays of two element strides
 * (token, head) or NULL for contiguous; demand fp32 [N,Hq] likewise.
 * cu_tokens: DEVICE [S+1] int32, starting at 0 and not decreasing; tokens from
 * cu_tokens[S] on are padding: their values are not used, their rows of q_out
 * not written.  q_out may be q itself (then contiguous); a q_out that lies over
 * rows of q, k, v or demand in any other way is DA_ERR_INVALID.
 * spec: NULL appends k and q unrotated.  positions: DEVICE [n_axes][N], or NULL
 * for the token's place in its sequence on every axis.
 * workspace: 256 bytes (dilution_attn_paged_append_workspace_size()). */
size_t dilution_attn_paged_append_workspace_size(void);

int dilution_attn_paged_append(const void *q, const int64_t *q_strides, const void *k, const int64_t *k_strides,
                               const void *v, const int64_t *v_strides, const float *demand,
                               const int64_t *demand_strides, void *q_out, const int32_t *cu_tokens, int N,
                               const dilution_attn_paged_cache *cache, const dilution_attn_rope_spec *spec,
                               const int32_t *positions, void *workspace, size_t workspace_bytes, void *stream);

/* One decode step of every sequence over the paged cache (the operator of
 * dilution_attn_decode_step; the new token has been appended, with demand 0):
 * q, out [S,Hq,d]; sequence s sees its seq_lens[s] keys, out is formed as in
 * steps 2-4 there and the demand of every key it sees grows by its bid.  A
 * sequence of length 0 (an idle slot) gets zeros and changes nothing.
 *
 * prefix_table (nullable): DEVICE [n_prefix_pages] page ids.  The first
 * n_prefix_pages * page_size tokens of EVERY sequence then live in those
 * pages, whose keys and values are read for 8 to 64 rows (sequence, query head)
 * of a key head at a time; short calls read them for every sequence, from L2 (the
 * first n_prefix_pages entries of each page_table row are not read).  Each
 * sequence keeps its own demand over them.  A length below the prefix's, other than 0,
 * records DA_ERR_INVALID.  The result is that of the same call with the
 * prefix's pages in every page_table row.
 *
 * max_len: host upper bound of seq_lens (at most max_pages * page_size); sizes
 * the workspace and the launch, and short bf16 calls (max_len up to 2048 at
 * d = 64, 1024 at d = 128, few sequences) run as one kernel.  The workspace's
 * size depends on whether there is a prefix, not on its length.  tau_bh: nullable device [S*Hq], index
 * s*Hq + h.  tau, eps, flags (DA_FLAG_EARLIER_DEMAND_ONLY) as for
 * dilution_attn_decode_step_ex; DA_BF16 needs eps >= 1e-18 as the forward.
 * Repeated calls give equal bits.  Errors as for dilution_attn_decode_step_ex.
 * DA_BF16: products of bf16 operands summed in fp32; the shares enter the value
 * product as two bf16 terms (2^-16 relative), exponentials and reciprocals are
 * the approximate instructions: besides the logits' own rounding, out is within
 * 2^-14 max |v| of the formula before its rounding to bf16.
 *
 * dilution_attn_paged_decode_ex records what the kernels find in `status` (DEVICE,
 * 256 bytes, 256-byte aligned, zeroed once by the caller) instead of the
 * workspace's first 256 bytes: for workspaces that do not outlive the call.
 * Calls that overlap on the GPU may share a status block. */
size_t dilution_attn_paged_decode_workspace_size(int S, int Hq, int Hkv, int d, int max_len, int n_prefix_pages,
                                                 int page_size, int dtype);

int dilution_attn_paged_decode(const void *q, const dilution_attn_paged_cache *cache, const int32_t *prefix_table,
                               int n_prefix_pages, int max_len, void *out, float tau, const float *tau_bh,
                               float eps, int flags, void *workspace, size_t workspace_bytes, void *stream);

int dilution_attn_paged_decode_ex(const void *q, const dilution_attn_paged_cache *cache, const int32_t *prefix_table,
                                  int n_prefix_pages, int max_len, void *out, float tau, const float *tau_bh,
                                  float eps, int flags, void *workspace, size_t workspace_bytes, void *status,
                                  void *stream);

/* Chunks of new tokens over the paged cache: several decode steps of every
 * sequence at once, for drafted tokens to be verified, for parts of long
 * prompts, and for whole prompts of different lengths packed one behind the
 * other.  Sequence s has n = cu_tokens[s+1] - cu_tokens[s] queries: its LAST n
 * tokens, which have been appended (with demand 0; seq_lens counts them).  For
 * query i of them, at place P + i with P = seq_lens[s] - n, over the keys
 * t <= P + i:
 *     p_t = softmax_t(tau q.k_t / sqrt(d)),   total_t += p_t,
 *     share_t = p_t / (total_t + eps),        out = sum share_t v_t / sum share_t,
 * query after query, where total_t begins as what the key's demand page holds and
 * goes back there after the last query.  (DA_FLAG_EARLIER_DEMAND_ONLY: the total
 * before p_t.)  That is n calls of dilution_attn_paged_decode, a token longer each
 * time; n = seq_lens[s] with demand 0 is dilution_attn_fwd of the prompt.
 * q, out [N,Hq,d] contiguous; out may be q.  cu_tokens: DEVICE [S+1] int32 as for
 * dilution_attn_paged_append; rows of q from cu_tokens[S] on are padding: not read,
 * and their rows of out not written.  A sequence without new tokens is left as it is.
 * max_new, max_len: host upper bounds of the sequences' new tokens and of seq_lens
 * (max_len at most max_pages * page_size and 2^30).  A sequence with more new tokens than
 * max_new or than its length, a length outside 0 .. max_len, cu_tokens that decrease
 * or pass N record DA_ERR_INVALID; such a sequence's rows of out are not written and
 * its demand stays.  A page id outside the pool records it too, and the sequence's
 * results are unspecified.
 * What is not finite in a new token's value reaches the outputs of the queries that see
 * the token, and no others; a NaN in a query or key its outputs, the totals of the keys
 * that its query sees, and through them the sequence's later queries (of that head).
 * tau_bh: nullable device [S*Hq], index s*Hq + h.  tau, eps, flags as for
 * dilution_attn_paged_decode.  status: DEVICE, 256 bytes, 256-byte aligned, zeroed
 * once by the caller, or NULL for the workspace's first 256 bytes.  The workspace is
 * overwritten from byte 256 on: calls that may overlap on the GPU need workspaces
 * of their own.  One that was sized for some N, max_new and max_len serves every call
 * of this cache within them.  It holds about 4 (d + 7) bytes for each query head of the
 * new tokens, and as much for each row of the longest sequence's in each of 152 CTAs
 * (DA_F32: 304, with few rows 456), in both of up to 8192 tokens of a sequence (longer
 * parts go by slices of those); and, in DA_BF16, the logits of up to d / 8 new tokens times
 * query heads a key head, up to 2 GB.  One prompt of any length from 8192 tokens on, 12
 * query heads, d = 128: 0.73 GB beside those logits, DA_F32 1.39 GB.  Pages that sequences
 * share are read for each of them.  Repeated calls give equal bits.  Errors as for
 * dilution_attn_paged_decode_ex.
 * DA_BF16: products, exponentials and reciprocals as in dilution_attn_paged_decode.  The
 * shares enter the value product as two bf16 terms (2^-16 relative), as there, for
 * sequences with up to 4 new tokens, also beside long parts, and for those with up to 64
 * rows a key head (the new tokens rounded up to 8, for each of its query heads); in larger
 * parts they are rounded to bf16 once, as in dilution_attn_fwd, which moves out by at
 * most 2^-8 of the values' mean distance from it. */
size_t dilution_attn_paged_chunk_workspace_size(int S, int Hq, int Hkv, int d, int N, int max_new, int max_len, int dtype);

int dilution_attn_paged_chunk(const void *q, const dilution_attn_paged_cache *cache, const int32_t *cu_tokens, int N,
                              int max_new, int max_len, void *out, float tau, const float *tau_bh, float eps, int flags,
                              void *workspace, size_t workspace_bytes, void *status, void *stream);

/* Eviction: the cache keeps the tokens that have received the most attention.
 * Sequence s keeps m = min(seq_lens[s], keep[s]) tokens of each key head: those with
 * the highest score, equal scores by the lower place.  A token's score is the sum
 * of the totals of the key head's query heads, added in fp32 in the heads' order;
 * the first `sinks` and the last `recent` tokens, and those whose score is NaN,
 * score +infinity.  The tokens that stay keep their order and become rows
 * 0 .. m - 1 (keys, values and totals move together, bit for bit), so that after
 * an eviction one row holds different tokens in different key heads: keys carry
 * their rotation, and later tokens need their positions passed to
 * dilution_attn_paged_append.  In place every row behind the first that goes moves, so
 * that one token costs about what many do (64 sequences of 4097 tokens, 4 key heads,
 * d = 128: 112 us for one token of each; a decode step reads all of them in about 80):
 * a serving loop lets sequences grow by some tokens between evictions.
 *   dst_page_table, dst_demand_table: both NULL: in place (pages that sequences share
 *       then hold only tokens that every key head of theirs keeps, as below).  Otherwise DEVICE
 *       [S][dst_max_pages] tables of the same pools, dst_max_pages * page_size at
 *       least min(max_keep, max_len), that receive the rows that stay, of
 *       sequences that lose nothing too.  A page named there is one that the call does
 *       not read, or the source's at the same place of the same sequence where every
 *       key head keeps all tokens of that page and before it (a prefix of at most
 *       `sinks` tokens, which sequences may share): only rows whose place changes are
 *       written.
 *   keep: DEVICE [S] int32.  max_keep, max_len: host upper bounds of m and of
 *       seq_lens (max_len at most max_pages * page_size and 2^30).
 *   new_lens: DEVICE [S] int32, receives m; may be cache->seq_lens itself.
 *   kept: nullable DEVICE [S][Hkv][max_keep] int32, receives the places that the
 *       rows had, then -1.
 * A length outside 0 .. max_len, a negative keep[s] or m > max_keep records
 * DA_ERR_INVALID; the sequence is left as it is, new_lens[s] is its length, kept all
 * -1.  A page id outside the pool records it too; its rows stay where they are, and
 * which tokens the sequence keeps is unspecified.
 * status and workspace as for dilution_attn_paged_chunk.  Repeated calls on equal
 * contents give equal bits. */
size_t dilution_attn_paged_evict_workspace_size(int S, int Hkv, int max_keep, int max_len);

int dilution_attn_paged_evict(const dilution_attn_paged_cache *cache, const int32_t *dst_page_table,
                              const int32_t *dst_demand_table, int dst_max_pages, const int32_t *keep, int max_keep,
                              int max_len, int sinks, int recent, int32_t *new_lens, int32_t *kept, void *workspace,
                              size_t workspace_bytes, void *status, void *stream);

/* ------------------------------------------------------------------------
 * Synchronises `stream`, reads the status word that kernels of the last call
 * on `workspace` may have set, clears it and returns it (DA_OK if none).
 * Returns DA_ERR_CUDA if the synchronisation or the copy fails.
 * ---------------------------------------------------------------------- */
int dilution_attn_get_error(void *workspace, void *stream);

/* Copies the workspace's 4-word status block to host `out` after a device
 * synchronisation: [0] status, and when a bounded wait timed out, [1] the
 * shared-memory offset of the mbarrier it waited on, [2] the block index,
 * [3] the thread index of the first wait that gave up.  Diagnostic only. */
int dilution_attn_debug_last_timeout(void *workspace, int32_t *out);

/* ------------------------------------------------------------------------
 * Test hook of the bounded waits (diagnostic only; no counterpart on the
 * pages).  Runs one decode step like dilution_attn_decode_step (same
 * arguments, tau_bh = NULL, flags = 0), except that
 *   - in the first kernel's block for key chunk `stall_chunk` (2048 keys per
 *     chunk) of head stall_bh (= b*H + h), one consumer warp keeps the first
 *     ring stage it read instead of handing it back, so the block's copy
 *     producer waits for a shared-memory slot that is never freed (the chunk
 *     needs at least three 256-key stages of cached keys before n_ctx);
 *   - every wait of that kernel gives up after wait_limit_ns (1e3 .. 1e9 ns).
 * The waits that run out record DA_ERR_TIMEOUT and their place
 * (dilution_attn_debug_last_timeout: status, barrier offset, block index =
 * stall_chunk, thread index) in the workspace status word; the blocks that
 * gave up finish without waiting further, so the call completes and the
 * device stays usable.  The step's outputs, the appended cache row and the
 * demand are then unspecified.  Errors: those of dilution_attn_decode_step,
 * and DA_ERR_INVALID for a wait_limit_ns outside the range, a negative
 * stall_chunk or a stall_bh outside [0, B*H).
 * ---------------------------------------------------------------------- */
int dilution_attn_debug_decode_stall(const void *q_new, const void *k_new, const void *v_new,
                                     void *k_cache, void *v_cache, float *demand,
                                     int n_ctx, int T_cap, void *out,
                                     int B, int H, int d, float tau, float eps, int dtype,
                                     void *workspace, size_t workspace_bytes, void *stream,
                                     int stall_chunk, int stall_bh, long long wait_limit_ns);

/* The same for the paged step: one decode step like dilution_attn_paged_decode
 * (tau_bh = NULL, flags = 0), except that in block `stall_block` of kernel
 * `stall_kernel` (0: logits, 1: shares of the streaming kernels; 2, 3: those of
 * a prefix with many rows) one warp keeps the first ring stage it read (3: the
 * first table of demand pages is not handed over), and every wait of that kernel
 * gives up after wait_limit_ns (1e3 .. 1e9 ns; kernel 3: after the ordinary 1 s,
 * as it has no register left for the limit).  It has an effect where the call runs
 * that kernel and the block has more tiles than ring stages (8).  The waits that
 * run out record as above; the call completes, the device stays usable, out and
 * the demand are unspecified, and the workspace's first 256 bytes have to be
 * zeroed again.  Errors: those of dilution_attn_paged_decode, and DA_ERR_INVALID
 * for a stall_kernel outside 0 .. 3, a negative stall_block or a wait_limit_ns
 * outside the range. */
int dilution_attn_debug_paged_decode_stall(const void *q, const dilution_attn_paged_cache *cache,
                                           const int32_t *prefix_table, int n_prefix_pages, int max_len, void *out,
                                           float tau, float eps, void *workspace, size_t workspace_bytes, void *stream,
                                           int stall_kernel, int stall_block, long long wait_limit_ns);

/* ------------------------------------------------------------------------
 * Host-only introspection of integer artefacts (no GPU needed).
 *
 * dilution_attn_debug_tile_schedule: the work order of the bf16 forward's and
 * backward's kernels for a problem of BH = B*H heads and T tokens.  kernel = 0 (row
 * statistics at d = 64: pairs of 128-row query tiles, heads in groups of
 * about 96 MB of Q and K), 1 (demand sweep at d = 64: 128-row query tiles,
 * 384-key spans), 2 (demand sweep at d = 128: 256-key spans), 3 (row
 * statistics at d = 128), or 4 + 2 * pass + (d == 128) for the tensor-core
 * backward's passes (pass 0: reverse pass, 1: light dK pass, one CTA per
 * 128-key tile; 2: dQ pass, one CTA per 128-query tile).  For each CTA index
 * c (in launch order), writes 4 int32 to out[4c..4c+3]: head index, first
 * query tile, number of query tiles (row stats: the query tiles it owns;
 * sweep and key-tile passes: the query tiles it walks, from its diagonal; dQ
 * pass: 1, its own), first key (sweep and key-tile passes) or 0.  Returns the number of CTAs; if cap (in
 * int32 elements) is too small, writes nothing and returns -(needed).
 *
 * dilution_attn_debug_tile_mask: the causal mask the kernels apply to the
 * 128 x 128 tile (query tile qt, key tile kt) of a T-token head: out[r*128+c]
 * = 1 if query qt*128+r may see key kt*128+c (key <= query < T), else 0.
 * ---------------------------------------------------------------------- */
int dilution_attn_debug_tile_schedule(int BH, int T, int kernel, int32_t *out, size_t cap);
int dilution_attn_debug_tile_mask(int T, int qt, int kt, uint8_t *out);

#ifdef __cplusplus
}
#endif

#endif /* DILUTION_ATTN_H */
