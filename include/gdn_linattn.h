/*
 * gdn_linattn.h: C ABI of linear attention with a decay for each head, beside the gated delta
 * rule of gdn.h (same conventions: layouts, ownership, asynchrony, errors, debug mode).
 *
 *     S_t = exp(g_t) S_{t-1} + k_t v_t^T,    o_t = scale * S_t^T q_t
 *
 * per head h of every packed sequence n, with the d x d state S reset at every sequence start to
 * that sequence's initial state (or zero).  It is the gated delta rule without the correction
 * along k_t; no passage of the pages applies to it.  The forward and backward work in 64-token
 * chunks (decays summed within a chunk, one masked 64 x 64 product, the state from chunk to chunk)
 * and split long sequences exactly: the state is linear in its start, so units of a sequence are
 * summed from zero side by side, joined, and run again from their true starts.
 *
 * Layouts, types and the initial and final states are those of gdn.h (q, k [T, Hk, d]; v, o
 * [T, H, d]; h0, ht fp32), with
 *   g     fp32 log decays: [T, H], one for each token and head, or [H] with head_decay = 1 (a
 *         constant decay per head).  g <= 0 in use; -inf empties the state.  Values that are
 *         finite but whose decay is zero in fp32 act as -inf and get a zero gradient.
 * Sums and states are fp32.  With bf16 inputs, what is not an input and enters a product (states,
 * decayed rows, the masked products of a chunk) does so as a sum of bf16 terms: to 2^-16 of each
 * element at least, to 2^-24 where the result stays fp32, whatever the units' length.  bf16 outputs
 * are rounded once.  dg_t is a difference of sums over its unit: its error is absolute, fp32's
 * rounding of the unit's |q_s . dq_s| and |k_s . dk_s|, not relative to a small dg_t.
 * Inputs are finite: a NaN or infinity in a token's k or v reaches the outputs of its own 64-token
 * chunk (also those before it) and of what follows in its sequence and head; no other sequence or
 * head.
 */
#ifndef GDN_LINATTN_H_
#define GDN_LINATTN_H_

#include "gdn.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct gdn_linattn_problem {
  int64_t total_tokens;  /* T = cu_seqlens[N] (>= 0) */
  int32_t num_seqs;      /* N >= 1 */
  int32_t num_heads;     /* H >= 1: heads of v, o, g and of the state */
  int32_t num_k_heads;   /* heads of q and k: 0 (= num_heads) or a divisor of num_heads; value head h
                          * reads key head h / (num_heads / num_k_heads) */
  int32_t head_dim;      /* 64 or 128 (d_k = d_v) */
  int32_t dtype;         /* GDN_DTYPE_* of q, k, v, o and their gradients */
  int32_t head_decay;    /* 0: g is [T, H]; 1: g is [H] */
  int32_t seg_chunks;    /* length in chunks of the units that sequences are split into; 0 = chosen
                          * from T, N and H, so by the sequences' mean length: set it (8 or so) for
                          * one long sequence among many short ones, which else is not split */
  int32_t num_slots;     /* workgroups that the choice plans for; 0 = the device's */
  float scale;           /* o_t = scale * S_t^T q_t */
  int32_t reserved;      /* must be 0 */
  int64_t h0_seq_stride; /* elements between consecutive sequences' h0; 0 = broadcast */
} gdn_linattn_problem;

/* Bytes of device workspace for the two calls below.  Host only; num_slots = 0 may query the
 * current device. */
gdn_status gdn_linattn_fwd_workspace_size(const gdn_linattn_problem *p, size_t *bytes);
gdn_status gdn_linattn_bwd_workspace_size(const gdn_linattn_problem *p, size_t *bytes);

/* Forward.  h0 may be NULL (zero initial states) and ht may be NULL (final states not written).
 * o and ht must not overlap an input. */
gdn_status gdn_linattn_fwd(const gdn_linattn_problem *p, const void *q, const void *k,
                           const void *v, const float *g, const int32_t *cu_seqlens,
                           const float *h0, void *o, float *ht, void *workspace,
                           size_t workspace_bytes, hipStream_t stream);

/* Backward: given dout [T, H, d] and optionally dht [N, H, d, d] fp32 (NULL = zero), writes dq,
 * dk [T, Hk, d] (sums over each key head's value heads) and dv [T, H, d] in dtype, dg in fp32
 * ([T, H], or [H] summed over all tokens with head_decay) and, unless NULL, dh0 (fp32, per sequence,
 * or one [H, d, d] summed over the sequences when h0_seq_stride is 0).  Outputs must not overlap
 * an input.  The states are recomputed, not stored by the forward. */
gdn_status gdn_linattn_bwd(const gdn_linattn_problem *p, const void *q, const void *k,
                           const void *v, const float *g, const int32_t *cu_seqlens,
                           const float *h0, const void *dout, const float *dht, void *dq, void *dk,
                           void *dv, float *dg, float *dh0, void *workspace,
                           size_t workspace_bytes, hipStream_t stream);

/* One token for each of `batch` rows: S <- exp(g) S + k v^T, o = scale S^T q, in place.  q, k
 * [batch, Hk, d], v, o [batch, H, d]; g [batch, H] or [H] (head_decay); state fp32.
 *   pages == NULL: state is [batch, H, d, d], row b's state is state[b] (num_pages is not used).
 *   pages: device int32 [batch]; state is a pool [num_pages, H, d, d] and row b's state is
 *     state[pages[b]].  -1 marks a row without a sequence (padding): its o is zero.  A page
 *     outside the pool, or one that an earlier row has (at most 2^16 rows), is treated as -1 and sets a fault flag
 *     (gdn_device_faults bits 2 and 4; in debug mode the call returns GDN_ERR_DEVICE_CHECK). */
gdn_status gdn_linattn_step(int32_t batch, int32_t num_heads, int32_t num_k_heads,
                            int32_t head_dim, int32_t dtype, int32_t head_decay, float scale,
                            const void *q, const void *k, const void *v, const float *g,
                            const int32_t *pages, int32_t num_pages, float *state, void *o,
                            hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* GDN_LINATTN_H_ */
