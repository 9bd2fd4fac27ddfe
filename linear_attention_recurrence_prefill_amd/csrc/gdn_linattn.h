// Internal interface of linear attention with a decay for each head (gdn_linattn.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace gdn {

// One linear-attention pass over all (unit, head) pairs: with x, y, z the query-, key- and
// value-like rows of the pass,
//   forward in time   out_t = s_out (e^{G_t} S^T x_t + sum_{i <= t} e^{G_t - G_i} (x_t . y_i) z_i)
//   backward in time  out_i = e^{G_C - G_i} R^T x_i + s_in sum_{t >= i} e^{G_t - G_i} (x_i . y_t) z_t
// per 64-token chunk, with the state carried from chunk to chunk.  The four output passes and the
// two that only sum a unit's state are the same kernel with other rows:
//   kLinFwd    x = q,  y = k,  z = v     out = o, final state = ht
//   kLinDq     x = do, y = v,  z = k     out = dq (state transposed), and dg's parts that need S
//   kLinDv     x = k,  y = q,  z = do    backward in time: out = dv, final state = dh0
//   kLinDk     x = v,  y = do, z = q     backward in time: out = dk (state transposed), k . dk
//   kLinSumFwd y = k,  z = v             the unit's state from zero
//   kLinSumRev y = q,  z = do            the same backward in time
enum LinPass { kLinFwd = 0, kLinDq, kLinDv, kLinDk, kLinSumFwd, kLinSumRev };

struct LinArgs {
  const void *q, *k, *v, *dout;
  const float *g;        // log decays: [T, H] or, with g_head, [H]
  int32_t g_head;
  const int32_t *cu;
  const float *h0;       // initial states, or null
  int64_t h0_stride;
  const float *dht;      // gradients of the final states [N, H, D, D], or null
  void *o, *dq, *dk, *dv;
  int32_t grad_f32;      // dq, dk as fp32 per value head [T, H, D] (grouped heads)
  float *ht, *dh0;       // per sequence [N, H, D, D], or null
  // split runs (L > 0): per unit and head, the states at the unit's start (unit_s) and the state
  // gradients at its end (unit_r), [units, H, D, D]; before the scan they hold the unit's own
  // contribution, with its whole decay in unit_decay ([2, units, H]: forward and reversed sums)
  float *unit_s, *unit_r, *unit_decay;
  int32_t *seq_unit;     // [N]: each sequence's first unit
  // dg's parts: pairs within a chunk, q . dq and k . dk of the states' shares, [H, T] each, and
  // <state, state gradient> at each unit's end, [units, H]
  float *dg_pairs, *dg_q, *dg_k, *unit_dot;
  double *dg_unit;       // with g_head: dg summed over each unit, [units, H]
  float *dg;             // [T, H], or [H] with g_head
  int64_t T;
  int32_t N, H, HK, L;
  int64_t units;
  // whole sequences (L = 0), at most kMaxLongestFirst: taken longest first, all heads of one before
  // the next, so that the last workgroups to start are the shortest
  int32_t longest_first;
  int32_t cus;           // of the device
  float scale;
};

// Workgroups of four waves that one CU holds at once (registers and LDS), which the units' length is
// planned for.  Launches differ: one of eight waves where there are no more workgroups than CUs and in
// fp32 with d = 128, three in the forward's sums with d = 128.
inline int linattn_blocks_per_cu(int D, bool bf16) { return bf16 || D == 64 ? 2 : 1; }
// The forward: the units' sums and the states at their starts (split runs), then the output.
hipError_t launch_linattn_fwd(const LinArgs &a, int D, bool bf16, hipStream_t stream);
// The backward: the same in both directions, dq, dk, dv and dg's parts, then dg.
hipError_t launch_linattn_bwd(const LinArgs &a, int D, bool bf16, hipStream_t stream);
// dq[t, hk] = sum over the H / HK value heads of a.dq[t, h] (fp32) for the tokens t of a's sequences,
// to the input type, and dk likewise.
hipError_t launch_linattn_group_sum(const LinArgs &a, int D, bool bf16, void *dq, void *dk,
                                    hipStream_t stream);
hipError_t launch_linattn_zero(float *x, int64_t n, hipStream_t stream);

// One token per row of a batch, on states in a batch or in the pages of a pool.
struct LinStepArgs {
  const void *q, *k, *v;
  const float *g;
  int32_t g_head;
  const int32_t *pages;  // [B] page of each row, -1 = no sequence; null: row b's state is state[b]
  int32_t num_pages;
  float *state;
  void *o;
  uint32_t *faults;
  int32_t B, H, HK;
  float scale;
};
hipError_t launch_linattn_step(const LinStepArgs &a, int D, bool bf16, hipStream_t stream);

}  // namespace gdn
