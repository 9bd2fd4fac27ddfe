// C ABI of linear attention with a decay for each head and of the operators on a pool's pages:
// argument validation, workspace layout and launches.  Declarations: include/gdn_linattn.h,
// include/gdn_pages.h.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>

#include "../../include/gdn_linattn.h"
#include "../../include/gdn_pages.h"
#include "gdn_api_util.h"
#include "gdn_internal.h"
#include "gdn_linattn.h"
#include "gdn_pages.h"

using namespace gdn::api;

namespace {

// Workgroups of at most 512 threads along a grid's first dimension stay below 2^32 threads.
constexpr int64_t kMaxUnits = (int64_t)1 << 23;
// Rows of a step on pages: each looks for its page in the rows before it (2^16 rows: 256 loads per
// thread).
constexpr int32_t kMaxPagedRows = 1 << 16;

gdn_status check_problem(const gdn_linattn_problem *p) {
  if (!p) return fail(GDN_ERR_NULL_ARG, "problem is NULL");
  if (p->total_tokens < 0 || p->total_tokens > INT32_MAX - gdn::kChunk)
    return fail(GDN_ERR_BAD_SHAPE, "total_tokens %lld out of range", (long long)p->total_tokens);
  if (p->num_seqs < 1) return fail(GDN_ERR_BAD_SHAPE, "num_seqs must be >= 1");
  if (p->num_heads < 1 || p->num_heads > 65535)
    return fail(GDN_ERR_BAD_SHAPE, "num_heads must be in [1, 65535]");
  if (p->num_k_heads < 0 || p->num_k_heads > p->num_heads ||
      (p->num_k_heads > 0 && p->num_heads % p->num_k_heads != 0))
    return fail(GDN_ERR_BAD_SHAPE, "num_k_heads must be 0 or a divisor of num_heads");
  if (p->head_dim != 64 && p->head_dim != 128)
    return fail(GDN_ERR_BAD_SHAPE, "head_dim must be 64 or 128");
  if (p->dtype != GDN_DTYPE_F32 && p->dtype != GDN_DTYPE_BF16)
    return fail(GDN_ERR_BAD_DTYPE, "dtype %d", p->dtype);
  if (p->head_decay != 0 && p->head_decay != 1)
    return fail(GDN_ERR_BAD_MODE, "head_decay must be 0 or 1");
  if (p->seg_chunks < 0 || p->num_slots < 0)
    return fail(GDN_ERR_BAD_SHAPE, "seg_chunks / num_slots out of range");
  if (p->reserved != 0) return fail(GDN_ERR_BAD_SHAPE, "reserved must be 0");
  if (p->h0_seq_stride < 0) return fail(GDN_ERR_BAD_SHAPE, "h0_seq_stride must be >= 0");
  if (!std::isfinite(p->scale)) return fail(GDN_ERR_BAD_SHAPE, "scale must be finite");
  return GDN_OK;
}

int32_t k_heads(const gdn_linattn_problem *p) {
  return p->num_k_heads > 0 ? p->num_k_heads : p->num_heads;
}

// Length in chunks of the units that sequences are split into (0: one unit per sequence).  A unit's
// chunks are a chain, run twice; each unit costs its state, written, joined and read.  The sum is
// least at a length proportional to sqrt(chunks x heads / slots), the latency model of "How to Speed
// Up GDN Kernels for Qwen Models", section "Lever 1"; the factors are fitted to sweeps of the length
// (bf16, d = 128: best at 1, 2, 5, 9, 16 chunks for 64, 256, 1024, 4096, 8192 chunks x heads, where the
// rule takes 1, 2, 5, 9, 17).  fp32's products are sixteen times dearer, so its chains are cut
// shorter.  Sequences that fill the slots by themselves, or are no longer than a unit, stay whole;
// the host knows their mean length only, so one long sequence among many short ones stays whole too
// (the caller can set seg_chunks).
gdn_status segment_chunks(const gdn_linattn_problem *p, int32_t *L) {
  *L = p->seg_chunks;
  if (*L > 0) return GDN_OK;
  int slots = p->num_slots;
  if (slots == 0) {
    gdn_status s = device_info(&slots);
    if (s != GDN_OK) return s;
    slots *= gdn::linattn_blocks_per_cu(p->head_dim, p->dtype == GDN_DTYPE_BF16);
  }
  const int64_t nc = ceil_div(p->total_tokens, gdn::kChunk);
  const double factor = p->dtype == GDN_DTYPE_BF16 ? 3.5 : 1.8;
  const double want = std::max(1.0, std::round(factor * std::sqrt((double)nc * p->num_heads / slots)));
  if ((int64_t)p->num_seqs * p->num_heads >= 2 * (int64_t)slots || nc <= want * p->num_seqs) return GDN_OK;
  // Units that nearly fill the slots a whole number of times are made to do so (32K tokens x 8 heads:
  // 9 chunks and 129 us instead of 10 and 135; 65K tokens, backward: 17 chunks and 663 us instead of 14
  // and 685): the last of a sequence is on average half a unit.
  const double partial = 0.5 * p->num_seqs;
  const double rounds = std::round((nc / want + partial) * p->num_heads / slots);
  const double units = rounds * slots / p->num_heads - partial;
  const double fit = units >= 1.0 ? std::ceil(nc / units) : want;
  *L = (int32_t)std::min<double>(fit, INT32_MAX);
  return GDN_OK;
}

struct Layout {
  int32_t L = 0;
  int64_t units = 0;
  size_t unit_s = 0, unit_r = 0, decay = 0, seq_unit = 0;  // split
  size_t dg_pairs = 0, dg_q = 0, dg_k = 0, unit_dot = 0, dg_unit = 0;
  size_t dq_part = 0, dk_part = 0, dh0_seq = 0;
  size_t total = 0;
};

gdn_status layout(const gdn_linattn_problem *p, bool bwd, Layout *l) {
  gdn_status s = segment_chunks(p, &l->L);
  if (s != GDN_OK) return s;
  const int64_t T = p->total_tokens, N = p->num_seqs, H = p->num_heads, D = p->head_dim;
  l->units = l->L > 0 ? ceil_div(ceil_div(T, gdn::kChunk) + N, l->L) + N : N;
  if (l->units >= kMaxUnits) return fail(GDN_ERR_BAD_SHAPE, "too many work units");
  size_t at = 0;
  const auto take = [&](size_t bytes) {
    const size_t here = at;
    at += align_up(bytes);
    return here;
  };
  if (T > 0) {
    if (l->L > 0) {
      l->unit_s = take((size_t)l->units * H * D * D * 4);
      if (bwd) l->unit_r = take((size_t)l->units * H * D * D * 4);
      l->decay = take((size_t)l->units * H * 2 * 4);
      l->seq_unit = take((size_t)N * 4);
    }
    if (bwd) {
      l->dg_pairs = take((size_t)T * H * 4);
      l->dg_q = take((size_t)T * H * 4);
      l->dg_k = take((size_t)T * H * 4);
      l->unit_dot = take((size_t)l->units * H * 4);
      if (p->head_decay) l->dg_unit = take((size_t)l->units * H * 8);
      if (k_heads(p) != H) {
        l->dq_part = take((size_t)T * H * D * 4);
        l->dk_part = take((size_t)T * H * D * 4);
      }
      if (p->h0_seq_stride == 0) l->dh0_seq = take((size_t)N * H * D * D * 4);
    }
  }
  l->total = at;
  return GDN_OK;
}

gdn::LinArgs base_args(const gdn_linattn_problem *p, const Layout &l, int cus, const void *q, const void *k,
                       const void *v, const float *g, const int32_t *cu, const float *h0, char *ws) {
  gdn::LinArgs a{};
  a.q = q;
  a.k = k;
  a.v = v;
  a.g = g;
  a.g_head = p->head_decay;
  a.cu = cu;
  a.h0 = h0;
  a.h0_stride = p->h0_seq_stride;
  a.T = p->total_tokens;
  a.N = p->num_seqs;
  a.H = p->num_heads;
  a.HK = k_heads(p);
  a.L = l.L;
  a.units = l.units;
  a.longest_first = l.L == 0 && p->num_seqs > 1 && p->num_seqs <= gdn::kMaxLongestFirst;
  a.cus = cus;
  a.scale = p->scale;
  if (l.L > 0) {
    a.unit_s = reinterpret_cast<float *>(ws + l.unit_s);
    a.unit_decay = reinterpret_cast<float *>(ws + l.decay);
    a.seq_unit = reinterpret_cast<int32_t *>(ws + l.seq_unit);
  }
  return a;
}

gdn_status check_all(const char *what, std::initializer_list<const void *> required,
                     std::initializer_list<const void *> aligned) {
  for (const void *x : required)
    if (!x) return fail(GDN_ERR_NULL_ARG, "%s are required", what);
  for (const void *x : aligned)
    if (!aligned16(x)) return fail(GDN_ERR_BAD_ALIGNMENT, "tensor pointers must be 16-byte aligned");
  return GDN_OK;
}

gdn_status after(hipStream_t stream) { return debug_on() ? debug_faults(stream) : GDN_OK; }

// The fault flags hold what earlier calls set: in debug mode a call reports only its own.
gdn_status clear_faults_for_debug(hipStream_t stream) {
  if (!debug_on()) return GDN_OK;
  uint32_t *w = fault_word();
  if (!w) return fail(GDN_ERR_HIP, "debug mode: check words");
  const uint32_t zero = 0;
  hipError_t e = hipMemcpyAsync(w, &zero, sizeof(zero), hipMemcpyHostToDevice, stream);
  if (e == hipSuccess) e = hipStreamSynchronize(stream);
  return e == hipSuccess ? GDN_OK : hip_fail(e, "debug mode: fault flags");
}

}  // namespace

#define LAUNCH(call, what)                         \
  do {                                             \
    const hipError_t e_ = (call);                  \
    if (e_ != hipSuccess) return hip_fail(e_, what); \
  } while (0)

extern "C" {

gdn_status gdn_linattn_fwd_workspace_size(const gdn_linattn_problem *p, size_t *bytes) {
  gdn_status s = check_problem(p);
  if (s != GDN_OK) return s;
  if (!bytes) return fail(GDN_ERR_NULL_ARG, "bytes is NULL");
  Layout l;
  s = layout(p, false, &l);
  if (s == GDN_OK) *bytes = l.total;
  return s;
}

gdn_status gdn_linattn_bwd_workspace_size(const gdn_linattn_problem *p, size_t *bytes) {
  gdn_status s = check_problem(p);
  if (s != GDN_OK) return s;
  if (!bytes) return fail(GDN_ERR_NULL_ARG, "bytes is NULL");
  Layout l;
  s = layout(p, true, &l);
  if (s == GDN_OK) *bytes = l.total;
  return s;
}

gdn_status gdn_linattn_fwd(const gdn_linattn_problem *p, const void *q, const void *k,
                           const void *v, const float *g, const int32_t *cu_seqlens,
                           const float *h0, void *o, float *ht, void *workspace,
                           size_t workspace_bytes, hipStream_t stream) {
  gdn_status s = check_problem(p);
  if (s != GDN_OK) return s;
  const int64_t T = p->total_tokens;
  s = check_all("g and cu_seqlens", {cu_seqlens, T > 0 ? (const void *)g : cu_seqlens},
                {q, k, v, h0, o, ht});
  if (s == GDN_OK && T > 0) s = check_all("q, k, v and o", {q, k, v, o}, {});
  if (s != GDN_OK) return s;
  int cus = 0;
  s = device_info(&cus);
  if (s != GDN_OK) return s;
  if (T == 0) {  // every sequence is empty: its final state is its initial state
    if (!ht) return GDN_OK;
    LAUNCH(gdn::launch_copy_states(h0, p->h0_seq_stride, p->num_seqs, p->num_heads, p->head_dim, ht,
                                   stream),
           "final states of empty sequences");
    return GDN_OK;
  }
  Layout l;
  s = layout(p, false, &l);
  if (s != GDN_OK) return s;
  if (workspace_bytes < l.total)
    return fail(GDN_ERR_WORKSPACE_TOO_SMALL, "workspace needs %zu bytes", l.total);
  if (l.total > 0) {
    s = check_all("workspace", {workspace}, {workspace});
    if (s != GDN_OK) return s;
  }
  if (debug_on()) {
    s = debug_validate(cu_seqlens, p->num_seqs, T, nullptr, stream);
    if (s != GDN_OK) return s;
  }
  gdn::LinArgs a = base_args(p, l, cus, q, k, v, g, cu_seqlens, h0, static_cast<char *>(workspace));
  a.o = o;
  a.ht = ht;
  LAUNCH(gdn::launch_linattn_fwd(a, p->head_dim, p->dtype == GDN_DTYPE_BF16, stream),
         "linear attention forward");
  return after(stream);
}

gdn_status gdn_linattn_bwd(const gdn_linattn_problem *p, const void *q, const void *k,
                           const void *v, const float *g, const int32_t *cu_seqlens,
                           const float *h0, const void *dout, const float *dht, void *dq, void *dk,
                           void *dv, float *dg, float *dh0, void *workspace,
                           size_t workspace_bytes, hipStream_t stream) {
  gdn_status s = check_problem(p);
  if (s != GDN_OK) return s;
  const int64_t T = p->total_tokens;
  s = check_all("g, dg and cu_seqlens",
                {cu_seqlens, T > 0 ? (const void *)g : cu_seqlens,
                 T > 0 || p->head_decay ? (const void *)dg : cu_seqlens},
                {q, k, v, h0, dout, dht, dq, dk, dv, dh0});
  if (s == GDN_OK && T > 0)
    s = check_all("q, k, v, dout, dq, dk and dv", {q, k, v, dout, dq, dk, dv}, {});
  if (s != GDN_OK) return s;
  int cus = 0;
  s = device_info(&cus);
  if (s != GDN_OK) return s;
  const int64_t H = p->num_heads, D = p->head_dim;
  const bool shared = p->h0_seq_stride == 0;
  Layout l;
  s = layout(p, true, &l);
  if (s != GDN_OK) return s;
  if (T == 0) {  // every sequence is empty: the gradient of its state passes through
    if (dh0) {
      if (shared && dht)
        LAUNCH(gdn::launch_sum_dh0(dht, p->num_seqs, p->num_heads, p->head_dim, dh0, stream),
               "dh0 of empty sequences");
      else
        LAUNCH(gdn::launch_copy_states(dht, H * D * D, shared ? 1 : p->num_seqs, p->num_heads,
                                       p->head_dim, dh0, stream),
               "dh0 of empty sequences");
    }
    if (p->head_decay) LAUNCH(gdn::launch_linattn_zero(dg, H, stream), "dg of empty sequences");
    return GDN_OK;
  }
  if (workspace_bytes < l.total)
    return fail(GDN_ERR_WORKSPACE_TOO_SMALL, "workspace needs %zu bytes", l.total);
  s = check_all("workspace", {workspace}, {workspace});
  if (s != GDN_OK) return s;
  if (debug_on()) {
    s = debug_validate(cu_seqlens, p->num_seqs, T, nullptr, stream);
    if (s != GDN_OK) return s;
  }
  char *ws = static_cast<char *>(workspace);
  gdn::LinArgs a = base_args(p, l, cus, q, k, v, g, cu_seqlens, h0, ws);
  a.dout = dout;
  a.dht = dht;
  if (l.L > 0) a.unit_r = reinterpret_cast<float *>(ws + l.unit_r);
  a.dg_pairs = reinterpret_cast<float *>(ws + l.dg_pairs);
  a.dg_q = reinterpret_cast<float *>(ws + l.dg_q);
  a.dg_k = reinterpret_cast<float *>(ws + l.dg_k);
  a.unit_dot = reinterpret_cast<float *>(ws + l.unit_dot);
  if (p->head_decay) a.dg_unit = reinterpret_cast<double *>(ws + l.dg_unit);
  a.dg = dg;
  const bool bf = p->dtype == GDN_DTYPE_BF16, grouped = k_heads(p) != p->num_heads;
  float *const dq_part = grouped ? reinterpret_cast<float *>(ws + l.dq_part) : nullptr;
  float *const dk_part = grouped ? reinterpret_cast<float *>(ws + l.dk_part) : nullptr;
  a.grad_f32 = grouped;
  a.dq = grouped ? dq_part : dq;
  a.dk = grouped ? dk_part : dk;
  a.dv = dv;
  a.dh0 = dh0 && shared ? reinterpret_cast<float *>(ws + l.dh0_seq) : dh0;
  LAUNCH(gdn::launch_linattn_bwd(a, D, bf, stream), "linear attention backward");
  if (grouped)
    LAUNCH(gdn::launch_linattn_group_sum(a, D, bf, dq, dk, stream),
           "linear attention: dq and dk of shared heads");
  if (dh0 && shared)
    LAUNCH(gdn::launch_sum_dh0(a.dh0, p->num_seqs, p->num_heads, D, dh0, stream),
           "linear attention: dh0 of a shared state");
  return after(stream);
}

gdn_status gdn_linattn_step(int32_t batch, int32_t num_heads, int32_t num_k_heads,
                            int32_t head_dim, int32_t dtype, int32_t head_decay, float scale,
                            const void *q, const void *k, const void *v, const float *g,
                            const int32_t *pages, int32_t num_pages, float *state, void *o,
                            hipStream_t stream) {
  if (batch < 1 || num_heads < 1 || (int64_t)batch * num_heads >= kMaxUnits)
    return fail(GDN_ERR_BAD_SHAPE, "batch and num_heads must be >= 1, and their product below 2^23");
  if (num_k_heads < 0 || num_k_heads > num_heads ||
      (num_k_heads > 0 && num_heads % num_k_heads != 0))
    return fail(GDN_ERR_BAD_SHAPE, "num_k_heads must be 0 or a divisor of num_heads");
  if (head_dim != 64 && head_dim != 128) return fail(GDN_ERR_BAD_SHAPE, "head_dim must be 64 or 128");
  if (dtype != GDN_DTYPE_F32 && dtype != GDN_DTYPE_BF16) return fail(GDN_ERR_BAD_DTYPE, "dtype %d", dtype);
  if (head_decay != 0 && head_decay != 1) return fail(GDN_ERR_BAD_MODE, "head_decay must be 0 or 1");
  if (!std::isfinite(scale)) return fail(GDN_ERR_BAD_SHAPE, "scale must be finite");
  if (pages && num_pages < 1) return fail(GDN_ERR_BAD_SHAPE, "num_pages must be >= 1");
  if (pages && batch > kMaxPagedRows)
    return fail(GDN_ERR_BAD_SHAPE, "at most %d rows of a step have pages", kMaxPagedRows);
  gdn_status s = check_all("q, k, v, g, state and o", {q, k, v, g, state, o}, {q, k, v, state, o});
  if (s != GDN_OK) return s;
  s = device_info(nullptr);
  if (s == GDN_OK) s = clear_faults_for_debug(stream);
  if (s != GDN_OK) return s;
  gdn::LinStepArgs a{};
  a.q = q;
  a.k = k;
  a.v = v;
  a.g = g;
  a.g_head = head_decay;
  a.pages = pages;
  a.num_pages = num_pages;
  a.state = state;
  a.o = o;
  a.faults = pages ? fault_word() : nullptr;
  a.B = batch;
  a.H = num_heads;
  a.HK = num_k_heads > 0 ? num_k_heads : num_heads;
  a.scale = scale;
  LAUNCH(gdn::launch_linattn_step(a, head_dim, dtype == GDN_DTYPE_BF16, stream), "step launch");
  return after(stream);
}

// ---- pages ----------------------------------------------------------------------------------

namespace {

gdn_status check_pool(const char *what, const void *pool, int32_t num_pages, int64_t page_bytes) {
  if (num_pages < 1) return fail(GDN_ERR_BAD_SHAPE, "%s must have at least one page", what);
  if (page_bytes < 16 || page_bytes % 16 != 0 || page_bytes > ((int64_t)1 << 40))
    return fail(GDN_ERR_BAD_SHAPE, "page_bytes must be a positive multiple of 16 (at most 2^40)");
  if (!pool) return fail(GDN_ERR_NULL_ARG, "%s is required", what);
  if (!aligned16(pool)) return fail(GDN_ERR_BAD_ALIGNMENT, "%s must be 16-byte aligned", what);
  return GDN_OK;
}

bool overlap(const int32_t *a, int64_t n, const int32_t *b, int64_t m) {
  return a < b + m && b < a + n;
}

gdn_status check_workspace(int32_t num_pages, int32_t count, const void *ws, size_t bytes) {
  size_t need = 0;
  gdn_status s = gdn_pages_workspace_size(num_pages, count, &need);
  if (s != GDN_OK) return s;
  if (bytes < need) return fail(GDN_ERR_WORKSPACE_TOO_SMALL, "workspace needs %zu bytes", need);
  return check_all("workspace", {ws}, {ws});
}

}  // namespace

gdn_status gdn_pages_workspace_size(int32_t num_pages, int32_t count, size_t *bytes) {
  if (!bytes) return fail(GDN_ERR_NULL_ARG, "bytes is NULL");
  if (num_pages < 0 || count < 0) return fail(GDN_ERR_BAD_SHAPE, "num_pages and count must be >= 0");
  // the free list, the moves (two lists of at most half the pages, and their number) or each
  // destination's first pair; a copy's two lists
  *bytes = align_up(sizeof(int32_t) * ((size_t)num_pages + 4)) + align_up(sizeof(int32_t) * 2 * (size_t)count);
  return GDN_OK;
}

gdn_status gdn_pages_copy(void *dst, int32_t dst_num_pages, const void *src, int32_t src_num_pages,
                          int64_t page_bytes, const int32_t *dst_pages, const int32_t *src_pages,
                          int32_t count, void *workspace, size_t workspace_bytes,
                          hipStream_t stream) {
  gdn_status s = check_pool("dst", dst, dst_num_pages, page_bytes);
  if (s == GDN_OK) s = check_pool("src", src, src_num_pages, page_bytes);
  if (s != GDN_OK) return s;
  if (count < 0) return fail(GDN_ERR_BAD_SHAPE, "count must be >= 0");
  const char *d = static_cast<const char *>(dst), *c = static_cast<const char *>(src);
  const bool same = d == c;
  if (!same && d < c + src_num_pages * page_bytes && c < d + dst_num_pages * page_bytes)
    return fail(GDN_ERR_BAD_SHAPE, "dst and src must be one pool or not overlap");
  if (count == 0) return GDN_OK;
  s = check_all("dst_pages and src_pages", {dst_pages, src_pages}, {});
  if (s == GDN_OK) s = check_workspace(dst_num_pages, count, workspace, workspace_bytes);
  if (s != GDN_OK) return s;
  int cus = 0;
  s = device_info(&cus);
  if (s == GDN_OK) s = clear_faults_for_debug(stream);
  if (s != GDN_OK) return s;
  int32_t *const to = static_cast<int32_t *>(workspace), *const from = to + count;
  int32_t *const first = from + count;
  LAUNCH(gdn::launch_pages_check(dst_pages, src_pages, count, dst_num_pages, src_num_pages, same, to,
                                 from, first, fault_word(), stream),
         "pages_copy: checks");
  gdn::PageCopyArgs a{static_cast<char *>(dst), c, dst_num_pages, src_num_pages, page_bytes,
                      to, from, count, nullptr};
  LAUNCH(gdn::launch_pages_copy(a, cus, stream), "pages_copy");
  return after(stream);
}

gdn_status gdn_pages_fork(void *pool, int32_t *live, int32_t num_pages, int64_t page_bytes,
                          const int32_t *parents, int32_t count, int32_t *children,
                          void *workspace, size_t workspace_bytes, hipStream_t stream) {
  gdn_status s = check_pool("pool", pool, num_pages, page_bytes);
  if (s != GDN_OK) return s;
  if (count < 0) return fail(GDN_ERR_BAD_SHAPE, "count must be >= 0");
  if (count == 0) return GDN_OK;
  s = check_all("live, parents and children", {live, parents, children}, {});
  if (s == GDN_OK) s = check_workspace(num_pages, 0, workspace, workspace_bytes);
  if (s != GDN_OK) return s;
  if (overlap(children, count, parents, count) || overlap(children, count, live, num_pages) ||
      overlap(parents, count, live, num_pages))
    return fail(GDN_ERR_BAD_SHAPE, "live, parents and children must not overlap");
  int cus = 0;
  s = device_info(&cus);
  if (s == GDN_OK) s = clear_faults_for_debug(stream);
  if (s != GDN_OK) return s;
  LAUNCH(gdn::launch_pages_fork_plan(live, num_pages, parents, count, children,
                                     static_cast<int32_t *>(workspace), fault_word(), stream),
         "pages_fork: plan");
  gdn::PageCopyArgs a{static_cast<char *>(pool), static_cast<const char *>(pool), num_pages,
                      num_pages, page_bytes, children, parents, count, nullptr};
  LAUNCH(gdn::launch_pages_copy(a, cus, stream), "pages_fork: copy");
  return after(stream);
}

gdn_status gdn_pages_free(int32_t *live, int32_t num_pages, const int32_t *pages, int32_t count,
                          hipStream_t stream) {
  if (num_pages < 1) return fail(GDN_ERR_BAD_SHAPE, "num_pages must be >= 1");
  if (count < 0) return fail(GDN_ERR_BAD_SHAPE, "count must be >= 0");
  if (count == 0) return GDN_OK;
  gdn_status s = check_all("live and pages", {live, pages}, {});
  if (s != GDN_OK) return s;
  if (overlap(live, num_pages, pages, count))
    return fail(GDN_ERR_BAD_SHAPE, "live and pages must not overlap");
  s = device_info(nullptr);
  if (s == GDN_OK) s = clear_faults_for_debug(stream);
  if (s != GDN_OK) return s;
  LAUNCH(gdn::launch_pages_free(live, num_pages, pages, count, fault_word(), stream), "pages_free");
  return after(stream);
}

gdn_status gdn_pages_compact(void *pool, int32_t *live, int32_t num_pages, int64_t page_bytes,
                             int32_t *remap, void *workspace, size_t workspace_bytes,
                             hipStream_t stream) {
  gdn_status s = check_pool("pool", pool, num_pages, page_bytes);
  if (s == GDN_OK) s = check_all("live and remap", {live, remap}, {});
  if (s == GDN_OK) s = check_workspace(num_pages, 0, workspace, workspace_bytes);
  if (s != GDN_OK) return s;
  if (overlap(live, num_pages, remap, num_pages))
    return fail(GDN_ERR_BAD_SHAPE, "live and remap must not overlap");
  int cus = 0;
  s = device_info(&cus);
  if (s == GDN_OK) s = clear_faults_for_debug(stream);
  if (s != GDN_OK) return s;
  const int32_t half = num_pages / 2 + 1;
  int32_t *const to = static_cast<int32_t *>(workspace), *const from = to + half;
  int32_t *const moves = from + half;
  LAUNCH(gdn::launch_pages_compact_plan(live, num_pages, remap, to, from, moves, stream),
         "pages_compact: plan");
  gdn::PageCopyArgs a{static_cast<char *>(pool), static_cast<const char *>(pool), num_pages,
                      num_pages, page_bytes, to, from, num_pages / 2, moves};
  LAUNCH(gdn::launch_pages_copy(a, cus, stream), "pages_compact: moves");
  return after(stream);
}

}  // extern "C"
