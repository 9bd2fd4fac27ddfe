// Linear attention's step of one token per sequence on gfx950, on fp32 states that are a batch or
// the pages of a pool: S <- e^g S + k v^T, o = scale S^T q, in place.
//
// The step reads and writes every state once (2 d^2 fp32 per head) and computes 5 flop per element:
// it is bound by HBM.  The columns of a state are independent (o_j needs column j only), so a
// workgroup takes 32 columns of one (row, head): 128-byte row pieces, four (d = 128) times as many
// workgroups as states, which is what a batch of one needs, and no sum crosses workgroups.
// 80 rows x 16 heads, d = 128: 27.9 us for 169 MB, 6.1 TB/s, as a large copy; one row x 8 heads: 4 us,
// a launch's latency.
// Thread (row group, 4 columns) keeps its rows in registers; o is summed over the row groups in
// LDS in a fixed order.
#include "gdn_device.h"
#include "gdn_internal.h"
#include "gdn_linattn.h"

namespace gdn {
namespace {

__device__ __forceinline__ float as_f32(const float *p, int64_t i) { return p[i]; }
__device__ __forceinline__ float as_f32(const bf16 *p, int64_t i) { return (float)p[i]; }

}  // namespace

template <int D, class E>
__global__ __launch_bounds__(256) void linattn_step_kernel(LinStepArgs a) {
  constexpr int RG = 32;        // row groups: 8 lanes cover 32 columns
  constexpr int RPT = D / RG;   // rows per thread
  __shared__ __attribute__((aligned(16))) float part[RG][36];
  const int tid = threadIdx.x, cg = tid & 7, rg = tid >> 3;
  const int b = blockIdx.x / a.H, h = blockIdx.x % a.H;
  const int col = 32 * blockIdx.y + 4 * cg;
  const int64_t bh = (int64_t)b * a.H + h;
  const int64_t bk = (int64_t)b * a.HK + h / (a.H / a.HK);
  const E *q = static_cast<const E *>(a.q) + bk * D;
  const E *k = static_cast<const E *>(a.k) + bk * D;
  const E *v = static_cast<const E *>(a.v) + bh * D;
  E *o = static_cast<E *>(a.o) + bh * D;
  int64_t page = b;
  if (a.pages) {
    // a page outside the pool, or one that an earlier row has, is not touched: its row gets zeros
    const int32_t p = a.pages[b];
    bool twice = false;
    for (int i = tid; i < b; i += 256) twice |= a.pages[i] == p;
    const bool in = p >= 0 && p < a.num_pages;
    const bool dup = __syncthreads_or(in && twice);
    if (!in || dup) {
      if (tid < 32) o[32 * blockIdx.y + tid] = (E)0.f;
      if (tid == 0 && a.faults && p != -1)
        atomicOr(a.faults, in ? kFaultPageTwice : kFaultPageRange);
      return;
    }
    page = p;
  }
  float *S = a.state + (page * a.H + h) * D * D + col;
  f32x4 x[RPT];
#pragma unroll
  for (int i = 0; i < RPT; ++i)
    x[i] = *reinterpret_cast<const f32x4 *>(S + (int64_t)(rg + RG * i) * D);
  f32x4 vv;
#pragma unroll
  for (int j = 0; j < 4; ++j) vv[j] = as_f32(v, col + j);
  const float eg = expf(a.g[a.g_head ? h : bh]);
  f32x4 s = zero4();
#pragma unroll
  for (int i = 0; i < RPT; ++i) {
    const int r = rg + RG * i;
    x[i] = eg * x[i] + as_f32(k, r) * vv;
    *reinterpret_cast<f32x4 *>(S + (int64_t)r * D) = x[i];
    s += as_f32(q, r) * x[i];
  }
  *reinterpret_cast<f32x4 *>(&part[rg][4 * cg]) = s;
  __syncthreads();
  if (tid < 32) {
    float t = 0.f;
#pragma unroll
    for (int g = 0; g < RG; ++g) t += part[g][tid];
    o[32 * blockIdx.y + tid] = (E)(a.scale * t);
  }
}

hipError_t launch_linattn_step(const LinStepArgs &a, int D, bool is_bf16, hipStream_t stream) {
  const dim3 grid((unsigned)((int64_t)a.B * a.H), D / 32), block(256);
  if (D == 128) {
    if (is_bf16) hipLaunchKernelGGL((linattn_step_kernel<128, bf16>), grid, block, 0, stream, a);
    else hipLaunchKernelGGL((linattn_step_kernel<128, float>), grid, block, 0, stream, a);
  } else {
    if (is_bf16) hipLaunchKernelGGL((linattn_step_kernel<64, bf16>), grid, block, 0, stream, a);
    else hipLaunchKernelGGL((linattn_step_kernel<64, float>), grid, block, 0, stream, a);
  }
  return hipGetLastError();
}

}  // namespace gdn
