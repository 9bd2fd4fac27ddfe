// Operators on the pages of a pool (a cache of states): copy, fork, free, compact.
//
// All of the data movement is one copy kernel over a list of (to, from) pages on the device; the
// lists are made by one workgroup from the pool's live flags, so nothing waits for the host.  The
// copy is bound by HBM (each page read once, written once); a list takes one short launch's latency
// (3 us for a hundred pages).  A workgroup moves 16 KiB pieces, four 16-byte loads per lane in
// flight: one page of 1 MiB forked 80 times 16 to 17 us, 85 MB read from the caches and written, 5.0
// to 5.2 TB/s (a fill of one large buffer reaches 6.9 TB/s, a copy 6.0).
#include <algorithm>

#include "gdn_device.h"
#include "gdn_internal.h"
#include "gdn_pages.h"

namespace gdn {
namespace {

typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));
constexpr int kPlanThreads = 1024;
constexpr int kPiece = 256 * 4;  // 16-byte units of a piece

__global__ __launch_bounds__(256) void pages_copy_kernel(PageCopyArgs a) {
  const int64_t units = a.page_bytes / 16, per = (units + kPiece - 1) / kPiece;
  const int64_t n = a.count_dev ? min(*a.count_dev, a.count) : a.count;
  for (int64_t item = blockIdx.x; item < n * per; item += gridDim.x) {
    const int64_t pair = item / per, u0 = item % per * kPiece + threadIdx.x;
    const int32_t to = a.to[pair], from = a.from[pair];
    if (to < 0 || to >= a.dst_pages || from >= a.src_pages) continue;
    u32x4 *d = reinterpret_cast<u32x4 *>(a.dst + to * a.page_bytes);
    const u32x4 *s = reinterpret_cast<const u32x4 *>(a.src + from * a.page_bytes);
    u32x4 x[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      x[j] = u32x4{0u, 0u, 0u, 0u};
      if (from >= 0 && u0 + 256 * j < units) x[j] = s[u0 + 256 * j];
    }
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (u0 + 256 * j < units) d[u0 + 256 * j] = x[j];
  }
}

// The pairs of a copy that can be done at once: first[d] is the first pair that names destination d.
// Linear in the list, whatever the pools' size: only the entries that a pair names are set.  One pool
// may be given with two page counts (a part of it as dst): `first` has an entry for each page of dst,
// and a source page past them is no pair's destination.
__global__ __launch_bounds__(kPlanThreads) void pages_check_kernel(const int32_t *dst_idx,
                                                                   const int32_t *src_idx, int count,
                                                                   int dst_pages, int src_pages,
                                                                   bool same_pool, int32_t *to,
                                                                   int32_t *from, int32_t *first,
                                                                   uint32_t *faults) {
  const auto in_range = [&](int32_t d, int32_t s) {
    return d >= -1 && d < dst_pages && s >= -1 && s < src_pages;
  };
  for (int64_t i = threadIdx.x; i < count; i += kPlanThreads) {
    const int32_t d = dst_idx[i], s = src_idx[i];
    if (!in_range(d, s)) continue;
    if (d >= 0) first[d] = INT32_MAX;
    if (same_pool && s >= 0 && s < dst_pages) first[s] = INT32_MAX;
  }
  __threadfence();
  __syncthreads();
  for (int64_t i = threadIdx.x; i < count; i += kPlanThreads) {
    const int32_t d = dst_idx[i], s = src_idx[i];
    if (in_range(d, s) && d >= 0) atomicMin(first + d, (int32_t)i);
  }
  __threadfence();
  __syncthreads();
  const auto first_of = [&](int32_t d) {  // past the caches that the stores above went through
    return __hip_atomic_load(first + d, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  };
  for (int64_t i = threadIdx.x; i < count; i += kPlanThreads) {
    const int32_t d = dst_idx[i], s = src_idx[i];
    uint32_t f = 0u;
    if (!in_range(d, s)) {
      f = kFaultPageRange;
    } else if (d >= 0) {
      bool races = first_of(d) != i;
      if (same_pool && s >= 0 && s < dst_pages && s != d) races |= first_of(s) != INT32_MAX;
      if (races) f = kFaultPageTwice;
    }
    to[i] = f || d < 0 || (same_pool && d == s) ? -1 : d;
    from[i] = f ? -1 : s;
    if (f && faults) atomicOr(faults, f);
  }
}

// Inclusive sum of x over the workgroup; *all gets the total.  Every thread calls it.
__device__ int block_scan(int x, int *all) {
  __shared__ int wave_sum[kPlanThreads / 64];
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  int s = x;
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) {
    const int y = __shfl_up(s, off, 64);
    if (lane >= off) s += y;
  }
  __syncthreads();  // the last call's sums have been read
  if (lane == 63) wave_sum[w] = s;
  __syncthreads();
  int before = 0, total = 0;
#pragma unroll
  for (int j = 0; j < kPlanThreads / 64; ++j) {
    const int y = wave_sum[j];
    before += j < w ? y : 0;
    total += y;
  }
  *all = total;
  return before + s;
}

__global__ __launch_bounds__(kPlanThreads) void pages_fork_plan_kernel(
    int32_t *live, int P, const int32_t *parents, int count, int32_t *children, int32_t *free_list,
    uint32_t *faults) {
  int nfree = 0;
  for (int p0 = 0; p0 < P; p0 += kPlanThreads) {  // the free pages in order
    const int p = p0 + threadIdx.x;
    const int is = p < P && live[p] == 0;
    int all;
    const int r = block_scan(is, &all);
    if (is) free_list[nfree + r - 1] = p;
    nfree += all;
  }
  __syncthreads();
  int taken = 0;
  for (int i0 = 0; i0 < count; i0 += kPlanThreads) {
    const int i = i0 + threadIdx.x;
    int ok = 0;
    if (i < count) {
      const int32_t p = parents[i];
      ok = p == -1 || (p >= 0 && p < P && live[p] != 0);
      if (!ok && faults) atomicOr(faults, kFaultPageRange);
    }
    int all;
    const int r = taken + block_scan(ok, &all) - 1;
    if (i < count) {
      children[i] = ok && r < nfree ? free_list[r] : -1;
      if (ok && r >= nfree && faults) atomicOr(faults, kFaultNoPage);
    }
    taken += all;
  }
  __syncthreads();  // every parent's flag has been read
  for (int r = threadIdx.x; r < min(taken, nfree); r += kPlanThreads) live[free_list[r]] = 1;
}

// The same for a pool and a list of at most one round (kPlanThreads entries each): the flags and the
// list are read at once, counted by one scan, and the free pages are listed in LDS (128 pages: 2.6 us
// instead of 3.8).
__global__ __launch_bounds__(kPlanThreads) void pages_fork_plan_small_kernel(
    int32_t *live, int P, const int32_t *parents, int count, int32_t *children, uint32_t *faults) {
  __shared__ int32_t s_live[kPlanThreads], s_free[kPlanThreads];
  const int i = threadIdx.x;
  const int32_t flag = i < P ? live[i] : 1, parent = i < count ? parents[i] : -2;
  s_live[i] = flag;
  __syncthreads();  // also: every flag has been read
  const bool ok = parent == -1 || (parent >= 0 && parent < P && s_live[parent] != 0);
  int all;  // pages in the low half, parents in the high one
  const int sums = block_scan((flag == 0) | (ok ? 1 << 16 : 0), &all);
  if (flag == 0) s_free[(sums & 0xffff) - 1] = i;
  __syncthreads();
  if (i >= count) return;
  const int r = (sums >> 16) - 1, nfree = all & 0xffff;
  const int32_t child = ok && r < nfree ? s_free[r] : -1;
  children[i] = child;
  if (child >= 0) live[child] = 1;
  else if (faults) atomicOr(faults, ok ? kFaultNoPage : kFaultPageRange);
}

__global__ __launch_bounds__(256) void pages_free_kernel(int32_t *live, int P,
                                                         const int32_t *__restrict__ pages,
                                                         int count, uint32_t *faults) {
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < count; i += (int64_t)gridDim.x * 256) {
    const int32_t p = pages[i];
    if (p >= 0 && p < P) live[p] = 0;
    else if (p != -1 && faults) atomicOr(faults, kFaultPageRange);
  }
}

__global__ __launch_bounds__(kPlanThreads) void pages_compact_plan_kernel(int32_t *live, int P,
                                                                         int32_t *remap, int32_t *to,
                                                                         int32_t *from,
                                                                         int32_t *moves) {
  int mine = 0, count;
  for (int p = threadIdx.x; p < P; p += kPlanThreads) mine += live[p] != 0;
  block_scan(mine, &count);
  int holes = 0, movers = 0;  // as many of one as of the other
  for (int p0 = 0; p0 < P; p0 += kPlanThreads) {
    const int p = p0 + threadIdx.x;
    const bool used = p < P && live[p] != 0;
    const int hole = p < count && !used, mover = p >= count && used;
    int all_h, all_m;
    const int rh = block_scan(hole, &all_h), rm = block_scan(mover, &all_m);
    if (hole) to[holes + rh - 1] = p;
    if (mover) from[movers + rm - 1] = p;
    if (p < P) remap[p] = used ? p : -1;
    holes += all_h;
    movers += all_m;
  }
  __syncthreads();  // the lists are complete, every flag has been read
  for (int i = threadIdx.x; i < movers; i += kPlanThreads) remap[from[i]] = to[i];
  for (int p = threadIdx.x; p < P; p += kPlanThreads) live[p] = p < count;
  if (threadIdx.x == 0) *moves = movers;
}

// The same for a pool of at most one round: one scan of the flags ranks the live pages, and with it the
// holes before L and the pages that move into them (128 pages: 2.7 us instead of 3.8).
__global__ __launch_bounds__(kPlanThreads) void pages_compact_plan_small_kernel(
    int32_t *live, int P, int32_t *remap, int32_t *to, int32_t *from, int32_t *moves) {
  __shared__ int32_t s_to[kPlanThreads];
  __shared__ int s_front;  // live pages before L
  const int p = threadIdx.x;
  const bool used = p < P && live[p] != 0;
  int count;
  const int before = block_scan(used, &count) - (used ? 1 : 0);
  if (p == count || (count == kPlanThreads && p == 0)) s_front = p == count ? before : count;
  if (p < count && !used) s_to[p - before] = p, to[p - before] = p;
  __syncthreads();
  if (p == 0) *moves = count - s_front;
  if (p >= P) return;
  int32_t where = used ? p : -1;
  if (used && p >= count) {
    where = s_to[before - s_front];
    from[before - s_front] = p;
  }
  remap[p] = where;
  live[p] = p < count;
}

}  // namespace

hipError_t launch_pages_check(const int32_t *dst_idx, const int32_t *src_idx, int32_t count,
                              int32_t dst_pages, int32_t src_pages, bool same_pool, int32_t *to,
                              int32_t *from, int32_t *first, uint32_t *faults, hipStream_t stream) {
  hipLaunchKernelGGL(pages_check_kernel, dim3(1), dim3(kPlanThreads), 0, stream, dst_idx, src_idx,
                     count, dst_pages, src_pages, same_pool, to, from, first, faults);
  return hipGetLastError();
}

hipError_t launch_pages_copy(const PageCopyArgs &a, int cus, hipStream_t stream) {
  const int64_t per = (a.page_bytes / 16 + kPiece - 1) / kPiece;
  const int64_t blocks = std::min<int64_t>((int64_t)a.count * per, (int64_t)cus * 16);
  if (blocks <= 0) return hipSuccess;
  hipLaunchKernelGGL(pages_copy_kernel, dim3((unsigned)blocks), dim3(256), 0, stream, a);
  return hipGetLastError();
}

hipError_t launch_pages_fork_plan(int32_t *live, int32_t num_pages, const int32_t *parents,
                                  int32_t count, int32_t *children, int32_t *free_list,
                                  uint32_t *faults, hipStream_t stream) {
  if (num_pages <= kPlanThreads && count <= kPlanThreads)
    hipLaunchKernelGGL(pages_fork_plan_small_kernel, dim3(1), dim3(kPlanThreads), 0, stream, live,
                       num_pages, parents, count, children, faults);
  else
    hipLaunchKernelGGL(pages_fork_plan_kernel, dim3(1), dim3(kPlanThreads), 0, stream, live, num_pages,
                     parents, count, children, free_list, faults);
  return hipGetLastError();
}

hipError_t launch_pages_free(int32_t *live, int32_t num_pages, const int32_t *pages, int32_t count,
                             uint32_t *faults, hipStream_t stream) {
  const int blocks = std::min((count + 255) / 256, 1024);
  hipLaunchKernelGGL(pages_free_kernel, dim3(blocks), dim3(256), 0, stream, live, num_pages, pages,
                     count, faults);
  return hipGetLastError();
}

hipError_t launch_pages_compact_plan(int32_t *live, int32_t num_pages, int32_t *remap, int32_t *to,
                                     int32_t *from, int32_t *moves, hipStream_t stream) {
  if (num_pages <= kPlanThreads)
    hipLaunchKernelGGL(pages_compact_plan_small_kernel, dim3(1), dim3(kPlanThreads), 0, stream, live,
                       num_pages, remap, to, from, moves);
  else
    hipLaunchKernelGGL(pages_compact_plan_kernel, dim3(1), dim3(kPlanThreads), 0, stream, live,
                     num_pages, remap, to, from, moves);
  return hipGetLastError();
}

}  // namespace gdn
