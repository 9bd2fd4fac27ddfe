// Internal interface of the operators on a pool's pages (gdn_pages.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace gdn {

struct PageCopyArgs {
  char *dst;
  const char *src;
  int32_t dst_pages, src_pages;  // pages of the two pools
  int64_t page_bytes;
  const int32_t *to, *from;      // [count] page of dst (-1: none) and of src (-1: zeros)
  int32_t count;
  const int32_t *count_dev;      // when not null, the number of pairs, at most count
};

// to[i], from[i] of the pairs that can be copied at once, -1 to of the others (see gdn_pages_copy);
// first: scratch, [dst_pages].
hipError_t launch_pages_check(const int32_t *dst_idx, const int32_t *src_idx, int32_t count,
                              int32_t dst_pages, int32_t src_pages, bool same_pool, int32_t *to,
                              int32_t *from, int32_t *first, uint32_t *faults, hipStream_t stream);
hipError_t launch_pages_copy(const PageCopyArgs &a, int cus, hipStream_t stream);
// children[i] = the pages that take parents[i] (-1: none), marked in live; free_list: [num_pages].
hipError_t launch_pages_fork_plan(int32_t *live, int32_t num_pages, const int32_t *parents,
                                  int32_t count, int32_t *children, int32_t *free_list,
                                  uint32_t *faults, hipStream_t stream);
hipError_t launch_pages_free(int32_t *live, int32_t num_pages, const int32_t *pages, int32_t count,
                             uint32_t *faults, hipStream_t stream);
// The moves that bring the live pages to the front: to, from [num_pages / 2] and their number.
hipError_t launch_pages_compact_plan(int32_t *live, int32_t num_pages, int32_t *remap, int32_t *to,
                                     int32_t *from, int32_t *moves, hipStream_t stream);

}  // namespace gdn
