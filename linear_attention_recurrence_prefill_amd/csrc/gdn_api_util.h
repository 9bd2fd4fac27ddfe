// What the library's C entry points share: error reporting, the device check, the debug mode.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/gdn.h"

namespace gdn {
namespace api {

// Stores the calling thread's error detail and returns s.
gdn_status fail(gdn_status s, const char *fmt, ...) __attribute__((format(printf, 2, 3)));
gdn_status hip_fail(hipError_t e, const char *what);
const char *last_error();

bool debug_on();
void set_debug_on(bool on);
// Debug mode: cu_seqlens checked on the device (and against the host copy) before a launch, and the
// fault flags read after the launches; both synchronise the stream.
gdn_status debug_validate(const int32_t *cu, int32_t N, int64_t T, const int32_t *cu_host,
                          hipStream_t stream);
gdn_status debug_faults(hipStream_t stream);
uint32_t *fault_word();

// The current device must be gfx950; *cus (when not null) gets its compute units.
gdn_status device_info(int *cus);

inline bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
constexpr size_t kAlign = 256;
inline size_t align_up(size_t x) { return (x + kAlign - 1) / kAlign * kAlign; }

}  // namespace api
}  // namespace gdn
