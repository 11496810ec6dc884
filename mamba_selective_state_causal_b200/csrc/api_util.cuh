// api_util.cuh -- what the entry points of the C ABI share (defined in ssd_api.cu): the last error
// of the calling thread, per-device lookups, the environment hooks and simple argument checks.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace ssd {

int api_fail(int code, const char *fmt, ...) __attribute__((format(printf, 2, 3)));
int api_ok();
unsigned int *api_status_ptr();
int api_sm_count();
uint64_t api_wait_limit_ns();
bool api_force_generic();
int64_t api_take_drop_unit();   // SSD_TEST_DROP_UNIT on the first scan or slot step of the process, else -1

inline size_t api_elem_size(int dtype) { return dtype == 1 ? 2 : 4; }
inline bool api_aligned(const void *p, size_t n = 16) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
inline size_t api_round256(size_t v) { return (v + 255) & ~size_t(255); }
inline bool api_pow2_dim(int v) { return v == 16 || v == 32 || v == 64 || v == 128; }

}  // namespace ssd
