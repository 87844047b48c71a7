// hcgr_host.h -- host-side helpers shared by the C ABI sources: the error
// record of the calling thread, pointer and overlap checks, and the device
// guard of every launching entry point. Defined in hcgr_api.hip. Not installed.
#pragma once

#include <cstddef>
#include <cstdint>

#include "../../include/hcgr.h"

namespace hcgr_host {

// Records the reason and returns st; ok() clears it and returns HCGR_OK.
hcgr_status fail(hcgr_status st, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
hcgr_status ok();

struct Range {
  uintptr_t lo, hi;  // [lo, hi)
  const char* name;
};
inline bool overlap(const Range& a, const Range& b) { return a.lo < b.hi && b.lo < a.hi; }
inline Range range_of(const void* p, uint64_t bytes, const char* name) {
  return Range{(uintptr_t)p, (uintptr_t)p + (uintptr_t)bytes, name};
}
// HCGR_ERR_ALIASING when a non-empty output overlaps another output or an input.
hcgr_status check_overlaps(const Range* outs, int nout, const Range* ins, int nin);

struct PtrCheck {
  const void* p;
  const char* name;
  size_t align;
};
hcgr_status check_ptrs(const PtrCheck* ptrs, int n);

// HCGR_OK when `device` exists and is a gfx950.
hcgr_status check_device(int device);

// Checks that `stream` (NULL: the default stream of `device`) belongs to `device`
// and makes that device current; *prev is the caller's device.
hcgr_status enter_device(int device, void* stream, int* prev);
void restore_device(int device, int prev);

}  // namespace hcgr_host
