// host.h -- host-side helpers shared by the translation units that define the C
// entry points: error text, launch events, tensor maps and the device's facts.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>

namespace mc2 {
namespace host {

// Records the formatted text as this thread's mc2_last_error() and returns `status`.
__attribute__((format(printf, 2, 3))) int fail(int status, const char *fmt, ...);
void clear_error();

inline bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

constexpr uint64_t kWaitLimitNs = 2000000000ull;  // 2 s per bounded device-side wait

// Records the events that mc2_set_launch_events installed on this thread around
// the kernel launches of one call, in launch order.
class LaunchMarks {
  public:
    explicit LaunchMarks(cudaStream_t s) : s_(s) { mark(); }
    // after each kernel launch of the call
    void launched() { mark(); }

  private:
    void mark();
    cudaStream_t s_;
    int next_ = 0;
};

struct DeviceInfo {
    int device = -1;
    int num_sms = 0;
};

// The current device's facts (cached); a negative status if it is none this library runs on.
int current_device(DeviceInfo *info);

// 2-D map over a row-major (outer, inner) matrix with 16-bit elements and a
// swizzle of the box's row, 128 bytes (64 columns) or 64 (32 columns); out-of-range box
// elements read as zero.  pitch: elements
// from row to row, 0 for contiguous rows (a multiple of 8 either way).
bool make_map16(CUtensorMap *m, const void *base, uint64_t inner, uint64_t outer, uint32_t box_inner,
                uint32_t box_outer, uint64_t pitch = 0);
// The same for an N-major operand as a 3-D map, `groups` 64-column slices a copy
// (inner % 64 == 0 only; false otherwise).
bool make_map16_nmajor3d(CUtensorMap *m, const void *base, uint64_t inner, uint64_t outer, uint32_t box_outer,
                         uint32_t groups, uint64_t pitch = 0);

}  // namespace host
}  // namespace mc2
