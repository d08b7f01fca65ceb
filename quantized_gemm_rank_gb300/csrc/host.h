// host.h -- host-side helpers shared by the translation units that define the C
// entry points: error text, launch events, tensor maps and the device's facts.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "mc2_gb300.h"
#include "num.cuh"

namespace mc2 {
namespace host {

// Records the formatted text as this thread's mc2_last_error() and returns `status`.
__attribute__((format(printf, 2, 3))) int fail(int status, const char *fmt, ...);
void clear_error();

inline bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

inline size_t elem_size(int dtype) { return dtype == MC2_F32 ? 4 : 2; }

inline int elem_kind(int dtype) {
    return dtype == MC2_F16 ? mc2::ELEM_F16 : (dtype == MC2_BF16 ? mc2::ELEM_BF16 : mc2::ELEM_F32);
}

// A matrix argument: its rows must not overlap and its elements must be aligned
// to their own size.  Optional ones are passed only when given.
inline int check_rows(const char *what, const void *p, int64_t ld, int64_t m, int64_t cols, size_t size) {
    if (ld < cols && m > 1)
        return fail(MC2_ERR_SHAPE, "%s: rows of %lld elements cannot be %lld elements apart", what, (long long)cols,
                    (long long)ld);
    if (ld > INT64_MAX / 4 / (m > 1 ? m : 1))
        return fail(MC2_ERR_SHAPE, "%s: a row stride of %lld elements is too large", what, (long long)ld);
    if (reinterpret_cast<uintptr_t>(p) % size != 0)
        return fail(MC2_ERR_UNSUPPORTED, "%s is not aligned to its %zu-byte elements", what, size);
    return MC2_OK;
}

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

// 2-D map over 8-bit elements: boxes of 128 columns x box_outer rows, 128-byte swizzle; pitch a multiple of 16.
bool make_map8(CUtensorMap *m, const void *base, uint64_t inner, uint64_t outer, uint32_t box_outer, uint64_t pitch);
// 3-D map over fp32 matrices (parts, outer, inner) with rows `pitch` elements apart (a multiple of 4): boxes of 32 columns x 32
// rows, 128-byte swizzle.
bool make_map32_parts(CUtensorMap *m, const void *base, uint64_t inner, uint64_t outer, uint64_t parts, uint64_t pitch);

}  // namespace host
}  // namespace mc2
