// What the library's source files share among themselves.
#ifndef GEMM_F32_INTERNAL_H
#define GEMM_F32_INTERNAL_H

#include <stdint.h>

namespace gemm_f32_internal {

constexpr int kMaxDevices = 64;   // whose properties and addresses are kept

// The device the work runs on, read once per device: its compute units
// (the unit the shape rules balance tiles over, and stream-K's worker count)
// and the dies (XCDs, 32 compute units each on MI355X) workgroups are dealt
// to round-robin.  A whole MI355X has 256 and 8; a partitioned one fewer.
// Without a usable device (plans described on a host without a GPU) the
// whole MI355X is assumed.
struct Device {
    int64_t cus;
    int xcds;
};
Device current_device();

}  // namespace gemm_f32_internal

#endif
