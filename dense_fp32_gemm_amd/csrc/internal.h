// What the library's source files share among themselves.
#ifndef GEMM_F32_INTERNAL_H
#define GEMM_F32_INTERNAL_H

#include <stdint.h>

namespace gemm_f32_internal {

// The current device's compute units, and the dies (XCDs) it deals
// workgroups to round-robin; read once per device.
struct Device {
    int64_t cus;
    int xcds;
};
Device current_device();

}  // namespace gemm_f32_internal

#endif
