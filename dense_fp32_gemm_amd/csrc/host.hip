// Host code that all entry points share: the device's properties and the texts of the
// return codes.  Apart from the kernels, whose committed counter records hold for
// their source file as it was measured.

#include <hip/hip_runtime.h>

#include <atomic>

#include "gemm_f32.h"
#include "internal.h"

namespace gemm_f32_internal {

static std::atomic<int> g_device_cus[kMaxDevices];   // 0: not read yet

Device current_device()
{
    constexpr int kDefaultCus = 256, kCusPerXcd = 32;
    int dev = -1, cu = 0;
    if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= kMaxDevices) {
        (void)hipGetLastError();
        cu = kDefaultCus;
    } else {
        cu = g_device_cus[dev].load(std::memory_order_relaxed);
        if (cu == 0) {
            if (hipDeviceGetAttribute(&cu, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess || cu <= 0) {
                (void)hipGetLastError();
                cu = kDefaultCus;
            }
            g_device_cus[dev].store(cu, std::memory_order_relaxed);
        }
    }
    return {cu, cu % kCusPerXcd == 0 ? cu / kCusPerXcd : 1};
}

}  // namespace gemm_f32_internal

extern "C" {

const char *gemm_f32_status_string(int status)
{
    switch (status) {
    case GEMM_F32_OK: return "ok";
    case GEMM_F32_ERR_DIM: return "M, N or K is negative or the problem is too large to tile";
    case GEMM_F32_ERR_LD: return "a leading dimension is smaller than its row length";
    case GEMM_F32_ERR_NULL: return "a required pointer is NULL";
    case GEMM_F32_ERR_LAUNCH: return "kernel launch failed";
    case GEMM_F32_ERR_CONFIG: return "unknown kernel configuration";
    case GEMM_F32_ERR_ALIGN: return "a pointer is not aligned to its elements (4 bytes for binary32)";
    case GEMM_F32_ERR_SCRATCH: return "the split plan needs more than the library's static scratch holds";
    case GEMM_F32_ERR_TYPE: return "unknown element type";
    case GEMM_F32_ERR_OPTION: return "an option is outside its range";
    case GEMM_F32_ERR_WORKSPACE: return "the workspace is NULL, too small or not 16-byte aligned";
    default: return "unknown status";
    }
}

}  // extern "C"
