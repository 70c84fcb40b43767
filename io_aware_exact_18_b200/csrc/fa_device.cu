// The device check of the entry points outside fa.h. They need no set-up beyond
// it: no status word, no tensor maps.
#include <cuda_runtime.h>

#include <atomic>

#include "fa_host.h"

namespace fa {

int device_ready() {
    constexpr int kMaxDevices = 64;
    static std::atomic<int8_t> known[kMaxDevices];           // 0 not yet, 1 sm_100, -1 other
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return FA_ERR_LAUNCH;
    if (dev < 0 || dev >= kMaxDevices) return FA_ERR_UNSUPPORTED;
    int8_t is = known[dev].load(std::memory_order_relaxed);
    if (is == 0) {
        int major = 0, minor = 0;
        if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
            cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess)
            return FA_ERR_LAUNCH;
        is = major == 10 && minor == 0 ? 1 : -1;
        known[dev].store(is, std::memory_order_relaxed);
    }
    if (is < 0) return FA_ERR_UNSUPPORTED;
    // launches are read back through cudaGetLastError: clear an error that an
    // unrelated runtime call left there
    (void)cudaGetLastError();
    return FA_OK;
}

}  // namespace fa
