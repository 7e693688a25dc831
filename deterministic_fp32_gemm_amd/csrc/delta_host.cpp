// Host side shared by the libraries' entry points: device and pointer checks, the last HIP error, status texts.
#include <hip/hip_runtime.h>

#include <cstdint>
#include <atomic>
#include <cstring>

#include "delta_host.h"

namespace sdm_delta {

namespace {
thread_local int t_last_hip_error = 0;
constexpr int kDevices = 64;
std::atomic<int> g_known[kDevices];     // per device: 0 not asked yet, 1 gfx950, 2 another
}  // namespace

int record_hip_error(hipError_t e) {
    t_last_hip_error = static_cast<int>(e);
    return SDM_GX_ERR_HIP;
}

int current_gfx950(int* dev) {
    hipError_t e = hipGetDevice(dev);
    if (e != hipSuccess) return record_hip_error(e);
    if (*dev < 0 || *dev >= kDevices) return SDM_GX_ERR_DEVICE;
    int k = g_known[*dev].load(std::memory_order_relaxed);
    if (!k) {
        hipDeviceProp_t prop;
        e = hipGetDeviceProperties(&prop, *dev);
        if (e != hipSuccess) return record_hip_error(e);
        k = std::strncmp(prop.gcnArchName, "gfx950", 6) == 0 ? 1 : 2;
        g_known[*dev].store(k, std::memory_order_relaxed);
    }
    return k == 1 ? SDM_GX_OK : SDM_GX_ERR_DEVICE;
}

int pointer_on(const void* p, int dev) {
    hipPointerAttribute_t at;
    if (hipPointerGetAttributes(&at, p) != hipSuccess) {
        (void)hipGetLastError();
        return SDM_GX_ERR_DEVICE;
    }
    return (at.type == hipMemoryTypeDevice || at.type == hipMemoryTypeManaged) && at.device == dev ? SDM_GX_OK
                                                                                                  : SDM_GX_ERR_DEVICE;
}

int last_hip_error() { return t_last_hip_error; }

const char* status_text(int code) {
    switch (code) {
        case SDM_GX_OK: return "ok";
        case SDM_GX_ERR_NULL: return "a required pointer is NULL";
        case SDM_GX_ERR_SHAPE: return "sizes out of range (see the header's limits)";
        case SDM_GX_ERR_ALIGN: return "a pointer is not aligned to its elements, or a workspace to 256 (norm, linear recurrence: 16) bytes";
        case SDM_GX_ERR_OVERLAP: return "an output overlaps an input or another output";
        case SDM_GX_ERR_STRIDE: return "stride out of range, or rows of an output that overlap each other";
        case SDM_GX_ERR_LIMIT: return "workspace too small, or the launch exceeds a device limit";
        case SDM_GX_ERR_HIP: return "HIP runtime error (see the library's last_hip_error call)";
        case SDM_GX_ERR_DEVICE: return "no gfx950 device, or a pointer is not on the current device";
        case SDM_GX_ERR_ARG: return "invalid argument";
        default: return "unknown status";
    }
}

}  // namespace sdm_delta
