// Makes a device current for a scope and the caller's current again after it.
#pragma once

#include <hip/hip_runtime.h>

namespace ss {

struct DeviceGuard {
    int before = -1;
    bool ok = false;
    bool moved = false;
    explicit DeviceGuard(int device) {
        if (hipGetDevice(&before) != hipSuccess) return;
        moved = before != device;
        ok = !moved || hipSetDevice(device) == hipSuccess;
    }
    ~DeviceGuard() {
        if (moved && ok) (void)hipSetDevice(before);
    }
    DeviceGuard(const DeviceGuard&) = delete;
    DeviceGuard& operator=(const DeviceGuard&) = delete;
};

}  // namespace ss
