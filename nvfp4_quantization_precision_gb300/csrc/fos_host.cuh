// fos_host.cuh -- host-side argument helpers shared by the C ABI entry points.
#pragma once

#include <cstdint>
#include <initializer_list>

#include <cuda_runtime.h>

#include "fos.h"
#include "fos_device.cuh"

namespace fos {

inline bool valid_dtype(int dt) { return dt == FOS_BF16 || dt == FOS_FP16 || dt == FOS_FP32; }

inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// Device that owns a pointer, or -1 when the pointer is not device memory.
inline int device_of(const void* p) {
    cudaPointerAttributes at;
    if (cudaPointerGetAttributes(&at, p) != cudaSuccess) {
        cudaGetLastError();
        return -1;
    }
    if (at.type != cudaMemoryTypeDevice && at.type != cudaMemoryTypeManaged) return -1;
    return at.device;
}

// Switches to the device owning the data for the lifetime of the object.
struct DeviceScope {
    int prev = -1;
    int dev = -1;
    bool switched = false;
    fos_status st = FOS_OK;
    explicit DeviceScope(int d) : dev(d) {
        if (cudaGetDevice(&prev) != cudaSuccess) {
            cudaGetLastError();
            st = FOS_ERR_CUDA;
            return;
        }
        if (prev != dev) {
            if (cudaSetDevice(dev) != cudaSuccess) {
                cudaGetLastError();
                st = FOS_ERR_CUDA;
                return;
            }
            switched = true;
        }
    }
    ~DeviceScope() {
        if (switched) cudaSetDevice(prev);
    }
};

// All listed device pointers must live on one device; returns it or -1.
inline int common_device(std::initializer_list<const void*> ptrs) {
    int dev = -1;
    for (const void* p : ptrs) {
        const int d = device_of(p);
        if (d < 0) return -1;
        if (dev >= 0 && d != dev) return -1;
        dev = d;
    }
    return dev;
}

inline fos_status cuda_status(cudaError_t e) {
    if (e == cudaSuccess) return FOS_OK;
    cudaGetLastError();
    return FOS_ERR_CUDA;
}

inline In in_of(fos_dtype dt) { return dt == FOS_BF16 ? In::BF16 : (dt == FOS_FP16 ? In::F16 : In::F32); }

}  // namespace fos
