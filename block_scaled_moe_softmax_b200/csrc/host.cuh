// host.cuh -- host-side helpers shared by the entry points' translation units: the error text,
// pointer checks, tensor-map encoding and the device switch of a call.  Defined in api.cu.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace moe_mx {

// Record the calling thread's error text and return `code`.
int fail(int code, const char *fmt, ...);
int cuda_fail(cudaError_t e, const char *what);
void clear_error();

bool is_device_ptr(const void *p, int dev);
// MOE_MX_OK, or MOE_MX_ERR_INVALID_ARG unless p is a 16-byte aligned device pointer on dev.
int check_ptr(const void *p, int dev, const char *name);

// Tensor map of `rank` dimensions (innermost first): dims in elements, strides in bytes of
// dimensions 1..rank-1, box in elements; 128-byte swizzle.
int encode_nd(CUtensorMap *map, CUtensorMapDataType dt, int rank, const void *ptr, const cuuint64_t *dims,
              const cuuint64_t *strides, const cuuint32_t *box);

inline int64_t round_up(int64_t v, int64_t m) { return (v + m - 1) / m * m; }

// The current device switched to `dev` for the lifetime of the object.
struct DeviceGuard {
    int prev = 0, dev;
    explicit DeviceGuard(int d) : dev(d)
    {
        cudaGetDevice(&prev);
        if (prev != dev)
            cudaSetDevice(dev);
    }
    ~DeviceGuard()
    {
        if (prev != dev)
            cudaSetDevice(prev);
    }
};

} // namespace moe_mx
