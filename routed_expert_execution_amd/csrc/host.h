// What the host files share: the context as C entry points see it.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/moe.h"

namespace moe {
namespace host {

// Note the message on the context (if there is one) and return the status.
moe_status fail(moe_ctx* c, moe_status st, const char* fmt, ...) __attribute__((format(printf, 3, 4)));
moe_status need_device(moe_ctx* c);  // MOE_EINVAL for a host-only context
int device_of(const moe_ctx* c);
int* error_word(const moe_ctx* c);   // device

// The device of the context is the current one while this lives.
struct DeviceGuard {
    int prev = -1;
    bool changed = false;
    explicit DeviceGuard(int dev) {
        if (dev >= 0 && hipGetDevice(&prev) == hipSuccess && prev != dev) {
            changed = hipSetDevice(dev) == hipSuccess;
        }
    }
    ~DeviceGuard() { if (changed) (void)hipSetDevice(prev); }
};

inline bool aligned_to(const void* p, size_t n) { return ((uintptr_t)p) % n == 0; }
inline bool dtype_valid(int32_t dtype) { return dtype == MOE_F32 || dtype == MOE_BF16; }
inline int elem_bytes(int32_t dtype) { return dtype == MOE_BF16 ? 2 : 4; }

}  // namespace host
}  // namespace moe
