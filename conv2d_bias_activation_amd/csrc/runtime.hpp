// Host-side state and checks that every C ABI source of the library shares (api.hip defines
// them): the per-thread error message, the registered workspace and the device query.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include <hip/hip_runtime.h>

namespace c2d {

// Sets the calling thread's conv2d_last_error() text and returns `code`.
int set_error(int code, const char *fmt, ...) __attribute__((format(printf, 2, 3)));
int set_ok();
int hip_fail(hipError_t e, const char *what);

int dtype_bytes(int dtype);  // 0 for an unknown code

inline bool aligned16(const void *p) { return ((uintptr_t)p & 15u) == 0; }

inline bool overlap(const void *a, long long abytes, const void *b, long long bbytes) {
    if (!a || !b) return false;
    uintptr_t a0 = (uintptr_t)a, b0 = (uintptr_t)b;
    return a0 < b0 + (uintptr_t)bbytes && b0 < a0 + (uintptr_t)abytes;
}

// Caller-owned workspace (device scratch) of the calls made from this thread on one
// device, registered by conv2d_set_workspace.
struct Workspace {
    char *p;
    size_t bytes;
};
Workspace current_ws();

int device_cus(int *out);  // compute units of the current device (queried once per device)

}  // namespace c2d
