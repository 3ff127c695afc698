// mx_check.h -- argument checks and device check shared by the entry points
// (mx_api.hip, mx_block_api.hip).  Everything here runs on the host before the
// first launch.
#pragma once
#include <atomic>
#include <string.h>

#include "mx.h"
#include "mx_internal.h"

namespace mx {

constexpr int kMaxDevices = 64;
inline std::atomic<int> g_arch_ok[kMaxDevices];  // 0 unknown, 1 gfx950, 2 other

// An enum parameter's value as the caller passed it.  A C caller may pass any
// int through an enum type, but in C++ a load of an enum object whose value
// lies outside its enumerators' range has no defined meaning; the entry
// points therefore read their enum parameters' bytes as an int and validate
// that.
template <class E>
inline int raw(const E &e) {
    static_assert(sizeof(E) == sizeof(int), "the ABI's enums are int-sized");
    int v;
    memcpy(&v, &e, sizeof v);
    return v;
}

inline bool fmt_ok(int f) { return f == MX_E4M3 || f == MX_E5M2 || f == MX_E2M1; }

inline int64_t code_bytes(int64_t n, int fmt) { return fmt == MX_E2M1 ? n / 2 : n; }

// half-open byte ranges [p, p + n) overlap
inline bool overlap(const void *p, int64_t n, const void *q, int64_t m) {
    if (n <= 0 || m <= 0) return false;
    const uintptr_t a = (uintptr_t)p, b = (uintptr_t)q;
    return a < b + (uintptr_t)m && b < a + (uintptr_t)n;
}

// Rows of wp bytes from p and of wq bytes from q, both one row every `stride` bytes, any number of them: every row
// of the second lies in the gap after a row of the first.
inline bool interleaved(const void *p, int64_t wp, const void *q, int64_t wq, int64_t stride) {
    int64_t d = (int64_t)((uintptr_t)q - (uintptr_t)p) % stride;
    if (d < 0) d += stride;
    return d >= wp && d + wq <= stride;
}

inline mx_status_t check_device() {
    int dev = -1;
    if (hipGetDevice(&dev) != hipSuccess || dev < 0) return MX_ERR_HIP;
    if (dev >= kMaxDevices) return MX_ERR_UNSUPPORTED;
    int st = g_arch_ok[dev].load(std::memory_order_relaxed);
    if (st == 0) {
        hipDeviceProp_t prop;
        if (hipGetDeviceProperties(&prop, dev) != hipSuccess) return MX_ERR_HIP;
        st = strncmp(prop.gcnArchName, "gfx950", 6) == 0 ? 1 : 2;
        g_arch_ok[dev].store(st, std::memory_order_relaxed);
    }
    return st == 1 ? MX_OK : MX_ERR_UNSUPPORTED;
}

inline mx_status_t launched(hipError_t e) { return e == hipSuccess ? MX_OK : MX_ERR_HIP; }

}  // namespace mx
