// mx_check.h -- argument checks and device check shared by the entry points
// (mx_api.hip, mx_block_api.hip, mx_rope_api.hip).  Everything here runs on the host before the
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

// `rows` rows of `width` used bytes, one every `stride` bytes (0: a single row); `n` bytes from the first of them to the
// end of the last, -1 if that leaves 64 bits
struct Range {
    const void *p;
    int64_t n, width, stride;
};
inline Range run(const void *p, int64_t n) { return {p, n, n, 0}; }
// row stride ld, `width` used, in units of `size` bytes
inline Range rows_at(const void *p, int64_t rows, int64_t ld, int64_t width, int64_t size) {
    if (rows <= 0 || width <= 0) return run(p, 0);
    if (width > INT64_MAX / size) return run(p, -1);
    if (rows == 1) return run(p, width * size);
    if (rows - 1 > (INT64_MAX / size - width) / ld) return run(p, -1);
    return {p, ((rows - 1) * ld + width) * size, width * size, ld * size};
}
// no byte belongs to both: their whole extents are disjoint, or the rows of one lie in the gaps of the other's
inline bool disjoint(const Range &a, const Range &b) {
    if (!overlap(a.p, a.n, b.p, b.n)) return true;
    return a.stride > 0 && a.stride == b.stride && interleaved(a.p, a.width, b.p, b.width, a.stride);
}
// every range exists (n >= 0) and no range from `first_out` on overlaps another one
inline mx_status_t check_ranges(const Range *r, int count, int first_out) {
    for (int i = 0; i < count; i++)
        if (r[i].n < 0) return MX_ERR_INVALID_ARG;
    for (int i = first_out; i < count; i++)
        for (int j = 0; j < i; j++)
            if (!disjoint(r[i], r[j])) return MX_ERR_INVALID_ARG;
    return MX_OK;
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
