// Host helpers shared by the C ABI's entry points (wl_abi.cpp, wl_layer_abi.cpp):
// status messages, alignment and overlap checks.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include "wl.h"

namespace wl {

// WL_LOG was set when the process first asked.
bool log_on();
// Records the calling thread's message (wl_last_error) and returns st.
wl_status fail(wl_status st, const char *fmt, ...) __attribute__((format(printf, 2, 3)));
// Clears it and returns WL_OK.
wl_status ok();
const char *last_message();

namespace abi {

constexpr size_t kAlign = 256;

inline size_t round_up(size_t v, size_t a) { return (v + a - 1) / a * a; }

inline bool aligned(const void *p, size_t a) { return ((uintptr_t)p & (a - 1)) == 0; }

struct Range {
    const void *p;
    size_t bytes;
};

inline bool overlaps(Range a, Range b) {
    if (!a.p || !b.p || a.bytes == 0 || b.bytes == 0) return false;
    const uintptr_t a0 = (uintptr_t)a.p, b0 = (uintptr_t)b.p;
    return a0 < b0 + b.bytes && b0 < a0 + a.bytes;
}

// Rows of `width` bytes, `ld` bytes apart.
struct Rows {
    const void *p;
    size_t rows, width, ld;
};

inline Range extent(Rows r) { return {r.p, r.rows ? (r.rows - 1) * r.ld + r.width : 0}; }

// Whether two sets of rows share a byte. Rows of one pitch whose columns are
// disjoint (Q, K and V side by side) do not; for unequal pitches it is enough
// that the extents meet.
inline bool rows_overlap(const Rows &a, const Rows &b) {
    if (!overlaps(extent(a), extent(b))) return false;
    if (a.ld != b.ld || a.ld == 0) return true;
    const size_t ld = a.ld;
    const uintptr_t a0 = (uintptr_t)a.p % ld, b0 = (uintptr_t)b.p % ld;
    const size_t delta = (b0 + ld - a0) % ld;   // b's first column behind a's, modulo the pitch
    return !(delta >= a.width && delta + b.width <= ld);
}

}  // namespace abi
}  // namespace wl
