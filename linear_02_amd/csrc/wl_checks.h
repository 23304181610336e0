// Argument checks shared by the operations around the projections
// (wl_layer_abi.cpp, wl_serve_abi.cpp): rows, overlaps, rotations.
#pragma once

#include <hip/hip_runtime.h>

#include <initializer_list>

#include "wl_abi.h"

namespace wl {
namespace abi {

constexpr int64_t kMaxElems = (int64_t)1 << 31;
constexpr int32_t kMaxTokens = 1 << 24;        // a wave each stays inside a launch's 2^32 threads
constexpr int32_t kMaxKeys = 1 << 30;          // key numbers stay in int32 a few tiles past the last
constexpr int64_t kMaxWorkgroups = (1 << 23) - 1;   // of up to 512 threads: fewer than 2^32 in a launch

inline wl_status check_dtype(int32_t dtype) {
    if (dtype != WL_DTYPE_BF16 && dtype != WL_DTYPE_F32)
        return fail(WL_ERR_UNSUPPORTED, "dtype=%d is neither WL_DTYPE_BF16 nor WL_DTYPE_F32", dtype);
    return WL_OK;
}

inline size_t bytes_of(int32_t dtype) { return dtype == WL_DTYPE_F32 ? 4 : 2; }

inline wl_status need(const void *p, size_t align, const char *name) {
    if (!p) return fail(WL_ERR_INVALID_ARG, "%s is NULL", name);
    if (!aligned(p, align)) return fail(WL_ERR_INVALID_ARG, "%s is not %zu-byte aligned", name, align);
    return WL_OK;
}

// A tensor of T rows of `width` elements, ld apart.
inline wl_status check_rows(const void *p, int32_t T, int64_t width, int32_t ld, const char *name) {
    const wl_status st = need(p, 16, name);
    if (st != WL_OK) return st;
    if (ld < width || ld % 8)
        return fail(WL_ERR_INVALID_ARG, "%s: ld=%d must be a multiple of 8 and at least %lld", name, ld, (long long)width);
    if ((int64_t)T * ld >= kMaxElems) return fail(WL_ERR_INVALID_ARG, "%s spans 2^31 or more elements", name);
    if (T > kMaxTokens) return fail(WL_ERR_UNSUPPORTED, "T=%d exceeds %d", T, kMaxTokens);
    return WL_OK;
}

struct Named {
    Rows r;
    const char *name;
};

inline Rows flat(const void *p, size_t bytes) { return {p, 1, bytes, bytes}; }

inline bool same(const Rows &a, const Rows &b) { return a.p == b.p && a.rows == b.rows && a.width == b.width && a.ld == b.ld; }

// `out` may not meet any of `ins` but `alias` (exactly).
inline wl_status check_out(const Named &out, std::initializer_list<Named> ins, std::initializer_list<const void *> alias = {}) {
    for (const Named &in : ins) {
        if (!in.r.p || !rows_overlap(out.r, in.r)) continue;
        bool allowed = false;
        for (const void *p : alias) allowed = allowed || (p == in.r.p && same(out.r, in.r));
        if (!allowed) return fail(WL_ERR_INVALID_ARG, "%s overlaps %s", out.name, in.name);
    }
    return WL_OK;
}

inline wl_status check_rotary(const wl_rotary *r, int32_t d, bool pos_needed) {
    wl_status st;
    if (!r) return WL_OK;
    if ((st = need(r->freq, 8, "freq")) != WL_OK) return st;
    if (pos_needed || r->pos)
        if ((st = need(r->pos, 4, "pos")) != WL_OK) return st;
    if (r->rot < 8 || r->rot % 8 || r->rot > d)
        return fail(WL_ERR_INVALID_ARG, "rot=%d must be a multiple of 8 from 8 to d=%d", r->rot, d);
    if (r->style != WL_ROPE_HALF && r->style != WL_ROPE_INTERLEAVED)
        return fail(WL_ERR_INVALID_ARG, "style=%d is neither WL_ROPE_HALF nor WL_ROPE_INTERLEAVED", r->style);
    return WL_OK;
}

inline Named row_set(const void *p, int32_t T, int64_t width, int32_t ld, int32_t dtype, const char *name) {
    return {{p, (size_t)T, (size_t)width * bytes_of(dtype), (size_t)ld * bytes_of(dtype)}, name};
}

inline wl_status launched(hipError_t e, const char *what) {
    if (e != hipSuccess) return fail(WL_ERR_HIP, "%s launch failed: %s", what, hipGetErrorString(e));
    return ok();
}

}  // namespace abi
}  // namespace wl
