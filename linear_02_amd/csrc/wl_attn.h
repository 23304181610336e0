// What the attention kernels share: which keys a query sees, where they lie, and
// the one-row routine that every other kernel falls back to.
#pragma once

#include "wl_device.h"
#include "wl_layer.h"

namespace wl {

constexpr float kNegInf = -__builtin_inff();

// One sequence of the batch.
struct Seq {
    int s, q0, rows, m;   // first row of q, rows with a result, new tokens
    int kv, ctx;          // keys, keys before the new tokens (may be negative)
};

__device__ __forceinline__ Seq seq_of(const AttnJob &a, int s) {
    Seq q;
    q.s = s;
    q.q0 = min(max(a.q_start[s], 0), a.T);
    const int end = min(max(a.q_start[s + 1], q.q0), a.T);
    q.m = end - q.q0;
    q.rows = min(q.m, a.max_q);
    const int64_t room = (int64_t)a.c.max_pages << a.c.page_shift;
    const int len = min(a.kv_len[s], a.max_kv);
    q.kv = max((int)(len < room ? len : room), 0);
    q.ctx = a.kv_len[s] - q.m;
    return q;
}

// What query i of a sequence sees: slots [lo, hi), and in the tree mask new token
// j (slot ctx + j) where bit j of `tree` is set.
struct Sees {
    int lo, hi;
    const uint32_t *tree;
};

__device__ __forceinline__ Sees sees(const AttnJob &a, const Seq &q, int i) {
    Sees v{0, 0, nullptr};
    if (i >= q.rows) return v;
    const int at = q.ctx + i;   // its own slot
    if (a.mask == kMaskFull) {
        v.hi = q.kv;
    } else if (a.mask == kMaskCausal) {
        v.hi = max(min(at + 1, q.kv), 0);
        if (a.window) v.lo = max(at - a.window + 1, 0);
    } else {
        const int t = q.q0 + i;
        v.hi = max(min(q.ctx, q.kv), 0);
        if (a.window) v.lo = (int)min(max((int64_t)(a.q_pos ? a.q_pos[t] : at) - a.window + 1, (int64_t)0), (int64_t)0x7FFFFFFF);
        v.tree = a.tree + (size_t)t * a.tree_words;
    }
    return v;
}

__device__ __forceinline__ bool visible(const AttnJob &a, const Seq &q, const Sees &v, int j) {
    if (j >= v.lo && j < v.hi) return true;
    if (!v.tree || j < q.ctx || j >= q.kv) return false;
    const int64_t b = (int64_t)j - q.ctx;
    return b < 32ll * a.tree_words && (v.tree[b >> 5] >> (b & 31) & 1u);
}

// Four elements of a cache row as fp32, at element `at` of the pool.
template <int F>
__device__ __forceinline__ void cache4(const void *pool, int64_t at, float *v) {
    if (F == kFmtBf16) {
        const u32x2 w = ldg(reinterpret_cast<const u32x2 *>(static_cast<const uint16_t *>(pool) + at));
        v[0] = bf16_f(w.x & 0xFFFFu), v[1] = __uint_as_float(w.x & 0xFFFF0000u);
        v[2] = bf16_f(w.y & 0xFFFFu), v[3] = __uint_as_float(w.y & 0xFFFF0000u);
    } else if (F == kFmtF32) {
        const f32x4 w = ldg(reinterpret_cast<const f32x4 *>(static_cast<const float *>(pool) + at));
        v[0] = w.x, v[1] = w.y, v[2] = w.z, v[3] = w.w;
    } else {
        const uint32_t c = ldg(reinterpret_cast<const uint32_t *>(static_cast<const uint8_t *>(pool) + at));
        if (F == kFmtInt8) {
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] = (float)(int8_t)(c >> (8 * e));
        } else {
            const auto lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)c, false), hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)c, true);
            v[0] = lo[0], v[1] = lo[1], v[2] = hi[0], v[3] = hi[1];
        }
    }
}

__device__ __forceinline__ void query4(const uint16_t *p, float *v) {
    const u32x2 w = ldg(reinterpret_cast<const u32x2 *>(p));
    v[0] = bf16_f(w.x & 0xFFFFu), v[1] = __uint_as_float(w.x & 0xFFFF0000u);
    v[2] = bf16_f(w.y & 0xFFFFu), v[3] = __uint_as_float(w.y & 0xFFFF0000u);
}
__device__ __forceinline__ void query4(const float *p, float *v) {
    const f32x4 w = ldg(reinterpret_cast<const f32x4 *>(p));
    v[0] = w.x, v[1] = w.y, v[2] = w.z, v[3] = w.w;
}

// One wave, one query row and head, keys [j0, j1): the definition, key by key,
// with the running maximum m (in powers of two) and sum l of a softmax. A key the
// query does not see is not read. Lane holds output elements 4 lane .. + 3 in acc
// (unnormalised).
template <class E, int F>
__device__ void one_row(const AttnJob &a, const Seq &q, int i, int h, int j0, int j1, float *acc, float &m, float &l) {
    const int lane = threadIdx.x & 63, d = a.c.d;
    const bool on = 4 * lane < d;
    const Sees v = sees(a, q, i);
    float qv[4] = {0, 0, 0, 0};
    if (on) query4(static_cast<const E *>(a.q) + (size_t)(q.q0 + i) * a.ldq + (size_t)h * d + 4 * lane, qv);
    m = kNegInf, l = 0.0f;
#pragma unroll
    for (int e = 0; e < 4; ++e) acc[e] = 0.0f;
    const int kvh = h / a.group;
    j0 = v.tree ? min(max(j0, min(v.lo, max(q.ctx, 0))), j1) : max(j0, v.lo);
    j1 = v.tree ? j1 : min(j1, v.hi);
    for (int j = j0; j < j1; ++j) {
        if (!visible(a, q, v, j)) continue;
        const int page = a.c.table[(int64_t)q.s * a.c.max_pages + (j >> a.c.page_shift)];
        if ((unsigned)page >= (unsigned)a.c.n_pages) continue;
        const int64_t row = (((int64_t)page * a.c.n_kv + kvh) << a.c.page_shift) + (j & ((1 << a.c.page_shift) - 1));
        float k[4] = {0, 0, 0, 0}, w[4] = {0, 0, 0, 0};
        if (on) {
            cache4<F>(a.c.k, row * d + 4 * lane, k);
            cache4<F>(a.c.v, row * d + 4 * lane, w);
        }
        float s = wave_sum(qv[0] * k[0] + qv[1] * k[1] + qv[2] * k[2] + qv[3] * k[3]);
        float vs = 1.0f;
        if (F == kFmtInt8 || F == kFmtE4m3) s *= a.c.k_scale[row], vs = a.c.v_scale[row];
        s *= a.scale2;
        if (s == kNegInf) continue;
        const float n = s > m ? s : m;   // a NaN score leaves m and makes p NaN
        const float up = m == n ? 1.0f : __builtin_amdgcn_exp2f(m - n);
        const float p = __builtin_amdgcn_exp2f(s - (n == kNegInf ? 0.0f : n));
        m = n;
        l = l * up + p;
        if (l != l) break;   // the row is NaN, whatever follows
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[e] = acc[e] * up + (p != 0.0f ? p * (vs * w[e]) : 0.0f);
    }
}

__device__ __forceinline__ void put4(uint16_t *p, const float *v) {
    *reinterpret_cast<u32x2 *>(p) =
        u32x2{f_bf16(v[0]) | (uint32_t)f_bf16(v[1]) << 16, f_bf16(v[2]) | (uint32_t)f_bf16(v[3]) << 16};
}
__device__ __forceinline__ void put4(float *p, const float *v) { *reinterpret_cast<f32x4 *>(p) = f32x4{v[0], v[1], v[2], v[3]}; }

}  // namespace wl
