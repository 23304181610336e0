// What the kernels of latent attention share: their job, and the one-row routine that
// the others fall back to.
#pragma once

#include <type_traits>

#include "wl_attn_mfma.h"
#include "wl_serve.h"

namespace wl {

// a: latent queries [T][heads][latent + rot] over one key/value head whose rows are
// the values too, first `latent` elements of them; a.o: [T][heads][latent], and the outputs of
// pieces of divided keys. What something is formed from yet (pieces to be joined, outputs that W^V
// is applied to) is fp32.
struct CoreArgs {
    AttnJob a;
    Split sp;
    int rot;
    int wide;   // a.o is fp32
};

// Which kernel: waves over tiles of 16 rows (the others over keys), whether queries are fp32, as
// the product into the latent space leaves them (else bf16, as given).
struct CoreKind {
    int row_waves;
    bool exact;
};
// Workgroups of it that share a CU. At a latent of 512 widened codes, and remainders of queries, take more
// registers than half a SIMD has.
constexpr int workgroups_per_cu(int fmt, int latent, int row_waves, bool exact) {
    return row_waves == 4 && (latent < 512 || (fmt == kFmtBf16 && !exact)) ? 2 : 1;
}
void launch_latent_tile(const CoreArgs &x, int fmt, const CoreKind &k, unsigned blocks, hipStream_t s);

// Products of every token and head (k_latent_heads.hip): into the latent space, where queries are
// fp32, and out of it, with the join of divided keys.
void launch_absorb(const LatentJob &a, float *out, hipStream_t s);
void launch_absorb_f32(const LatentJob &a, float *out, hipStream_t s);
void launch_up(const LatentJob &a, const CoreArgs &x, bool f32, hipStream_t s);
void launch_join(const CoreArgs &x, bool f32, hipStream_t s);

// The core in fp32 (k_latent_f32.hip).
void launch_latent_f32(const CoreArgs &x, const CoreKind &k, unsigned blocks, hipStream_t s);

// The expanded form, of heads first .. first + heads - 1 (k_latent_expand.hip). a: the call's
// own q and o, [T][n_q][nope + rot] and [T][n_q][value].
struct ExpandArgs {
    AttnJob a;
    const void *w;
    uint16_t *k, *v;       // [n_seq][heads][keys][nope], [value], fp16
    float *scales;         // [n_seq][heads][keys / 32][2][32]: what a row of k, and of v, is to be multiplied with
    int rot, first, heads;
    int keys;              // room of a sequence, a multiple of 128
    int blocks, tiles;     // of 128 keys, of 128 queries of a sequence, at most
};
void launch_expanded(const ExpandArgs &x, int d, hipStream_t s);

// The power of two that brings a row's largest element to 2^14 .. 2^15 in fp16, and its inverse. What lies up
// to 2^28 below the largest has fp16's full precision then, 2^-11; an infinity stays one.
struct HalfScale {
    float up, down;
};
__device__ __forceinline__ HalfScale half_scale(float most) {
    const int k = 14 - min(max((int)(__float_as_uint(most) >> 23) - 127, -112), 127);
    return {__uint_as_float((uint32_t)(127 + k) << 23), __uint_as_float((uint32_t)(127 - k) << 23)};
}

// Bytes of a cache row.
template <int F>
__device__ __forceinline__ int latent_row_bytes(int latent, int rot) {
    return F == kFmtE4m3 ? latent + 2 * rot : (latent + rot) * (F == kFmtF32 ? 4 : 2);
}

__device__ __forceinline__ float element(const uint16_t *p) { return bf16_f(ldg(p)); }
__device__ __forceinline__ float element(const float *p) { return ldg(p); }

// One wave, one query row (token i, head h), keys [j0, j1): the definition, key by key,
// with the running maximum m (in powers of two) and sum l of a softmax. A key that the
// query does not see is not read. Lane holds output elements 8 lane .. + 7 in acc
// (unnormalised).
template <class E, int F>
__device__ void latent_row(const AttnJob &a, int rot, const Seq &q, int i, int h, int j0, int j1, float (&acc)[8], float &m, float &l) {
    typedef typename std::conditional<F == kFmtF32, float, uint16_t>::type C;   // of the key
    const int lane = threadIdx.x & 63, L = a.c.d;
    const bool on = 8 * lane < L, key = lane < rot;
    const Sees v = sees(a, q, i);
    float qv[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    const E *qp = static_cast<const E *>(a.q) + (size_t)(q.q0 + i) * a.ldq + (size_t)h * (L + rot);
    if (on) {
        query4(qp + 8 * lane, qv);
        query4(qp + 8 * lane + 4, qv + 4);
    }
    const float qr = key ? element(qp + L + lane) : 0.0f;
    m = kNegInf, l = 0.0f;
#pragma unroll
    for (int e = 0; e < 8; ++e) acc[e] = 0.0f;
    const int bytes = latent_row_bytes<F>(L, rot);
    j0 = v.tree ? min(max(j0, min(v.lo, max(q.ctx, 0))), j1) : max(j0, v.lo);
    j1 = v.tree ? j1 : min(j1, v.hi);
    for (int j = j0; j < j1; ++j) {
        if (!visible(a, q, v, j)) continue;
        const int page = a.c.table[(int64_t)q.s * a.c.max_pages + (j >> a.c.page_shift)];
        if ((unsigned)page >= (unsigned)a.c.n_pages) continue;
        const int64_t row = ((int64_t)page << a.c.page_shift) + (j & ((1 << a.c.page_shift) - 1));
        const char *at = static_cast<const char *>(a.c.k) + row * bytes;
        float k[8] = {0, 0, 0, 0, 0, 0, 0, 0};
        if (on) {
            cache4<F>(at, 8 * lane, k);
            cache4<F>(at, 8 * lane + 4, k + 4);
        }
        const float r = key ? element(reinterpret_cast<const C *>(at + (F == kFmtE4m3 ? L : L * (int)sizeof(C))) + lane) : 0.0f;
        float s = 0.0f, scale = 1.0f;
#pragma unroll
        for (int e = 0; e < 8; ++e) s += qv[e] * k[e];
        if (F == kFmtE4m3) s *= scale = a.c.k_scale[row];
        s = wave_sum(s + qr * r) * a.scale2;
        if (s == kNegInf) continue;
        const float n = s > m ? s : m;   // a NaN score leaves m and makes p NaN
        const float up = m == n ? 1.0f : __builtin_amdgcn_exp2f(m - n);
        const float p = __builtin_amdgcn_exp2f(s - (n == kNegInf ? 0.0f : n));
        m = n;
        l = l * up + p;
        if (l != l) break;   // the row is NaN, whatever follows
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[e] = acc[e] * up + (p != 0.0f ? p * (scale * k[e]) : 0.0f);
    }
}

}  // namespace wl
