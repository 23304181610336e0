// Norms around a block, fused with its gate and its residual:
//
//   p  = post ? rms(y) (post + offset) : y
//   x' = res_scale x + branch_scale gate p
//   n  = rms(x') (pre + offset),    rms(z) = z / sqrt(mean z^2 + eps)
//
// Bound by memory: x, y (and a per-token gate) are read once, x' and n written
// once; a row stays in registers between its two sums, in fp32. Rows of up to 2048
// elements belong to one wave (no barrier; four rows per workgroup), longer ones to
// a workgroup of one thread per 8 elements, up to 1024 threads: the fewer pieces a
// thread holds, the more rows a CU has under way. Every load of a row, weights too,
// is issued before the first sum: a single row is one round trip to memory and two
// reductions. Large results are stored past the caches.
// 2048 rows of 5376 in bf16, gated per token (110 MB): 34.4 us with four waves of
// three pieces and plain stores, 25.8 us with streaming stores, 24.3 us with twelve
// waves of one piece too (4.5 TB/s; a large copy reaches 5.1 TB/s). One row of
// 1152: 3.9 us.
#include "wl_device.h"
#include "wl_layer.h"

namespace wl {

namespace {

__device__ __forceinline__ void load8(const uint16_t *p, float *v) {
    const u32x4 w = ldg(reinterpret_cast<const u32x4 *>(p));
    const uint32_t r[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        v[2 * e] = bf16_f(r[e] & 0xFFFFu);
        v[2 * e + 1] = __uint_as_float(r[e] & 0xFFFF0000u);
    }
}
__device__ __forceinline__ void load8(const float *p, float *v) {
    const f32x4 a = ldg(reinterpret_cast<const f32x4 *>(p)), b = ldg(reinterpret_cast<const f32x4 *>(p) + 1);
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
    v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
}
template <bool S, class V>
__device__ __forceinline__ void put(V *p, V v) {
    if (S)
        __builtin_nontemporal_store(v, p);
    else
        *p = v;
}
template <bool S>
__device__ __forceinline__ void store8(uint16_t *p, const float *v) {
    uint32_t r[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) r[e] = f_bf16(v[2 * e]) | (uint32_t)f_bf16(v[2 * e + 1]) << 16;
    put<S>(reinterpret_cast<u32x4 *>(p), u32x4{r[0], r[1], r[2], r[3]});
}
template <bool S>
__device__ __forceinline__ void store8(float *p, const float *v) {
    put<S>(reinterpret_cast<f32x4 *>(p), f32x4{v[0], v[1], v[2], v[3]});
    put<S>(reinterpret_cast<f32x4 *>(p) + 1, f32x4{v[4], v[5], v[6], v[7]});
}

// Sum over the WAVES waves that hold a row, in wave order, returned everywhere.
template <int WAVES>
__device__ __forceinline__ float row_sum(float v, float *slot) {
    v = wave_sum(v);
    if (WAVES == 1) return v;
    if ((threadIdx.x & 63) == 0) slot[threadIdx.x >> 6] = v;
    __syncthreads();
    float s = slot[0];
#pragma unroll
    for (int w = 1; w < WAVES; ++w) s += slot[w];
    return s;
}

// NP 8-element pieces per thread, WAVES waves per row, S: results past the caches.
template <class E, int NP, int WAVES, bool S>
__global__ __launch_bounds__(WAVES == 1 ? 256 : WAVES * 64) void norm_kernel(NormJob a) {
    __shared__ float sums[2][16];
    constexpr int kThreads = WAVES * 64;
    const int t = WAVES == 1 ? blockIdx.x * 4 + (threadIdx.x >> 6) : blockIdx.x;
    if (WAVES == 1 && t >= a.T) return;
    const int tid = WAVES == 1 ? threadIdx.x & 63 : threadIdx.x;
    const size_t row = (size_t)t * a.d;
    const E *x = static_cast<const E *>(a.x) + row, *y = static_cast<const E *>(a.y) + row;
    const E *gate = static_cast<const E *>(a.gate) + (size_t)t * a.gate_ld;
    const E *post = static_cast<const E *>(a.post), *pre = static_cast<const E *>(a.pre);

    const float pre_offset = a.pre ? a.offset : 0.0f;   // an absent weight is 1, whatever the offset

    float r[NP][8], p[NP][8], g[NP][8], wp[NP][8], wn[NP][8];
#pragma unroll
    for (int i = 0; i < NP; ++i) {
        const int at = (tid + i * kThreads) * 8;
#pragma unroll
        for (int e = 0; e < 8; ++e) r[i][e] = p[i][e] = 0.0f, g[i][e] = wp[i][e] = wn[i][e] = 1.0f;
        if (at >= a.d) continue;
        load8(x + at, r[i]);
        if (a.y) load8(y + at, p[i]);
        if (a.y && a.gate) load8(gate + at, g[i]);
        if (a.y && a.post) load8(post + at, wp[i]);
        if (a.n_out && a.pre) load8(pre + at, wn[i]);
    }
    if (a.y && a.post) {
        float s = 0.0f;
#pragma unroll
        for (int i = 0; i < NP; ++i)
#pragma unroll
            for (int e = 0; e < 8; ++e) s += p[i][e] * p[i][e];
        const float inv = rsqrtf(row_sum<WAVES>(s, sums[0]) / a.d + a.eps);
#pragma unroll
        for (int i = 0; i < NP; ++i)
#pragma unroll
            for (int e = 0; e < 8; ++e) p[i][e] *= inv * (wp[i][e] + a.offset);
    }
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < NP; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            r[i][e] = a.res_scale * r[i][e];
            if (a.y) r[i][e] += a.branch_scale * g[i][e] * p[i][e];
            s += r[i][e] * r[i][e];
        }
    float inv = 0.0f;
    if (a.n_out) inv = rsqrtf(row_sum<WAVES>(s, sums[1]) / a.d + a.eps);
    E *xo = static_cast<E *>(a.x_out) + row, *no = static_cast<E *>(a.n_out) + row;
#pragma unroll
    for (int i = 0; i < NP; ++i) {
        const int at = (tid + i * kThreads) * 8;
        if (at >= a.d) continue;
        if (a.x_out) store8<S>(xo + at, r[i]);
        if (a.n_out) {
#pragma unroll
            for (int e = 0; e < 8; ++e) r[i][e] *= inv * (wn[i][e] + pre_offset);
            store8<S>(no + at, r[i]);
        }
    }
}

template <class E, int NP, int WAVES>
void run(const NormJob &a, hipStream_t stream) {
    const int blocks = WAVES == 1 ? (a.T + 3) / 4 : a.T;
    const dim3 grid(blocks), block(WAVES == 1 ? 256 : WAVES * 64);
    const size_t written = (size_t)a.T * a.d * sizeof(E) * ((a.x_out != nullptr) + (a.n_out != nullptr));
    if (written > kStreamBytes)
        hipLaunchKernelGGL((norm_kernel<E, NP, WAVES, true>), grid, block, 0, stream, a);
    else
        hipLaunchKernelGGL((norm_kernel<E, NP, WAVES, false>), grid, block, 0, stream, a);
}

template <class E>
void pick(const NormJob &a, hipStream_t stream) {
    const int d = a.d;
    if (d <= 512) return run<E, 1, 1>(a, stream);
    if (d <= 1024) return run<E, 2, 1>(a, stream);
    if (d <= 1536) return run<E, 3, 1>(a, stream);
    if (d <= 2048) return run<E, 4, 1>(a, stream);
    if (d <= 4096) return run<E, 1, 8>(a, stream);
    if (d <= 6144) return run<E, 1, 12>(a, stream);
    if (d <= 8192) return run<E, 1, 16>(a, stream);
    if (d <= 16384) return run<E, 2, 16>(a, stream);
    run<E, 4, 16>(a, stream);
}

}  // namespace

hipError_t launch_norm(const NormJob &a, bool f32, hipStream_t stream) {
    if (f32)
        pick<float>(a, stream);
    else
        pick<uint16_t>(a, stream);
    return hipGetLastError();
}

}  // namespace wl
