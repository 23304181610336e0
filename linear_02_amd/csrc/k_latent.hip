// Attention over the latent cache: which form and kernels run, and the join of divided keys.
#include <type_traits>

#include "wl_latent.h"

namespace wl {

namespace {

// Every query row by a wave of its own, key by key.
template <class E, int F>
__global__ __launch_bounds__(256) void rows_kernel(CoreArgs x) {
    const AttnJob &a = x.a;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    const int64_t w = (int64_t)blockIdx.x * 4 + wave, per = (int64_t)a.max_q * a.group;
    const int s = (int)(w / per), r = (int)(w - (int64_t)s * per);
    if (s >= a.c.n_seq) return;
    const Seq q = seq_of(a, s);
    if (r >= q.rows * a.group) return;
    const int i = r / a.group, h = r - i * a.group;
    float acc[8], m, l;
    latent_row<E, F>(a, x.rot, q, i, h, 0, q.kv, acc, m, l);
    if (8 * lane >= a.c.d) return;
#pragma unroll
    for (int e = 0; e < 8; ++e) acc[e] = l == 0.0f ? 0.0f : acc[e] / l;
    E *o = static_cast<E *>(a.o) + (size_t)(q.q0 + i) * a.ldo + (size_t)h * a.c.d + 8 * lane;
    put4(o, acc);
    put4(o + 4, acc + 4);
}

// q' = W^K^T q of every token and head, its rotated part beside it.
template <class E>
__global__ __launch_bounds__(256) void absorb_kernel(LatentJob a, E *out) {
    __shared__ float qs[256];
    const int t = blockIdx.x / a.a.n_q, h = blockIdx.x - t * a.a.n_q, L = a.a.c.d, N = a.nope, R = a.rot;
    const E *q = static_cast<const E *>(a.q) + (size_t)t * a.ldq + (size_t)h * (N + R);
    E *o = out + ((size_t)t * a.a.n_q + h) * (L + R);
    if ((int)threadIdx.x < N) qs[threadIdx.x] = element(q + threadIdx.x);
    if ((int)threadIdx.x < R) o[L + threadIdx.x] = q[N + threadIdx.x];
    __syncthreads();
    const E *w = static_cast<const E *>(a.w) + (size_t)h * (N + a.value) * L;
    for (int l = threadIdx.x; l < L; l += 256) {
        float s = 0.0f;
        for (int n = 0; n < N; ++n) s += qs[n] * element(w + (size_t)n * L + l);
        o[l] = std::is_same<E, float>::value ? (E)s : (E)f_bf16(s);
    }
}

// o = W^V o' of every token and head that has a result: of a sequence's first max_q rows.
template <class E>
__global__ __launch_bounds__(256) void up_kernel(LatentJob a, const E *in) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int t = blockIdx.x / a.a.n_q, h = blockIdx.x - t * a.a.n_q, L = a.a.c.d, N = a.nope, V = a.value;
    if (!has_result(a.a, t)) return;
    const E *x = in + ((size_t)t * a.a.n_q + h) * L;
    const E *w = static_cast<const E *>(a.w) + ((size_t)h * (N + V) + N) * L;
    E *o = static_cast<E *>(a.o) + (size_t)t * a.ldo + (size_t)h * V;
    for (int v = wave; v < V; v += 4) {
        float s = 0.0f;
        for (int l = lane; l < L; l += 64) s += element(x + l) * element(w + (size_t)v * L + l);
        s = wave_sum(s);
        if (lane == 0) o[v] = std::is_same<E, float>::value ? (E)s : (E)f_bf16(s);
    }
}

size_t pad(size_t b) { return (b + 255) & ~(size_t)255; }

size_t element_bytes(bool f32) { return f32 ? 4 : 2; }

}  // namespace

bool latent_can_expand(const LatentJob &, bool) { return false; }

LatentNeeds latent_needs(const LatentJob &a, int, bool f32, int) {
    const size_t rows = (size_t)a.a.T * a.a.n_q;
    LatentNeeds n{0, ((int64_t)a.a.c.n_seq * a.a.max_q * a.a.group + 3) / 4};
    if (a.w) {
        n.scratch = pad(rows * (a.a.c.d + a.rot) * element_bytes(f32)) + pad(rows * a.a.c.d * element_bytes(f32));
        if ((int64_t)rows > n.workgroups) n.workgroups = rows;
    }
    return n;
}

namespace {

template <class E, int F>
hipError_t run(LatentJob a, void *ws, hipStream_t s) {
    const size_t rows = (size_t)a.a.T * a.a.n_q;
    E *q = static_cast<E *>(ws), *o = reinterpret_cast<E *>(static_cast<char *>(ws) + pad(rows * (a.a.c.d + a.rot) * sizeof(E)));
    hipError_t e;
    if (a.w) {
        hipLaunchKernelGGL((absorb_kernel<E>), dim3((unsigned)rows), dim3(256), 0, s, a, q);
        if ((e = hipGetLastError()) != hipSuccess) return e;
        a.a.q = q, a.a.ldq = a.a.n_q * (a.a.c.d + a.rot);
        a.a.o = o, a.a.ldo = a.a.n_q * a.a.c.d;
    }
    const int64_t waves = (int64_t)a.a.c.n_seq * a.a.max_q * a.a.group;
    hipLaunchKernelGGL((rows_kernel<E, F>), dim3((unsigned)((waves + 3) / 4)), dim3(256), 0, s, CoreArgs{a.a, Split{}, a.rot});
    if ((e = hipGetLastError()) != hipSuccess || !a.w) return e;
    hipLaunchKernelGGL((up_kernel<E>), dim3((unsigned)rows), dim3(256), 0, s, a, o);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_latent(const LatentJob &a, int fmt, bool, int, void *ws, hipStream_t s) {
    switch (fmt) {
        case kFmtBf16: return run<uint16_t, kFmtBf16>(a, ws, s);
        case kFmtF32: return run<float, kFmtF32>(a, ws, s);
        default: return run<uint16_t, kFmtE4m3>(a, ws, s);
    }
}

}  // namespace wl
