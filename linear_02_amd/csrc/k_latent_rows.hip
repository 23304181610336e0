// Rows of the latent cache: written, with the latent's norm and the rotation of its key
// (and of Q beside it) in the same launch, and read back.
//
// A row is a token's latent vector and a key that all heads share; of a head of Q, the
// last `rot` elements are rotated. Angles, styles and codes as in k_rows.hip: turns in
// fp64 reduced to a fraction of one, code = round(448 x / most) by one correctly rounded
// quotient.
//
// Bound by memory at prompts (2048 tokens with 128 heads of Q 40 us, 5.2 TB/s), by latency at a few
// tokens (32 of 16 heads 4.4 us). A workgroup takes a token, or
// part of its heads where tokens are few, and forms the token's angles once, in LDS.
// Rows and heads pass as pieces of eight elements; a piece of the rotated part in the
// half style is four elements and their partners, so a pair never leaves its thread and
// q_out may be q. One wave of the first workgroup takes the cache's row, eight elements
// of the latent a lane.
#include <type_traits>

#include "wl_device.h"
#include "wl_serve.h"

namespace wl {

namespace {

constexpr int kThreads = 256;
constexpr int kWorkgroupsWanted = 1024;

__device__ __forceinline__ void load4(const uint16_t *p, float *v) {
    const u32x2 w = ldg(reinterpret_cast<const u32x2 *>(p));
    v[0] = bf16_f(w.x & 0xFFFFu), v[1] = __uint_as_float(w.x & 0xFFFF0000u);
    v[2] = bf16_f(w.y & 0xFFFFu), v[3] = __uint_as_float(w.y & 0xFFFF0000u);
}
__device__ __forceinline__ void load4(const float *p, float *v) {
    const f32x4 w = ldg(reinterpret_cast<const f32x4 *>(p));
    v[0] = w.x, v[1] = w.y, v[2] = w.z, v[3] = w.w;
}
__device__ __forceinline__ void store4(uint16_t *p, const float *v) {
    *reinterpret_cast<u32x2 *>(p) =
        u32x2{f_bf16(v[0]) | (uint32_t)f_bf16(v[1]) << 16, f_bf16(v[2]) | (uint32_t)f_bf16(v[3]) << 16};
}
__device__ __forceinline__ void store4(float *p, const float *v) { *reinterpret_cast<f32x4 *>(p) = f32x4{v[0], v[1], v[2], v[3]}; }

// Place of a token's row in the pool, -1: none.
__device__ __forceinline__ int64_t find_row(const LatentRef &c, int seq, int slot) {
    const int at = slot >> c.page_shift;
    if ((unsigned)seq >= (unsigned)c.n_seq || slot < 0 || at >= c.max_pages) return -1;
    const int page = c.table[(int64_t)seq * c.max_pages + at];
    if ((unsigned)page >= (unsigned)c.n_pages) return -1;
    return ((int64_t)page << c.page_shift) + (slot & ((1 << c.page_shift) - 1));
}

template <int F>
__device__ __forceinline__ int row_bytes(const LatentRef &c) {
    return F == kFmtE4m3 ? c.latent + 2 * c.rot : (c.latent + c.rot) * (F == kFmtF32 ? 4 : 2);
}

// Where piece j of the rotated part lies: elements [o0, o0 + 4) and [o1, o1 + 4).
struct Places {
    int o0, o1;
};
__device__ __forceinline__ Places places(int j, int rot, bool halves) {
    return halves ? Places{4 * j, rot / 2 + 4 * j} : Places{8 * j, 8 * j + 4};
}

// Piece j turned by the token's angles.
__device__ __forceinline__ void turn(float *v, int j, bool halves, const float *cs, const float *sn) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const float c = cs[4 * j + e], s = sn[4 * j + e];
        const float p = halves ? v[e] : v[2 * e], q = halves ? v[e + 4] : v[2 * e + 1];
        const float np = p * c - q * s, nq = p * s + q * c;
        if (halves)
            v[e] = np, v[e + 4] = nq;
        else
            v[2 * e] = np, v[2 * e + 1] = nq;
    }
}

template <class E, int F>
__global__ __launch_bounds__(kThreads) void write_kernel(LatentWriteJob a) {
    __shared__ float cs[kMaxRot / 2], sn[kMaxRot / 2];
    const int t = blockIdx.x / a.parts, part = blockIdx.x - t * a.parts;
    const int seq = a.seq[t];
    if ((unsigned)seq >= (unsigned)a.c.n_seq) return;   // a padding token
    const int slot = a.slot[t], R = a.c.rot, L = a.c.latent;
    const bool turned = a.freq, halves = turned && !a.interleaved;
    if (turned && (int)threadIdx.x < R / 2) {
        double turns = (double)(a.pos ? a.pos[t] : slot) * a.freq[threadIdx.x] * 0.15915494309189533577;   // 1 / (2 pi)
        turns -= rint(turns);
        float s, c;
        sincospif((float)(2.0 * turns), &s, &c);
        cs[threadIdx.x] = c * a.turn_scale, sn[threadIdx.x] = s * a.turn_scale;
    }
    __syncthreads();
    // Q: the heads' pieces, shared by the token's workgroups.
    const int width = a.nope + R, per = width / 8, kept = a.nope / 8;
    const E *q = static_cast<const E *>(a.q) + (size_t)t * a.ldq;
    E *q_out = static_cast<E *>(a.q_out) + (size_t)t * a.ldq_out;
    for (int p = part * kThreads + threadIdx.x; p < a.n_q * per; p += a.parts * kThreads) {
        const int h = p / per, j = p - h * per, at = h * width;
        float v[8];
        if (j < kept) {
            load4(q + at + 8 * j, v);
            load4(q + at + 8 * j + 4, v + 4);
            store4(q_out + at + 8 * j, v);
            store4(q_out + at + 8 * j + 4, v + 4);
        } else {
            const Places o = places(j - kept, R, halves);
            const int from = at + a.nope;
            load4(q + from + o.o0, v);
            load4(q + from + o.o1, v + 4);
            if (turned) turn(v, j - kept, halves, cs, sn);
            store4(q_out + from + o.o0, v);
            store4(q_out + from + o.o1, v + 4);
        }
    }
    // The cache's row, by the last wave.
    if (part != a.parts - 1 || threadIdx.x < kThreads - 64) return;
    const int64_t row = find_row(a.c, seq, slot);
    if (row < 0) return;
    const int lane = threadIdx.x & 63;
    const E *in = static_cast<const E *>(a.in) + (size_t)t * a.ldc;
    char *out = static_cast<char *>(a.c.rows) + row * row_bytes<F>(a.c);
    const bool on = 8 * lane < L;
    float v[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    if (on) {
        load4(in + 8 * lane, v);
        load4(in + 8 * lane + 4, v + 4);
    }
    if (a.norm) {
        float s = 0.0f;
#pragma unroll
        for (int e = 0; e < 8; ++e) s += v[e] * v[e];
        const float inv = rsqrtf(wave_sum(s) / L + a.eps);
        if (on) {
            float g[8];
            load4(static_cast<const E *>(a.norm) + 8 * lane, g);
            load4(static_cast<const E *>(a.norm) + 8 * lane + 4, g + 4);
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] *= inv * (g[e] + a.offset);
        }
    }
    typedef typename std::conditional<F == kFmtF32, float, uint16_t>::type C;   // of the key
    if (F == kFmtE4m3) {
        uint32_t top = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e) top = max(top, __float_as_uint(v[e]) & 0x7FFFFFFFu);   // NaN is above infinity
#pragma unroll
        for (int x = 1; x < 64; x <<= 1) top = max(top, (uint32_t)__shfl_xor((int)top, x));
        const float most = __uint_as_float(top);
        // Both are scaled by the same power of two where the product or a small divisor would leave fp32's range.
        const float s = most > 0x1p64f ? 0x1p-64f : most < 0x1p-64f ? 0x1p64f : 1.0f;
        float y[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] = most == 0.0f ? 0.0f : v[e] * s * 448.0f / (most * s);
        if (on) {
            int lo = __builtin_amdgcn_cvt_pk_fp8_f32(y[0], y[1], 0, false), hi = __builtin_amdgcn_cvt_pk_fp8_f32(y[4], y[5], 0, false);
            lo = __builtin_amdgcn_cvt_pk_fp8_f32(y[2], y[3], lo, true);
            hi = __builtin_amdgcn_cvt_pk_fp8_f32(y[6], y[7], hi, true);
            *reinterpret_cast<u32x2 *>(out + 8 * lane) = u32x2{(uint32_t)lo, (uint32_t)hi};
        }
        if (lane == 0) a.c.scale[row] = most / 448.0f;
        out += L;
    } else {
        if (on) {
            store4(reinterpret_cast<C *>(out) + 8 * lane, v);
            store4(reinterpret_cast<C *>(out) + 8 * lane + 4, v + 4);
        }
        out += L * sizeof(C);
    }
    if (8 * lane < R) {
        const Places o = places(lane, R, halves);
        load4(in + L + o.o0, v);
        load4(in + L + o.o1, v + 4);
        if (turned) turn(v, lane, halves, cs, sn);
        store4(reinterpret_cast<C *>(out) + o.o0, v);
        store4(reinterpret_cast<C *>(out) + o.o1, v + 4);
    }
}

// A wave a token.
template <class E, int F>
__global__ __launch_bounds__(kThreads) void read_kernel(LatentReadJob a) {
    const int t = __builtin_amdgcn_readfirstlane(blockIdx.x * (kThreads / 64) + (threadIdx.x >> 6)), lane = threadIdx.x & 63;
    if (t >= a.T) return;
    const int64_t row = find_row(a.c, a.seq[t], a.slot[t]);
    if (row < 0) return;
    const int L = a.c.latent, R = a.c.rot;
    const char *in = static_cast<const char *>(a.c.rows) + row * row_bytes<F>(a.c);
    E *out = static_cast<E *>(a.out) + (size_t)t * a.ld;
    for (int j = lane; j < (L + R) / 8; j += 64) {
        float v[8];
        if (F == kFmtE4m3 && 8 * j < L) {
            const u32x2 w = ldg(reinterpret_cast<const u32x2 *>(in + 8 * j));
            const float s = a.c.scale[row];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const int c = (int)(k ? w.y : w.x);
                const auto lo = __builtin_amdgcn_cvt_pk_f32_fp8(c, false), hi = __builtin_amdgcn_cvt_pk_f32_fp8(c, true);
                v[4 * k] = lo[0] * s, v[4 * k + 1] = lo[1] * s, v[4 * k + 2] = hi[0] * s, v[4 * k + 3] = hi[1] * s;
            }
        } else {
            typedef typename std::conditional<F == kFmtF32, float, uint16_t>::type C;
            const C *p = F == kFmtE4m3 ? reinterpret_cast<const C *>(in + L) + 8 * j - L : reinterpret_cast<const C *>(in) + 8 * j;
            load4(p, v);
            load4(p + 4, v + 4);
        }
        store4(out + 8 * j, v);
        store4(out + 8 * j + 4, v + 4);
    }
}

}  // namespace

hipError_t launch_latent_write(LatentWriteJob a, int fmt, hipStream_t s) {
    // Workgroups per token: no more than its pieces fill.
    const int pieces = a.n_q * ((a.nope + a.c.rot) / 8), most = (pieces + kThreads - 1) / kThreads;
    const int want = (kWorkgroupsWanted + a.T - 1) / a.T;
    a.parts = want < most ? want : most > 1 ? most : 1;
    const dim3 g((unsigned)((int64_t)a.T * a.parts)), b(kThreads);
    switch (fmt) {
        case kFmtBf16: hipLaunchKernelGGL((write_kernel<uint16_t, kFmtBf16>), g, b, 0, s, a); break;
        case kFmtF32: hipLaunchKernelGGL((write_kernel<float, kFmtF32>), g, b, 0, s, a); break;
        default: hipLaunchKernelGGL((write_kernel<uint16_t, kFmtE4m3>), g, b, 0, s, a);
    }
    return hipGetLastError();
}

hipError_t launch_latent_read(const LatentReadJob &a, int fmt, hipStream_t s) {
    const dim3 g((unsigned)((a.T + 3) / 4)), b(kThreads);
    switch (fmt) {
        case kFmtBf16: hipLaunchKernelGGL((read_kernel<uint16_t, kFmtBf16>), g, b, 0, s, a); break;
        case kFmtF32: hipLaunchKernelGGL((read_kernel<float, kFmtF32>), g, b, 0, s, a); break;
        default: hipLaunchKernelGGL((read_kernel<uint16_t, kFmtE4m3>), g, b, 0, s, a);
    }
    return hipGetLastError();
}

}  // namespace wl
