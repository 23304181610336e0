// Rows of heads: the per-head norm and rotation of Q and K, and the paged cache,
// written (with that norm and rotation in the same launch) and read back.
//
// Rotation: pair (a, b) -> scale (a cos t - b sin t, a sin t + b cos t) with
// t = position * freq. t is formed in turns in fp64 and reduced to a fraction of
// a turn there, so a position of a million loses nothing; cos and sin are fp32.
// Quantised rows: most = max |x| over a head; scale = most / top; code =
// round(top x / most), top = 127 or 448. The quotient is a correctly rounded
// fp32 division of the exact product top * x (bf16 inputs), so a value that lies
// exactly between two codes goes to the even one, which x / scale would decide
// by the rounding of scale.
//
// Bound by memory at prompts (every element read and written once), by latency at
// a few tokens. A head belongs to a power of two of lanes, eight elements each:
// in the half style a lane holds four elements of the first half and their
// partners of the second, so a pair never leaves its lane, and the sum or
// maximum over a head is a few DPP steps. A wave takes 64 / lanes heads at once
// and, at prompts, walks all heads of its token, so that a token's angles are
// formed once; with few tokens the heads are spread over waves.
#include <type_traits>

#include "wl_device.h"
#include "wl_layer.h"

namespace wl {

namespace {

constexpr int kThreads = 256;
// Waves that a call is spread over where its tokens alone are fewer: four per
// SIMD cover the latency of a chunk's loads. 2048 tokens, 48 heads of 256 into an
// int8 cache took 33.2 us on 2048 waves, 27.2 on 4096, 24.7 on 8192, 26.2 on 16384;
// 40 heads rotated alone 18.9, 15.9, 15.7, 16.9.
constexpr int kWavesWanted = 8192;

__device__ __forceinline__ void load4(const uint16_t *p, float *v) {
    const u32x2 w = ldg(reinterpret_cast<const u32x2 *>(p));
    v[0] = bf16_f(w.x & 0xFFFFu), v[1] = __uint_as_float(w.x & 0xFFFF0000u);
    v[2] = bf16_f(w.y & 0xFFFFu), v[3] = __uint_as_float(w.y & 0xFFFF0000u);
}
__device__ __forceinline__ void load4(const float *p, float *v) {
    const f32x4 w = ldg(reinterpret_cast<const f32x4 *>(p));
    v[0] = w.x, v[1] = w.y, v[2] = w.z, v[3] = w.w;
}
// S: past the caches.
template <bool S, class V>
__device__ __forceinline__ void put(V *p, V v) {
    if (S)
        __builtin_nontemporal_store(v, p);
    else
        *p = v;
}
template <bool S = false>
__device__ __forceinline__ void store4(uint16_t *p, const float *v) {
    put<S>(reinterpret_cast<u32x2 *>(p),
           u32x2{f_bf16(v[0]) | (uint32_t)f_bf16(v[1]) << 16, f_bf16(v[2]) | (uint32_t)f_bf16(v[3]) << 16});
}
template <bool S = false>
__device__ __forceinline__ void store4(float *p, const float *v) {
    put<S>(reinterpret_cast<f32x4 *>(p), f32x4{v[0], v[1], v[2], v[3]});
}

__device__ __forceinline__ uint32_t swap16(uint32_t v) { return __builtin_amdgcn_ds_swizzle(v, 0x401F); }   // lane ^ 16

// Sum and maximum over the L lanes of a head, returned in each of them.
template <int L>
__device__ __forceinline__ float head_sum(float v) {
    v += dpp<0xB1>(v);    // lane ^ 1
    v += dpp<0x4E>(v);    // lane ^ 2
    v += dpp<0x141>(v);   // the other quad of eight
    if (L >= 16) v += dpp<0x140>(v);   // the other half of sixteen
    if (L >= 32) v += __uint_as_float(swap16(__float_as_uint(v)));
    return v;
}
// Of bit patterns of magnitudes: NaN is above infinity, so it survives.
template <int L>
__device__ __forceinline__ uint32_t head_max(uint32_t v) {
    auto step = [&](uint32_t o) { v = v > o ? v : o; };
    step(__float_as_uint(dpp<0xB1>(__uint_as_float(v))));
    step(__float_as_uint(dpp<0x4E>(__uint_as_float(v))));
    step(__float_as_uint(dpp<0x141>(__uint_as_float(v))));
    if (L >= 16) step(__float_as_uint(dpp<0x140>(__uint_as_float(v))));
    if (L >= 32) step(swap16(v));
    return v;
}

// Where a token's rows lie; false: nowhere.
__device__ __forceinline__ bool find_row(const CacheRef &c, int seq, int slot, int64_t &first, int &off) {
    const int at = slot >> c.page_shift;
    if ((unsigned)seq >= (unsigned)c.n_seq || slot < 0 || at >= c.max_pages) return false;
    const int page = c.table[(int64_t)seq * c.max_pages + at];
    if ((unsigned)page >= (unsigned)c.n_pages) return false;
    off = slot & ((1 << c.page_shift) - 1);
    first = (int64_t)page * c.n_kv;   // + head: rows of a page and head
    return true;
}

// Four codes of x top / most, packed. Both are scaled by the same power of two
// first where the product or a small divisor would leave fp32's range.
template <int F>
__device__ __forceinline__ uint32_t code4(const float *x, float s, float most) {
    constexpr float top = F == kFmtInt8 ? 127.0f : 448.0f;
    float y[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) y[e] = x[e] * s * top / most;
    if (F == kFmtInt8) {
        uint32_t r = 0;
#pragma unroll
        for (int e = 0; e < 4; ++e) r |= ((uint32_t)(int)rintf(y[e]) & 0xFFu) << (8 * e);
        return r;
    }
    int r = __builtin_amdgcn_cvt_pk_fp8_f32(y[0], y[1], 0, false);
    return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(y[2], y[3], r, true);
}

// E: element type of the rows, F: cache format (kFmtNone: rotation only), L:
// lanes per head.
template <class E, int F, int L>
__global__ __launch_bounds__(kThreads) void rows_kernel(RowsJob a) {
    constexpr int HW = 64 / L;
    const int lane = threadIdx.x & 63, j = lane & (L - 1), sub = lane / L;
    const int wave = __builtin_amdgcn_readfirstlane(blockIdx.x * (kThreads / 64) + (threadIdx.x >> 6));
    const int t = wave / a.waves, part = wave - t * a.waves;
    if (t >= a.T) return;
    bool stored = false;
    int64_t first = 0;
    int off = 0, slot = 0;
    if (F != kFmtNone) {
        const int seq = a.seq[t];
        if ((unsigned)seq >= (unsigned)a.c.n_seq) return;   // a padding token
        slot = a.slot[t];
        stored = find_row(a.c, seq, slot, first, off);
    }
    // This lane's elements: [o0, o0 + 4) and [o1, o1 + 4).
    const bool turned = a.freq && 8 * j < a.rot;
    const bool halves = turned && !a.interleaved;
    const int o0 = halves ? 4 * j : 8 * j, o1 = halves ? a.rot / 2 + 4 * j : 8 * j + 4;
    const bool mine = 8 * j < a.d;
    float cs[4], sn[4];
    if (turned) {
        const double p = (double)(F != kFmtNone && !a.pos ? slot : a.pos[t]);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            double turns = p * a.freq[4 * j + e] * 0.15915494309189533577;   // 1 / (2 pi)
            turns -= rint(turns);
            float s, c;
            sincospif((float)(2.0 * turns), &s, &c);
            cs[e] = c * a.turn_scale, sn[e] = s * a.turn_scale;
        }
    }
    const int heads = a.n_q + a.n_k + (F != kFmtNone ? a.n_v : 0);
    for (int h0 = part * HW; h0 < heads; h0 += a.waves * HW) {
        const int h = h0 + sub;
        const bool is_q = h < a.n_q, is_k = !is_q && h < a.n_q + a.n_k;
        const int hk = h - a.n_q, hv = hk - a.n_k;
        const bool on = mine && h < heads;
        float v[8] = {0, 0, 0, 0, 0, 0, 0, 0};
        const E *in = is_q ? static_cast<const E *>(a.q) + (size_t)t * a.ldq + (size_t)h * a.d
                    : is_k ? static_cast<const E *>(a.k) + (size_t)t * a.ldk + (size_t)hk * a.d
                           : static_cast<const E *>(a.v) + (size_t)t * a.ldv + (size_t)hv * a.d;
        if (on) {
            load4(in + o0, v);
            load4(in + o1, v + 4);
        }
        const E *w = static_cast<const E *>(is_q ? a.q_weight : is_k ? a.k_weight : nullptr);
        if (a.q_weight || a.k_weight) {
            float s = 0.0f;
#pragma unroll
            for (int e = 0; e < 8; ++e) s += v[e] * v[e];
            const float inv = rsqrtf(head_sum<L>(s) / a.d + a.eps);
            if (on && w) {
                float g[8];
                load4(w + o0, g);
                load4(w + o1, g + 4);
#pragma unroll
                for (int e = 0; e < 8; ++e) v[e] *= inv * (g[e] + a.offset);
            }
        }
        if (turned && (is_q || is_k)) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                // pair e: (v[e], v[e + 4]) in halves, (v[2e], v[2e + 1]) interleaved
                const float p = halves ? v[e] : v[2 * e], q = halves ? v[e + 4] : v[2 * e + 1];
                const float np = p * cs[e] - q * sn[e], nq = p * sn[e] + q * cs[e];
                if (halves)
                    v[e] = np, v[e + 4] = nq;
                else
                    v[2 * e] = np, v[2 * e + 1] = nq;
            }
        }
        if (is_q || F == kFmtNone) {
            E *out = is_q ? static_cast<E *>(a.q_out) + (size_t)t * a.ldq_out + (size_t)h * a.d
                          : static_cast<E *>(a.k_out) + (size_t)t * a.ldk_out + (size_t)hk * a.d;
            if (on) {
                store4(out + o0, v);
                store4(out + o1, v + 4);
            }
        }
        if (F == kFmtNone || h0 + HW <= a.n_q) continue;
        const int hc = is_k ? hk : hv;
        const int64_t row = ((first + hc) << a.c.page_shift) + off;
        void *pool = is_k ? a.c.k : a.c.v;
        if (F == kFmtBf16 || F == kFmtF32) {
            typedef typename std::conditional<F == kFmtF32, float, uint16_t>::type C;
            if (on && !is_q && stored) {
                C *out = static_cast<C *>(pool) + row * a.d;
                store4(out + o0, v);
                store4(out + o1, v + 4);
            }
        } else {
            uint32_t top = 0;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const uint32_t b = __float_as_uint(v[e]) & 0x7FFFFFFFu;
                top = top > b ? top : b;
            }
            const float most = __uint_as_float(head_max<L>(top));
            if (on && !is_q && stored) {
                const float s = most > 0x1p64f ? 0x1p-64f : most < 0x1p-64f ? 0x1p64f : 1.0f;
                uint8_t *out = static_cast<uint8_t *>(pool) + row * a.d;
                const bool zero = most == 0.0f;
                *reinterpret_cast<uint32_t *>(out + o0) = zero ? 0u : code4<F>(v, s, most * s);
                *reinterpret_cast<uint32_t *>(out + o1) = zero ? 0u : code4<F>(v + 4, s, most * s);
                if (j == 0) (is_k ? a.c.k_scale : a.c.v_scale)[row] = most / (F == kFmtInt8 ? 127.0f : 448.0f);
            }
        }
    }
}

// Eight elements of a cache row as fp32.
template <int F>
__device__ __forceinline__ void cache8(const void *pool, int64_t at, float *v) {
    if (F == kFmtBf16) {
        const uint16_t *p = static_cast<const uint16_t *>(pool) + at;
        load4(p, v);
        load4(p + 4, v + 4);
    } else if (F == kFmtF32) {
        const float *p = static_cast<const float *>(pool) + at;
        load4(p, v);
        load4(p + 4, v + 4);
    } else {
        const u32x2 w = ldg(reinterpret_cast<const u32x2 *>(static_cast<const uint8_t *>(pool) + at));
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            const uint32_t c = q ? w.y : w.x;
            if (F == kFmtInt8) {
#pragma unroll
                for (int e = 0; e < 4; ++e) v[4 * q + e] = (float)(int8_t)(c >> (8 * e));
            } else {
                const auto lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)c, false), hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)c, true);
                v[4 * q] = lo[0], v[4 * q + 1] = lo[1], v[4 * q + 2] = hi[0], v[4 * q + 3] = hi[1];
            }
        }
    }
}

// S: the results go past the caches (8191 rows of 16 heads of 256 out of an e4m3
// cache, 101 MB: 25.2 us without, 20.1 us with).
template <class E, int F, int L, bool S>
__global__ __launch_bounds__(kThreads) void read_kernel(ReadJob a) {
    constexpr int HW = 64 / L;
    const int lane = threadIdx.x & 63, j = lane & (L - 1), sub = lane / L;
    const int wave = __builtin_amdgcn_readfirstlane(blockIdx.x * (kThreads / 64) + (threadIdx.x >> 6));
    const int t = wave / a.waves, part = wave - t * a.waves;
    if (t >= a.T) return;
    int64_t first;
    int off;
    if (!find_row(a.c, a.seq[t], a.slot[t], first, off)) return;
    const int d = a.c.d;
    for (int h0 = part * HW; h0 < 2 * a.c.n_kv; h0 += a.waves * HW) {
        const int h = h0 + sub;
        const bool is_k = h < a.c.n_kv;
        const int hc = is_k ? h : h - a.c.n_kv;
        E *out = static_cast<E *>(is_k ? a.k_out : a.v_out);
        if (h >= 2 * a.c.n_kv || 8 * j >= d || !out) continue;
        const int64_t row = ((first + hc) << a.c.page_shift) + off;
        float v[8];
        cache8<F>(is_k ? a.c.k : a.c.v, row * d + 8 * j, v);
        if (F == kFmtInt8 || F == kFmtE4m3) {
            const float s = (is_k ? a.c.k_scale : a.c.v_scale)[row];
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] *= s;
        }
        out += (size_t)t * (is_k ? a.ldk : a.ldv) + (size_t)hc * d + 8 * j;
        store4<S>(out, v);
        store4<S>(out + 4, v + 4);
    }
}

// Waves per token: one where tokens alone are enough, else up to one per chunk of
// heads.
int waves_per_token(int T, int heads, int lanes) {
    const int chunks = (heads * lanes + 63) / 64, want = kWavesWanted / T;
    return want < 1 ? 1 : want > chunks ? chunks : want;
}

int lanes_of(int d) { return d <= 64 ? 8 : d <= 128 ? 16 : 32; }

dim3 grid_of(int T, int waves) { return dim3((unsigned)(((int64_t)T * waves + 3) / 4)); }

template <class E, int F>
void run_rows(const RowsJob &a, hipStream_t s) {
    const dim3 g = grid_of(a.T, a.waves), b(kThreads);
    switch (lanes_of(a.d)) {
        case 8: hipLaunchKernelGGL((rows_kernel<E, F, 8>), g, b, 0, s, a); break;
        case 16: hipLaunchKernelGGL((rows_kernel<E, F, 16>), g, b, 0, s, a); break;
        default: hipLaunchKernelGGL((rows_kernel<E, F, 32>), g, b, 0, s, a);
    }
}

template <class E, int F, bool S>
void run_read(const ReadJob &a, hipStream_t s) {
    const dim3 g = grid_of(a.T, a.waves), b(kThreads);
    switch (lanes_of(a.c.d)) {
        case 8: hipLaunchKernelGGL((read_kernel<E, F, 8, S>), g, b, 0, s, a); break;
        case 16: hipLaunchKernelGGL((read_kernel<E, F, 16, S>), g, b, 0, s, a); break;
        default: hipLaunchKernelGGL((read_kernel<E, F, 32, S>), g, b, 0, s, a);
    }
}

template <class E, int F>
void run_read(const ReadJob &a, hipStream_t s) {
    const size_t written = (size_t)a.T * a.c.n_kv * a.c.d * sizeof(E) * ((a.k_out != nullptr) + (a.v_out != nullptr));
    written > kStreamBytes ? run_read<E, F, true>(a, s) : run_read<E, F, false>(a, s);
}

}  // namespace

hipError_t launch_rows(RowsJob a, int fmt, bool f32, hipStream_t s) {
    a.waves = waves_per_token(a.T, a.n_q + a.n_k + (fmt != kFmtNone ? a.n_v : 0), lanes_of(a.d));
    switch (fmt) {
        case kFmtNone: f32 ? run_rows<float, kFmtNone>(a, s) : run_rows<uint16_t, kFmtNone>(a, s); break;
        case kFmtBf16: run_rows<uint16_t, kFmtBf16>(a, s); break;
        case kFmtF32: run_rows<float, kFmtF32>(a, s); break;
        case kFmtInt8: f32 ? run_rows<float, kFmtInt8>(a, s) : run_rows<uint16_t, kFmtInt8>(a, s); break;
        default: f32 ? run_rows<float, kFmtE4m3>(a, s) : run_rows<uint16_t, kFmtE4m3>(a, s);
    }
    return hipGetLastError();
}

hipError_t launch_cache_read(ReadJob a, int fmt, bool f32, hipStream_t s) {
    a.waves = waves_per_token(a.T, 2 * a.c.n_kv, lanes_of(a.c.d));
    switch (fmt) {
        case kFmtBf16: run_read<uint16_t, kFmtBf16>(a, s); break;
        case kFmtF32: run_read<float, kFmtF32>(a, s); break;
        case kFmtInt8: f32 ? run_read<float, kFmtInt8>(a, s) : run_read<uint16_t, kFmtInt8>(a, s); break;
        default: f32 ? run_read<float, kFmtE4m3>(a, s) : run_read<uint16_t, kFmtE4m3>(a, s);
    }
    return hipGetLastError();
}

}  // namespace wl
