// Attention in fp32: fp32 queries over an fp32, int8 or e4m3 cache, for any number
// of query rows.
//
// v_mfma_f32_16x16x4_f32 has the same result layout as the bf16 product and takes
// one value per lane: A[m = l & 15][k = g], B[k = g][n = l & 15]. Scores are formed
// transposed as there (16 keys x 16 query rows), and register i of a score tile,
// keys 4 g + i, is the B operand of the step over those four keys, so the weights
// stay where they are. A workgroup holds 64 rows, 16 per wave; keys and values go
// through LDS 16 at a time as fp32, the next 16 waiting in registers. At prompts
// bound by the fp32 matrix rate (32 cycles per product and SIMD, a sixteenth of
// the bf16 rate); with few rows by the latency of a step, so the keys are divided
// over workgroups.
#include "wl_attn_mfma.h"

namespace wl {

namespace {

__device__ __forceinline__ f32x4 mfma4(float a, float b, f32x4 c) { return __builtin_amdgcn_mfma_f32_16x16x4f32(a, b, c, 0, 0, 0); }

template <int F, int DT>
__global__ __launch_bounds__(256, 2) void f32_kernel(TileArgs x) {
    constexpr int kBlocks = DT / 16, kRow = 4 * DT, kSide = 16 * kRow;   // bytes of a row and of 16 keys
    constexpr int kPieces = DT / 4, kLoads = 16 * kPieces / 256;         // 16-byte pieces of a row; per thread and side
    const AttnJob &a = x.a;
    __shared__ __align__(16) char lds[2 * kSide + 2 * 64 + 32];
    float *k_scale = reinterpret_cast<float *>(lds + 2 * kSide), *v_scale = k_scale + 16;
    int(*range)[4] = reinterpret_cast<int(*)[4]>(lds + 2 * kSide + 128);
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int n = lane & 15, g = lane >> 4;
    const int kvh = (int)blockIdx.x % a.c.n_kv;
    Seq q;
    const Work work = work_of(a, x.sp, (int)blockIdx.x / a.c.n_kv, q);
    const int tile = work.tile, s = work.s;
    if (s < 0) return;
    auto rows_of = [](int tile, int) { return WaveRows{(tile * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6)) * 16, 1}; };
    const int rows = q.rows * a.group, d = a.c.d, r = rows_of(tile, 0).first + n;
    if (tile * kF32Rows >= rows) return;

    // Queries of this lane's row: elements 16 j + 4 g .. + 3 are those of step (j, e).
    f32x4 qf[kBlocks], o[1][kBlocks];
    float m[1] = {kNegInf}, l[1] = {0.0f};
    const float sign = a.scale2 < 0.0f ? -1.0f : 1.0f, scale2 = fmaxf(fabsf(a.scale2), 0x1p-126f);
    const int i = r / a.group;
    const bool on = r < rows;
    const float *qp = static_cast<const float *>(a.q) + (size_t)(q.q0 + (on ? i : 0)) * a.ldq + (size_t)(kvh * a.group + (on ? r - i * a.group : 0)) * d;
#pragma unroll
    for (int j = 0; j < kBlocks; ++j) {
        qf[j] = o[0][j] = f32x4{0, 0, 0, 0};
        if (on && 16 * j < d) qf[j] = ldg(reinterpret_cast<const f32x4 *>(qp + 16 * j + 4 * g)) * sign;
    }
    int lo = 0x7FFFFFFF, hi = 0;
    if (on) {
        const Sees v = sees(a, q, i);
        lo = v.tree ? min(v.lo, max(q.ctx, 0)) : v.lo;
        hi = v.tree ? q.kv : v.hi;
    }
#pragma unroll
    for (int b = 1; b < 16; b <<= 1) {
        lo = min(lo, __shfl_xor(lo, b));
        hi = max(hi, __shfl_xor(hi, b));
    }
    if (lane == 0) range[0][wave] = lo, range[1][wave] = hi;
    __syncthreads();
    const int wlo = __builtin_amdgcn_readfirstlane(lo), whi = __builtin_amdgcn_readfirstlane(hi);
    lo = min(min(range[0][0], range[0][1]), min(range[0][2], range[0][3]));
    hi = max(max(range[1][0], range[1][1]), max(range[1][2], range[1][3]));
    lo = __builtin_amdgcn_readfirstlane(lo) & ~31;
    hi = __builtin_amdgcn_readfirstlane(hi);
    const int64_t c0 = (int64_t)lo + work.from;
    const int k0 = c0 < hi ? (int)c0 : hi, k1 = (int)min((int64_t)hi, c0 + work.chunk), last = k1 - 1;

    if (k0 < k1) {
        const int32_t *table = a.c.table + (int64_t)s * a.c.max_pages;
        const int shift = a.c.page_shift, pmask = (1 << shift) - 1;
        float kr[kLoads][4], vr[kLoads][4], scale_in = 0.0f;
        bool paged = false, paged_in;
        // The next 16 keys, all of one page; rows behind the last key read that key again.
        auto fetch = [&](int j0) {
            const int page = table[j0 >> shift];
            paged_in = (unsigned)page < (unsigned)a.c.n_pages;
            const int64_t first = ((((int64_t)(paged_in ? page : 0) * a.c.n_kv + kvh) << shift) + (j0 & pmask));
#pragma unroll
            for (int b = 0; b < kLoads; ++b) {
                const int p = threadIdx.x + b * 256, row = min(p / kPieces, last - j0), c = min(p % kPieces * 4, d - 4);
                cache4<F>(a.c.k, (first + row) * d + c, kr[b]);
                cache4<F>(a.c.v, (first + row) * d + c, vr[b]);
            }
            if (F != kFmtF32 && threadIdx.x < 32) scale_in = (threadIdx.x < 16 ? a.c.k_scale : a.c.v_scale)[first + min((int)threadIdx.x & 15, last - j0)];
        };
        // LDS places: K piece c of row r at c ^ r (a pass of a read takes 16 rows of one
        // piece), V's at c ^ 4 (r / 4) (a pass takes 16 columns of rows 4 g + i).
        auto land = [&]() {
#pragma unroll
            for (int b = 0; b < kLoads; ++b) {
                const int p = threadIdx.x + b * 256, row = p / kPieces, c = p % kPieces;
                *reinterpret_cast<f32x4 *>(lds + row * kRow + ((c ^ row) & (kPieces - 1)) * 16) = f32x4{kr[b][0], kr[b][1], kr[b][2], kr[b][3]};
                *reinterpret_cast<f32x4 *>(lds + kSide + row * kRow + ((c ^ (row & 12)) & (kPieces - 1)) * 16) = f32x4{vr[b][0], vr[b][1], vr[b][2], vr[b][3]};
            }
            if (F != kFmtF32 && threadIdx.x < 32) k_scale[threadIdx.x] = scale_in;
            paged = paged_in;
        };
        fetch(k0);
        for (int j0 = k0; j0 < k1; j0 += 16) {
            land();
            __syncthreads();
            if (j0 + 16 < k1) fetch(j0 + 16);
            if (j0 + 15 >= wlo && j0 < whi) {
                f32x4 sc{0, 0, 0, 0};
#pragma unroll
                for (int j = 0; j < kBlocks; ++j) {
                    const f32x4 kf = *reinterpret_cast<const f32x4 *>(lds + n * kRow + (((4 * j + g) ^ n) & (kPieces - 1)) * 16);
                    sc = mfma4(kf.x, qf[j].x, sc);
                    sc = mfma4(kf.y, qf[j].y, sc);
                    sc = mfma4(kf.z, qf[j].z, sc);
                    sc = mfma4(kf.w, qf[j].w, sc);
                }
                const uint32_t vis = !paged ? 0u : seen(x, work, rows_of, 0, j0) & bits(0, k1 - j0);
                f32x4 vs{1, 1, 1, 1};
                if (F != kFmtF32) {
                    sc *= *reinterpret_cast<const f32x4 *>(k_scale + 4 * g);
                    vs = *reinterpret_cast<const f32x4 *>(v_scale + 4 * g);
                }
                float p[4], top = kNegInf;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    p[e] = vis >> (4 * g + e) & 1u ? sc[e] * scale2 : kNegInf;
                    top = fmaxf(top, p[e]);
                }
                top = groups_max(top);
                if (__any(top > m[0])) {
                    const float now = fmaxf(m[0], top), up = now == m[0] ? 1.0f : __builtin_amdgcn_exp2f(m[0] - now);
                    m[0] = now;
                    l[0] *= up;
#pragma unroll
                    for (int b = 0; b < kBlocks; ++b) o[0][b] *= up;
                }
                const float at = m[0] == kNegInf ? 0.0f : m[0];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    p[e] = __builtin_amdgcn_exp2f(p[e] - at);
                    l[0] += p[e];
                    p[e] = p[e] == 0.0f ? 0.0f : p[e] * vs[e];
                }
#pragma unroll
                for (int b = 0; b < kBlocks; ++b)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int c = ((4 * b + (n >> 2)) ^ (4 * g)) & (kPieces - 1);
                        const float vf = *reinterpret_cast<const float *>(lds + kSide + (4 * g + e) * kRow + c * 16 + 4 * (n & 3));
                        o[0][b] = mfma4(vf, p[e], o[0][b]);
                    }
            }
            __syncthreads();
        }
    }
    finish<float, F, DT, 1>(argument_again<TileArgs>(), work, rows_of, o, m, l, k0, k1);
}

template <int F, int DT>
void run(const AttnJob &a, const Split &sp, hipStream_t s) {
    hipLaunchKernelGGL((f32_kernel<F, DT>), dim3((unsigned)sp.items * a.c.n_kv), dim3(256), 0, s, TileArgs{a, sp});
}

template <int F>
void pick(const AttnJob &a, const Split &sp, hipStream_t s) {
    if (a.c.d <= 64)
        run<F, 64>(a, sp, s);
    else if (a.c.d <= 128)
        run<F, 128>(a, sp, s);
    else
        run<F, 256>(a, sp, s);
}

}  // namespace

void launch_f32(const AttnJob &a, int fmt, const Split &sp, hipStream_t s) {
    switch (fmt) {
        case kFmtF32: pick<kFmtF32>(a, sp, s); break;
        case kFmtInt8: pick<kFmtInt8>(a, sp, s); break;
        default: pick<kFmtE4m3>(a, sp, s);
    }
}

}  // namespace wl
