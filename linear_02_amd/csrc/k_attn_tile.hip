// Attention with many query rows per key/value head (prompts, larger trees).
//
// A workgroup takes 128 query rows of one key/value head, a row being a new token
// and one of the query heads that share the key/value head, so that those heads
// share every key that is staged; its four waves hold 32 rows each. Keys and
// values pass through LDS 32 at a time, in two buffers: while the waves work on
// one, the next 32 are on their way into the other. Queries, scores, weights and
// outputs stay in registers from the first key to the last.
#include "wl_attn_mfma.h"

namespace wl {

namespace {

constexpr int kRowsPerWave = 32, kNT = kRowsPerWave / 16;

template <int F, int DT>
__global__ __launch_bounds__(256, 2) void tile_kernel(AttnJob a, Split sp, int tiles) {
    constexpr bool kCodes = F == kFmtInt8 || F == kFmtE4m3;
    constexpr int kSteps = DT / 32, kBlocks = DT / 16;
    constexpr int kRow = 2 * DT, kSide = 32 * kRow;          // LDS bytes of a row, of 32 keys
    constexpr int kPieces = DT / 8;                          // 16-byte pieces of a row
    constexpr int kMaskV = DT >= 128 ? 7 : 3;
    __shared__ __align__(16) char lds[2][2][kSide];          // [buffer][K, V]
    __shared__ __align__(16) float lds_scale[2][2][32];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int n = lane & 15, g = lane >> 4;
    int u = blockIdx.x;
    const int kvh = u % a.c.n_kv;
    u /= a.c.n_kv;
    const int split = u % sp.n_split;
    u /= sp.n_split;
    const int tile = tiles - 1 - u % tiles, s = u / tiles;   // the longest rows first
    const Seq q = seq_of(a, s);
    const int rows = q.rows * a.group, d = a.c.d, r0 = tile * 128 + wave * kRowsPerWave;
    if (tile * 128 >= rows) return;

    u32x4 qf[kNT][kSteps];
    f32x4 o[kNT][kBlocks];
    float m[kNT], l[kNT];
    Sees see[kNT];
    int lo = 0x7FFFFFFF, hi = 0;
    const uint32_t sign = a.scale2 < 0.0f ? 0x80008000u : 0u;   // a negative scale goes into the queries
    const float scale2 = fmaxf(fabsf(a.scale2), 0x1p-126f);   // not 0: -inf marks an unseen key
#pragma unroll
    for (int t = 0; t < kNT; ++t) {
        const int r = r0 + 16 * t + n, i = r / a.group;
        const bool on = r < rows;
        const uint16_t *qp = static_cast<const uint16_t *>(a.q) + (size_t)(q.q0 + (on ? i : 0)) * a.ldq +
                             (size_t)(kvh * a.group + (on ? r - i * a.group : 0)) * d;
#pragma unroll
        for (int k = 0; k < kSteps; ++k) {
            const int at = 32 * k + 8 * g;
            qf[t][k] = u32x4{0, 0, 0, 0};
            if (on && at < d) qf[t][k] = ldg(reinterpret_cast<const u32x4 *>(qp + at)) ^ sign;
        }
        see[t] = sees(a, q, i);
        if (on) {
            lo = min(lo, see[t].tree ? min(see[t].lo, max(q.ctx, 0)) : see[t].lo);
            hi = max(hi, see[t].tree ? q.kv : see[t].hi);
        } else {
            see[t] = Sees{0, 0x7FFFFFFF, nullptr};   // an unused column: never the reason to mask
        }
#pragma unroll
        for (int b = 0; b < kBlocks; ++b) o[t][b] = f32x4{0, 0, 0, 0};
        m[t] = kNegInf, l[t] = 0.0f;
    }
#pragma unroll
    for (int x = 1; x < 16; x <<= 1) {
        lo = min(lo, __shfl_xor(lo, x));
        hi = max(hi, __shfl_xor(hi, x));
    }
    // Keys of this wave's rows, of the workgroup's, and the piece of them that is this workgroup's.
    __shared__ int range[2][4];
    if (lane == 0) range[0][wave] = lo, range[1][wave] = hi;
    __syncthreads();
    const int wlo = __builtin_amdgcn_readfirstlane(lo), whi = __builtin_amdgcn_readfirstlane(hi);
    lo = min(min(range[0][0], range[0][1]), min(range[0][2], range[0][3]));
    hi = max(max(range[1][0], range[1][1]), max(range[1][2], range[1][3]));
    lo = __builtin_amdgcn_readfirstlane(lo) & ~31;
    hi = __builtin_amdgcn_readfirstlane(hi);
    const int64_t c0 = (int64_t)lo + (int64_t)split * sp.chunk;
    const int k0 = c0 < hi ? (int)c0 : hi, k1 = (int)min((int64_t)hi, c0 + sp.chunk), last = k1 - 1;

    if (k0 < k1) {
        const int pmask = (1 << a.c.page_shift) - 1;
        const int32_t *table = a.c.table + (int64_t)s * a.c.max_pages;
        const int bytes = d * (kCodes ? 1 : 2);              // of a cache row
        int page[2];                                         // of the keys that are staged next
        auto look = [&](int j0) {
#pragma unroll
            for (int b = 0; b < 2; ++b) page[b] = table[min(j0 + 16 * b, last) >> a.c.page_shift];
        };
        // The 16 keys of half b: element row of the first, and whether they have a page.
        auto base = [&](int j0, int b, bool &ok) {
            ok = (unsigned)page[b] < (unsigned)a.c.n_pages;
            return (((int64_t)(ok ? page[b] : 0) * a.c.n_kv + kvh) << a.c.page_shift) + (min(j0 + 16 * b, last) & pmask & ~15);
        };
        // Within a half: rows behind the last key read that key again.
        auto row_at = [&](int j0, int b, int r) { return min(r, last - min(j0 + 16 * b, last & ~15)); };
        // bf16: 64 pieces per load, straight into LDS; piece c of row r lies at c ^ f(r).
        constexpr int kDma = kPieces * 32 / 256;             // loads per wave and side
        // codes: 16 bytes per load and lane, widened when they are put down.
        constexpr int kCodeLoads = kCodes ? (2 * DT + 255) / 256 : 1;   // per lane and side: 32 rows of DT / 16 pieces over 256 lanes
        u32x4 kc[kCodeLoads], vc[kCodeLoads];
        float scale_in = 0.0f;
        uint32_t valid_in = 0;
        auto fetch = [&](int j0, int buf) {
            int64_t first[2];
            bool ok[2];
#pragma unroll
            for (int b = 0; b < 2; ++b) first[b] = base(j0, b, ok[b]);
            valid_in = (ok[0] ? 0xFFFFu : 0u) | (ok[1] ? 0xFFFF0000u : 0u);
            if (!kCodes) {
#pragma unroll
                for (int i = 0; i < kDma; ++i) {
                    const int p0 = (wave * kDma + i) * 64, b = p0 / (16 * kPieces);   // a load's rows are of one half
                    const int p = p0 + lane, r = p / kPieces, c = p % kPieces;
                    const int from = row_at(j0, b, r & 15) * bytes;
                    const int ck = (c ^ (r & 7)) * 16, cv = (c ^ ((r & kMaskV) << 1)) * 16;
                    const char *k = static_cast<const char *>(a.c.k) + first[b] * bytes, *v = static_cast<const char *>(a.c.v) + first[b] * bytes;
                    lds_dma16(reinterpret_cast<const u32x4 *>(k + (from + (ck < bytes ? ck : 0))),
                              reinterpret_cast<u32x4 *>(lds[buf][0] + p0 * 16));
                    lds_dma16(reinterpret_cast<const u32x4 *>(v + (from + (cv < bytes ? cv : 0))),
                              reinterpret_cast<u32x4 *>(lds[buf][1] + p0 * 16));
                }
            } else {
#pragma unroll
                for (int i = 0; i < kCodeLoads; ++i) {
                    const int p = threadIdx.x + i * 256, r = (p / (DT / 16)) & 31, c = p % (DT / 16) * 16, b = r >> 4;
                    const int64_t from = first[b] * bytes + row_at(j0, b, r & 15) * bytes + (c < bytes ? c : 0);
                    kc[i] = ldg(reinterpret_cast<const u32x4 *>(static_cast<const char *>(a.c.k) + from));
                    vc[i] = ldg(reinterpret_cast<const u32x4 *>(static_cast<const char *>(a.c.v) + from));
                }
                if (threadIdx.x < 64) {
                    const int r = lane & 31;
                    const int64_t from = first[r >> 4] + row_at(j0, r >> 4, r & 15);
                    scale_in = (lane < 32 ? a.c.k_scale : a.c.v_scale)[from];
                }
            }
        };
        auto land = [&](int buf) {
            if (!kCodes) {
                wait_vm<0>();
                return;
            }
#pragma unroll
            for (int i = 0; i < kCodeLoads; ++i) {
                const int p = threadIdx.x + i * 256, r = p / (DT / 16), c = p % (DT / 16) * 2;
                if (DT == 64 && r >= 32) break;
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    *reinterpret_cast<u32x4 *>(lds[buf][0] + r * kRow + ((c + e) ^ (r & 7)) * 16) =
                        e ? widen8<F>(kc[i].z, kc[i].w) : widen8<F>(kc[i].x, kc[i].y);
                    *reinterpret_cast<u32x4 *>(lds[buf][1] + r * kRow + ((c + e) ^ ((r & kMaskV) << 1)) * 16) =
                        e ? widen8<F>(vc[i].z, vc[i].w) : widen8<F>(vc[i].x, vc[i].y);
                }
            }
            if (threadIdx.x < 64) lds_scale[buf][lane >> 5][lane & 31] = scale_in;
        };
        // Operand addresses within a buffer.
        int at_k[2], at_v[8];
#pragma unroll
        for (int x = 0; x < 2; ++x) at_k[x] = n * kRow + (((4 * x + g) ^ (n & 7)) << 4);
#pragma unroll
        for (int x = 0; x < 8; ++x) {
            const int key = 4 * g + (n >> 2);
            at_v[x] = key * kRow + (((x ^ key) & kMaskV) << 5) + 8 * (n & 3);
        }
        look(k0);
        fetch(k0, 0);
        uint32_t valid = valid_in;
        if (k0 + 32 < k1) look(k0 + 32);
        land(0);
        __syncthreads();
        int buf = 0;
        for (int j0 = k0; j0 < k1; j0 += 32, buf ^= 1) {
            const bool more = j0 + 32 < k1;
            if (more) {
                fetch(j0 + 32, buf ^ 1);
                look(min(j0 + 64, last));
            }
            if (j0 + 31 >= wlo && j0 < whi) {
                const char *kb = lds[buf][0], *vb = lds[buf][1];
                f32x4 sc[kNT][2];
#pragma unroll
                for (int b = 0; b < 2; ++b) {
#pragma unroll
                    for (int t = 0; t < kNT; ++t) sc[t][b] = f32x4{0, 0, 0, 0};
#pragma unroll
                    for (int k = 0; k < kSteps; ++k) {
                        const u32x4 kf = *reinterpret_cast<const u32x4 *>(kb + at_k[k & 1] + (k >> 1) * 128 + b * 16 * kRow);
#pragma unroll
                        for (int t = 0; t < kNT; ++t) sc[t][b] = mfma16(kf, qf[t][k], sc[t][b]);
                    }
                }
                f32x4 vm[2];
                if (kCodes) {
#pragma unroll
                    for (int b = 0; b < 2; ++b) {
                        const f32x4 ks = *reinterpret_cast<const f32x4 *>(&lds_scale[buf][0][16 * b + 4 * g]);
                        vm[b] = *reinterpret_cast<const f32x4 *>(&lds_scale[buf][1][16 * b + 4 * g]);
#pragma unroll
                        for (int t = 0; t < kNT; ++t) sc[t][b] *= ks;
                    }
                }
                u32x4 ph[kNT];
#pragma unroll
                for (int t = 0; t < kNT; ++t) {
                    float x[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) x[e] = sc[t][e >> 2][e & 3];
                    const uint32_t vis = visible32(a, q, see[t], j0) & valid & bits(0, k1 - j0);
                    if (__any(vis != 0xFFFFFFFFu)) {
                        const uint32_t mine = vis >> (4 * g);
#pragma unroll
                        for (int e = 0; e < 8; ++e) x[e] = mine & (1u << (16 * (e >> 2) + (e & 3))) ? x[e] : kNegInf;
                    }
                    float top = x[0];
#pragma unroll
                    for (int e = 1; e < 8; ++e) top = fmaxf(top, x[e]);
                    top = groups_max(top);
                    top = top == kNegInf ? top : top * scale2;
                    if (__any(top > m[t] + 8.0f)) {
                        // The reference moves only when a score passes it by 2^8: sums stay in range.
                        const float now = fmaxf(m[t], top), up = now == m[t] ? 1.0f : __builtin_amdgcn_exp2f(m[t] - now);
                        m[t] = now;
                        l[t] *= up;
#pragma unroll
                        for (int b = 0; b < kBlocks; ++b) o[t][b] *= up;
                    }
                    const float ref = m[t] == kNegInf ? 0.0f : m[t];
                    float p[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        p[e] = __builtin_amdgcn_exp2f(__builtin_fmaf(x[e], scale2, -ref));
                        if (kCodes) {
                            l[t] += p[e];
                            p[e] = p[e] == 0.0f ? 0.0f : p[e] * vm[e >> 2][e & 3];
                        }
                    }
                    ph[t] = u32x4{pack2(p[0], p[1]), pack2(p[2], p[3]), pack2(p[4], p[5]), pack2(p[6], p[7])};
                    if (!kCodes) {
                        // the sum of the weights as the product will use them
                        constexpr uint32_t kOnes = 0x3F803F80u;
                        l[t] = dot2(ph[t].x, kOnes, l[t]);
                        l[t] = dot2(ph[t].y, kOnes, l[t]);
                        l[t] = dot2(ph[t].z, kOnes, l[t]);
                        l[t] = dot2(ph[t].w, kOnes, l[t]);
                    }
                }
#pragma unroll
                for (int b = 0; b < kBlocks; ++b) {
                    const char *p = vb + at_v[b & 7] + (b >> 3) * 256;
                    const u32x2 x = read_tr16(p), y = read_tr16(p + 16 * kRow);
#pragma unroll
                    for (int t = 0; t < kNT; ++t) o[t][b] = mfma16(u32x4{x.x, x.y, y.x, y.y}, ph[t], o[t][b]);
                }
            }
            if (more) land(buf ^ 1);
            valid = valid_in;
            __syncthreads();
        }
    }

    // Outputs: lane (n, g) holds elements 16 b + 4 g .. + 3 of row n.
#pragma unroll
    for (int t = 0; t < kNT; ++t) {
        const int r = r0 + 16 * t + n, i = r / a.group;
        l[t] = groups_sum(l[t]);
        float check = l[t] * 0.0f;
#pragma unroll
        for (int b = 0; b < kBlocks; ++b)
            if (16 * b < d) check += o[t][b].x * 0.0f + o[t][b].y * 0.0f + o[t][b].z * 0.0f + o[t][b].w * 0.0f;
        // A row with an infinity or a NaN is done again key by key: one that it does
        // not see may have got in as 0 * NaN.
        uint64_t odd = __ballot(r < rows && check != 0.0f);
        odd |= odd >> 32;
        odd |= odd >> 16;
        const uint32_t again = (uint32_t)odd & 0xFFFFu;
        const int64_t part = ((int64_t)(s * (int64_t)a.c.n_kv + kvh) * sp.n_split + split) * sp.rows;
        auto row_out = [&](int r) {
            const int i = r / a.group;
            return static_cast<uint16_t *>(a.o) + (size_t)(q.q0 + i) * a.ldo + (size_t)(kvh * a.group + r - i * a.group) * d;
        };
        if (r < rows && !(again >> n & 1u)) {
            const float inv = l[t] == 0.0f ? 0.0f : 1.0f / l[t];
#pragma unroll
            for (int b = 0; b < kBlocks; ++b) {
                const int at = 16 * b + 4 * g;
                if (at >= d) break;
                if (sp.n_split > 1) {
                    *reinterpret_cast<f32x4 *>(sp.part + (part + r) * d + at) = o[t][b];
                } else {
                    const float v[4] = {o[t][b].x * inv, o[t][b].y * inv, o[t][b].z * inv, o[t][b].w * inv};
                    put4(row_out(r) + at, v);
                }
            }
            if (sp.n_split > 1 && g == 0) sp.ml[part + r] = make_float2(m[t], l[t]);
        }
        for (uint32_t left = again; left; left &= left - 1) {
            const int rr = r0 + 16 * t + __ffs(left) - 1, ii = rr / a.group;
            float acc[4], mm, ll;
            one_row<uint16_t, F>(a, q, ii, kvh * a.group + rr - ii * a.group, k0, k1, acc, mm, ll);
            if (4 * lane < d) {
                if (sp.n_split > 1) {
                    *reinterpret_cast<f32x4 *>(sp.part + (part + rr) * d + 4 * lane) = f32x4{acc[0], acc[1], acc[2], acc[3]};
                } else {
#pragma unroll
                    for (int e = 0; e < 4; ++e) acc[e] = ll == 0.0f ? 0.0f : acc[e] / ll;
                    put4(row_out(rr) + 4 * lane, acc);
                }
            }
            if (sp.n_split > 1 && lane == 0) sp.ml[part + rr] = make_float2(mm, ll);
        }
        (void)i;
    }
}

template <int F, int DT>
void run(const AttnJob &a, const Split &sp, hipStream_t s) {
    const int tiles = (sp.rows + kTileRows - 1) / kTileRows;
    const int64_t blocks = (int64_t)a.c.n_seq * tiles * sp.n_split * a.c.n_kv;
    hipLaunchKernelGGL((tile_kernel<F, DT>), dim3((unsigned)blocks), dim3(256), 0, s, a, sp, tiles);
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

void launch_tile(const AttnJob &a, int fmt, const Split &sp, hipStream_t s) {
    switch (fmt) {
        case kFmtBf16: pick<kFmtBf16>(a, sp, s); break;
        case kFmtInt8: pick<kFmtInt8>(a, sp, s); break;
        default: pick<kFmtE4m3>(a, sp, s);
    }
}

}  // namespace wl
