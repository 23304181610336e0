// Latent attention in fp32: the core over fp32 rows on the fp32 matrix instructions.
//
// v_mfma_f32_16x16x4_f32, D = A B + C: lane l holds A[m = l & 15][k = l >> 4], B[k][n = l & 15]
// and C[m = 4 (l >> 4) + i][n] (i = 0..3). As in bf16 (k_latent_tile.hip), scores are formed
// transposed, a lane owns a query row, and a row in LDS is key and value at once. A key
// operand is read 16 bytes at a time: of elements 16 k + 4 g + s, step s of four products
// takes one a lane, queries lie the same way. Weights are, as they lie, the operand of the
// second product: its step i takes keys 4 g + i. A value operand is four neighbouring
// columns of a key; column 4 m + j of 64 goes to product j, which only permutes the outputs.
//   over 16 rows   four waves of 16 rows share 16 keys at a time, in two buffers
//   16 rows        every wave with keys of its own, joined in LDS at the end
// Bound by the fp32 matrix instructions (2 x 16 x 16 x 4 operations in 32 cycles of a SIMD)
// where rows are many, by latency where they are few (4 streams of 3 tokens, 16 heads and a latent of 256 over
// up to 1024 keys 19 us).
#include "wl_latent.h"

namespace wl {

namespace {

template <int L>
struct Tile {
    static constexpr int kLatent = L / 4;                    // pieces of 16 bytes of a row's latent
    static constexpr int kRow = 16 * kLatent, kKeys = 16 * kRow, kBytes = kKeys + 16 * 256;
    static constexpr int kPer = kLatent < 64 ? 64 / kLatent : 1, kEach = kLatent > 64 ? kLatent / 64 : 1;   // rows of a load, loads of a row
};
// Piece c of row r lies at c ^ r, within groups of 16: the 16 rows of a key operand meet all banks.

template <int L, int kRW, int kKW>
__global__ __launch_bounds__(256, 1) void latent_f32_kernel(CoreArgs x) {
    typedef Tile<L> T;
    constexpr int kSteps = L / 16, kGroups = L / 64, kBuffers = kKW == 1 ? 2 : 1;
    constexpr int kTiles = kKW * kBuffers * T::kBytes, kJoin = kKW > 1 ? 4 * kGroups * 4096 : 0;
    constexpr int kMain = kTiles > kJoin ? kTiles : kJoin;
    __shared__ __align__(16) char lds_all[kMain + 512];
    // The waves' key ranges and what their join exchanges lie apart: a workgroup without keys meets no barrier between
    // the reads of the one and the first write of the other.
    int (*range)[4] = reinterpret_cast<int (*)[4]>(lds_all + kMain);   // [lo, hi][wave]
    float *shared = reinterpret_cast<float *>(lds_all + kMain + 256);  // [wave][row]
    const AttnJob &a = x.a;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int n = lane & 15, g = lane >> 4, rw = wave % kRW, kw = wave / kRW;
    Seq q;
    const Work work = work_of(a, x.sp, (int)blockIdx.x, q);
    const int tile = work.tile, s = work.s;
    if (s < 0) return;
    const int rows = q.rows * a.group, R = x.rot;
    if (tile * 16 * kRW >= rows) return;
    const int r0 = tile * 16 * kRW + 16 * rw, row = r0 + n, token = row / a.group;
    const bool on = row < rows;
    f32x4 qf[kSteps + 4];
    {
        const float *qp = static_cast<const float *>(a.q) + (int64_t)(q.q0 + (on ? token : 0)) * a.ldq + (int64_t)(on ? row - token * a.group : 0) * (L + R) + 4 * g;
#pragma unroll
        for (int k = 0; k < kSteps + 4; ++k) {
            // Of a row that there is not, and of elements behind the head's: read somewhere, and not used.
            const f32x4 v = ldg(reinterpret_cast<const f32x4 *>(qp + (k < kSteps ? 16 * k : min(16 * k, L + R - 16))));
            const bool kept = on && 16 * k < L + R;
            qf[k] = f32x4{kept ? v.x : 0.0f, kept ? v.y : 0.0f, kept ? v.z : 0.0f, kept ? v.w : 0.0f};
        }
    }
    f32x4 o[kGroups][4];
#pragma unroll
    for (int b = 0; b < kGroups; ++b)
#pragma unroll
        for (int j = 0; j < 4; ++j) o[b][j] = f32x4{0, 0, 0, 0};
    float m = kNegInf, l = 0.0f;
    const Sees see = sees(a, q, token);
    int lo = on ? (see.tree ? min(see.lo, max(q.ctx, 0)) : see.lo) : 0x7FFFFFFF, hi = on ? (see.tree ? q.kv : see.hi) : 0;
#pragma unroll
    for (int y = 1; y < 16; y <<= 1) lo = min(lo, __shfl_xor(lo, y)), hi = max(hi, __shfl_xor(hi, y));
    if (lane == 0) range[0][wave] = lo, range[1][wave] = hi;
    __syncthreads();
    const int wlo = __builtin_amdgcn_readfirstlane(lo), whi = __builtin_amdgcn_readfirstlane(hi);
#pragma unroll
    for (int w = 0; w < 4; ++w) lo = min(lo, range[0][w]), hi = max(hi, range[1][w]);
    lo = __builtin_amdgcn_readfirstlane(lo) & ~31;
    hi = __builtin_amdgcn_readfirstlane(hi);
    const int64_t c0 = (int64_t)lo + work.from;
    const int k0 = c0 < hi ? (int)c0 : hi, k1 = (int)min((int64_t)hi, c0 + work.chunk), last = k1 - 1;
    if (k0 < k1) {
        const int32_t *table = a.c.table + (int64_t)s * a.c.max_pages;
        const int shift = a.c.page_shift, pmask = (1 << shift) - 1, n_pages = a.c.n_pages, bytes = (L + R) * 4;
        // 16 keys lie within one page; a group's waves share their loads.
        int first_page = -64, entries = 0;   // lane i holds entry first_page + i of the table
        auto page_of = [&](int j0) {
            const int e = min(j0, last) >> shift;
            if (e - first_page >= 64) {
                first_page = e;
                entries = table[min(e + lane, last >> shift)];
                __builtin_amdgcn_s_waitcnt(0x0F70);   // vmcnt(0)
            }
            return __builtin_amdgcn_readlane(entries, e - first_page);
        };
        auto fetch = [&](int j0, int step, int page) {
            const bool has = (unsigned)page < (unsigned)n_pages;
            const int off = min(j0, last) & pmask & ~15, most = last - min(j0, last & ~15);
            const char *from = scalar(static_cast<const char *>(a.c.k) + ((((int64_t)(has ? page : 0)) << shift) + off) * bytes);
            const uint32_t to = lds_byte(lds_all) + (kw * kBuffers + (kBuffers == 2 ? step & 1 : 0)) * T::kBytes;
            constexpr int kLoads = 16 * T::kEach / T::kPer;
#pragma unroll
            for (int i = 0; i < kLoads / kRW; ++i) {
                const int at = i * kRW + rw, r = T::kPer > 1 ? at * T::kPer + lane / T::kLatent : at / T::kEach;
                const int c = T::kPer > 1 ? lane % T::kLatent : at % T::kEach * 64 + lane;
                load_to_lds(from, min(r, most) * bytes + ((c ^ r) << 4), to + at * 1024);
            }
            if (rw == kRW - 1)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int r = 4 * i + g, piece = (n ^ r) & 15;
                    load_to_lds(from, min(r, most) * bytes + T::kRow + min(piece, R / 4 - 1) * 16, to + T::kKeys + i * 1024);
                }
            return has;
        };
        auto attend = [&](int j0, int step, bool has) {
            const char *in = lds_all + (kw * kBuffers + (kBuffers == 2 ? step & 1 : 0)) * T::kBytes;
            f32x4 sc[2] = {{0, 0, 0, 0}, {0, 0, 0, 0}};
#pragma unroll
            for (int k = 0; k < kSteps + 4; ++k) {
                if (k >= kSteps && 16 * k >= L + R) break;
                const f32x4 kf = k < kSteps ? *reinterpret_cast<const f32x4 *>(in + n * T::kRow + (((4 * k + g) ^ n) << 4))
                                            : *reinterpret_cast<const f32x4 *>(in + T::kKeys + n * 256 + (((4 * (k - kSteps) + g) ^ n) << 4));
#pragma unroll
                for (int e = 0; e < 4; ++e) sc[e & 1] = __builtin_amdgcn_mfma_f32_16x16x4f32(kf[e], qf[k][e], sc[e & 1], 0, 0, 0);
            }
            sc[0] += sc[1];
            float v[4];
            const uint32_t mine = has ? (visible32(a, q, see, j0) & bits(0, min(16, k1 - j0))) >> (4 * g) : 0u;
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = on && mine >> i & 1u ? sc[0][i] * a.scale2 : kNegInf;
            const float top = groups_max(fmaxf(fmaxf(v[0], v[1]), fmaxf(v[2], v[3])));
            if (__any(top > m + 8.0f)) {
                // The reference moves only when a score passes it by 2^8: sums stay in range.
                const float now = fmaxf(m, top), up = now == m ? 1.0f : __builtin_amdgcn_exp2f(m - now);
                m = now;
                l *= up;
#pragma unroll
                for (int b = 0; b < kGroups; ++b)
#pragma unroll
                    for (int j = 0; j < 4; ++j) o[b][j] *= up;
            }
            const float ref = m == kNegInf ? 0.0f : m;
#pragma unroll
            for (int i = 0; i < 4; ++i) l += v[i] = __builtin_amdgcn_exp2f(v[i] - ref);
#pragma unroll
            for (int b = 0; b < kGroups; ++b)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const f32x4 vf = *reinterpret_cast<const f32x4 *>(in + (4 * g + i) * T::kRow + (((16 * b + n) ^ (4 * g + i)) << 4));
#pragma unroll
                    for (int j = 0; j < 4; ++j) o[b][j] = __builtin_amdgcn_mfma_f32_16x16x4f32(vf[j], v[i], o[b][j], 0, 0, 0);
                }
        };
        if (kKW == 1) {
            bool has = fetch(k0, 0, page_of(k0));
            wait_loads();
            __syncthreads();
            int step = 0;
            for (int j0 = k0; j0 < k1; j0 += 16, ++step) {
                const bool more = j0 + 16 < k1;
                bool next = false;
                if (more) next = fetch(j0 + 16, step + 1, page_of(j0 + 16));
                if (j0 + 15 >= wlo && j0 < whi) attend(j0, step, has);
                has = next;
                wait_loads();
                __syncthreads();
            }
        } else {
            for (int j0 = k0 + 16 * kw; j0 < k1; j0 += 16 * kKW) {
                const bool has = fetch(j0, 0, page_of(j0));
                wait_loads();
                if (j0 + 15 >= wlo && j0 < whi) attend(j0, 0, has);
                asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");   // read before the next rows come in
            }
            __syncthreads();
        }
    }
    const Split &sp = x.sp;
    auto place = [&](int r) {
        const int i = r / a.group;
        return sp.n_split > 1 ? sp.part + part_row(a, sp, work.part, 0, tile, r) * L
                              : static_cast<float *>(a.o) + (size_t)(q.q0 + i) * a.ldo + (size_t)(r - i * a.group) * L;
    };
    auto put_stat = [&](int r, float mm, float ll) {
        if (sp.n_split > 1) sp.ml[part_row(a, sp, work.part, 0, tile, r)] = make_float2(mm, ll);
    };
    l = groups_sum(l);
    // A row with an infinity or a NaN is done again key by key: one that it does not see may
    // have got in as 0 * NaN.
    float check = l * 0.0f;
#pragma unroll
    for (int b = 0; b < kGroups; ++b)
#pragma unroll
        for (int j = 0; j < 4; ++j) check += o[b][j].x * 0.0f + o[b][j].y * 0.0f + o[b][j].z * 0.0f + o[b][j].w * 0.0f;
    uint64_t odd = __ballot(on && check != 0.0f);
    odd |= odd >> 32;
    odd |= odd >> 16;
    uint32_t again = (uint32_t)odd & 0xFFFFu;
    float up[kKW] = {1.0f}, sum = l, top = m;
    if (kKW > 1) {
        f32x4 *mine = reinterpret_cast<f32x4 *>(lds_all);
#pragma unroll
        for (int c = 0; c < 4 * kGroups; ++c) mine[(wave * 4 * kGroups + c) * 64 + lane] = o[c >> 2][c & 3];
        if (g == 0) shared[wave * 16 + n] = m;
        __syncthreads();
        float ms[kKW];
        top = kNegInf;
#pragma unroll
        for (int w = 0; w < kKW; ++w) ms[w] = shared[w * 16 + n], top = fmaxf(top, ms[w]);
        __syncthreads();
        if (g == 0) shared[wave * 16 + n] = l;
        __syncthreads();
        sum = 0.0f;
#pragma unroll
        for (int w = 0; w < kKW; ++w) {
            up[w] = ms[w] == kNegInf ? 0.0f : __builtin_amdgcn_exp2f(ms[w] - top);
            sum += up[w] * shared[w * 16 + n];
        }
        __syncthreads();
        if (lane == 0) reinterpret_cast<uint32_t *>(shared)[wave] = again;
        __syncthreads();
        again = 0;
#pragma unroll
        for (int w = 0; w < kKW; ++w) again |= reinterpret_cast<const uint32_t *>(shared)[w];
        again = __builtin_amdgcn_readfirstlane(again);
    }
    if (on && !(again >> n & 1u)) {
        const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
        float *to = place(row) + 16 * g;
#pragma unroll
        for (int b = 0; b < kGroups; ++b) {
            if (b % kKW != kw) continue;   // (one group of waves: all of them)
            f32x4 v[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                v[j] = o[b][j];
                if (kKW > 1) {
                    v[j] = f32x4{0, 0, 0, 0};
#pragma unroll
                    for (int w = 0; w < kKW; ++w) v[j] += reinterpret_cast<const f32x4 *>(lds_all)[(w * 4 * kGroups + 4 * b + j) * 64 + lane] * up[w];
                }
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) *reinterpret_cast<f32x4 *>(to + 64 * b + 4 * i) = f32x4{v[0][i], v[1][i], v[2][i], v[3][i]} * inv;
        }
        if (kw == 0 && g == 0) put_stat(row, top, sum);
    }
    if (kw == 0)
        for (uint32_t left = again; left; left &= left - 1) {
            const int rr = r0 + __ffs(left) - 1, ii = rr / a.group;
            float acc[8], mm, ll;
            latent_row<float, kFmtF32>(a, R, q, ii, rr - ii * a.group, k0, k1, acc, mm, ll);
            if (8 * lane < L) {
#pragma unroll
                for (int e = 0; e < 8; ++e) acc[e] = ll == 0.0f ? 0.0f : acc[e] / ll;
                put4(place(rr) + 8 * lane, acc);
                put4(place(rr) + 8 * lane + 4, acc + 4);
            }
            if (lane == 0) put_stat(rr, mm, ll);
        }
}

template <int L>
void run(const CoreArgs &x, const CoreKind &k, unsigned blocks, hipStream_t s) {
    if (k.row_waves == 4)
        hipLaunchKernelGGL((latent_f32_kernel<L, 4, 1>), dim3(blocks), dim3(256), 0, s, x);
    else
        hipLaunchKernelGGL((latent_f32_kernel<L, 1, 4>), dim3(blocks), dim3(256), 0, s, x);
}

}  // namespace

void launch_latent_f32(const CoreArgs &x, const CoreKind &k, unsigned blocks, hipStream_t s) {
    switch (x.a.c.d) {
        case 128: run<128>(x, k, blocks, s); break;
        case 256: run<256>(x, k, blocks, s); break;
        default: run<512>(x, k, blocks, s);
    }
}

}  // namespace wl
