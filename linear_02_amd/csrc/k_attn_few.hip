// Attention with few query rows per key/value head (single tokens, small trees):
// at most 32 rows (16 of heads wider than 128), a row being a new token and
// one of the query heads that share the key/value head.
//
// Bound by reading the keys and values once. Every wave works alone on a stretch
// of keys, 32 at a time, with no barrier in its loop: K and V come as whole rows,
// past the caches, into registers and from there into a patch of LDS of the wave's
// own, where K is read as the operand of the score product and V through the
// transposing reads. The next 32 keys' loads are issued as soon as the registers
// are free, so 32 keys of K and V per wave are under way while the present ones are
// worked on. The matrix cores do 16 rows for the price of one, so the weights are
// fed as a bf16 head plus a bf16 remainder, off by 2^-16 at most. The four waves of a
// workgroup join their outputs in LDS; workgroups that divide a long sequence
// leave partial outputs that a second launch joins.
//
// 32 streams of 2048 to 8192 keys, 32 query and 8 key/value heads of 256, one token
// each: bf16 226 us (1.37 GB, 6.1 TB/s), int8 136 us, e4m3 130 us (0.69 GB, 5.3 TB/s);
// a large copy moves 5.1 TB/s. Reading K straight into operand layout (16 rows x 64
// bytes per load) gave 278 and 169 us; V alone as whole rows 262 and 146, both
// 227 and 136.
#include "wl_attn_mfma.h"

namespace wl {

namespace {

constexpr int kWaves = 4;

// F: cache format; DT: padded head width; NT: tiles of 16 query rows.
template <int F, int DT, int NT>
struct Few {
    static constexpr bool kCodes = F == kFmtInt8 || F == kFmtE4m3;
    static constexpr int kSteps = DT / 32;              // 32-wide steps of the score product
    static constexpr int kLoads = kCodes ? DT / 64 : DT / 32;   // 16-byte pieces per key row and lane
    static constexpr int kBlocks = DT / 16;             // 16-wide blocks of the output
    static constexpr int kRow = kCodes ? DT : 2 * DT;   // bytes of a V row in LDS
    // Two workgroups per CU where 256 registers hold the 32 keys' K and V beside the outputs.
    static constexpr int kPerCu = DT == 256 && !kCodes ? 1 : 2;
    static_assert(DT < 256 || NT == 1, "32 rows of 256 do not fit the registers");
    static constexpr int kPatch = 64 * kRow > 64 * DT ? 64 * kRow : 64 * DT;   // LDS bytes per wave: 32 rows of V and of K, or 16 output rows fp32
    u32x4 q[NT][kSteps];
    f32x4 o[NT][kBlocks];
    float m[NT], l[NT];
};

// Which of keys j0 .. j0 + 31 this lane's row of tile t sees, for trees: from the
// arguments in memory, at the few steps that reach the tree.
__device__ __forceinline__ uint32_t few_seen(const TileArgs &x, int s, int t, int j0) {
    const Seq q = seq_of(x.a, s);
    return visible32(x.a, q, sees(x.a, q, (16 * t + (threadIdx.x & 15)) / x.a.group), j0);
}

// Joins the four waves' outputs, 16 rows at a time: row n of a wave's patch holds
// what it has of row n.
template <int F, int DT, int NT>
__device__ __forceinline__ void join_waves(const TileArgs &args, const Work &work, const Seq &q, Few<F, DT, NT> &st, char *lds, int k0, int k1) {
    typedef Few<F, DT, NT> P;
    const AttnJob &a = args.a;
    const Split &sp = args.sp;
    __shared__ float2 ml[kWaves][16];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), n = lane & 15, g = lane >> 4;
    const int kvh = (int)blockIdx.x % a.c.n_kv;
    const int rows = q.rows * a.group, d = a.c.d;
    char *patch = lds + wave * P::kPatch;
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        if (16 * t >= rows) break;
        st.l[t] = groups_sum(st.l[t]);
        float check = st.l[t] * 0.0f;
        float *out = reinterpret_cast<float *>(patch);
#pragma unroll
        for (int b = 0; b < P::kBlocks; ++b) {
            if (16 * b < d) check += st.o[t][b].x * 0.0f + st.o[t][b].y * 0.0f + st.o[t][b].z * 0.0f + st.o[t][b].w * 0.0f;
            *reinterpret_cast<f32x4 *>(out + n * DT + 16 * b + 4 * g) = st.o[t][b];
        }
        if (g == 0) ml[wave][n] = make_float2(st.m[t], st.l[t]);
        // A row with an infinity or a NaN is done again key by key: one that it does
        // not see may have got in as 0 * NaN.
        uint64_t odd = __ballot(16 * t + n < rows && check != 0.0f);
        odd |= odd >> 32;
        odd |= odd >> 16;
        for (uint32_t left = (uint32_t)odd & 0xFFFFu; left; left &= left - 1) {
            const int c = __ffs(left) - 1, r = 16 * t + c, i = r / a.group;
            float acc[4], m, l;
            one_row<uint16_t, F>(a, q, i, kvh * a.group + r - i * a.group, k0, k1, acc, m, l);
            if (4 * lane < DT) *reinterpret_cast<f32x4 *>(out + c * DT + 4 * lane) = f32x4{acc[0], acc[1], acc[2], acc[3]};
            if (lane == 0) ml[wave][c] = make_float2(m, l);
        }
        __syncthreads();
        for (int x = threadIdx.x; x < 16 * DT / 4; x += 256) {
            const int c = x / (DT / 4), at = 4 * (x % (DT / 4)), r = 16 * t + c;
            if (r >= rows || at >= d) continue;
            float m = kNegInf, l = 0.0f;
#pragma unroll
            for (int w = 0; w < kWaves; ++w) m = fmaxf(m, ml[w][c].x);
            f32x4 sum{0, 0, 0, 0};
#pragma unroll
            for (int w = 0; w < kWaves; ++w) {
                const float2 v = ml[w][c];
                if (v.x == kNegInf && v.y == 0.0f) continue;
                const float up = __builtin_amdgcn_exp2f(v.x - m);
                l += up * v.y;
                sum += *reinterpret_cast<const f32x4 *>(lds + w * P::kPatch + (c * DT + at) * 4) * up;
            }
            if (sp.n_split > 1) {
                const int64_t row = part_row(a, sp, work.part, kvh, 0, r);
                *reinterpret_cast<f32x4 *>(sp.part + row * d + at) = sum;
                if (at == 0) sp.ml[row] = make_float2(m, l);
            } else {
                const float v[4] = {sum.x, sum.y, sum.z, sum.w};
                float w[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) w[e] = l == 0.0f ? 0.0f : v[e] / l;
                const int i = r / a.group;
                put4(static_cast<uint16_t *>(a.o) + (size_t)(q.q0 + i) * a.ldo + (size_t)(kvh * a.group + r - i * a.group) * d + at, w);
            }
        }
        if (NT > 1) __syncthreads();
    }
}

template <int F, int DT, int NT>
__global__ __launch_bounds__(256, (Few<F, DT, NT>::kPerCu)) void few_kernel(TileArgs args) {
    const AttnJob &a = args.a;
    typedef Few<F, DT, NT> P;
    constexpr bool kCodes = P::kCodes;
    __shared__ __align__(16) char lds[kWaves * P::kPatch];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int n = lane & 15, g = lane >> 4;
    const int kvh = (int)blockIdx.x % a.c.n_kv;
    Seq q;
    const Work work = work_of(a, args.sp, (int)blockIdx.x / a.c.n_kv, q);
    const int s = work.s;
    if (s < 0) return;
    const int rows = q.rows * a.group, d = a.c.d;
    const bool tree = a.mask == kMaskTree;
    if (rows == 0) return;

    // Query rows of this lane's columns, and what they see.
    P st;
    int lo = 0x7FFFFFFF, hi = 0, flo = 0, fhi = 0x7FFFFFFF;   // some row sees [lo, hi), every row [flo, fhi)
    int row_lo[NT], row_hi[NT];                              // this lane's rows; trees besides
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        const int r = 16 * t + n, i = r / a.group;
        const bool on = r < rows;
        const uint16_t *qp = static_cast<const uint16_t *>(a.q) + (size_t)(q.q0 + (on ? i : 0)) * a.ldq +
                             (size_t)(kvh * a.group + (on ? r - i * a.group : 0)) * d;
#pragma unroll
        for (int k = 0; k < P::kSteps; ++k) {
            const int at = kCodes ? 64 * (k >> 1) + 16 * g + 8 * (k & 1) : 32 * k + 8 * g;
            st.q[t][k] = u32x4{0, 0, 0, 0};
            if (on && at < d) st.q[t][k] = ldg(reinterpret_cast<const u32x4 *>(qp + at));
        }
        const Sees see = sees(a, q, i);
        if (on) {   // an unused column is never the reason to mask
            lo = min(lo, see.tree ? min(see.lo, max(q.ctx, 0)) : see.lo);
            hi = max(hi, see.tree ? q.kv : see.hi);
            flo = max(flo, see.lo);
            fhi = min(fhi, see.hi);
        }
        row_lo[t] = on ? see.lo : 0, row_hi[t] = on ? see.hi : 0x7FFFFFFF;
#pragma unroll
        for (int b = 0; b < P::kBlocks; ++b) st.o[t][b] = f32x4{0, 0, 0, 0};
        st.m[t] = kNegInf, st.l[t] = 0.0f;
    }
#pragma unroll
    for (int x = 1; x < 16; x <<= 1) {
        lo = min(lo, __shfl_xor(lo, x));
        hi = max(hi, __shfl_xor(hi, x));
        flo = max(flo, __shfl_xor(flo, x));
        fhi = min(fhi, __shfl_xor(fhi, x));
    }
    flo = __builtin_amdgcn_readfirstlane(flo);
    fhi = __builtin_amdgcn_readfirstlane(fhi);
    lo = __builtin_amdgcn_readfirstlane(lo) & ~31;
    hi = __builtin_amdgcn_readfirstlane(hi);
    // This workgroup's keys, and this wave's: a stretch of whole 32s.
    const int64_t c0 = (int64_t)lo + work.from;
    const int w0 = c0 < hi ? (int)c0 : hi, w1 = (int)min((int64_t)hi, c0 + work.chunk);
    const int per = ((w1 - w0 + kWaves * 32 - 1) / (kWaves * 32)) * 32;
    const int k0 = min(w0 + wave * per, w1), k1 = min(k0 + per, w1), last = k1 - 1;

    char *patch = lds + wave * P::kPatch;
    if (k0 < k1) {
        u32x4 kr[2][P::kLoads], vr[2][P::kLoads];
        f32x4 ks[2], vs[2];
        uint32_t valid;
        const int32_t *table = a.c.table + (int64_t)s * a.c.max_pages;
        const int shift = a.c.page_shift, pmask = (1 << shift) - 1, n_pages = a.c.n_pages, bytes = d * (kCodes ? 1 : 2);
        const int64_t head = (int64_t)kvh << shift, pitch = (int64_t)a.c.n_kv << shift;   // rows: of this head in a page, of a page
        // Page numbers come from a register: lane i holds entry first_page + i of the
        // table, read anew every 64 pages. A load per step would be waited for behind
        // the keys and values that are on their way.
        int first_page = -64, pages = 0;
        // Where 32 keys lie, in two halves of 16, each within one page. Past the last
        // key the last one is read again, so no load leaves the pages.
        int64_t first[2];   // element row of the half's first key
        uint32_t rows_in[2];   // rows of the half behind its first, to the last key
        uint32_t valid_in;
        auto look = [&](int j0) {
            const int e0 = min(j0, last) >> shift, e1 = min(j0 + 16, last) >> shift;
            if (e1 - first_page >= 64) {
                first_page = e0;
                pages = table[min(e0 + lane, last >> shift)];
                __builtin_amdgcn_s_waitcnt(0x0F70);   // vmcnt(0)
            }
            valid_in = 0;
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                const int page = __builtin_amdgcn_readlane(pages, (b ? e1 : e0) - first_page), j = min(j0 + 16 * b, last);
                const bool ok = (unsigned)page < (unsigned)n_pages;
                if (ok) valid_in |= 0xFFFFu << (16 * b);
                first[b] = (ok ? page : 0) * pitch + head + (j & pmask & ~15);
                rows_in[b] = last - (j & ~15);
            }
        };
        // Whole rows by neighbouring lanes, and not kept in the caches: 64 bytes of 16
        // rows each, as the score product takes them, cost a fifth of the bandwidth.
        constexpr int kPieces = P::kRow / 16, kRows = 64 / kPieces;   // 16-byte pieces of a row, rows per load
        int my_row = lane / kPieces, my_piece = lane % kPieces;
        auto load = [&](const void *pool, u32x4 (&to)[2][P::kLoads]) {
            const uint32_t c = min(my_piece * 16, bytes - 16);
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                const char *row = scalar(static_cast<const char *>(pool) + first[b] * bytes);
#pragma unroll
                for (int i = 0; i < P::kLoads; ++i)
                    to[b][i] = __builtin_nontemporal_load((const __attribute__((address_space(1))) u32x4 *)(row + (min((uint32_t)(i * kRows + my_row), rows_in[b]) * bytes + c)));
            }
        };
        auto load_scale = [&](const float *pool, f32x4 (&to)[2]) {
#pragma unroll
            for (int b = 0; b < 2; ++b) to[b] = ldg(reinterpret_cast<const f32x4 *>(pool + first[b] + 4 * g));
        };
        // LDS places. V row of key r: 16-byte piece c at c ^ f(r), so that the rows
        // one transposing read takes together lie on different banks.
        constexpr int kMask = DT >= 128 ? 7 : 3;
        int get[8];
        auto put = [&](int b, int i) {
            const int r = i * kRows + my_row, f = kCodes ? ((r & 3) | b << 2) & kMask : (r & kMask) << 1;
            return (16 * b + r) * P::kRow + ((my_piece ^ f) << 4);
        };
        // K piece c of row r at c ^ fk(r): the 16 rows of one pass of a read meet all banks.
        constexpr int kShare = kPieces < 16 ? 16 / kPieces : 1;
        auto fk = [&](int r) { return r / kShare & ((kPieces < 16 ? kPieces : 16) - 1); };
        auto put_k = [&](int b, int i) {
            const int r = i * kRows + my_row;
            return 32 * P::kRow + (16 * b + r) * P::kRow + ((my_piece ^ fk(r)) << 4);
        };
        const int get_k = 32 * P::kRow + n * P::kRow + ((g ^ fk(n)) << 4);   // piece 4 i + g: ^ (i << 6)
#pragma unroll
        for (int x = 0; x < 8; ++x) {
            if (kCodes) {
                const int e = n >> 1, key = 16 * (e >> 2) + 4 * g + (e & 3);
                get[x] = key * P::kRow + (((x ^ e) & kMask) << 4) + 8 * (n & 1);
            } else {
                const int key = 4 * g + (n >> 2);
                get[x] = key * P::kRow + (((x ^ key) & kMask) << 5) + 8 * (n & 3);
            }
        }
        look(k0);
        load(a.c.k, kr);
        if (kCodes) load_scale(a.c.k_scale, ks);
        load(a.c.v, vr);
        if (kCodes) load_scale(a.c.v_scale, vs);
        for (int j0 = k0; j0 < k1; j0 += 32) {
            valid = valid_in;
            asm volatile("" : "+v"(my_row), "+v"(my_piece));   // places are formed anew, not held in registers
            look(min(j0 + 32, last & ~31));
            // scores
#pragma unroll
            for (int b = 0; b < 2; ++b)
#pragma unroll
                for (int i = 0; i < P::kLoads; ++i) *reinterpret_cast<u32x4 *>(patch + put_k(b, i)) = kr[b][i];
            f32x4 kscale[2];
            if (kCodes) kscale[0] = ks[0], kscale[1] = ks[1];
            load(a.c.k, kr);
            if (kCodes) load_scale(a.c.k_scale, ks);
            f32x4 sc[NT][2];
#pragma unroll
            for (int t = 0; t < NT; ++t) sc[t][0] = sc[t][1] = f32x4{0, 0, 0, 0};
#pragma unroll
            for (int b = 0; b < 2; ++b)
#pragma unroll
                for (int i = 0; i < P::kLoads; ++i) {
                    const u32x4 w = *reinterpret_cast<const u32x4 *>(patch + (get_k ^ ((i & 3) << 6)) + (i >> 2) * 256 + b * 16 * P::kRow);
#pragma unroll
                    for (int e = 0; e < (kCodes ? 2 : 1); ++e) {
                        const u32x4 kf = kCodes ? (e ? widen8<F>(w.z, w.w) : widen8<F>(w.x, w.y)) : w;
#pragma unroll
                        for (int t = 0; t < NT; ++t) sc[t][b] = mfma16(kf, st.q[t][kCodes ? 2 * i + e : i], sc[t][b]);
                    }
                }
            f32x4 mul[2] = {f32x4{a.scale2, a.scale2, a.scale2, a.scale2}, f32x4{a.scale2, a.scale2, a.scale2, a.scale2}};
            if (kCodes) mul[0] *= kscale[0], mul[1] *= kscale[1];
            // V into the patch
#pragma unroll
            for (int b = 0; b < 2; ++b)
#pragma unroll
                for (int i = 0; i < P::kLoads; ++i)
                    *reinterpret_cast<u32x4 *>(patch + put(b, i)) = vr[b][i];
            f32x4 vm[2];
            if (kCodes) vm[0] = vs[0], vm[1] = vs[1];
            load(a.c.v, vr);
            if (kCodes) load_scale(a.c.v_scale, vs);
            // weights
            u32x4 ph[NT], pl[NT];
            const bool all = j0 >= flo && j0 + 32 <= min(fhi, k1) && valid == 0xFFFFFFFFu;
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                float x[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) x[e] = sc[t][e >> 2][e & 3] * mul[e >> 2][e & 3];
                if (!all) {
                    uint32_t vis = bits(row_lo[t] - j0, row_hi[t] - j0);
                    if (tree) vis = few_seen(argument_again<TileArgs>(), s, t, j0);
                    const uint32_t mine = (vis & valid & bits(0, k1 - j0)) >> (4 * g);
#pragma unroll
                    for (int e = 0; e < 8; ++e) x[e] = mine & (1u << (16 * (e >> 2) + (e & 3))) ? x[e] : kNegInf;
                }
                float top = x[0];
#pragma unroll
                for (int e = 1; e < 8; ++e) top = fmaxf(top, x[e]);
                top = groups_max(top);
                if (__any(top > st.m[t] + 8.0f)) {
                    // The reference moves only when a score passes it by 2^8: sums stay in range.
                    const float now = fmaxf(st.m[t], top), up = now == st.m[t] ? 1.0f : __builtin_amdgcn_exp2f(st.m[t] - now);
                    st.m[t] = now;
                    st.l[t] *= up;
#pragma unroll
                    for (int b = 0; b < P::kBlocks; ++b) st.o[t][b] *= up;
                }
                const float ref = st.m[t] == kNegInf ? 0.0f : st.m[t];
                float p[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    p[e] = __builtin_amdgcn_exp2f(x[e] - ref);
                    st.l[t] += p[e];
                    if (kCodes) p[e] = p[e] == 0.0f ? 0.0f : p[e] * vm[e >> 2][e & 3];
                }
                uint32_t h[4], r[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    h[e] = pack2(p[2 * e], p[2 * e + 1]);
                    r[e] = pack2(p[2 * e] - bf16_f(h[e] & 0xFFFFu), p[2 * e + 1] - __uint_as_float(h[e] & 0xFFFF0000u));
                }
                ph[t] = u32x4{h[0], h[1], h[2], h[3]};
                pl[t] = u32x4{r[0], r[1], r[2], r[3]};
            }
            // outputs
#pragma unroll
            for (int b = 0; b < P::kBlocks; ++b) {
                u32x4 vf;
                if (kCodes) {
                    const u32x2 w = read_tr8(patch + get[b & 7] + (b >> 3) * 128);
                    vf = widen8<F>(w.x, w.y);
                } else {
                    const char *p = patch + get[b & 7] + (b >> 3) * 256;
                    const u32x2 x = read_tr16(p), y = read_tr16(p + 16 * P::kRow);
                    vf = u32x4{x.x, x.y, y.x, y.y};
                }
#pragma unroll
                for (int t = 0; t < NT; ++t) {
                    st.o[t][b] = mfma16(vf, ph[t], st.o[t][b]);
                    st.o[t][b] = mfma16(vf, pl[t], st.o[t][b]);
                }
            }
        }
    }

    join_waves<F, DT, NT>(args, work, q, st, lds, k0, k1);
}

template <int F, int DT, int NT>
void run(const AttnJob &a, const Split &sp, hipStream_t s) {
    hipLaunchKernelGGL((few_kernel<F, DT, NT>), dim3((unsigned)sp.items * a.c.n_kv), dim3(256), 0, s, TileArgs{a, sp});
}

template <int F>
void pick(const AttnJob &a, const Split &sp, hipStream_t s) {
    const bool two = a.max_q * a.group > 16;
    if (a.c.d <= 64)
        two ? run<F, 64, 2>(a, sp, s) : run<F, 64, 1>(a, sp, s);
    else if (a.c.d <= 128)
        two ? run<F, 128, 2>(a, sp, s) : run<F, 128, 1>(a, sp, s);
    else
        run<F, 256, 1>(a, sp, s);
}

}  // namespace

void launch_few(const AttnJob &a, int fmt, const Split &sp, hipStream_t s) {
    switch (fmt) {
        case kFmtBf16: pick<kFmtBf16>(a, sp, s); break;
        case kFmtInt8: pick<kFmtInt8>(a, sp, s); break;
        default: pick<kFmtE4m3>(a, sp, s);
    }
}

}  // namespace wl
