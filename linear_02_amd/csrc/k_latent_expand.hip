// Latent attention in the expanded form, for prompts over bf16 rows: every head's keys and
// values formed once per call, then attention over them head by head.
//
// Expanded, a pair of a query and a key takes nope + rot + value products instead of the 4
// latent + rot of the latent space with its remainders, for latent (nope + value) more per key:
// less from some 75 queries of a sequence on (latent 512, heads of 128 and 64), where the
// products are equally fast.
//   expand  [W^K; W^V] of a head times 128 keys' latents, a matrix product with both sides
//           through LDS 64 elements at a time, in two buffers. A wave has 64 rows of the
//           weight and all keys; rows are dealt to the matrix instruction so that a lane gets
//           eight neighbouring ones of a key.
//   attend  128 queries of a head a workgroup, 32 a wave, over keys of nope elements from the
//           workspace and `rot` from the cache (they are the same for all heads), 32 at a time
//           through two LDS buffers; two workgroups share a CU, so that one's softmax falls into
//           the other's products.
// Expanded rows are fp16 times a power of two of each row's own, weights fp16 too: an eighth of the error of bf16,
// which put outputs at 1.5 to 1.8 times what their own rounding costs (1.02 now), in as many products. A scale of
// more than one row would let a row that a query does not see take precision from those that it sees.
// 2048 tokens over 4000 keys, 32 heads of 128 + 64, latent 512, traced: 62 to 66 us for the first, 194 to 203 for
// the second, the matrix products and the softmax between them, 229 us for the untraced call.
#include "wl_latent.h"

namespace wl {

namespace {

constexpr int kBlock = 128;   // keys of a workgroup that expands

// First and last key of a sequence that any of its queries sees.
struct Span {
    int lo, hi;
};
__device__ __forceinline__ Span span_of(const AttnJob &a, const Seq &q) {
    const int lo = a.mask == kMaskCausal && a.window && q.ctx >= a.window ? min(q.ctx - a.window + 1, q.kv) : 0;
    return {lo, a.mask == kMaskCausal ? max(min(q.ctx + q.rows, q.kv), 0) : q.kv};
}

// kD: nope and value.
template <int kD>
__global__ __launch_bounds__(256) void expand_kernel(ExpandArgs x) {
    constexpr int kRows = 2 * kD, kPairs = kD / 64;              // of the weight; of 32 rows, of a wave
    constexpr int kSide = kBlock * 128, kBuffer = kSide + kRows * 128;
    __shared__ __align__(16) char lds[2 * kBuffer];
    const AttnJob &a = x.a;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), n = lane & 15, g = lane >> 4;
    const int head = (int)(blockIdx.x % x.heads), unit = (int)(blockIdx.x / x.heads), s = unit / x.blocks, j0 = (unit - s * x.blocks) * kBlock;
    const Seq q = seq_of(a, s);
    if (q.rows == 0) return;
    const Span see = span_of(a, q);
    if (j0 >= see.hi || j0 + kBlock <= see.lo) return;
    const int L = a.c.d, last = see.hi - 1, shift = a.c.page_shift, pmask = (1 << shift) - 1, bytes = 2 * (L + x.rot);
    // The wave fetches keys 32 wave .. + 31: two pages' worth of 16.
    const char *from[2];
    int most[2];
    uint32_t has = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int j = j0 + 16 * i, page = __builtin_amdgcn_readfirstlane(a.c.table[(int64_t)s * a.c.max_pages + (min(j, last) >> shift)]);
        const bool there = (unsigned)page < (unsigned)a.c.n_pages;
        has |= (there ? 1u : 0u) << i;
        if (i / 2 != wave) continue;
        from[i & 1] = scalar(static_cast<const char *>(a.c.k) + ((((int64_t)(there ? page : 0)) << shift) + (min(j, last) & pmask & ~15)) * bytes);
        most[i & 1] = last - min(j, last & ~15);
    }
    const char *w = scalar(static_cast<const char *>(x.w) + (size_t)(x.first + head) * kRows * L * 2);
    auto turn_w = [](int r) { return (r >> 1 & 1) | (r >> 3 & 3) << 1; };
    auto fetch = [&](int k, int buffer) {
        const uint32_t to = lds_byte(lds) + buffer * kBuffer;
        const int r = lane >> 3, c = lane & 7;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int row = 8 * (i & 1) + r;
            load_to_lds(from[i >> 1], min(row, most[i >> 1]) * bytes + k * 128 + ((c ^ (row >> 1 & 7)) << 4), to + (32 * wave + 8 * i) * 128);
        }
#pragma unroll
        for (int i = 0; i < kRows / 32; ++i) {
            const int first = wave * (kRows / 4) + 8 * i, row = first + r;
            load_to_lds(w, (uint32_t)row * L * 2 + k * 128 + ((c ^ turn_w(row)) << 4), to + kSide + first * 128);
        }
    };
    f32x4 o[2 * kPairs][8];
#pragma unroll
    for (int b = 0; b < 2 * kPairs; ++b)
#pragma unroll
        for (int i = 0; i < 8; ++i) o[b][i] = f32x4{0, 0, 0, 0};
    const int steps = L / 64;
    fetch(0, 0);
    wait_loads();
    __syncthreads();
    for (int k = 0; k < steps; ++k) {
        if (k + 1 < steps) fetch(k + 1, (k + 1) & 1);
        const char *in = lds + (k & 1) * kBuffer;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            u32x4 wf[2 * kPairs];
#pragma unroll
            for (int b = 0; b < 2 * kPairs; ++b) {
                const int row = wave * (kRows / 4) + 32 * (b >> 1) + 8 * (n >> 2) + 4 * (b & 1) + (n & 3);
                wf[b] = *reinterpret_cast<const u32x4 *>(in + kSide + row * 128 + (((4 * h + g) ^ turn_w(row)) << 4));
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const u32x4 c = *reinterpret_cast<const u32x4 *>(in + (16 * i + n) * 128 + (((4 * h + g) ^ (n >> 1 & 7)) << 4));
#pragma unroll
                for (int b = 0; b < 2 * kPairs; ++b) o[b][i] = mfma16(wf[b], c, o[b][i]);
            }
        }
        wait_loads();
        __syncthreads();
    }
    // Two waves share a key's row: its largest finite element decides over the scale.
    float *largest = reinterpret_cast<float *>(lds);   // [wave][key]
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        float top = 0.0f;
#pragma unroll
        for (int b = 0; b < 2 * kPairs; ++b)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float a = fabsf(o[b][i][e]);
                top = fmaxf(top, a < __builtin_inff() ? a : 0.0f);
            }
        top = groups_max(top);
        if (g == 0) largest[wave * kBlock + 16 * i + n] = top;
    }
    __syncthreads();
    const size_t unit_rows = ((size_t)s * x.heads + head) * x.keys;
    uint16_t *base = (wave < 2 ? x.k : x.v) + unit_rows * kD + (wave & 1) * (kD / 2) + 8 * g;
    float *scales = x.scales + 2 * (unit_rows + j0) + 32 * (wave >> 1);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int at = 16 * i + n, j = j0 + at;
        const HalfScale to = half_scale(fmaxf(largest[wave * kBlock + at], largest[(wave ^ 1) * kBlock + at]));
        if (g == 0 && (wave & 1) == 0) scales[(at >> 5) * 64 + (at & 31)] = to.down;   // of every key of the block: all are read
        if (j >= see.hi) continue;
        const bool there = has >> i & 1u;
#pragma unroll
        for (int p = 0; p < kPairs; ++p) {
            const f32x4 u = o[2 * p][i] * to.up, v = o[2 * p + 1][i] * to.up;
            const u32x4 e = {pack_half2(u.x, u.y), pack_half2(u.z, u.w), pack_half2(v.x, v.y), pack_half2(v.z, v.w)};
            *reinterpret_cast<u32x4 *>(base + (size_t)j * kD + 32 * p) = there ? e : u32x4{0, 0, 0, 0};
        }
    }
}

__device__ __forceinline__ float half_element(const uint16_t *p) { return (float)__builtin_bit_cast(_Float16, ldg(p)); }

// One wave, one query row: the definition, key by key, over the expanded keys and values.
// Lane holds output elements 2 lane, 2 lane + 1 (unnormalised).
template <int kD>
__device__ void expanded_row(const ExpandArgs &x, const Seq &q, int i, int head, const uint16_t *kp, const uint16_t *vp, float (&acc)[2], float &l) {
    const AttnJob &a = x.a;
    const int lane = threadIdx.x & 63;
    const bool on = 2 * lane < kD, key = lane < x.rot;
    const Sees v = sees(a, q, i);
    const uint16_t *qp = static_cast<const uint16_t *>(a.q) + (size_t)(q.q0 + i) * a.ldq + (size_t)(x.first + head) * (kD + x.rot);
    const float q0 = on ? element(qp + 2 * lane) : 0.0f, q1 = on ? element(qp + 2 * lane + 1) : 0.0f, qr = key ? element(qp + kD + lane) : 0.0f;
    float m = kNegInf;
    l = 0.0f, acc[0] = acc[1] = 0.0f;
    const Span span = span_of(a, q);
    const float *scales = x.scales + 2 * ((size_t)q.s * x.heads + head) * x.keys;
    const int j0 = v.tree ? min(v.lo, max(q.ctx, 0)) : v.lo, j1 = v.tree ? q.kv : v.hi;
    for (int j = max(j0, span.lo); j < min(j1, span.hi); ++j) {
        if (!visible(a, q, v, j)) continue;
        const int page = a.c.table[(int64_t)q.s * a.c.max_pages + (j >> a.c.page_shift)];
        if ((unsigned)page >= (unsigned)a.c.n_pages) continue;
        const int64_t row = ((int64_t)page << a.c.page_shift) + (j & ((1 << a.c.page_shift) - 1));
        const uint16_t *rp = static_cast<const uint16_t *>(a.c.k) + row * (a.c.d + x.rot) + a.c.d;
        const float *scale = scales + (size_t)(j >> 5) * 64 + (j & 31);
        const float ks = scale[0], vs = scale[32];
        float s = key ? qr * element(rp + lane) : 0.0f;
        if (on) s += q0 * (ks * half_element(kp + (size_t)j * kD + 2 * lane)) + q1 * (ks * half_element(kp + (size_t)j * kD + 2 * lane + 1));
        s = wave_sum(s) * a.scale2;
        if (s == kNegInf) continue;
        const float top = s > m ? s : m;   // a NaN score leaves m and makes p NaN
        const float up = m == top ? 1.0f : __builtin_amdgcn_exp2f(m - top);
        const float p = __builtin_amdgcn_exp2f(s - (top == kNegInf ? 0.0f : top));
        m = top;
        l = l * up + p;
        if (l != l) break;   // the row is NaN, whatever follows
        if (on)
#pragma unroll
            for (int e = 0; e < 2; ++e) acc[e] = acc[e] * up + (p != 0.0f ? p * (vs * half_element(vp + (size_t)j * kD + 2 * lane + e)) : 0.0f);
    }
}

template <int kD>
__global__ __launch_bounds__(256, 2) void attend_kernel(ExpandArgs x) {
    constexpr int kSteps = kD / 32, kBlocks = kD / 16, kRow = 2 * kD, kPieces = kD / 8, kPer = 64 / kPieces;   // rows of a load
    constexpr int kK = 32 * kRow, kBuffer = 2 * kK + 32 * 128;   // keys, values, rotated keys
    constexpr int kAhead = 4;
    constexpr int kScales = 2 * kBuffer, kRange = kScales + 2 * 256;   // [step % 2][of keys, of values][32]
    __shared__ __align__(16) char lds[kRange + 64];
    int (*range)[4] = reinterpret_cast<int (*)[4]>(lds + kRange);
    const AttnJob &a = x.a;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), n = lane & 15, g = lane >> 4;
    const int head = (int)(blockIdx.x % x.heads), unit = (int)(blockIdx.x / x.heads);
    // Later queries see more keys under a causal mask: the longest first, so that the short ones fill in.
    const int s = unit / x.tiles, tile = x.tiles - 1 - (unit - s * x.tiles);
    const Seq q = seq_of(a, s);
    if (tile * 128 >= q.rows) return;
    const int R = x.rot, r0 = tile * 128 + 32 * wave;
    const uint16_t *kp = x.k + ((size_t)s * x.heads + head) * x.keys * kD, *vp = x.v + ((size_t)s * x.heads + head) * x.keys * kD;
    u32x4 qf[2][kSteps + 2];
    f32x4 o[2][kBlocks];
    // References, sums; of a row's scores; outputs and sums are held times 2^in_o, which brings weights times their
    // values' scales into fp16's range.
    float m[2], l[2], scale2[2];
    int in_o[2];
    int lo = 0x7FFFFFFF, hi = 0, flo = 0, fhi = 0x7FFFFFFF;   // some row sees [lo, hi), every row [flo, fhi)
    const uint32_t sign = a.scale2 < 0.0f ? 0x80008000u : 0u;
#pragma unroll
    for (int t = 0; t < 2; ++t) {
        const int i = r0 + 16 * t + n;
        const bool on = i < q.rows;
        const uint16_t *qp = static_cast<const uint16_t *>(a.q) + (size_t)(q.q0 + (on ? i : 0)) * a.ldq + (size_t)(x.first + head) * (kD + R) + 8 * g;
        float most = 0.0f;
#pragma unroll
        for (int k = 0; k < kSteps + 2; ++k) {
            const uint32_t kept = on && 32 * k < kD + R ? 0xFFFFFFFFu : 0u;
            qf[t][k] = (ldg(reinterpret_cast<const u32x4 *>(qp + min(32 * k, kD + R - 32))) ^ sign) & kept;
            if (k < kSteps)
#pragma unroll
                for (int e = 0; e < 4; ++e) most = fmaxf(most, fmaxf(fabsf(bf16_f(qf[t][k][e] & 0xFFFFu)), fabsf(__uint_as_float(qf[t][k][e] & 0xFFFF0000u))));
        }
        // Queries are multiplied by a power of two of the row's, the rotated ones, which stay bf16, by the same. (Where all are
        // below 2^-46 it is no larger: scale2 stays a number then.)
        const HalfScale to = half_scale(fmaxf(groups_max(most), 0x1p-46f));
        scale2[t] = fmaxf(fabsf(a.scale2) * to.down, 0x1p-126f), in_o[t] = -90;
#pragma unroll
        for (int k = 0; k < kSteps + 2; ++k)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float q0 = bf16_f(qf[t][k][e] & 0xFFFFu) * to.up, q1 = __uint_as_float(qf[t][k][e] & 0xFFFF0000u) * to.up;
                qf[t][k][e] = k < kSteps ? pack_half2(q0, q1) : pack2(q0, q1);
            }
        const Sees see = sees(a, q, i);
        if (on) {
            lo = min(lo, see.tree ? min(see.lo, max(q.ctx, 0)) : see.lo);
            hi = max(hi, see.tree ? q.kv : see.hi);
            flo = max(flo, see.lo);
            fhi = min(fhi, see.hi);
        }
#pragma unroll
        for (int b = 0; b < kBlocks; ++b) o[t][b] = f32x4{0, 0, 0, 0};
        m[t] = kNegInf, l[t] = 0.0f;
    }
#pragma unroll
    for (int y = 1; y < 16; y <<= 1) {
        lo = min(lo, __shfl_xor(lo, y));
        hi = max(hi, __shfl_xor(hi, y));
        flo = max(flo, __shfl_xor(flo, y));
        fhi = min(fhi, __shfl_xor(fhi, y));
    }
    flo = __builtin_amdgcn_readfirstlane(flo);
    fhi = __builtin_amdgcn_readfirstlane(fhi);
    if (lane == 0) range[0][wave] = lo, range[1][wave] = hi;
    __syncthreads();
    const int wlo = __builtin_amdgcn_readfirstlane(lo), whi = __builtin_amdgcn_readfirstlane(hi);
#pragma unroll
    for (int w = 0; w < 4; ++w) lo = min(lo, range[0][w]), hi = max(hi, range[1][w]);
    const Span span = span_of(a, q);
    lo = max(__builtin_amdgcn_readfirstlane(lo), span.lo);
    const int k1 = min(__builtin_amdgcn_readfirstlane(hi), span.hi), k0 = lo & ~31, last = k1 - 1;
    if (k0 < k1) {
        const int32_t *table = a.c.table + (int64_t)s * a.c.max_pages;
        const int shift = a.c.page_shift, pmask = (1 << shift) - 1, n_pages = a.c.n_pages, bytes = 2 * (a.c.d + R);
        int page[2], first_page = -64, entries = 0;   // lane i holds entry first_page + i of the table
        auto look = [&](int j0) {
            const int e0 = min(j0, last) >> shift, e1 = min(j0 + 16, last) >> shift;
            if (e1 - first_page >= 64) {
                first_page = e0;
                entries = table[min(e0 + lane, last >> shift)];
                __builtin_amdgcn_s_waitcnt(0x0F70);   // vmcnt(0)
            }
            page[0] = __builtin_amdgcn_readlane(entries, e0 - first_page);
            page[1] = __builtin_amdgcn_readlane(entries, e1 - first_page);
        };
        auto turn_k = [](int r) { return kD == 128 ? r & 15 : r >> 1 & 7; };
        auto turn_v = [](int r) { return kD == 128 ? (r & 7) << 1 : (r >> 1 & 3) << 1; };
        const char *kpool = scalar(reinterpret_cast<const char *>(kp)), *vpool = scalar(reinterpret_cast<const char *>(vp));
        const char *spool = scalar(reinterpret_cast<const char *>(x.scales + 2 * ((size_t)s * x.heads + head) * x.keys));
        uint32_t valid_in = 0;
        auto fetch = [&](int j0, int step) {
            valid_in = ((unsigned)page[0] < (unsigned)n_pages ? 0xFFFFu : 0u) | ((unsigned)page[1] < (unsigned)n_pages ? 0xFFFF0000u : 0u);
            const uint32_t to = lds_byte(lds) + (step & 1) * kBuffer;
            const int most = last - j0;   // rows behind the last key read that key again
            int ln = lane;
            asm volatile("" : "+v"(ln));
            const char *kf = scalar(kpool + (int64_t)j0 * kRow), *vf = scalar(vpool + (int64_t)j0 * kRow);
#pragma unroll
            for (int i = 0; i < 8 / kPer; ++i) {
                const int first = 8 * wave + i * kPer, r = first + ln / kPieces, c = ln % kPieces, at = min(r, most) * kRow;
                load_to_lds(kf, at + ((c ^ turn_k(r)) << 4), to + first * kRow);
                load_to_lds(vf, at + ((c ^ turn_v(r)) << 4), to + kK + first * kRow);
            }
            const int half = wave >> 1, jh = j0 + 16 * half, pg = half ? page[1] : page[0], off = min(jh, last) & pmask & ~15;
            const char *rf = scalar(static_cast<const char *>(a.c.k) + ((((int64_t)((unsigned)pg < (unsigned)n_pages ? pg : 0)) << shift) + off) * bytes + 2 * a.c.d);
            const int r = 8 * (wave & 1) + (ln >> 3), piece = (ln & 7) ^ (r >> 1 & 7);
            load_to_lds(rf, min(r, last - min(jh, last & ~15)) * bytes + min(piece, R / 8 - 1) * 16, to + 2 * kK + 8 * wave * 128);
            if (wave == 0) load_to_lds4(scalar(spool + (int64_t)j0 * 8), ln * 4, lds_byte(lds) + kScales + (step & 1) * 256);
        };
        const int key_v = 4 * g + (n >> 2);
        const uint32_t second = R > 32 ? 0xFFFFFFFFu : 0u;
        auto attend = [&](const int &j0, const int &step, const uint32_t &valid) {
            const int in = (step & 1) * kBuffer;
            int kb = in + n * kRow + ((g ^ turn_k(n)) << 4), rb = in + 2 * kK + n * 128 + ((g ^ (n >> 1 & 7)) << 4);
            asm volatile("" : "+v"(kb), "+v"(rb));
            f32x4 sc[2][2], rotated[2][2];
#pragma unroll
            for (int t = 0; t < 2; ++t) sc[t][0] = sc[t][1] = rotated[t][0] = rotated[t][1] = f32x4{0, 0, 0, 0};
            constexpr int kEach = kSteps + 2, kAll = 2 * kEach;
            // Rows n and 16 + n are turned alike: bit 4 is in neither turn.
            auto operand = [&](int i) {
                const int b = i / kEach, k = i % kEach;
                if (k < kSteps) return *reinterpret_cast<const u32x4 *>(lds + (kb ^ k << 6) + b * 16 * kRow);
                return *reinterpret_cast<const u32x4 *>(lds + (rb ^ (k - kSteps) << 6) + b * 16 * 128);
            };
            u32x4 kf[kAhead];
            __builtin_amdgcn_s_setprio(1);
#pragma unroll
            for (int i = 0; i < kAhead; ++i) kf[i] = operand(i);
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int i = 0; i < kAll; ++i) {
                const int b = i / kEach, k = i % kEach;
                const u32x4 here = k > kSteps ? kf[i % kAhead] & second : kf[i % kAhead];
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    if (k < kSteps)
                        sc[t][b] = mfma16_half(here, qf[t][k], sc[t][b]);
                    else
                        rotated[t][b] = mfma16(here, qf[t][k], rotated[t][b]);
                }
                if (i + kAhead < kAll) kf[i % kAhead] = operand(i + kAhead);
                __builtin_amdgcn_sched_barrier(0);
            }
            __builtin_amdgcn_s_setprio(0);
            u32x4 ph[2];
            const char *scales = lds + kScales + (step & 1) * 256 + 16 * g;
            f32x4 ks[2], vs[2];
#pragma unroll
            for (int b = 0; b < 2; ++b) ks[b] = *reinterpret_cast<const f32x4 *>(scales + 64 * b), vs[b] = *reinterpret_cast<const f32x4 *>(scales + 128 + 64 * b);
            float most = vs[0].x;
#pragma unroll
            for (int e = 1; e < 8; ++e) most = fmaxf(most, vs[e >> 2][e & 3]);
            const bool all = j0 >= flo && j0 + 32 <= min(fhi, k1) && valid == 0xFFFFFFFFu;
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                float v[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) v[e] = __builtin_fmaf(sc[t][e >> 2][e & 3], ks[e >> 2][e & 3], rotated[t][e >> 2][e & 3]);
                if (__builtin_expect(!all, 0)) {
                    const ExpandArgs again = argument_again<ExpandArgs>();
                    const Seq qq = seq_of(again.a, s);
                    const uint32_t mine = (visible32(again.a, qq, sees(again.a, qq, r0 + 16 * t + n), j0) & valid & bits(0, k1 - j0)) >> (4 * g);
#pragma unroll
                    for (int e = 0; e < 8; ++e) v[e] = mine & (1u << (16 * (e >> 2) + (e & 3))) ? v[e] : kNegInf;
                }
                float top = v[0];
#pragma unroll
                for (int e = 1; e < 8; ++e) top = fmaxf(top, v[e]);
                top = groups_max(top);
                top = top == kNegInf ? top : top * scale2[t];
                if (__builtin_expect(__any(top > m[t] + 8.0f || ldexpf(most, in_o[t]) > 128.0f), 0)) {
                    // The reference moves only when a score passes it by 2^8: sums stay in range. in_o moves with it, or
                    // when a weight times its value's scale might pass fp16's range: the largest of them so far becomes 2^3 to 2^4.
                    const float now = fmaxf(m[t], top), up = now == m[t] ? 1.0f : __builtin_amdgcn_exp2f(m[t] - now);
                    const float ref = now == kNegInf ? 0.0f : now;
                    float large = 0.0f;
#pragma unroll
                    for (int e = 0; e < 8; ++e) large = fmaxf(large, __builtin_amdgcn_exp2f(__builtin_fmaf(v[e], scale2[t], -ref)) * vs[e >> 2][e & 3]);
                    large = fmaxf(groups_max(large), ldexpf(8.0f * up, -in_o[t]));
                    const int is = min(max(130 - (int)(__float_as_uint(large) >> 23), -90), 90);
                    const float by = ldexpf(up, is - in_o[t]);
                    m[t] = now, in_o[t] = is;
                    l[t] *= by;
#pragma unroll
                    for (int b = 0; b < kBlocks; ++b) o[t][b] *= by;
                }
                const float ref = (float)in_o[t] - (m[t] == kNegInf ? 0.0f : m[t]);
                float p[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    l[t] += p[e] = __builtin_amdgcn_exp2f(__builtin_fmaf(v[e], scale2[t], ref));
                    p[e] *= vs[e >> 2][e & 3];
                }
                ph[t] = u32x4{pack_half2(p[0], p[1]), pack_half2(p[2], p[3]), pack_half2(p[4], p[5]), pack_half2(p[6], p[7])};
            }
            int vb = in + kK + key_v * kRow + ((turn_v(key_v) | (n >> 1 & 1)) << 4) + 8 * (n & 1);
            asm volatile("" : "+v"(vb));
            __builtin_amdgcn_s_setprio(1);
#pragma unroll
            for (int b = 0; b < kBlocks; ++b) {
                const char *p = lds + (vb ^ b << 5);
                const u32x2 u = read_tr16(p), w = read_tr16(p + 16 * kRow);
#pragma unroll
                for (int t = 0; t < 2; ++t) o[t][b] = mfma16_half(u32x4{u.x, u.y, w.x, w.y}, ph[t], o[t][b]);
            }
            __builtin_amdgcn_sched_group_barrier(0x100, 2 * kAhead, 1);
#pragma unroll
            for (int i = 0; i < kBlocks; ++i) {
                __builtin_amdgcn_sched_group_barrier(0x008, 2, 1);
                if (i + kAhead < kBlocks) __builtin_amdgcn_sched_group_barrier(0x100, 2, 1);
            }
            __builtin_amdgcn_s_setprio(0);
        };
        look(k0);
        fetch(k0, 0);
        uint32_t valid = valid_in;
        wait_loads();
        __syncthreads();
        int step = 0;
        for (int j0 = k0; j0 < k1; j0 += 32, ++step) {
            const bool more = j0 + 32 < k1;
            if (more) {
                look(j0 + 32);
                fetch(j0 + 32, step + 1);
            }
            if (j0 + 31 >= wlo && j0 < whi) attend(j0, step, valid);
            valid = valid_in;
            wait_loads();
            __syncthreads();
        }
    }
    const ExpandArgs y = argument_again<ExpandArgs>();
#pragma unroll
    for (int t = 0; t < 2; ++t) {
        const int i = r0 + 16 * t + n;
        l[t] = groups_sum(l[t]);
        float check = l[t] * 0.0f;
#pragma unroll
        for (int b = 0; b < kBlocks; ++b) check += o[t][b].x * 0.0f + o[t][b].y * 0.0f + o[t][b].z * 0.0f + o[t][b].w * 0.0f;
        // A row with an infinity or a NaN is done again key by key: one that it does not see may have got in as 0 * NaN.
        uint64_t odd = __ballot(i < q.rows && (check != 0.0f || beyond(m[t])));
        odd |= odd >> 32;
        odd |= odd >> 16;
        const uint32_t again = (uint32_t)odd & 0xFFFFu;
        auto place = [&](int i) { return static_cast<uint16_t *>(y.a.o) + (size_t)(q.q0 + i) * y.a.ldo + (size_t)(y.first + head) * kD; };
        if (i < q.rows && !(again >> n & 1u)) {
            const float inv = l[t] == 0.0f ? 0.0f : 1.0f / l[t];
#pragma unroll
            for (int b = 0; b < kBlocks; ++b) {
                const float v[4] = {o[t][b].x * inv, o[t][b].y * inv, o[t][b].z * inv, o[t][b].w * inv};
                put4(place(i) + 16 * b + 4 * g, v);
            }
        }
        for (uint32_t left = again; left; left &= left - 1) {
            const int ii = r0 + 16 * t + __ffs(left) - 1;
            float acc[2], ll;
            expanded_row<kD>(y, q, ii, head, kp, vp, acc, ll);
            if (2 * lane < kD)
#pragma unroll
                for (int e = 0; e < 2; ++e) place(ii)[2 * lane + e] = f_bf16(ll == 0.0f ? 0.0f : acc[e] / ll);
        }
    }
}

template <int kD>
void run(const ExpandArgs &x, hipStream_t s) {
    if (x.blocks) hipLaunchKernelGGL((expand_kernel<kD>), dim3((unsigned)((int64_t)x.a.c.n_seq * x.blocks * x.heads)), dim3(256), 0, s, x);
    hipLaunchKernelGGL((attend_kernel<kD>), dim3((unsigned)((int64_t)x.a.c.n_seq * x.tiles * x.heads)), dim3(256), 0, s, x);
}

}  // namespace

void launch_expanded(const ExpandArgs &x, int d, hipStream_t s) { d == 128 ? run<128>(x, s) : run<64>(x, s); }

}  // namespace wl
