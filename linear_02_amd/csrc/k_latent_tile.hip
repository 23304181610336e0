// Attention of latent queries on the matrix cores, over bf16 and e4m3 rows.
//
// All heads share a row, and a row is key and value at once: a workgroup takes a tile
// of (token, head) rows and brings every cache row once into LDS, 32 at a time, where
// its first `latent` elements serve both products. Queries, scores, weights and outputs
// stay in registers from the first key to the last; at a latent of 512 that is 128 of
// outputs, 72 of queries and 64 of their remainders for the 16 rows that a wave has.
//   many rows  four waves of 16 rows share a tile of keys, two workgroups per CU where
//              registers allow, so that one's softmax falls into the other's products
//   32 rows    two pairs of waves, each pair with keys of its own
//   16 rows    every wave with keys of its own, which it fetches for itself and waits
//              for alone; joined in LDS at the end. Where two buffers of latents fit, the
//              rotated keys, which only the scores need, are read first, and the next rows
//              come in behind that (e4m3, 64 streams of 16 heads over up to 16384 keys,
//              whole call, with queries in two products: 150 us with one buffer, 132 us so)
// Rows of e4m3 stay codes in LDS and are widened as operands: half the LDS traffic, and
// the vector units have the time beside the products.
// Few rows are bound by memory (64 streams of 16 heads over up to 16384 e4m3 keys 106 us, 4.3 TB/s), many at a
// latent of 512 by what one wave per SIMD waits for between its products, which remainders double (32 streams of
// 128 heads over up to 8192 bf16 keys 114 to 129 us, some 750 TFLOP/s of them). Two workgroups a CU, which
// queries rounded to bf16 would leave room for, took 119 us for that call instead of 127, 98 instead of 110 for 4
// trees of 32 tokens and 32 heads, 653 instead of 862 for 2048 tokens over 4000 keys; 32 rows a wave, with weights'
// remainders alone, 124, 108 and 755.
// Nothing is rounded to bf16 but the output: weights, and queries that the product into the latent space left in
// fp32, are multiplied as a bf16 head and its remainder (2^-16 off), queries of codes as fp16 (2^-11). With
// both rounded to bf16 outputs were off by 1.6 times what their own rounding costs, with queries alone 1.41.
#include "wl_latent.h"

namespace wl {

namespace {

// The tile in LDS: 32 rows of the latent, kLatent pieces of 16 bytes each, then 32 rows of 8
// pieces of the key. Piece c of row r lies at c ^ turn(r) (c ^ (r / 2 % 8) of the key), so that
// every pass of the operands' reads meets all 64 banks once: 16 rows and one piece of a key
// operand; 8 rows and two pieces of a transposing read; rows 0 .. 7 and 16 .. 23 and one piece
// of an 8-bit one. (128 wide codes have half a row of banks, and two passes.)
template <int F, int L>
struct Tile {
    static constexpr bool kCodes = F == kFmtE4m3;
    static constexpr int kLatent = kCodes ? L / 16 : L / 8;
    static constexpr int kRow = 16 * kLatent, kKeys = 32 * kRow;
    static constexpr int kLoads = 16 * kLatent / 64;          // of the latents of 16 rows
    static constexpr int kPer = 64 / kLatent;                 // rows of a load
    static __device__ __forceinline__ int turn(int r) { return ((r & 7) << 1 | ((r >> 3 ^ r >> 4) & 1)) & (kLatent - 1); }
};

// kRW x kKW waves: over tiles of 16 rows, and over keys. kExact: queries are fp32. Over bf16 rows they
// are multiplied as a bf16 head and its remainder; over codes, which fp16 holds too, as fp16 times a power of
// two of the row's own, in one product. Weights are multiplied with their remainders.
template <int F, int L, int kRW, int kKW, bool kExact>
__global__ __launch_bounds__(256, workgroups_per_cu(F, L, kRW, kExact)) void latent_kernel(CoreArgs x) {
    typedef Tile<F, L> T;
    constexpr bool kCodes = T::kCodes, kHalf = kExact && kCodes, kSplit = kExact && !kCodes;
    constexpr int kSteps = L / 32, kBlocks = L / 16;
    // Waves with keys of their own: two buffers of latents and one of keys, where LDS has room.
    constexpr bool kKeysFirst = kKW == 4 && T::kKeys <= 16384;
    constexpr int kBuffers = kKW < 4 || kKeysFirst ? 2 : 1, kKeyBuffers = kKW < 4 ? 2 : 1;
    constexpr int kGroup = kBuffers * T::kKeys + kKeyBuffers * 32 * 128;
    constexpr int kAhead = 4;                                 // operands read ahead of the products
    constexpr int kScales = kCodes ? kKW * 2 * 32 * 4 : 0;    // [group][step % 2][32]
    constexpr int kTiles = kKW * kGroup, kJoin = kKW > 1 ? 4 * kBlocks * 1024 : 0;
    constexpr int kMain = kTiles + kScales > kJoin ? kTiles + kScales : kJoin;
    __shared__ __align__(16) char lds_all[kMain + 512];
    // Behind the tiles, the waves' key ranges and what their join exchanges. These lie apart: a workgroup without keys
    // meets no barrier between the reads of the one and the first write of the other.
    int (*range)[4] = reinterpret_cast<int (*)[4]>(lds_all + kMain);                   // [lo, hi][wave]
    float *shared = reinterpret_cast<float *>(lds_all + kMain + 256);                  // [wave][row]
    constexpr bool kAccum = workgroups_per_cu(F, L, kRW, kExact) == 1;   // one wave per SIMD
    const AttnJob &a = x.a;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int n = lane & 15, g = lane >> 4;
    const int rw = wave % kRW, kw = wave / kRW;
    Seq q;
    const Work work = work_of(a, x.sp, (int)blockIdx.x, q);
    const int tile = work.tile, s = work.s;
    if (s < 0) return;
    const int rows = q.rows * a.group, R = x.rot;
    if (tile * 16 * kRW >= rows) return;
    auto first_row = [](int tile) { return 16 * (tile * kRW + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) % kRW); };
    const int r0 = first_row(tile);

    // Outputs live in accumulation registers then. Said where paths meet and where
    // anything but a product writes them: else the compiler moves all of them there and back in every step.
    auto keep = [](f32x4 &v) {
        if (kAccum) asm("" : "+a"(v));
    };
    u32x4 qf[kSteps + 2], ql[kSplit ? kSteps : 1];
    float unscale = 1.0f;   // of fp16 queries
    f32x4 o[kBlocks];
    float m = kNegInf, l = 0.0f;
    auto keep_all = [&]() {
#pragma unroll
        for (int b = 0; b < kBlocks; ++b) keep(o[b]);
    };
    int lo = 0x7FFFFFFF, hi = 0, flo = 0, fhi = 0x7FFFFFFF;   // some row sees [lo, hi), every row [flo, fhi)
    const uint32_t sign = a.scale2 < 0.0f ? 0x80008000u : 0u;   // a negative scale goes into the queries
    const float scale2 = fmaxf(fabsf(a.scale2), 0x1p-126f);   // not 0: -inf marks an unseen key
    {
        const int r = r0 + n, i = r / a.group;
        const bool on = r < rows;
        const int64_t at = (int64_t)(q.q0 + (on ? i : 0)) * a.ldq + (int64_t)(on ? r - i * a.group : 0) * (L + R) + 8 * g;
        // Of a row that there is not, and of elements behind the head's: read somewhere, and masked.
        auto place = [&](int k) { return k < kSteps ? 32 * k : min(32 * k, L + R - 32); };
        auto kept = [&](int k) { return on && (k <= kSteps || R > 32) ? 0xFFFFFFFFu : 0u; };
        if (!kExact) {
            const uint16_t *qp = static_cast<const uint16_t *>(a.q) + at;
#pragma unroll
            for (int k = 0; k < kSteps + 2; ++k) qf[k] = (ldg(reinterpret_cast<const u32x4 *>(qp + place(k))) ^ sign) & kept(k);
        } else {
            // fp32 queries; the rotated part is exact in bf16.
            const float *qp = static_cast<const float *>(a.q) + at;
            f32x4 v[kSteps + 2][2];
#pragma unroll
            for (int k = 0; k < kSteps + 2; ++k)
#pragma unroll
                for (int e = 0; e < 2; ++e) v[k][e] = ldg(reinterpret_cast<const f32x4 *>(qp + place(k) + 4 * e));
            float scale = 1.0f;
            if (kHalf) {   // with an infinity the row is done again
                float most = 0.0f;
#pragma unroll
                for (int k = 0; k < kSteps; ++k)
#pragma unroll
                    for (int e = 0; e < 8; ++e) most = fmaxf(most, fabsf(v[k][e >> 2][e & 3]));
                const HalfScale to = half_scale(groups_max(most));
                scale = to.up, unscale = to.down;
            }
#pragma unroll
            for (int k = 0; k < kSteps + 2; ++k) {
                uint32_t h[4], w[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float v0 = v[k][e >> 1][2 * (e & 1)], v1 = v[k][e >> 1][2 * (e & 1) + 1];
                    h[e] = kHalf && k < kSteps ? pack_half2(v0 * scale, v1 * scale) : pack2(v0, v1);
                    w[e] = pack2(v0 - bf16_f(h[e] & 0xFFFFu), v1 - __uint_as_float(h[e] & 0xFFFF0000u));
                }
                qf[k] = (u32x4{h[0], h[1], h[2], h[3]} ^ sign) & kept(k);
                if (kSplit && k < kSteps) ql[k] = (u32x4{w[0], w[1], w[2], w[3]} ^ sign) & kept(k);
            }
        }
        const Sees see = sees(a, q, i);
        if (on) {   // an unused column is never the reason to mask
            lo = see.tree ? min(see.lo, max(q.ctx, 0)) : see.lo;
            hi = see.tree ? q.kv : see.hi;
            flo = see.lo;
            fhi = see.hi;
        }
#pragma unroll
        for (int b = 0; b < kBlocks; ++b) {
            o[b] = f32x4{0, 0, 0, 0};
            keep(o[b]);
        }
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
    lo = __builtin_amdgcn_readfirstlane(lo) & ~31;
    hi = __builtin_amdgcn_readfirstlane(hi);
    const int64_t c0 = (int64_t)lo + work.from;
    const int k0 = c0 < hi ? (int)c0 : hi, k1 = (int)min((int64_t)hi, c0 + work.chunk), last = k1 - 1;

    if (k0 < k1) {
        const int32_t *table = a.c.table + (int64_t)s * a.c.max_pages;
        const int shift = a.c.page_shift, pmask = (1 << shift) - 1, n_pages = a.c.n_pages;
        const int pieces = kCodes ? (L + 2 * R) / 16 : (L + R) / 8, bytes = 16 * pieces;   // of a cache row
        const int64_t page_bytes = (int64_t)bytes << shift;
        // Keys come in halves of 16, each within one page; a wave fetches kHalves of them, or half of one.
        constexpr int kHalves = kRW == 1 ? 2 : 1, kShare = kRW == 4 ? 2 : 1;
        constexpr int kMine = T::kLoads / kShare, kMineKeys = 2 / kShare;                  // loads of a half
        const int half0 = kRW == 1 ? 0 : rw / (kRW / 2), share = kRW == 4 ? rw % 2 : 0;
        int page[2];
        int first_page = -64, entries = 0;   // lane i holds entry first_page + i of the table
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
        auto has_page = [&](int b) { return (unsigned)page[b] < (unsigned)n_pages; };
        uint32_t valid_in = 0;
        auto fetch = [&](int j0, int step) {
            valid_in = (has_page(0) ? 0xFFFFu : 0u) | (has_page(1) ? 0xFFFF0000u : 0u);
            const uint32_t to = lds_byte(lds_all) + kw * kGroup + (kBuffers == 2 ? step & 1 : 0) * T::kKeys;
            const uint32_t key_to = lds_byte(lds_all) + kw * kGroup + kBuffers * T::kKeys + (kKeyBuffers == 2 ? step & 1 : 0) * 32 * 128;
            int ln = lane;
            asm volatile("" : "+v"(ln));   // what follows from it is not kept through the loop
#pragma unroll
            for (int hh = 0; hh < kHalves; ++hh) {
                const int half = half0 + hh, jh = j0 + 16 * half;
                const int pg = half ? page[1] : page[0], off = min(jh, last) & pmask & ~15;
                const int most = last - min(jh, last & ~15);   // rows behind the last key read that key again
                const char *from = scalar(static_cast<const char *>(a.c.k) + ((unsigned)pg < (unsigned)n_pages ? pg : 0) * page_bytes + (int64_t)off * bytes);
                const int sub = ln / T::kLatent, c = ln % T::kLatent, first = share * kMine * T::kPer;
                const uint32_t lds_to = to + half * 16 * T::kRow + share * kMine * 1024;
                const uint32_t turned = (uint32_t)(c ^ T::turn(16 * half) ^ T::turn(first) ^ T::turn(sub)) << 4;
                if (most >= 15) {
                    const uint32_t at = (uint32_t)(first + sub) * bytes;
#pragma unroll
                    for (int i = 0; i < kMine; ++i)
                        load_to_lds(from, at + i * T::kPer * bytes + (turned ^ (uint32_t)T::turn(i * T::kPer) << 4), lds_to + i * 1024);
                } else {
#pragma unroll 1
                    for (int i = 0; i < kMine; ++i) {
                        const int r = first + i * T::kPer + sub;
                        load_to_lds(from, min(r, most) * bytes + (turned ^ (uint32_t)T::turn(i * T::kPer) << 4), __builtin_amdgcn_readfirstlane(lds_to + i * 1024));
                    }
                }
#pragma unroll
                for (int i = 0; i < kMineKeys; ++i) {
                    const int r = 8 * (share * kMineKeys + i) + (ln >> 3), piece = (ln & 7) ^ (r >> 1 & 7);
                    load_to_lds(from, min(r, most) * bytes + T::kRow + min(piece, R / 8 - 1) * 16,
                                key_to + (16 * half + 8 * (share * kMineKeys + i)) * 128);
                }
                if (kCodes && rw == (kRW == 1 ? 0 : kRW / 2 * half)) {
                    const char *sc = scalar(reinterpret_cast<const char *>(a.c.k_scale + (((int64_t)((unsigned)pg < (unsigned)n_pages ? pg : 0) << shift) + off)));
                    if (ln < 16) load_to_lds4(sc, min(ln, most) * 4, lds_byte(lds_all) + kTiles + ((kw * 2 + (step & 1)) * 32 + 16 * half) * 4);
                }
            }
        };
        const int key_v = 4 * g + (n >> 2), key_c = n < 8 ? 4 * g + (n >> 1) : 16 + 4 * g + ((n - 8) >> 1);
        auto attend = [&](const int &j0, const int &step, const uint32_t &valid, auto &&fetch_next) {
            keep_all();
            const int in = kw * kGroup + (kBuffers == 2 ? step & 1 : 0) * T::kKeys;
            const int keys_in = kw * kGroup + kBuffers * T::kKeys + (kKeyBuffers == 2 ? step & 1 : 0) * 32 * 128;
            const float *scales = reinterpret_cast<const float *>(lds_all + kTiles) + (kw * 2 + (step & 1)) * 32;
            // Operands' places, formed anew in every step: held through the loop, they would take registers.
            int kb = in + n * T::kRow + ((T::kCodes ? g >> 1 : g) ^ T::turn(n)) * 16 + (T::kCodes ? 8 * (g & 1) : 0);
            int rb = keys_in + n * 128 + ((g ^ (n >> 1 & 7)) << 4);
            asm volatile("" : "+v"(kb), "+v"(rb));
            const uint32_t second = R > 32 ? 0xFFFFFFFFu : 0u;
            f32x4 sc[2] = {{0, 0, 0, 0}, {0, 0, 0, 0}};
            // Key operand i: rows 16 (i % 2) .., elements 32 (i / 2) .. of them, the rotated ones last. Both halves in
            // turn, so that a product does not wait for the one before it.
            constexpr int kEach = kKeysFirst ? kSteps : kSteps + 2, kAll = 2 * kEach;
            auto operand = [&](int i) {
                const int b = i & 1, k = i >> 1;
                if (k >= kSteps) {
                    u32x4 kf = *reinterpret_cast<const u32x4 *>(lds_all + (rb ^ (k - kSteps) << 6) + b * 16 * 128);
                    return kf;
                }
                const int c = (kCodes ? 2 : 4) * k;
                const char *p = lds_all + (kb ^ (((c & 15) ^ b) & (T::kLatent - 1)) << 4) + (c >> 4) * 256 + b * 16 * T::kRow;
                if (!kCodes) return *reinterpret_cast<const u32x4 *>(p);
                const u32x2 w = *reinterpret_cast<const u32x2 *>(p);
                return u32x4{w.x, w.y, 0, 0};
            };
            // Reads run kAhead ahead of the products, in this order: left to itself the compiler reads each
            // operand right before its use.
            u32x4 kf[kAhead];
            f32x4 rotated[2];
            if (kKeysFirst) {
                // The rotated part first: with it read, the wave's next rows may come in.
#pragma unroll
                for (int i = 0; i < 4; ++i) kf[i] = operand(2 * kSteps + i);
                asm volatile("s_waitcnt lgkmcnt(0)" : "+v"(kf[0]), "+v"(kf[1]), "+v"(kf[2]), "+v"(kf[3])::"memory");
                fetch_next();
#pragma unroll
                for (int b = 0; b < 2; ++b) {
                    rotated[b] = mfma16(kf[b], qf[kSteps], f32x4{0, 0, 0, 0});
                    rotated[b] = mfma16(kf[2 + b] & second, qf[kSteps + 1], rotated[b]);
                    if (!kCodes) sc[b] = rotated[b];
                }
            }
            __builtin_amdgcn_s_setprio(1);
#pragma unroll
            for (int i = 0; i < kAhead; ++i) kf[i] = operand(i);
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int i = 0; i < kAll; ++i) {
                const int b = i & 1, k = i >> 1;
                u32x4 here = kf[i % kAhead];
                if (kCodes && k < kSteps) here = kHalf ? widen_half8(here.x, here.y) : widen8<kFmtE4m3>(here.x, here.y);
                if (k > kSteps) here &= second;   // what lies in the place of elements that there are not may be anything
                if (kCodes && k == kSteps) sc[b] = sc[b] * unscale * *reinterpret_cast<const f32x4 *>(scales + 16 * b + 4 * g);
                sc[b] = kHalf && k < kSteps ? mfma16_half(here, qf[k], sc[b]) : mfma16(here, qf[k], sc[b]);
                if (kSplit && k < kSteps) sc[b] = mfma16(here, ql[k < kSteps ? k : 0], sc[b]);
                if (i + kAhead < kAll) kf[i % kAhead] = operand(i + kAhead);
                __builtin_amdgcn_sched_barrier(0);
            }
            __builtin_amdgcn_s_setprio(0);
            if (kKeysFirst && kCodes) {
#pragma unroll
                for (int b = 0; b < 2; ++b) {
                    const f32x4 ks = *reinterpret_cast<const f32x4 *>(scales + 16 * b + 4 * g);
#pragma unroll
                    for (int e = 0; e < 4; ++e) sc[b][e] = __builtin_fmaf(sc[b][e] * unscale, ks[e], rotated[b][e]);
                }
            }
            const bool all = j0 >= flo && j0 + 32 <= min(fhi, k1) && valid == 0xFFFFFFFFu;
            float v[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = sc[e >> 2][e & 3];
            if (__builtin_expect(!all, 0)) {
                const CoreArgs again = argument_again<CoreArgs>();
                const Seq qq = seq_of(again.a, work.s);
                const int r = first_row(work.tile) + (threadIdx.x & 15);
                const uint32_t mine = (visible32(again.a, qq, sees(again.a, qq, r / again.a.group), j0) & valid & bits(0, k1 - j0)) >> (4 * g);
#pragma unroll
                for (int e = 0; e < 8; ++e) v[e] = mine & (1u << (16 * (e >> 2) + (e & 3))) ? v[e] : kNegInf;
            }
            float top = v[0];
#pragma unroll
            for (int e = 1; e < 8; ++e) top = fmaxf(top, v[e]);
            top = groups_max(top);
            top = top == kNegInf ? top : top * scale2;
            if (__builtin_expect(__any(top > m + 8.0f), 0)) {
                // The reference moves only when a score passes it by 2^8: sums stay in range.
                const float now = fmaxf(m, top), up = now == m ? 1.0f : __builtin_amdgcn_exp2f(m - now);
                m = now;
                l *= up;
#pragma unroll
                for (int b = 0; b < kBlocks; ++b) {
                    o[b] *= up;
                    keep(o[b]);
                }
            }
            keep_all();
            const float ref = m == kNegInf ? 0.0f : m;
            float p[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) l += p[e] = __builtin_amdgcn_exp2f(__builtin_fmaf(v[e], scale2, -ref));
            if (kCodes) {
#pragma unroll
                for (int b = 0; b < 2; ++b) {
                    const f32x4 vs = *reinterpret_cast<const f32x4 *>(scales + 16 * b + 4 * g);
#pragma unroll
                    for (int e = 0; e < 4; ++e) p[4 * b + e] = p[4 * b + e] == 0.0f ? 0.0f : p[4 * b + e] * vs[e];
                }
            }
            const u32x4 ph = {pack2(p[0], p[1]), pack2(p[2], p[3]), pack2(p[4], p[5]), pack2(p[6], p[7])};
            u32x4 pl;
#pragma unroll
            for (int e = 0; e < 4; ++e) pl[e] = pack2(p[2 * e] - bf16_f(ph[e] & 0xFFFFu), p[2 * e + 1] - __uint_as_float(ph[e] & 0xFFFF0000u));
            __builtin_amdgcn_s_setprio(1);
            const int kv = kCodes ? key_c : key_v;
            int vb = in + kv * T::kRow + ((T::kCodes ? 0 : n >> 1 & 1) ^ T::turn(kv)) * 16 + 8 * (n & 1);
            asm volatile("" : "+v"(vb));
#pragma unroll
            for (int b = 0; b < kBlocks; ++b) {
                const int c = kCodes ? b : 2 * b;
                const char *p = lds_all + (vb ^ (c & 15 & (T::kLatent - 1)) << 4) + (c >> 4) * 256;
                u32x4 vf;
                if (kCodes) {
                    const u32x2 w = read_tr8(p);
                    vf = widen8<kFmtE4m3>(w.x, w.y);
                } else {
                    // rows kv and 16 + kv, whose turns differ in bit 0
                    const u32x2 u = read_tr16(p), w = read_tr16(lds_all + (vb ^ ((c & 15) ^ 1) << 4) + (c >> 4) * 256 + 16 * T::kRow);
                    vf = u32x4{u.x, u.y, w.x, w.y};
                }
                o[b] = mfma16(vf, ph, o[b]);
                o[b] = mfma16(vf, pl, o[b]);
            }
            constexpr int kReads = kCodes ? 1 : 2;   // of an operand
            __builtin_amdgcn_sched_group_barrier(0x100, kReads * kAhead, 1);
#pragma unroll
            for (int i = 0; i < kBlocks; ++i) {
                __builtin_amdgcn_sched_group_barrier(0x008, 2, 1);
                if (i + kAhead < kBlocks) __builtin_amdgcn_sched_group_barrier(0x100, kReads, 1);
            }
            __builtin_amdgcn_s_setprio(0);
        };
        if (kKW < 4) {
            // A group's tile of step n is fetched into buffer n % 2 while that of step n - 1 is
            // worked on. All groups take as many steps, and meet at the same barriers.
            constexpr int kStride = 32 * kKW;
            const int steps = (k1 - k0 + kStride - 1) / kStride;
            auto at = [&](int step) { return k0 + (step * kKW + kw) * 32; };
            uint32_t valid = 0;
            look(min(at(0), last));
            if (at(0) < k1) fetch(at(0), 0);
            valid = valid_in;
            wait_loads();
            __syncthreads();
            for (int step = 0; step < steps; ++step) {
                const int j0 = at(step), next = j0 + kStride;
                if (next < k1) {
                    look(next);
                    fetch(next, step + 1);
                }
                if (j0 < k1 && j0 + 31 >= wlo && j0 < whi) attend(j0, step, valid, [] {});
                keep_all();
                valid = valid_in;
                wait_loads();
                __syncthreads();
            }
        } else {
            // The wave's own keys, 32 of every 128: nothing to meet for.
            int j0 = k0 + 32 * kw;
            auto come = [&](int j, int step) {
                if (j < k1) {
                    look(j);
                    fetch(j, step);
                }
            };
            if (kKeysFirst) come(j0, 0);
            for (int step = 0; j0 < k1; j0 += 128, ++step) {
                if (!kKeysFirst) come(j0, step);
                wait_loads();
                const uint32_t valid = valid_in;
                attend(j0, step, valid, [&] { come(j0 + 128, step + 1); });
                keep_all();
                if (!kKeysFirst) asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");   // read before the next rows come in
            }
            __syncthreads();
        }
    }

    keep_all();
    // Outputs, of a piece of the keys or of all: normalised, with the reference and the sum of a piece.
    const CoreArgs y = argument_again<CoreArgs>();
    const AttnJob &b = y.a;
    const Split &sp = y.sp;
    const Seq qq = seq_of(b, s);
    const bool wide = sp.n_split > 1 || y.wide;
    auto put = [&](int r, int at, const float *v) {
        const int i = r / b.group;
        const size_t in_o = (size_t)(qq.q0 + i) * b.ldo + (size_t)(r - i * b.group) * L;
        if (wide)
            put4((sp.n_split > 1 ? sp.part + part_row(b, sp, work.part, 0, tile, r) * L : static_cast<float *>(b.o) + in_o) + at, v);
        else
            put4(static_cast<uint16_t *>(b.o) + in_o + at, v);
    };
    auto put_stat = [&](int r, float mm, float ll) {
        if (sp.n_split > 1) sp.ml[part_row(b, sp, work.part, 0, tile, r)] = make_float2(mm, ll);
    };
    // A row with an infinity or a NaN is done again key by key: one that it does not see may
    // have got in as 0 * NaN.
    auto redo = [&](uint32_t again, int first) {
        for (uint32_t left = again; left; left &= left - 1) {
            const int rr = first + __ffs(left) - 1, ii = rr / b.group;
            float acc[8], mm, ll;
            latent_row<typename std::conditional<kExact, float, uint16_t>::type, F>(b, y.rot, qq, ii, rr - ii * b.group, k0, k1, acc, mm, ll);
            if (8 * lane < L) {
#pragma unroll
                for (int e = 0; e < 8; ++e) acc[e] = ll == 0.0f ? 0.0f : acc[e] / ll;
                put(rr, 8 * lane, acc);
                put(rr, 8 * lane + 4, acc + 4);
            }
            if (lane == 0) put_stat(rr, mm, ll);
        }
    };
    l = groups_sum(l);
    float check = l * 0.0f;
#pragma unroll
    for (int c = 0; c < kBlocks; ++c) check += o[c].x * 0.0f + o[c].y * 0.0f + o[c].z * 0.0f + o[c].w * 0.0f;
    const int r = r0 + n;
    uint64_t odd = __ballot(r < rows && (check != 0.0f || beyond(m)));
    odd |= odd >> 32;
    odd |= odd >> 16;
    uint32_t again = (uint32_t)odd & 0xFFFFu;
    if constexpr (kKW == 1) {
        if (r < rows && !(again >> n & 1u)) {
            const float inv = l == 0.0f ? 0.0f : 1.0f / l;
#pragma unroll
            for (int c = 0; c < kBlocks; ++c) {
                const float v[4] = {o[c].x * inv, o[c].y * inv, o[c].z * inv, o[c].w * inv};
                put(r, 16 * c + 4 * g, v);
            }
            if (g == 0) put_stat(r, m, l);
        }
        redo(again, r0);
    } else {
        // The groups' outputs meet in LDS, each wave joins a part of the columns.
        constexpr int kOwn = kBlocks / kKW;
        f32x4 *mine = reinterpret_cast<f32x4 *>(lds_all);
#pragma unroll
        for (int c = 0; c < kBlocks; ++c) mine[(wave * kBlocks + c) * 64 + lane] = o[c];
        if (g == 0) shared[wave * 16 + n] = m;
        __syncthreads();
        float ms[kKW], top = kNegInf;
#pragma unroll
        for (int w = 0; w < kKW; ++w) {
            ms[w] = shared[(w * kRW + rw) * 16 + n];
            top = fmaxf(top, ms[w]);
        }
        __syncthreads();
        if (g == 0) shared[wave * 16 + n] = l;
        __syncthreads();
        float sum = 0.0f, up[kKW];
#pragma unroll
        for (int w = 0; w < kKW; ++w) {
            up[w] = ms[w] == kNegInf ? 0.0f : __builtin_amdgcn_exp2f(ms[w] - top);
            sum += up[w] * shared[(w * kRW + rw) * 16 + n];
        }
        __syncthreads();
        if (lane == 0) reinterpret_cast<uint32_t *>(shared)[wave] = again;
        __syncthreads();
        again = 0;
#pragma unroll
        for (int w = 0; w < kKW; ++w) again |= reinterpret_cast<const uint32_t *>(shared)[w * kRW + rw];
        again = __builtin_amdgcn_readfirstlane(again);
        if (r < rows && !(again >> n & 1u)) {
            const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
#pragma unroll
            for (int c = 0; c < kOwn; ++c) {
                const int at = kw * kOwn + c;
                f32x4 v{0, 0, 0, 0};
#pragma unroll
                for (int w = 0; w < kKW; ++w) v += mine[((w * kRW + rw) * kBlocks + at) * 64 + lane] * up[w];
                const float e[4] = {v.x * inv, v.y * inv, v.z * inv, v.w * inv};
                put(r, 16 * at + 4 * g, e);
            }
            if (kw == 0 && g == 0) put_stat(r, top, sum);
        }
        if (kw == 0) redo(again, r0);
    }
}

template <int F, int L, int kRW, int kKW>
void launch(const CoreArgs &x, const CoreKind &k, unsigned blocks, hipStream_t s) {
    const dim3 g(blocks), b(256);
    if (k.exact)
        hipLaunchKernelGGL((latent_kernel<F, L, kRW, kKW, true>), g, b, 0, s, x);
    else
        hipLaunchKernelGGL((latent_kernel<F, L, kRW, kKW, false>), g, b, 0, s, x);
}

template <int F, int L>
void run(const CoreArgs &x, const CoreKind &k, unsigned blocks, hipStream_t s) {
    if (k.row_waves == 4)
        launch<F, L, 4, 1>(x, k, blocks, s);
    else if (k.row_waves == 2)
        launch<F, L, 2, 2>(x, k, blocks, s);
    else
        launch<F, L, 1, 4>(x, k, blocks, s);
}

template <int F>
void run(const CoreArgs &x, const CoreKind &k, unsigned blocks, hipStream_t s) {
    switch (x.a.c.d) {
        case 128: run<F, 128>(x, k, blocks, s); break;
        case 256: run<F, 256>(x, k, blocks, s); break;
        default: run<F, 512>(x, k, blocks, s);
    }
}

}  // namespace

void launch_latent_tile(const CoreArgs &x, int fmt, const CoreKind &k, unsigned blocks, hipStream_t s) {
    fmt == kFmtE4m3 ? run<kFmtE4m3>(x, k, blocks, s) : run<kFmtBf16>(x, k, blocks, s);
}

}  // namespace wl
