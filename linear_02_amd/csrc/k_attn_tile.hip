// Attention with many query rows per key/value head (prompts, larger trees).
//
// A workgroup takes 128 query rows of one key/value head, a row being a new token
// and one of the query heads that share the key/value head, so that those heads
// share every key that is staged; its four waves hold up to 32 each. (64 rows, 16
// a wave, where a head has no more or the call is small.) Keys and
// values pass through LDS 32 at a time, in two buffers: while the waves work on
// one, the next 32 are on their way into the other. Queries, scores, weights and
// outputs stay in registers from the first key to the last, which at heads of 256
// fills them: 128 for outputs, 64 for queries, 16 for scores, the rest for
// operands on their way. Two workgroups share a CU, so that one's softmax and
// barriers fall into the other's products.
// int8 and e4m3 keys are widened to bf16 between two barriers (one workgroup's
// widening under the other's products), or with 129 to 256 rows, as larger trees
// have, by eight waves that share the widened keys.
//
// Bound by the issue of matrix products and of the softmax between them: 2048
// tokens over 4000 keys, 32 query and 8 key/value heads of 256, causal: bf16
// 201 us (200 GFLOP, 996 TFLOP/s; a large library product reaches 1335), e4m3
// 268 us; 8192 over 8192 in bf16 989 us (1112 TFLOP/s). Trees of up to 48 tokens of
// 4 sequences over up to 16384 int8 keys: 126 us with the join, of whose cycles the
// matrix cores work in 20 %, the vector units in 32 %, LDS in 27 % (and 4 % of
// conflicts): eight waves of one workgroup that wait for each other every 32 keys.
#include "wl_attn_mfma.h"

namespace wl {

namespace {

template <int N>
struct Tiles {
    static constexpr int n = N;
};

// kNT: tiles of 16 query rows per wave, at most. kExact: weights as a bf16 head plus a
// bf16 remainder, 16 bits of them, for which one tile leaves registers; else as one bf16.
template <int F, int DT, int NW, int kNT, bool kExact>
__global__ __launch_bounds__(64 * NW, 2) void tile_kernel(TileArgs x) {
    const AttnJob &a = x.a;
    constexpr bool kCodes = F == kFmtInt8 || F == kFmtE4m3;
    constexpr int kSteps = DT / 32, kBlocks = DT / 16;
    constexpr int kRow = 2 * DT, kSide = 32 * kRow;          // LDS bytes of a row, of 32 keys
    constexpr int kPieces = DT / 8;                          // 16-byte pieces of a row
    constexpr int kMaskV = DT >= 128 ? 7 : 3;
    // Operands read ahead of the products. 2048 tokens over 4000 keys, 32 heads of
    // 256, in us for 2, 3, 4, 6: bf16 213, 207, 208, 260; e4m3 266, 295, 294, 323 (the
    // registers that more would take are not there).
    constexpr int kAhead = kNT == 1 ? 4 : kCodes ? 2 : 3;
    static_assert(!kExact || kNT == 1, "two tiles leave no registers for the remainders");
    // LDS place of 16-byte piece c of a row: c ^ f(row), such that the 16 lanes that
    // one pass of a read serves meet all 64 banks.
    auto fk = [](int r) { return DT >= 128 ? r & 15 : (r >> 1) & 7; };
    auto fv = [](int r) { return (r & kMaskV) << 1; };
    // One LDS object: beside a second one the compiler waits for the loads into
    // LDS that are still on their way before every read.
    constexpr bool kTwo = !kCodes || NW == 8;                // two buffers of keys and values, or one and more workgroups
    constexpr int kRaw0 = (kTwo ? 4 : 2) * kSide, kTail = kRaw0 + (kCodes ? kSide : 0);
    __shared__ __align__(16) char lds_all[kTail + 1024 + 8 * NW];
    char (*lds)[2][kSide] = reinterpret_cast<char (*)[2][kSide]>(lds_all);   // [buffer][K, V]
    char *raw = lds_all + kRaw0;                                             // codes as fetched: K, then V
    float (*lds_scale)[2][32] = reinterpret_cast<float (*)[2][32]>(lds_all + kTail);   // [step % 4][K, V]
    int (*range)[NW] = reinterpret_cast<int (*)[NW]>(lds_all + kTail + 1024);
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int n = lane & 15, g = lane >> 4;
    const int kvh = (int)blockIdx.x % a.c.n_kv;
    Seq q;
    const Work work = work_of(a, x.sp, (int)blockIdx.x / a.c.n_kv, q);
    const int tile = work.tile, s = work.s;
    if (s < 0) return;
    const int rows = q.rows * a.group, d = a.c.d;
    if (tile * NW * 16 * kNT >= rows) return;
    // The four SIMDs share the rows alike: 16 for each of the first four waves, as
    // many for each of the next four, and so on, up to 32 per wave. With 32 per wave
    // from the first on, two SIMDs had twice the work at 192 rows, and the trees above
    // took 157 us; at 48 rows only two SIMDs had any (8 trees of 12 tokens over up to
    // 8192 int8 keys: 89, now 74 us). bf16 keys come as fast as memory gives them at so
    // few rows (97 and 94 us), and prompts lose 1 % to the second loop.
    auto rows_of = [](int tile, int rows) {
        const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), tile0 = tile * NW * 16 * kNT;
        if (!kCodes || kNT == 1) return WaveRows{tile0 + 16 * kNT * w, kNT};
        const int all = (rows - tile0 + 15) / 16, early = all > NW ? 2 : 1;
        if (NW == 4 || w < 4) return WaveRows{tile0 + 16 * w * early, early};
        const int late = all > 12 ? 2 : 1;
        return WaveRows{tile0 + 16 * (4 * early + (w - 4) * late), late};
    };
    const int r0 = rows_of(tile, rows).first, nt = rows_of(tile, rows).tiles;

    u32x4 qf[kNT][kSteps];
    f32x4 o[kNT][kBlocks];
    float m[kNT], l[kNT];
    int lo = 0x7FFFFFFF, hi = 0, flo = 0, fhi = 0x7FFFFFFF;   // some row sees [lo, hi), every row [flo, fhi)
    const uint32_t sign = a.scale2 < 0.0f ? 0x80008000u : 0u;   // a negative scale goes into the queries
    const float scale2 = fmaxf(fabsf(a.scale2), 0x1p-126f);   // not 0: -inf marks an unseen key
#pragma unroll
    for (int t = 0; t < kNT; ++t) {
        const int r = r0 + 16 * t + n, i = r / a.group;
        const bool on = t < nt && r < rows;
        const uint16_t *qp = static_cast<const uint16_t *>(a.q) + (size_t)(q.q0 + (on ? i : 0)) * a.ldq +
                             (size_t)(kvh * a.group + (on ? r - i * a.group : 0)) * d;
#pragma unroll
        for (int k = 0; k < kSteps; ++k) {
            const int at = 32 * k + 8 * g;
            qf[t][k] = u32x4{0, 0, 0, 0};
            if (on && at < d) qf[t][k] = ldg(reinterpret_cast<const u32x4 *>(qp + at)) ^ sign;
        }
        const Sees see = sees(a, q, i);
        if (on) {   // an unused column is never the reason to mask
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
    for (int x = 1; x < 16; x <<= 1) {
        lo = min(lo, __shfl_xor(lo, x));
        hi = max(hi, __shfl_xor(hi, x));
        flo = max(flo, __shfl_xor(flo, x));
        fhi = min(fhi, __shfl_xor(fhi, x));
    }
    flo = __builtin_amdgcn_readfirstlane(flo);
    fhi = __builtin_amdgcn_readfirstlane(fhi);
    // Keys of this wave's rows, of the workgroup's, and the piece of them that is this workgroup's.
    if (lane == 0) range[0][wave] = lo, range[1][wave] = hi;
    __syncthreads();
    const int wlo = __builtin_amdgcn_readfirstlane(lo), whi = __builtin_amdgcn_readfirstlane(hi);
#pragma unroll
    for (int w = 0; w < NW; ++w) lo = min(lo, range[0][w]), hi = max(hi, range[1][w]);
    lo = __builtin_amdgcn_readfirstlane(lo) & ~31;
    hi = __builtin_amdgcn_readfirstlane(hi);
    const int64_t c0 = (int64_t)lo + work.from;
    const int k0 = c0 < hi ? (int)c0 : hi, k1 = (int)min((int64_t)hi, c0 + work.chunk), last = k1 - 1;

    if (k0 < k1) {
        const int32_t *table = a.c.table + (int64_t)s * a.c.max_pages;
        const int shift = a.c.page_shift, pmask = (1 << shift) - 1, n_pages = a.c.n_pages;
        const int bytes = d * (kCodes ? 1 : 2);              // of a cache row
        const int64_t head = (int64_t)kvh << shift, pitch = (int64_t)a.c.n_kv << shift;   // rows: of this head in a page, of a page
        const char *kpool = static_cast<const char *>(a.c.k) + head * bytes;
        const int64_t to_v = static_cast<const char *>(a.c.v) - static_cast<const char *>(a.c.k), page_bytes = pitch * bytes;
        // Keys come in halves of 16, each within one page. A wave fetches kMine rows: its half, its first row there.
        constexpr int kMine = 32 / NW;
        const int half = wave / (NW / 2), row0 = kMine * (wave % (NW / 2));
        int page[2];                                         // of the keys that are fetched next
        // Page numbers come from a register: lane i holds entry first_page + i of the
        // table, read anew every 64 pages. A load per step would have to be waited
        // for behind the step's own loads.
        int first_page = -64, pages = 0;
        auto look = [&](int j0) {
            const int e0 = min(j0, last) >> shift, e1 = min(j0 + 16, last) >> shift;
            if (e1 - first_page >= 64) {
                first_page = e0;
                pages = table[min(e0 + lane, last >> shift)];
                __builtin_amdgcn_s_waitcnt(0x0F70);   // vmcnt(0)
            }
            page[0] = __builtin_amdgcn_readlane(pages, e0 - first_page);
            page[1] = __builtin_amdgcn_readlane(pages, e1 - first_page);
        };
        auto has_page = [&](int b) { return (unsigned)page[b] < (unsigned)n_pages; };
        // First of the 16 keys of half b, within its page. Rows behind the last key read that key again.
        auto off_of = [&](int j0, int b) { return min(j0 + 16 * b, last) & pmask & ~15; };
        auto row_at = [&](int j0, int b, int r) { return min(r, last - min(j0 + 16 * b, last & ~15)); };
        // bf16: 64 pieces per load, straight to their places.
        constexpr int kDma = kPieces * kMine / 64;           // loads per wave and side
        // codes: as they lie, into a patch that the wave which fetched them widens from.
        constexpr int kCodePieces = DT / 16, kRaw = (kMine * kCodePieces + 63) / 64;   // pieces of a row; loads per wave and side
        uint32_t valid_in = 0;
        auto fetch = [&](int j0, int step) {
            valid_in = (has_page(0) ? 0xFFFFu : 0u) | (has_page(1) ? 0xFFFF0000u : 0u);
            const int pg = half ? page[1] : page[0];
            const char *kp = scalar(kpool + ((unsigned)pg < (unsigned)n_pages ? pg : 0) * page_bytes + off_of(j0, half) * bytes);
            const char *vp = kp + to_v;
            const bool whole = j0 + 32 <= k1;
            int ln = lane;
            asm volatile("" : "+v"(ln));   // what follows from it is not kept through the loop
            if (!kCodes) {
                constexpr int kStep = 64 / kPieces;          // rows per load
                const int dr = ln / kPieces, c = ln % kPieces;
                const uint32_t to = lds_byte(lds_all) + (step & 1) * 2 * kSide + wave * kMine * kRow;
                auto piece = [&](int i, bool v) {
                    const int r = row0 + i * kStep + dr;
                    return (uint32_t)min((c ^ (v ? fv(r) : fk(r))) * 16, bytes - 16);
                };
                if (whole) {
                    const uint32_t at = (row0 + dr) * bytes;
#pragma unroll
                    for (int i = 0; i < kDma; ++i) {
                        load_to_lds(kp, at + i * kStep * bytes + piece(i, false), to + i * 1024);
                        load_to_lds(vp, at + i * kStep * bytes + piece(i, true), to + kSide + i * 1024);
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < kDma; ++i) {
                        const uint32_t at = row_at(j0, half, row0 + i * kStep + dr) * bytes;
                        load_to_lds(kp, at + piece(i, false), to + i * 1024);
                        load_to_lds(vp, at + piece(i, true), to + kSide + i * 1024);
                    }
                }
            } else {
#pragma unroll
                for (int i = 0; i < kRaw; ++i) {
                    const int p = i * 64 + ln, c = min(p % kCodePieces * 16, bytes - 16);
                    if (p >= kMine * kCodePieces) break;
                    const uint32_t at = row_at(j0, half, row0 + p / kCodePieces) * bytes + c;
                    load_to_lds(kp, at, lds_byte(raw) + (wave * kMine * kCodePieces + i * 64) * 16);
                    load_to_lds(vp, at, lds_byte(raw) + 32 * DT + (wave * kMine * kCodePieces + i * 64) * 16);
                }
                // 16 scales of K or V each by four waves
                if (wave < 4) {
                    const int h = wave >> 1, pg = h ? page[1] : page[0];
                    const char *scales = reinterpret_cast<const char *>(wave & 1 ? a.c.v_scale : a.c.k_scale);
                    const int64_t from = ((unsigned)pg < (unsigned)n_pages ? pg : 0) * pitch + head + off_of(j0, h);
                    if (ln < 16)
                        load_to_lds4(scalar(scales + from * 4), row_at(j0, h, ln) * 4, lds_byte(lds_scale[step & 3][wave & 1] + 16 * h));
                }
            }
        };
        // What fetch(.., step) began is there; codes are widened into their buffer.
        auto land = [&](int step) {
            wait_loads();
            if (!kCodes) return;
            char *to = lds_all + (kTwo ? (step & 1) * 2 * kSide : 0);
#pragma unroll
            for (int i = 0; i < kRaw; ++i) {
                if (i * 64 + lane >= kMine * kCodePieces) break;
                const int p = wave * kMine * kCodePieces + i * 64 + lane, r = p / kCodePieces, c = p % kCodePieces * 2;
                const u32x4 k = *reinterpret_cast<const u32x4 *>(raw + p * 16), v = *reinterpret_cast<const u32x4 *>(raw + 32 * DT + p * 16);
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    *reinterpret_cast<u32x4 *>(to + r * kRow + ((c + e) ^ fk(r)) * 16) =
                        e ? widen8<F>(k.z, k.w) : widen8<F>(k.x, k.y);
                    *reinterpret_cast<u32x4 *>(to + kSide + r * kRow + ((c + e) ^ fv(r)) * 16) =
                        e ? widen8<F>(v.z, v.w) : widen8<F>(v.x, v.y);
                }
            }
        };
        // Operand addresses within a buffer.
        const int at_k = n * kRow + ((g ^ fk(n)) << 4);      // piece 4 k + g: ^ (k << 6)
        const int key_v = 4 * g + (n >> 2), at_v = key_v * kRow + ((key_v & kMaskV) << 5) + 8 * (n & 3);   // block b: ^ (b << 5)
        // 32 keys for the first N tiles of this wave's rows.
        auto attend = [&](auto tiles, const int &j0, const int &step, const uint32_t &valid) {
            constexpr int N = decltype(tiles)::n;
            // Formed anew in every step: held in registers through the loop, the
            // places of all operands would leave none to read ahead into.
            const int in = kTwo ? (step & 1) * 2 * kSide : 0;
            int kb = at_k + in, vb = at_v + in + kSide;
            asm volatile("" : "+v"(kb), "+v"(vb));
            // The products at a higher wave priority than the softmax between them: the
            // other wave of the SIMD does its softmax meanwhile (and the compiler keeps the
            // phases apart: 322 -> 294 us for the prompt above in e4m3).
            __builtin_amdgcn_s_setprio(1);
            f32x4 sc[N][2];
#pragma unroll
            for (int b = 0; b < 2; ++b) {
#pragma unroll
                for (int t = 0; t < N; ++t) sc[t][b] = f32x4{0, 0, 0, 0};
#pragma unroll
                for (int k = 0; k < kSteps; ++k) {
                    const u32x4 kf = *reinterpret_cast<const u32x4 *>(lds_all + (kb ^ ((k & 3) << 6)) + (k >> 2) * 256 + b * 16 * kRow);
#pragma unroll
                    for (int t = 0; t < N; ++t) sc[t][b] = mfma16(kf, qf[t][k], sc[t][b]);
                }
            }
            // Operand reads run kAhead ahead of the products: left to itself the
            // compiler reads each operand right before its use.
            __builtin_amdgcn_sched_group_barrier(0x100, kAhead, 0);
#pragma unroll
            for (int i = 0; i < 2 * kSteps; ++i) {
                __builtin_amdgcn_sched_group_barrier(0x008, N, 0);
                if (i + kAhead < 2 * kSteps) __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
            }
            __builtin_amdgcn_s_setprio(0);
            if (kCodes) {
#pragma unroll
                for (int b = 0; b < 2; ++b) {
                    const f32x4 ks = *reinterpret_cast<const f32x4 *>(&lds_scale[step & 3][0][16 * b + 4 * g]);
#pragma unroll
                    for (int t = 0; t < N; ++t) sc[t][b] *= ks;
                }
            }
            u32x4 ph[N], pl[N];
            const bool all = j0 >= flo && j0 + 32 <= min(fhi, k1) && valid == 0xFFFFFFFFu;
#pragma unroll
            for (int t = 0; t < N; ++t) {
                float x[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) x[e] = sc[t][e >> 2][e & 3];
                if (!all) {
                    const uint32_t mine = (seen(argument_again<TileArgs>(), work, rows_of, t, j0) & valid & bits(0, k1 - j0)) >> (4 * g);
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
                f32x4 vm[2];
                if (kCodes) {
#pragma unroll
                    for (int b = 0; b < 2; ++b) vm[b] = *reinterpret_cast<const f32x4 *>(&lds_scale[step & 3][1][16 * b + 4 * g]);
                }
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    p[e] = __builtin_amdgcn_exp2f(__builtin_fmaf(x[e], scale2, -ref));
                    if (kCodes || kExact) l[t] += p[e];
                    if (kCodes) p[e] = p[e] == 0.0f ? 0.0f : p[e] * vm[e >> 2][e & 3];
                }
                ph[t] = u32x4{pack2(p[0], p[1]), pack2(p[2], p[3]), pack2(p[4], p[5]), pack2(p[6], p[7])};
                if (kExact) {
                    uint32_t r[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        r[e] = pack2(p[2 * e] - bf16_f(ph[t][e] & 0xFFFFu), p[2 * e + 1] - __uint_as_float(ph[t][e] & 0xFFFF0000u));
                    pl[t] = u32x4{r[0], r[1], r[2], r[3]};
                } else if (!kCodes) {
                    // the sum of the weights as the product will use them
                    constexpr uint32_t kOnes = 0x3F803F80u;
                    l[t] = dot2(ph[t].x, kOnes, l[t]);
                    l[t] = dot2(ph[t].y, kOnes, l[t]);
                    l[t] = dot2(ph[t].z, kOnes, l[t]);
                    l[t] = dot2(ph[t].w, kOnes, l[t]);
                }
            }
            __builtin_amdgcn_s_setprio(1);
#pragma unroll
            for (int b = 0; b < kBlocks; ++b) {
                const char *p = lds_all + (vb ^ ((b & 7) << 5)) + (b >> 3) * 256;
                const u32x2 x = read_tr16(p), y = read_tr16(p + 16 * kRow);
#pragma unroll
                for (int t = 0; t < N; ++t) {
                    o[t][b] = mfma16(u32x4{x.x, x.y, y.x, y.y}, ph[t], o[t][b]);
                    if (kExact) o[t][b] = mfma16(u32x4{x.x, x.y, y.x, y.y}, pl[t], o[t][b]);
                }
            }
            __builtin_amdgcn_sched_group_barrier(0x100, 2 * kAhead, 1);
#pragma unroll
            for (int i = 0; i < kBlocks; ++i) {
                __builtin_amdgcn_sched_group_barrier(0x008, kExact ? 2 * N : N, 1);
                if (i + kAhead < kBlocks) __builtin_amdgcn_sched_group_barrier(0x100, 2, 1);
            }
            __builtin_amdgcn_s_setprio(0);
        };
        // Step n is fetched into buffer n % 2 while step n - 1 is worked on, and has
        // landed for every wave behind the barrier at that step's end. Codes take one
        // more step: fetched, then widened into their buffer. With eight waves the two
        // that share a SIMD do that at opposite ends of a step, so that one widens
        // while the other feeds the matrix cores; with four waves and one buffer it
        // is done between two barriers, and the other workgroup of the CU goes on.
        look(k0);
        fetch(k0, 0);
        uint32_t valid = valid_in, valid_next = 0;
        if (k0 + 32 < k1) look(k0 + 32);
        if (kTwo) land(0);
        if (kCodes && kTwo && k0 + 32 < k1) {
            fetch(k0 + 32, 1);
            valid_next = valid_in;
            look(min(k0 + 64, last));
        }
        __syncthreads();
        // Waves of a workgroup with one and with two tiles walk in loops of their own and
        // meet at every barrier: each loop has the same ones, as often.
        auto walk = [&](auto tiles) {
            int step = 0;
            for (int j0 = k0; j0 < k1; j0 += 32, ++step) {
                const bool more = j0 + 32 < k1;
                // Codes of the step after next, once the next step's are widened.
                auto advance = [&]() {
                    if (!more) return;
                    land(step + 1);
                    if (j0 + 64 < k1) {
                        fetch(j0 + 64, step + 2);
                        look(min(j0 + 96, last));
                    }
                };
                if (kCodes && !kTwo) {
                    land(step);
                    valid = valid_in;
                }
                if (!(kCodes && kTwo)) {
                    if (more) {
                        fetch(j0 + 32, step + 1);
                        look(min(j0 + 64, last));
                    }
                } else if (wave < 4) {
                    advance();
                }
                if (kCodes && !kTwo) __syncthreads();
                if (j0 + 31 >= wlo && j0 < whi) {
                    attend(tiles, j0, step, valid);
                }
                if (!kCodes && more) land(step + 1);
                if (kCodes && kTwo && wave >= 4) advance();
                if (kTwo) valid = kCodes ? valid_next : valid_in, valid_next = valid_in;
                __syncthreads();
            }
        };
        if (!kCodes || kNT == 1 || nt == kNT)
            walk(Tiles<kNT>());
        else
            walk(Tiles<1>());
    }

    finish<uint16_t, F, DT, kNT>(argument_again<TileArgs>(), work, rows_of, o, m, l, k0, k1);
}

template <int F, int DT, int NW, int NT, bool EX>
void run(const AttnJob &a, const Split &sp, hipStream_t s) {
    hipLaunchKernelGGL((tile_kernel<F, DT, NW, NT, EX>), dim3((unsigned)sp.items * a.c.n_kv), dim3(64 * NW), 0, s, TileArgs{a, sp});
}

template <int F, int NW, int NT, bool EX>
void pick(const AttnJob &a, const Split &sp, hipStream_t s) {
    if (a.c.d <= 64)
        run<F, 64, NW, NT, EX>(a, sp, s);
    else if (a.c.d <= 128)
        run<F, 128, NW, NT, EX>(a, sp, s);
    else
        run<F, 256, NW, NT, EX>(a, sp, s);
}

template <int F>
void pick(const AttnJob &a, const Split &sp, int waves, int tiles, bool exact, hipStream_t s) {
    if (tiles == 1)
        exact ? pick<F, 4, 1, true>(a, sp, s) : pick<F, 4, 1, false>(a, sp, s);
    else if (waves == 8)
        pick<F, F == kFmtBf16 ? 4 : 8, 2, false>(a, sp, s);
    else
        pick<F, 4, 2, false>(a, sp, s);
}

}  // namespace

void launch_tile(const AttnJob &a, int fmt, const Split &sp, int waves, int tiles, bool exact, hipStream_t s) {
    switch (fmt) {
        case kFmtBf16: pick<kFmtBf16>(a, sp, waves, tiles, exact, s); break;
        case kFmtInt8: pick<kFmtInt8>(a, sp, waves, tiles, exact, s); break;
        default: pick<kFmtE4m3>(a, sp, waves, tiles, exact, s);
    }
}

}  // namespace wl
