// Matrix-core pieces of the attention kernels for bf16 queries.
//
// v_mfma_f32_16x16x32_bf16, D = A B + C: lane l holds A[m = l & 15][k = 8 g + e],
// B[k = 8 g + e][n = l & 15] (e = 0..7) and C[m = 4 g + i][n = l & 15] (i = 0..3),
// with g = l >> 4. Scores are formed transposed, S^T = K Q^T (A = 16 keys, B = 16
// query rows), so that a lane owns one query row: its maximum and sum are lane
// values, joined over the four lane groups by two swaps. Two such tiles (keys
// 4 g + i and 16 + 4 g + i) are, as they lie, the B operand of O^T = V^T P^T over
// 32 keys when slot (g, e) of that product stands for key 16 (e / 4) + 4 g + e % 4:
// the weights never leave their lane. V^T's operand with that key order comes from
// LDS rows of V by the transposing reads.
#pragma once

#include "wl_attn.h"

namespace wl {

__device__ __forceinline__ f32x4 mfma16(u32x4 a, u32x4 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}

// Maximum and sum over the four lanes l, l ^ 16, l ^ 32, l ^ 48.
__device__ __forceinline__ float groups_max(float v) {
    u32x2 r = __builtin_bit_cast(u32x2, __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false));
    v = fmaxf(__uint_as_float(r.x), __uint_as_float(r.y));
    r = __builtin_bit_cast(u32x2, __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false));
    return fmaxf(__uint_as_float(r.x), __uint_as_float(r.y));
}
__device__ __forceinline__ float groups_sum(float v) {
    u32x2 r = __builtin_bit_cast(u32x2, __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false));
    v = __uint_as_float(r.x) + __uint_as_float(r.y);
    r = __builtin_bit_cast(u32x2, __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false));
    return __uint_as_float(r.x) + __uint_as_float(r.y);
}

// Two fp32 as packed bf16.
__device__ __forceinline__ uint32_t pack2(float a, float b) {
    typedef float f32x2 __attribute__((ext_vector_type(2)));
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{a, b}, bf16x2));
}

// Eight one-byte codes as bf16 (every code is exact there).
template <int F>
__device__ __forceinline__ u32x4 widen8(uint32_t lo, uint32_t hi) {
    if (F == kFmtE4m3) {
        auto two = [](uint32_t w, bool up) {
            return up ? __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.0f, true))
                      : __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.0f, false));
        };
        return u32x4{two(lo, false), two(lo, true), two(hi, false), two(hi, true)};
    }
    auto f = [](uint32_t w, int e) { return (float)(int)(int8_t)(w >> (8 * e)); };
    return u32x4{pack2(f(lo, 0), f(lo, 1)), pack2(f(lo, 2), f(lo, 3)), pack2(f(hi, 0), f(hi, 1)), pack2(f(hi, 2), f(hi, 3))};
}

// The same in fp16.
__device__ __forceinline__ f32x4 mfma16_half(u32x4 a, u32x4 b, f32x4 c) {
    typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
}
__device__ __forceinline__ uint32_t pack_half2(float a, float b) {
    typedef float f32x2 __attribute__((ext_vector_type(2)));
    typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{a, b}, f16x2));
}
// Eight e4m3 codes as fp16 (every code is exact there too).
__device__ __forceinline__ u32x4 widen_half8(uint32_t lo, uint32_t hi) {
    return u32x4{__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, 1.0f, false)),
                 __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, 1.0f, true)),
                 __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, 1.0f, false)),
                 __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, 1.0f, true))};
}

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef int i32x2 __attribute__((ext_vector_type(2)));
#define WL_LDS __attribute__((address_space(3)))

// Transposing reads. 16-bit: the 16 lanes of a group address 4 rows x 16 columns,
// lane i row i / 4, columns 4 (i % 4) .. + 3; lane i receives column i's 4 rows.
// 8-bit: 8 rows x 16 columns, lane i row i / 2, columns 8 (i % 2) .. + 7; lane i
// receives column i's 8 rows.
__device__ __forceinline__ u32x2 read_tr16(const void *lds) {
    return __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((WL_LDS s16x4 *)lds));
}
__device__ __forceinline__ u32x2 read_tr8(const void *lds) {
    return __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr8_b64_v2i32((WL_LDS i32x2 *)lds));
}

// Each lane's 16 bytes at base + off (base the same in all lanes) into LDS byte
// lds + 16 * lane. It writes no register, so nothing of it can be overwritten while
// it is on its way; the wave waits with wait_loads before the barrier behind which
// the bytes are read. Through the builtin the compiler takes such a load for one
// that may finish out of order with LDS reads, and then drains every read of an
// operand to 0 instead of counting.
__device__ __forceinline__ void load_to_lds(const char *base, uint32_t off, uint32_t lds) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2" ::"s"(lds), "v"(off), "s"(base) : "memory");
}
// The same with 4 bytes per lane.
__device__ __forceinline__ void load_to_lds4(const char *base, uint32_t off, uint32_t lds) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dword %1, %2" ::"s"(lds), "v"(off), "s"(base) : "memory");
}
// A pointer that is the same in all lanes, in scalar registers.
__device__ __forceinline__ const char *scalar(const char *p) {
    const uint64_t v = (uint64_t)(uintptr_t)p;
    const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)v), hi = __builtin_amdgcn_readfirstlane((uint32_t)(v >> 32));
    return (const char *)(uintptr_t)((uint64_t)hi << 32 | lo);
}
__device__ __forceinline__ void wait_loads() { asm volatile("s_waitcnt vmcnt(0)" ::: "memory"); }
__device__ __forceinline__ uint32_t lds_byte(const void *p) { return (uint32_t)(uintptr_t)(WL_LDS const char *)p; }

// Bits [a, e) of 32.
__device__ __forceinline__ uint32_t bits(int a, int e) {
    a = min(max(a, 0), 32), e = min(max(e, 0), 32);
    return e > a ? (0xFFFFFFFFu >> (32 - (e - a))) << a : 0u;
}

// Which of keys j0 .. j0 + 31 a query sees.
__device__ __forceinline__ uint32_t visible32(const AttnJob &a, const Seq &q, const Sees &v, int j0) {
    uint32_t r = bits(v.lo - j0, v.hi - j0);
    if (!v.tree || j0 + 31 < q.ctx) return r;
    const int64_t b = (int64_t)j0 - q.ctx;
    auto word = [&](int64_t w) { return w < a.tree_words ? v.tree[w] : 0u; };
    uint32_t x;
    if (b < 0)
        x = word(0) << (int)-b;
    else
        x = (word(b >> 5) >> (b & 31)) | ((b & 31) ? word((b >> 5) + 1) << (32 - (b & 31)) : 0u);
    return r | (x & bits(q.ctx - j0 > 0 ? q.ctx - j0 : 0, q.kv - j0));
}

// How the work of a call is divided. A workgroup takes a tile of one sequence's
// query rows, of one key/value head, over all its keys or a piece of them, counted
// from the first key that a row of the tile sees. Pieces are of `chunk` keys, or
// (planned) of a length that the workgroups derive from the lengths of all
// sequences, which only the device knows.
// part: [tile and piece][head][rows][d] unnormalised outputs; ml: the same without
// [d], the reference maximum (power of two) and sum of each row.
struct Split {
    int n_split;      // most pieces of a tile's keys; 1: undivided
    int planned;      // whether the device chooses them
    int chunk;        // keys of a piece, not planned
    int step, least;  // a piece is a multiple of so many keys, and at least so many
    int want, places; // workgroups wanted, workgroups that run at once
    int tiles;        // of rows, most of a sequence
    int tile_rows, rows;   // rows of a tile, rows kept of one (fewer if no sequence has so many)
    int items;        // tiles and pieces at most, over all sequences
    int all_fit;      // whether all workgroups are on the card at once
    float *part;
    float2 *ml;
};

// The kernel's one argument, read from memory again: what only the end of a
// kernel needs would otherwise hold scalar registers all through its loop.
template <class T>
__device__ __forceinline__ T argument_again() {
    auto p = (const __attribute__((address_space(4))) char *)__builtin_amdgcn_kernarg_segment_ptr();
    asm volatile("" : "+s"(p));
    return *(const T *)p;
}

constexpr int kWorkgroups = 512;   // wanted: two per CU

constexpr int kTileRows = 16;     // query rows of a tile of the many-row kernel
constexpr int kF32Rows = 64;      // of the fp32 kernel

void launch_few(const AttnJob &a, int fmt, const Split &sp, hipStream_t s);
void launch_tile(const AttnJob &a, int fmt, const Split &sp, int waves, int tiles, bool exact, hipStream_t s);
void launch_f32(const AttnJob &a, int fmt, const Split &sp, hipStream_t s);

// ---- kernels whose workgroups of four waves take tiles of 64 NT query rows -------

struct TileArgs {
    AttnJob a;
    Split sp;
};

// Which rows and keys a workgroup works on: keys from + 0 .. chunk - 1 behind the
// first that a row sees. s < 0: none. part: place of its partial outputs.
struct Work {
    int s, tile, part, from, chunk;
};

// The lengths that a plan divides: this lane's sequence.
struct Lengths {
    int keys, tiles;   // keys that a tile's rows see at most, tiles of rows
    Seq q;
};
__device__ __forceinline__ Lengths lengths_of(const AttnJob &a, const Split &sp, int lane) {
    Lengths v{0, 0, seq_of(a, min(lane, a.c.n_seq - 1))};
    if (lane >= a.c.n_seq || v.q.rows == 0) return v;
    v.tiles = sp.tiles == 1 ? 1 : (unsigned)(v.q.rows * a.group + sp.tile_rows - 1) / sp.tile_rows;
    v.keys = v.q.kv;
    if (a.mask == kMaskCausal && a.window) v.keys = (int)min((int64_t)v.keys, (int64_t)a.window + v.q.rows + 31);
    return v;
}

constexpr int kMaxSplit = 64;      // most pieces: one lane each in the join
constexpr float kPieceCost = 96;   // of beginning and ending a piece, in keys

// Keys of a piece at up to 64 sequences, a lane each: of 64 lengths, from that which
// gives as many pieces as are wanted to three times that, the one with the least
// time, rounds of workgroups x the time of one. Never shorter than the first, so
// that there are at most want / n_kv + (all tiles) pieces; where 2^29 cuts it short,
// no sequence has more than two.
__device__ __forceinline__ int chunk_of(const AttnJob &a, const Split &sp, const Lengths &v, int lane) {
#pragma clang fp contract(off)
    // The kernels and the join have to come to the same bits: nothing is fused here.
    const float heads = (float)a.c.n_kv;
    const float ideal = wave_sum((float)v.keys * (float)v.tiles) * heads * __builtin_amdgcn_rcpf((float)sp.want) * 1.0001f + 1.0f;
    const float at = ideal * (1.0f + (float)lane * (1.0f / 32));
    const int mine = max(((int)fminf(at, 0x1p29f) & -sp.step) + sp.step, sp.least);
    const float inv = __builtin_amdgcn_rcpf((float)mine);
    float pieces = 0.0f;
    for (int j = 0; j < a.c.n_seq; ++j) {
        const float keys = (float)__builtin_amdgcn_readlane(v.keys, j), tiles = (float)__builtin_amdgcn_readlane(v.tiles, j);
        pieces += tiles * __builtin_ceilf(keys * inv);
    }
    const float cost = __builtin_ceilf(pieces * heads * __builtin_amdgcn_rcpf((float)sp.places) * (1.0f - 0x1p-20f)) * ((float)mine + kPieceCost);
    float best = -cost;
    best = fmaxf(best, dpp<0xB1>(best));    // quad_perm [1,0,3,2]
    best = fmaxf(best, dpp<0x4E>(best));    // quad_perm [2,3,0,1]
    best = fmaxf(best, dpp<0x141>(best));   // row_half_mirror
    best = fmaxf(best, dpp<0x140>(best));   // row_mirror
    best = groups_max(best);
    const uint64_t which = __ballot(best == -cost);
    return __builtin_amdgcn_readlane(mine, which ? __ffsll((unsigned long long)which) - 1 : 0);
}

// Pieces of this lane's sequence: never more than the keys over chunk rounded up
// (the factor makes up for the reciprocal's error), and at least 1 if there are keys.
__device__ __forceinline__ int pieces_of(const Lengths &v, int chunk) {
#pragma clang fp contract(off)
    return (int)fminf(__builtin_ceilf((float)v.keys * __builtin_amdgcn_rcpf((float)chunk) * (1.0f - 0x1p-20f)), kMaxSplit);
}

__device__ __forceinline__ Work find_work(const AttnJob &a, const Split &sp, int i, Seq &q) {
    Work w;
    if (!sp.planned) {
        const int split = i % sp.n_split, u = i / sp.n_split;
        // Under a causal mask later rows have more keys. The longest first, so that the
        // short ones fill in; where all are on the card at once, two on a CU, the
        // second half from the shortest up, so that a long and a short one share a CU.
        const int t = u % sp.tiles, half = (sp.tiles + 1) / 2;
        w.tile = sp.all_fit && t >= half ? t - half : sp.tiles - 1 - t;
        w.s = u / sp.tiles;
        w.part = (w.s * sp.tiles + w.tile) * sp.n_split + split;
        w.chunk = sp.chunk;
        w.from = split * sp.chunk;
        q = seq_of(a, w.s);
        return w;
    }
    const int lane = threadIdx.x & 63;
    const Lengths v = lengths_of(a, sp, lane);
    const int n = pieces_of(v, chunk_of(a, sp, v, lane)), all = n * v.tiles;
    int first = 0;
    w.s = -1;
    for (int j = 0; j < a.c.n_seq; ++j) {
        const int here = __builtin_amdgcn_readlane(all, j);
        if (i < first + here) {
            w.s = j;
            break;
        }
        first += here;
    }
    if (w.s < 0) return w;
    const int pieces = __builtin_amdgcn_readlane(n, w.s), keys = __builtin_amdgcn_readlane(v.keys, w.s);
    const int t = sp.tiles == 1 ? 0 : (unsigned)(i - first) / pieces, split = i - first - t * pieces;
    w.tile = __builtin_amdgcn_readlane(v.tiles, w.s) - 1 - t;
    w.part = first + w.tile * pieces + split;
    w.chunk = (int)((unsigned)(keys + pieces - 1) / pieces + sp.step - 1) & -sp.step;   // all pieces alike
    q = {w.s, __builtin_amdgcn_readlane(v.q.q0, w.s), __builtin_amdgcn_readlane(v.q.rows, w.s), __builtin_amdgcn_readlane(v.q.m, w.s),
         __builtin_amdgcn_readlane(v.q.kv, w.s), __builtin_amdgcn_readlane(v.q.ctx, w.s)};
    w.from = split * w.chunk;
    return w;
}

// Work of the i-th tile and piece of a call, in scalar registers.
__device__ __forceinline__ Work work_of(const AttnJob &a, const Split &sp, int i, Seq &q) {
    const Work w = find_work(a, sp, i, q);
    return {__builtin_amdgcn_readfirstlane(w.s), __builtin_amdgcn_readfirstlane(w.tile), __builtin_amdgcn_readfirstlane(w.part),
            __builtin_amdgcn_readfirstlane(w.from), __builtin_amdgcn_readfirstlane(w.chunk)};
}

// Where the pieces of a tile lie, for the join: n from `first` on.
struct Parts {
    int first, n;
};
__device__ __forceinline__ Parts parts_of(const AttnJob &a, const Split &sp, int s, int tile) {
    if (!sp.planned) return {(s * sp.tiles + tile) * sp.n_split, sp.n_split};
    const int lane = threadIdx.x & 63;
    const Lengths v = lengths_of(a, sp, lane);
    const int n = pieces_of(v, chunk_of(a, sp, v, lane)), all = n * v.tiles;
    int first = 0;
    for (int j = 0; j < s; ++j) first += __builtin_amdgcn_readlane(all, j);
    const int pieces = __builtin_amdgcn_readlane(n, s);
    return {first + tile * pieces, pieces};
}

// Row r of a sequence in the partial outputs.
__device__ __forceinline__ int64_t part_row(const AttnJob &a, const Split &sp, int part, int kvh, int tile, int r) {
    return ((int64_t)part * a.c.n_kv + kvh) * sp.rows + r - tile * sp.tile_rows;
}

// Rows of a wave: `tiles` tiles of 16 from `first` on.
struct WaveRows {
    int first, tiles;
};

// Which of keys j0 .. j0 + 31 this lane's row of the wave's tile t sees. Only
// at the edges of what the wave's rows see, so from the arguments in memory.
template <class R>
__device__ __forceinline__ uint32_t seen(const TileArgs &x, const Work &work, R rows_of, int t, int j0) {
    const Seq q = seq_of(x.a, work.s);
    const int r = rows_of(work.tile, q.rows * x.a.group).first + 16 * t + (threadIdx.x & 15);
    return visible32(x.a, q, sees(x.a, q, r / x.a.group), j0);
}

// Writes a wave's outputs: lane (n, g) holds elements 16 b + 4 g .. + 3 of row n.
template <class E, int F, int DT, int NT, class R>
__device__ __forceinline__ void finish(const TileArgs &x, const Work &work, R rows_of, f32x4 (&o)[NT][DT / 16], float (&m)[NT], float (&l)[NT], int k0, int k1) {
    constexpr int kBlocks = DT / 16;
    const AttnJob &a = x.a;
    const Split &sp = x.sp;
    const int lane = threadIdx.x & 63, n = lane & 15, g = lane >> 4;
    const int kvh = (int)blockIdx.x % a.c.n_kv, tile = work.tile, s = work.s;
    const Seq q = seq_of(a, s);
    const int rows = q.rows * a.group, d = a.c.d;
    const WaveRows mine = rows_of(tile, rows);
    const int r0 = mine.first;
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        if (t >= mine.tiles) break;
        const int r = r0 + 16 * t + n;
        l[t] = groups_sum(l[t]);
        float check = l[t] * 0.0f;
#pragma unroll
        for (int b = 0; b < kBlocks; ++b)
            if (16 * b < d) check += o[t][b].x * 0.0f + o[t][b].y * 0.0f + o[t][b].z * 0.0f + o[t][b].w * 0.0f;
        // A row with an infinity or a NaN is done again key by key: one that it does
        // not see may have got in as 0 * NaN.
        uint64_t odd = __ballot(r < rows && (check != 0.0f || beyond(m[t])));
        odd |= odd >> 32;
        odd |= odd >> 16;
        const uint32_t again = (uint32_t)odd & 0xFFFFu;
        const int64_t part = part_row(a, sp, work.part, kvh, tile, 0);
        auto row_out = [&](int r) {
            const int i = r / a.group;
            return static_cast<E *>(a.o) + (size_t)(q.q0 + i) * a.ldo + (size_t)(kvh * a.group + r - i * a.group) * d;
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
            one_row<E, F>(a, q, ii, kvh * a.group + rr - ii * a.group, k0, k1, acc, mm, ll);
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
    }
}

}  // namespace wl
