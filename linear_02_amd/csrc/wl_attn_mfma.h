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

// How the keys of a call are divided: every sequence and key/value head has
// n_split pieces of `chunk` keys, counted from the first key any of its queries
// sees. part: [unit][n_split][rows][d] unnormalised outputs, ml: the same without
// [d], the reference maximum (power of two) and sum of each row.
struct Split {
    int n_split, chunk, rows;
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
constexpr int kMaxSplit = 64;     // one lane each in the join

constexpr int kTileRows = 32;     // query rows per wave of the many-row kernel
constexpr int kF32Rows = 64;      // of the fp32 kernel

void launch_few(const AttnJob &a, int fmt, const Split &sp, hipStream_t s);
void launch_tile(const AttnJob &a, int fmt, const Split &sp, int waves, hipStream_t s);
void launch_f32(const AttnJob &a, int fmt, const Split &sp, hipStream_t s);

// ---- kernels whose workgroups of four waves take tiles of 64 NT query rows -------

struct TileArgs {
    AttnJob a;
    Split sp;
    int tiles;     // of rows, per sequence and key/value head
    int all_fit;   // whether all workgroups are on the card at once
};

// Which rows and keys a workgroup works on.
struct Work {
    int kvh, split, tile, s;
};
__device__ __forceinline__ Work work_of(const TileArgs &x) {
    Work w;
    int u = blockIdx.x;
    w.kvh = u % x.a.c.n_kv;
    u /= x.a.c.n_kv;
    w.split = u % x.sp.n_split;
    u /= x.sp.n_split;
    // Under a causal mask later rows have more keys. The longest first, so that the
    // short ones fill in; where all are on the card at once, two on a CU, the
    // second half from the shortest up, so that a long and a short one share a CU.
    const int i = u % x.tiles, half = (x.tiles + 1) / 2;
    w.tile = x.all_fit && i >= half ? i - half : x.tiles - 1 - i;
    w.s = u / x.tiles;
    return w;
}

// Which of keys j0 .. j0 + 31 this lane's row of tile `first` (0 or 16) sees. Only
// at the edges of what the wave's rows see, so from the arguments in memory.
template <int NT, int NW>
__device__ __forceinline__ uint32_t seen(const TileArgs &x, int first, int j0) {
    const Work work = work_of(x);
    const Seq q = seq_of(x.a, work.s);
    const int r = (work.tile * NW + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6)) * 16 * NT + first + (threadIdx.x & 15);
    return visible32(x.a, q, sees(x.a, q, r / x.a.group), j0);
}

// Writes a wave's outputs: lane (n, g) holds elements 16 b + 4 g .. + 3 of row n.
template <class E, int F, int DT, int NT, int NW>
__device__ __forceinline__ void finish(const TileArgs &x, f32x4 (&o)[NT][DT / 16], float (&m)[NT], float (&l)[NT], int k0, int k1) {
    constexpr int kBlocks = DT / 16;
    const AttnJob &a = x.a;
    const Split &sp = x.sp;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), n = lane & 15, g = lane >> 4;
    const Work work = work_of(x);
    const int kvh = work.kvh, split = work.split, tile = work.tile, s = work.s;
    const Seq q = seq_of(a, s);
    const int rows = q.rows * a.group, d = a.c.d, r0 = (tile * NW + wave) * 16 * NT;
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        const int r = r0 + 16 * t + n;
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
