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
constexpr int kFewRows = 32;      // most query rows per key/value head of the few-row kernel
constexpr int kMaxSplit = 64;     // one lane each in the join

constexpr int kTileRows = 128;    // query rows per workgroup of the many-row kernel

void launch_few(const AttnJob &a, int fmt, const Split &sp, hipStream_t s);
void launch_tile(const AttnJob &a, int fmt, const Split &sp, hipStream_t s);

}  // namespace wl
