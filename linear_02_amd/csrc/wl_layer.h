// Jobs and launchers of the operations between the projections: norms with a
// block's residual, rotary positions, the paged cache, attention over it.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace wl {

// Results larger than this are stored past the caches (twice the L2 of one XCD):
// they would push out what the call still reads.
constexpr size_t kStreamBytes = (size_t)8 << 20;

// ---- norms (k_norm.hip) -----------------------------------------------------
constexpr int kNormMaxD = 32768;

struct NormJob {
    const void *x, *y, *post, *pre, *gate;
    void *x_out, *n_out;
    int T, d, gate_ld;
    float eps, offset, res_scale, branch_scale;
};
hipError_t launch_norm(const NormJob &a, bool f32, hipStream_t stream);

// ---- rows of heads: rotation, cache write and read (k_rows.hip) ---------------
constexpr int kMaxHeadDim = 256;

// Cache element formats as in the C ABI; kFmtNone: rotation only.
enum : int { kFmtNone = -1, kFmtBf16 = 0, kFmtF32 = 1, kFmtInt8 = 2, kFmtE4m3 = 3 };

struct CacheRef {
    void *k, *v;
    float *k_scale, *v_scale;
    const int32_t *table;
    int n_pages, page_shift, n_kv, d, n_seq, max_pages;
};

struct RowsJob {
    const void *q, *k, *v, *q_weight, *k_weight;
    void *q_out, *k_out;   // k_out: rotation only
    const double *freq;    // NULL: no rotation
    const int32_t *pos;    // NULL: the slots
    const int32_t *seq, *slot;
    CacheRef c;
    int T, n_q, n_k, n_v, d, ldq, ldk, ldv, ldq_out, ldk_out;
    int rot, interleaved;
    int waves;   // per token, set by the launch
    float turn_scale, eps, offset;
};
hipError_t launch_rows(RowsJob a, int fmt, bool f32, hipStream_t stream);

struct ReadJob {
    const int32_t *seq, *slot;
    CacheRef c;
    void *k_out, *v_out;
    int T, ldk, ldv;
    int waves;   // per token, set by the launch
};
hipError_t launch_cache_read(ReadJob a, int fmt, bool f32, hipStream_t stream);

// ---- attention (k_attn.hip) ----------------------------------------------------
enum : int { kMaskCausal = 0, kMaskTree = 1, kMaskFull = 2 };

struct AttnJob {
    CacheRef c;
    const void *q;
    void *o;
    const int32_t *q_start, *kv_len, *q_pos;
    const uint32_t *tree;
    int T, n_q, group, ldq, ldo, max_q, max_kv, mask, window, tree_words;
    float scale2;   // scale * log2(e): scores are kept as powers of two
};
hipError_t launch_attention(const AttnJob &a, int fmt, bool f32, void *ws, hipStream_t stream);
int64_t attention_workgroups(const AttnJob &a, int fmt, bool f32);
// Bytes of scratch the launch needs.
size_t attention_scratch(const AttnJob &a, int fmt, bool f32);

}  // namespace wl
