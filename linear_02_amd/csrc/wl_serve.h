// Jobs and launchers of the operations around a serving batch: its plan, the
// latent cache with its attention, the verification of drafted tokens.
#pragma once

#include "wl_layer.h"

namespace wl {

// ---- the batch's rows and pages (k_plan.hip) ---------------------------------
struct PlanJob {
    int32_t *table, *held, *free_pages, *n_free;
    const int32_t *past, *n_new;
    int32_t *q_start, *kv_len, *seq, *slot;
    int T, n_seq, max_pages, n_pages, page_shift;
};
// Bytes of scratch; 0: one launch without.
size_t plan_scratch(const PlanJob &a);
hipError_t launch_plan(const PlanJob &a, void *ws, hipStream_t stream);

// ---- drafted tokens (k_verify.hip) ---------------------------------------------
constexpr int kVerifyRows = 1024;    // most rows of a sequence
constexpr int kVerifyChunks = 64;    // most chunks of a row: a lane each

struct VerifyJob {
    const void *target, *draft;
    const int32_t *token, *q_start, *parent;
    const float2 *u;
    const float *temperature;
    int32_t *out, *path, *n_out, *len;
    int T, n_seq, vocab, ld_target, ld_draft, max_q, logits;
    int chunks, groups;   // of a row; 16-byte groups of a chunk: set by the launch
};
int64_t verify_workgroups(const VerifyJob &a, bool f32);
size_t verify_scratch(const VerifyJob &a, bool f32);
hipError_t launch_verify(VerifyJob a, bool f32, void *ws, hipStream_t stream);
// Of a batch without rows: n_out of its sequences.
hipError_t launch_verify_no_rows(const VerifyJob &a, hipStream_t stream);

// ---- the latent cache (k_latent_rows.hip) ----------------------------------------
constexpr int kMaxLatent = 512, kMaxRot = 64;

struct LatentRef {
    void *rows;
    float *scale;
    const int32_t *table;
    int n_pages, page_shift, latent, rot, n_seq, max_pages;
};

struct LatentWriteJob {
    LatentRef c;
    const void *in, *norm, *q;
    void *q_out;
    const double *freq;   // NULL: no rotation
    const int32_t *pos, *seq, *slot;
    int T, n_q, nope, ldc, ldq, ldq_out, interleaved;
    int parts;            // workgroups per token, set by the launch
    float turn_scale, eps, offset;
};
hipError_t launch_latent_write(LatentWriteJob a, int fmt, hipStream_t stream);

struct LatentReadJob {
    LatentRef c;
    const int32_t *seq, *slot;
    void *out;
    int T, ld;
};
hipError_t launch_latent_read(const LatentReadJob &a, int fmt, hipStream_t stream);

// ---- attention over it (k_latent.hip) ---------------------------------------------
enum : int { kFormAuto = 0, kFormAbsorbed = 1, kFormExpanded = 2 };

// a: the attention of latent queries, one key/value head of c.d = latent whose rows
// go on with the key's `rot` elements (c.k = c.v = the pool, c.k_scale its scales);
// q and o are set by the launch where there are weights.
struct LatentJob {
    AttnJob a;
    const void *q, *w;    // w NULL: q and o are latent
    void *o;
    int rot, nope, value, ldq, ldo;
    float scale;
};
// What the launch does, and what of it is to be checked on the host.
struct LatentNeeds {
    size_t scratch;       // bytes
    int64_t workgroups;   // of the largest launch
};
bool latent_can_expand(const LatentJob &a, int fmt);
LatentNeeds latent_needs(const LatentJob &a, int fmt, bool f32, int form);
hipError_t launch_latent(const LatentJob &a, int fmt, bool f32, int form, void *ws, hipStream_t stream);

}  // namespace wl
