// Host side of the operations between the projections (include/wl.h): argument
// checks and launches of norms with a block's residual, rotary positions, the
// paged cache and attention over it.
#include <hip/hip_runtime.h>

#include <cmath>

#include "wl_abi.h"
#include "wl_checks.h"
#include "wl_layer.h"

using namespace wl::abi;
using wl::fail;
using wl::log_on;
using wl::ok;

static_assert(WL_CACHE_BF16 == wl::kFmtBf16 && WL_CACHE_F32 == wl::kFmtF32 && WL_CACHE_INT8 == wl::kFmtInt8 &&
                  WL_CACHE_E4M3 == wl::kFmtE4m3, "cache formats");
static_assert(WL_ATTN_CAUSAL == wl::kMaskCausal && WL_ATTN_TREE == wl::kMaskTree && WL_ATTN_FULL == wl::kMaskFull,
              "attention masks");

namespace {

wl_status check_cache(const wl_cache *c, int32_t dtype) {
    wl_status st;
    if (!c) return fail(WL_ERR_INVALID_ARG, "cache is NULL");
    if (c->format < WL_CACHE_BF16 || c->format > WL_CACHE_E4M3)
        return fail(WL_ERR_UNSUPPORTED, "cache format=%d is unknown", c->format);
    if ((c->format == WL_CACHE_BF16 && dtype != WL_DTYPE_BF16) || (c->format == WL_CACHE_F32 && dtype != WL_DTYPE_F32))
        return fail(WL_ERR_UNSUPPORTED, "dtype=%d does not go with cache format=%d", dtype, c->format);
    if (c->n_pages < 1 || c->n_kv < 1 || c->n_seq < 1 || c->max_pages < 1)
        return fail(WL_ERR_INVALID_ARG, "cache: n_pages=%d n_kv=%d n_seq=%d max_pages=%d must be >= 1", c->n_pages,
                    c->n_kv, c->n_seq, c->max_pages);
    if (c->page < 16 || c->page > 1024 || (c->page & (c->page - 1)))
        return fail(WL_ERR_INVALID_ARG, "cache: page=%d is not a power of two from 16 to 1024", c->page);
    if (c->d < 16 || c->d % 16) return fail(WL_ERR_INVALID_ARG, "cache: d=%d is not a positive multiple of 16", c->d);
    if (c->d > wl::kMaxHeadDim) return fail(WL_ERR_UNSUPPORTED, "cache: d=%d exceeds %d", c->d, wl::kMaxHeadDim);
    if (c->n_kv > 65535 / 8 || (int64_t)c->n_kv * c->d >= kMaxElems)
        return fail(WL_ERR_UNSUPPORTED, "cache: n_kv=%d is too large", c->n_kv);
    if ((st = need(c->k, 16, "cache k")) != WL_OK || (st = need(c->v, 16, "cache v")) != WL_OK ||
        (st = need(c->table, 4, "cache table")) != WL_OK)
        return st;
    if (c->format >= WL_CACHE_INT8)
        if ((st = need(c->k_scale, 16, "cache k_scale")) != WL_OK || (st = need(c->v_scale, 16, "cache v_scale")) != WL_OK)
            return st;
    return WL_OK;
}

// Bytes of a cache's pools (k, v) and scales.
size_t pool_rows(const wl_cache *c) { return (size_t)c->n_pages * c->n_kv * c->page; }
Named pool(const wl_cache *c, bool v) {
    const size_t e = c->format == WL_CACHE_BF16 ? 2 : c->format == WL_CACHE_F32 ? 4 : 1;
    return {flat(v ? c->v : c->k, pool_rows(c) * c->d * e), v ? "cache v" : "cache k"};
}
Named scales(const wl_cache *c, bool v) {
    return {flat(c->format >= WL_CACHE_INT8 ? (v ? c->v_scale : c->k_scale) : nullptr, pool_rows(c) * 4),
            v ? "cache v_scale" : "cache k_scale"};
}
Named table(const wl_cache *c) { return {flat(c->table, (size_t)c->n_seq * c->max_pages * 4), "cache table"}; }

wl::CacheRef cache_ref(const wl_cache *c) {
    int shift = 0;
    while ((1 << shift) < c->page) ++shift;
    return {c->k, c->v, c->k_scale, c->v_scale, c->table, c->n_pages, shift, c->n_kv, c->d, c->n_seq, c->max_pages};
}

void set_rotary(wl::RowsJob &j, const wl_rotary *r) {
    if (!r) return;
    j.freq = r->freq;
    j.pos = r->pos;
    j.rot = r->rot;
    j.interleaved = r->style == WL_ROPE_INTERLEAVED;
    j.turn_scale = r->scale;
}

// Everything of an attention call but its workspace. T == 0 is accepted.
wl_status check_attention(const wl_attention_args *a, wl::AttnJob *job) {
    wl_status st;
    if (!a) return fail(WL_ERR_INVALID_ARG, "arguments are NULL");
    if ((st = check_dtype(a->dtype)) != WL_OK || (st = check_cache(a->cache, a->dtype)) != WL_OK) return st;
    const wl_cache *c = a->cache;
    if (a->T < 0 || a->max_q < 0 || a->max_kv < 0)
        return fail(WL_ERR_INVALID_ARG, "T=%d, max_q=%d or max_kv=%d is negative", a->T, a->max_q, a->max_kv);
    if (a->max_kv > kMaxKeys) return fail(WL_ERR_UNSUPPORTED, "max_kv=%d exceeds %d", a->max_kv, kMaxKeys);
    if (a->n_q < 1 || a->n_q % c->n_kv)
        return fail(WL_ERR_INVALID_ARG, "n_q=%d is not a positive multiple of n_kv=%d", a->n_q, c->n_kv);
    if (a->mask < WL_ATTN_CAUSAL || a->mask > WL_ATTN_FULL) return fail(WL_ERR_INVALID_ARG, "mask=%d is unknown", a->mask);
    if (a->window < 0 || (a->window && a->mask == WL_ATTN_FULL))
        return fail(WL_ERR_INVALID_ARG, "window=%d is negative, or given with WL_ATTN_FULL", a->window);
    if (a->mask == WL_ATTN_TREE) {
        if (a->tree_words < 1) return fail(WL_ERR_INVALID_ARG, "tree_words=%d must be >= 1", a->tree_words);
        if ((int64_t)a->T * a->tree_words >= kMaxElems) return fail(WL_ERR_INVALID_ARG, "tree has 2^31 or more words");
    }
    if (!std::isfinite(a->scale)) return fail(WL_ERR_INVALID_ARG, "scale is not finite");
    if (a->T == 0) return WL_OK;
    const int64_t width = (int64_t)a->n_q * c->d;
    if ((st = check_rows(a->q, a->T, width, a->ldq, "q")) != WL_OK || (st = check_rows(a->o, a->T, width, a->ldo, "o")) != WL_OK ||
        (st = need(a->q_start, 4, "q_start")) != WL_OK || (st = need(a->kv_len, 4, "kv_len")) != WL_OK)
        return st;
    if (a->mask == WL_ATTN_TREE) {
        if ((st = need(a->tree, 4, "tree")) != WL_OK) return st;
        if (a->q_pos && (st = need(a->q_pos, 4, "q_pos")) != WL_OK) return st;
    }
    const bool tree = a->mask == WL_ATTN_TREE;
    st = check_out(row_set(a->o, a->T, width, a->ldo, a->dtype, "o"),
                   {row_set(a->q, a->T, width, a->ldq, a->dtype, "q"), pool(c, false), pool(c, true), scales(c, false),
                    scales(c, true), table(c), {flat(a->q_start, ((size_t)c->n_seq + 1) * 4), "q_start"},
                    {flat(a->kv_len, (size_t)c->n_seq * 4), "kv_len"},
                    {flat(tree ? a->tree : nullptr, (size_t)a->T * (tree ? a->tree_words : 0) * 4), "tree"},
                    {flat(tree ? a->q_pos : nullptr, (size_t)a->T * 4), "q_pos"}},
                   {a->q});
    if (st != WL_OK) return st;
    wl::AttnJob j{};
    j.c = cache_ref(c);
    j.q = a->q;
    j.o = a->o;
    j.q_start = a->q_start;
    j.kv_len = a->kv_len;
    j.q_pos = a->q_pos;
    j.tree = a->tree;
    j.T = a->T;
    j.n_q = a->n_q;
    j.group = a->n_q / c->n_kv;
    j.ldq = a->ldq;
    j.ldo = a->ldo;
    j.max_q = a->max_q < a->T ? a->max_q : a->T;
    j.max_kv = a->max_kv;
    j.mask = a->mask;
    j.window = a->window;
    j.tree_words = a->tree_words;
    j.scale2 = (float)(a->scale * 1.4426950408889634);   // log2(e)
    const int64_t blocks = wl::attention_workgroups(j, c->format, a->dtype == WL_DTYPE_F32);
    if (blocks > kMaxWorkgroups)
        return fail(WL_ERR_UNSUPPORTED, "n_seq=%d, n_kv=%d and max_q=%d ask for %lld workgroups, more than %lld", c->n_seq, c->n_kv,
                    a->max_q, (long long)blocks, (long long)kMaxWorkgroups);
    *job = j;
    return WL_OK;
}

}  // namespace

extern "C" {

wl_status wl_norm_residual(const wl_norm_args *a, void *hip_stream) {
    wl_status st;
    if (!a) return fail(WL_ERR_INVALID_ARG, "arguments are NULL");
    if ((st = check_dtype(a->dtype)) != WL_OK) return st;
    if (a->T < 0) return fail(WL_ERR_INVALID_ARG, "T=%d is negative", a->T);
    if (a->d < 8 || a->d % 8) return fail(WL_ERR_INVALID_ARG, "d=%d is not a positive multiple of 8", a->d);
    if (a->d > wl::kNormMaxD) return fail(WL_ERR_UNSUPPORTED, "d=%d exceeds %d", a->d, wl::kNormMaxD);
    if (a->T == 0) return ok();
    if (!a->x_out && !a->n_out) return fail(WL_ERR_INVALID_ARG, "x_out and n_out are both NULL");
    const int32_t T = a->T, d = a->d;
    const size_t e = bytes_of(a->dtype);
    if ((st = check_rows(a->x, T, d, d, "x")) != WL_OK) return st;
    if (a->y && (st = check_rows(a->y, T, d, d, "y")) != WL_OK) return st;
    if (a->x_out && (st = check_rows(a->x_out, T, d, d, "x_out")) != WL_OK) return st;
    if (a->n_out && (st = check_rows(a->n_out, T, d, d, "n_out")) != WL_OK) return st;
    if (a->post && (st = need(a->post, 16, "post")) != WL_OK) return st;
    if (a->pre && (st = need(a->pre, 16, "pre")) != WL_OK) return st;
    if (a->gate) {
        if ((st = need(a->gate, 16, "gate")) != WL_OK) return st;
        if (a->gate_ld && (st = check_rows(a->gate, T, d, a->gate_ld, "gate")) != WL_OK) return st;
    }
    const Named x = row_set(a->x, T, d, d, a->dtype, "x"), y = row_set(a->y, T, d, d, a->dtype, "y");
    const Named gate = !a->gate ? Named{flat(nullptr, 0), "gate"}
                       : a->gate_ld ? row_set(a->gate, T, d, a->gate_ld, a->dtype, "gate")
                                    : Named{flat(a->gate, d * e), "gate"};
    const Named post{flat(a->post, d * e), "post"}, pre{flat(a->pre, d * e), "pre"};
    const Named xo = row_set(a->x_out, T, d, d, a->dtype, "x_out"), no = row_set(a->n_out, T, d, d, a->dtype, "n_out");
    if (a->x_out && (st = check_out(xo, {x, y, gate, post, pre}, {a->x, a->y})) != WL_OK) return st;
    if (a->n_out && (st = check_out(no, {x, y, gate, post, pre}, {a->x, a->y})) != WL_OK) return st;
    if (a->x_out && a->n_out && (st = check_out(no, {xo})) != WL_OK) return st;
    wl::NormJob j{a->x, a->y, a->post, a->pre, a->gate, a->x_out, a->n_out, T, d, a->gate_ld,
                  a->eps, a->offset, a->res_scale, a->branch_scale};
    return launched(wl::launch_norm(j, a->dtype == WL_DTYPE_F32, static_cast<hipStream_t>(hip_stream)), "norm");
}

wl_status wl_rope_frequencies(int32_t rot, double base, int32_t scaling, double factor, double original, double slow,
                              double fast, double *freq, float *scale) {
    if (!freq || !scale) return fail(WL_ERR_INVALID_ARG, "freq or scale is NULL");
    if (rot < 8 || rot % 8 || rot > wl::kMaxHeadDim)
        return fail(WL_ERR_INVALID_ARG, "rot=%d must be a multiple of 8 from 8 to %d", rot, wl::kMaxHeadDim);
    if (!(base > 1.0) || !std::isfinite(base)) return fail(WL_ERR_INVALID_ARG, "base must be finite and above 1");
    if (scaling < WL_ROPE_PLAIN || scaling > WL_ROPE_PARTS) return fail(WL_ERR_INVALID_ARG, "scaling=%d is unknown", scaling);
    if (scaling != WL_ROPE_PLAIN && (!(factor >= 1.0) || !std::isfinite(factor)))
        return fail(WL_ERR_INVALID_ARG, "factor must be finite and at least 1");
    if (scaling == WL_ROPE_PARTS && !(original > 0.0 && fast > slow && std::isfinite(original) && std::isfinite(fast) && std::isfinite(slow)))
        return fail(WL_ERR_INVALID_ARG, "original must be positive and fast above slow, all finite");
    if (scaling == WL_ROPE_BASE) base *= std::pow(factor, (double)rot / (rot - 2));
    *scale = scaling == WL_ROPE_PARTS ? (float)(0.1 * std::log(factor) + 1.0) : 1.0f;
    for (int e = 0; e < rot / 2; ++e) {
        double f = std::pow(base, -2.0 * e / rot);
        if (scaling == WL_ROPE_LINEAR) f /= factor;
        if (scaling == WL_ROPE_PARTS) {
            const double g = (original * f / 6.283185307179586 - slow) / (fast - slow);
            const double kept = g < 0.0 ? 0.0 : g > 1.0 ? 1.0 : g;
            f = f * kept + f / factor * (1.0 - kept);
        }
        freq[e] = f;
    }
    return ok();
}

wl_status wl_rope(const wl_rope_args *a, void *hip_stream) {
    wl_status st;
    if (!a) return fail(WL_ERR_INVALID_ARG, "arguments are NULL");
    if ((st = check_dtype(a->dtype)) != WL_OK) return st;
    if (a->T < 0) return fail(WL_ERR_INVALID_ARG, "T=%d is negative", a->T);
    if (a->n_q < 0 || a->n_k < 0 || a->n_q + (int64_t)a->n_k < 1 || a->n_q + (int64_t)a->n_k > (1 << 20))
        return fail(WL_ERR_INVALID_ARG, "n_q=%d or n_k=%d is out of range", a->n_q, a->n_k);
    if (a->d < 8 || a->d % 8) return fail(WL_ERR_INVALID_ARG, "d=%d is not a positive multiple of 8", a->d);
    if (a->d > wl::kMaxHeadDim) return fail(WL_ERR_UNSUPPORTED, "d=%d exceeds %d", a->d, wl::kMaxHeadDim);
    if (a->T == 0) return ok();
    if ((st = check_rotary(a->rotary, a->d, true)) != WL_OK) return st;
    const int32_t T = a->T;
    const int64_t wq = (int64_t)a->n_q * a->d, wk = (int64_t)a->n_k * a->d;
    const size_t e = bytes_of(a->dtype);
    if (a->n_q && ((st = check_rows(a->q, T, wq, a->ldq, "q")) != WL_OK || (st = check_rows(a->q_out, T, wq, a->ldq_out, "q_out")) != WL_OK))
        return st;
    if (a->n_k && ((st = check_rows(a->k, T, wk, a->ldk, "k")) != WL_OK || (st = check_rows(a->k_out, T, wk, a->ldk_out, "k_out")) != WL_OK))
        return st;
    if (a->n_q && a->q_weight && (st = need(a->q_weight, 16, "q_weight")) != WL_OK) return st;
    if (a->n_k && a->k_weight && (st = need(a->k_weight, 16, "k_weight")) != WL_OK) return st;
    const wl_rotary *r = a->rotary;
    const Named none{flat(nullptr, 0), ""};
    const Named q = a->n_q ? row_set(a->q, T, wq, a->ldq, a->dtype, "q") : none;
    const Named k = a->n_k ? row_set(a->k, T, wk, a->ldk, a->dtype, "k") : none;
    const Named qw{flat(a->n_q ? a->q_weight : nullptr, a->d * e), "q_weight"}, kw{flat(a->n_k ? a->k_weight : nullptr, a->d * e), "k_weight"};
    const Named fr{flat(r ? r->freq : nullptr, r ? (size_t)r->rot * 4 : 0), "freq"}, ps{flat(r ? r->pos : nullptr, (size_t)T * 4), "pos"};
    const Named qo = row_set(a->q_out, T, wq, a->ldq_out, a->dtype, "q_out"), ko = row_set(a->k_out, T, wk, a->ldk_out, a->dtype, "k_out");
    if (a->n_q && (st = check_out(qo, {q, k, qw, kw, fr, ps}, {a->q})) != WL_OK) return st;
    if (a->n_k && (st = check_out(ko, {k, q, qw, kw, fr, ps}, {a->k})) != WL_OK) return st;
    if (a->n_q && a->n_k && (st = check_out(ko, {qo})) != WL_OK) return st;
    wl::RowsJob j{};
    j.q = a->q, j.k = a->k, j.q_out = a->q_out, j.k_out = a->k_out;
    j.q_weight = a->n_q ? a->q_weight : nullptr, j.k_weight = a->n_k ? a->k_weight : nullptr;
    j.T = T, j.n_q = a->n_q, j.n_k = a->n_k, j.d = a->d;
    j.ldq = a->ldq, j.ldk = a->ldk, j.ldq_out = a->ldq_out, j.ldk_out = a->ldk_out;
    j.eps = a->eps, j.offset = a->offset;
    set_rotary(j, r);
    return launched(wl::launch_rows(j, wl::kFmtNone, a->dtype == WL_DTYPE_F32, static_cast<hipStream_t>(hip_stream)), "rope");
}

wl_status wl_cache_write(const wl_cache_write_args *a, void *hip_stream) {
    wl_status st;
    if (!a) return fail(WL_ERR_INVALID_ARG, "arguments are NULL");
    if ((st = check_dtype(a->dtype)) != WL_OK || (st = check_cache(a->cache, a->dtype)) != WL_OK) return st;
    if (a->T < 0) return fail(WL_ERR_INVALID_ARG, "T=%d is negative", a->T);
    if (a->n_q < 0 || a->n_q > (1 << 20)) return fail(WL_ERR_INVALID_ARG, "n_q=%d is out of range", a->n_q);
    if (a->T == 0) return ok();
    const wl_cache *c = a->cache;
    const int32_t T = a->T;
    const int64_t wq = (int64_t)a->n_q * c->d, wk = (int64_t)c->n_kv * c->d;
    const size_t e = bytes_of(a->dtype);
    const wl_rotary *r = a->rotary;
    if ((st = check_rotary(r, c->d, false)) != WL_OK) return st;
    if ((st = check_rows(a->k, T, wk, a->ldk, "k")) != WL_OK || (st = check_rows(a->v, T, wk, a->ldv, "v")) != WL_OK ||
        (st = need(a->seq, 4, "seq")) != WL_OK || (st = need(a->slot, 4, "slot")) != WL_OK)
        return st;
    if (a->n_q && ((st = check_rows(a->q, T, wq, a->ldq, "q")) != WL_OK || (st = check_rows(a->q_out, T, wq, a->ldq_out, "q_out")) != WL_OK))
        return st;
    if (a->n_q && a->q_weight && (st = need(a->q_weight, 16, "q_weight")) != WL_OK) return st;
    if (a->k_weight && (st = need(a->k_weight, 16, "k_weight")) != WL_OK) return st;
    const Named none{flat(nullptr, 0), ""};
    const Named q = a->n_q ? row_set(a->q, T, wq, a->ldq, a->dtype, "q") : none;
    const Named k = row_set(a->k, T, wk, a->ldk, a->dtype, "k"), v = row_set(a->v, T, wk, a->ldv, a->dtype, "v");
    const Named qw{flat(a->n_q ? a->q_weight : nullptr, c->d * e), "q_weight"}, kw{flat(a->k_weight, c->d * e), "k_weight"};
    const Named fr{flat(r ? r->freq : nullptr, r ? (size_t)r->rot * 4 : 0), "freq"}, ps{flat(r ? r->pos : nullptr, (size_t)T * 4), "pos"};
    const Named sq{flat(a->seq, (size_t)T * 4), "seq"}, sl{flat(a->slot, (size_t)T * 4), "slot"};
    const Named qo = a->n_q ? row_set(a->q_out, T, wq, a->ldq_out, a->dtype, "q_out") : none;
    if (a->n_q && (st = check_out(qo, {q, k, v, qw, kw, fr, ps, sq, sl, table(c)}, {a->q})) != WL_OK) return st;
    const Named outs[4] = {pool(c, false), pool(c, true), scales(c, false), scales(c, true)};
    for (int i = 0; i < 4; ++i) {
        if (!outs[i].r.p) continue;
        if ((st = check_out(outs[i], {q, k, v, qw, kw, fr, ps, sq, sl, table(c), qo})) != WL_OK) return st;
        for (int l = 0; l < i; ++l)
            if (outs[l].r.p && (st = check_out(outs[i], {outs[l]})) != WL_OK) return st;
    }
    wl::RowsJob j{};
    j.q = a->q, j.k = a->k, j.v = a->v, j.q_out = a->q_out;
    j.q_weight = a->n_q ? a->q_weight : nullptr, j.k_weight = a->k_weight;
    j.seq = a->seq, j.slot = a->slot;
    j.c = cache_ref(c);
    j.T = T, j.n_q = a->n_q, j.n_k = c->n_kv, j.n_v = c->n_kv, j.d = c->d;
    j.ldq = a->ldq, j.ldk = a->ldk, j.ldv = a->ldv, j.ldq_out = a->ldq_out;
    j.eps = a->eps, j.offset = a->offset;
    set_rotary(j, r);
    return launched(wl::launch_rows(j, c->format, a->dtype == WL_DTYPE_F32, static_cast<hipStream_t>(hip_stream)), "cache write");
}

wl_status wl_cache_read(const wl_cache_read_args *a, void *hip_stream) {
    wl_status st;
    if (!a) return fail(WL_ERR_INVALID_ARG, "arguments are NULL");
    if ((st = check_dtype(a->dtype)) != WL_OK || (st = check_cache(a->cache, a->dtype)) != WL_OK) return st;
    if (a->T < 0) return fail(WL_ERR_INVALID_ARG, "T=%d is negative", a->T);
    if (a->T == 0) return ok();
    if (!a->k_out && !a->v_out) return fail(WL_ERR_INVALID_ARG, "k_out and v_out are both NULL");
    const wl_cache *c = a->cache;
    const int32_t T = a->T;
    const int64_t w = (int64_t)c->n_kv * c->d;
    if ((st = need(a->seq, 4, "seq")) != WL_OK || (st = need(a->slot, 4, "slot")) != WL_OK) return st;
    if (a->k_out && (st = check_rows(a->k_out, T, w, a->ldk, "k_out")) != WL_OK) return st;
    if (a->v_out && (st = check_rows(a->v_out, T, w, a->ldv, "v_out")) != WL_OK) return st;
    const Named sq{flat(a->seq, (size_t)T * 4), "seq"}, sl{flat(a->slot, (size_t)T * 4), "slot"};
    const Named ko = row_set(a->k_out, T, w, a->ldk, a->dtype, "k_out"), vo = row_set(a->v_out, T, w, a->ldv, a->dtype, "v_out");
    for (const Named *o : {&ko, &vo})
        if (o->r.p && (st = check_out(*o, {pool(c, false), pool(c, true), scales(c, false), scales(c, true), table(c), sq, sl})) != WL_OK)
            return st;
    if (a->k_out && a->v_out && (st = check_out(vo, {ko})) != WL_OK) return st;
    wl::ReadJob j{};
    j.seq = a->seq, j.slot = a->slot;
    j.c = cache_ref(c);
    j.k_out = a->k_out, j.v_out = a->v_out;
    j.T = T, j.ldk = a->ldk, j.ldv = a->ldv;
    return launched(wl::launch_cache_read(j, c->format, a->dtype == WL_DTYPE_F32, static_cast<hipStream_t>(hip_stream)), "cache read");
}

size_t wl_attention_workspace_bytes(const wl_attention_args *a) {
    wl::AttnJob j{};
    if (check_attention(a, &j) != WL_OK || a->T == 0) return 0;
    const size_t b = wl::attention_scratch(j, a->cache->format, a->dtype == WL_DTYPE_F32);
    return b ? WL_SYNC_BYTES + round_up(b, kAlign) : 0;
}

wl_status wl_attention(const wl_attention_args *a, void *ws, size_t ws_bytes, void *hip_stream) {
    wl::AttnJob j{};
    wl_status st = check_attention(a, &j);
    if (st != WL_OK) return st;
    if (a->T == 0 || j.max_q == 0) return ok();
    const wl_cache *c = a->cache;
    const bool f32 = a->dtype == WL_DTYPE_F32;
    const size_t scratch = wl::attention_scratch(j, c->format, f32);
    char *at = nullptr;
    if (scratch) {
        const size_t want = WL_SYNC_BYTES + round_up(scratch, kAlign);
        if (!ws) return fail(WL_ERR_WORKSPACE, "no workspace, %zu bytes needed", want);
        if (!aligned(ws, kAlign)) return fail(WL_ERR_INVALID_ARG, "the workspace is not 256-byte aligned");
        if (ws_bytes < want) return fail(WL_ERR_WORKSPACE, "workspace of %zu bytes, %zu needed", ws_bytes, want);
        at = static_cast<char *>(ws) + WL_SYNC_BYTES;
        const int64_t width = (int64_t)a->n_q * c->d;
        const bool tree = a->mask == WL_ATTN_TREE;
        st = check_out({flat(at, scratch), "workspace"},
                       {row_set(a->q, a->T, width, a->ldq, a->dtype, "q"), row_set(a->o, a->T, width, a->ldo, a->dtype, "o"),
                        pool(c, false), pool(c, true), scales(c, false), scales(c, true), table(c),
                        {flat(a->q_start, ((size_t)c->n_seq + 1) * 4), "q_start"}, {flat(a->kv_len, (size_t)c->n_seq * 4), "kv_len"},
                        {flat(tree ? a->tree : nullptr, (size_t)a->T * (tree ? a->tree_words : 0) * 4), "tree"},
                        {flat(tree ? a->q_pos : nullptr, (size_t)a->T * 4), "q_pos"}});
        if (st != WL_OK) return st;
    }
    return launched(wl::launch_attention(j, c->format, f32, at, static_cast<hipStream_t>(hip_stream)), "attention");
}

}  // extern "C"
