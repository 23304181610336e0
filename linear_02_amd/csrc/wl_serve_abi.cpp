// Host side of the operations around a serving batch (include/wl.h): argument checks
// and launches of the batch's plan, the latent cache with its attention, and the
// verification of drafted tokens.
#include <hip/hip_runtime.h>

#include <cmath>

#include "wl_abi.h"
#include "wl_checks.h"
#include "wl_serve.h"

using namespace wl::abi;
using wl::fail;
using wl::ok;

static_assert(WL_LATENT_AUTO == wl::kFormAuto && WL_LATENT_ABSORBED == wl::kFormAbsorbed && WL_LATENT_EXPANDED == wl::kFormExpanded,
              "forms of latent attention");

namespace {

Named array(const void *p, size_t n, const char *name) { return {flat(p, n * 4), name}; }

int shift_of(int32_t page) {
    int shift = 0;
    while ((1 << shift) < page) ++shift;
    return shift;
}

wl_status check_page(int32_t page) {
    if (page < 16 || page > 1024 || (page & (page - 1)))
        return fail(WL_ERR_INVALID_ARG, "page=%d is not a power of two from 16 to 1024", page);
    return WL_OK;
}

// Scratch behind the sync area of a workspace.
size_t ws_of(size_t scratch) { return scratch ? WL_SYNC_BYTES + round_up(scratch, kAlign) : 0; }

wl_status check_scratch(void *ws, size_t ws_bytes, size_t scratch, void **at) {
    *at = nullptr;
    if (!scratch) return WL_OK;
    const size_t want = ws_of(scratch);
    if (!ws) return fail(WL_ERR_WORKSPACE, "no workspace, %zu bytes needed", want);
    if (!aligned(ws, kAlign)) return fail(WL_ERR_INVALID_ARG, "the workspace is not 256-byte aligned");
    if (ws_bytes < want) return fail(WL_ERR_WORKSPACE, "workspace of %zu bytes, %zu needed", ws_bytes, want);
    *at = static_cast<char *>(ws) + WL_SYNC_BYTES;
    return WL_OK;
}

// ---- the batch's plan ---------------------------------------------------------

constexpr int32_t kMaxPlanned = 1 << 16;

wl_status check_plan(const wl_batch_plan_args *a, wl::PlanJob *job, void *scratch, size_t bytes) {
    wl_status st;
    if (!a) return fail(WL_ERR_INVALID_ARG, "arguments are NULL");
    if (a->T < 0) return fail(WL_ERR_INVALID_ARG, "T=%d is negative", a->T);
    if (a->T > kMaxTokens) return fail(WL_ERR_UNSUPPORTED, "T=%d exceeds %d", a->T, kMaxTokens);
    if (a->n_seq < 1 || a->max_pages < 1 || a->n_pages < 1)
        return fail(WL_ERR_INVALID_ARG, "n_seq=%d max_pages=%d n_pages=%d must be >= 1", a->n_seq, a->max_pages, a->n_pages);
    if (a->n_seq > kMaxPlanned) return fail(WL_ERR_UNSUPPORTED, "n_seq=%d exceeds %d", a->n_seq, kMaxPlanned);
    if ((st = check_page(a->page)) != WL_OK) return st;
    if ((int64_t)a->n_seq * a->max_pages >= kMaxElems) return fail(WL_ERR_INVALID_ARG, "table has 2^31 or more entries");
    if ((int64_t)a->max_pages * a->page > kMaxKeys)
        return fail(WL_ERR_UNSUPPORTED, "max_pages=%d of %d hold more than %d keys", a->max_pages, a->page, kMaxKeys);
    const size_t n = a->n_seq;
    const Named outs[] = {array(a->table, n * a->max_pages, "table"), array(a->held, n, "held"),
                          array(a->free_pages, a->n_pages, "free_pages"), array(a->n_free, 1, "n_free"),
                          array(a->q_start, n + 1, "q_start"), array(a->kv_len, n, "kv_len"),
                          array(a->T ? a->seq : nullptr, a->T, "seq"), array(a->T ? a->slot : nullptr, a->T, "slot"),
                          {flat(scratch, bytes), "workspace"}};
    const Named past = array(a->past, n, "past"), fresh = array(a->n_new, n, "n_new");
    for (int i = 0; i < 8; ++i)
        if (i < 6 || a->T)
            if ((st = need(outs[i].r.p, 4, outs[i].name)) != WL_OK) return st;
    if ((st = need(a->past, 4, "past")) != WL_OK || (st = need(a->n_new, 4, "n_new")) != WL_OK) return st;
    for (int i = 0; i < 9; ++i) {
        if (!outs[i].r.p) continue;
        if ((st = check_out(outs[i], {past, fresh})) != WL_OK) return st;
        for (int l = 0; l < i; ++l)
            if (outs[l].r.p && (st = check_out(outs[i], {outs[l]})) != WL_OK) return st;
    }
    *job = {a->table, a->held, a->free_pages, a->n_free, a->past, a->n_new, a->q_start, a->kv_len, a->seq, a->slot,
            a->T, a->n_seq, a->max_pages, a->n_pages, shift_of(a->page)};
    return WL_OK;
}

// ---- the latent cache -----------------------------------------------------------

wl_status check_latent_cache(const wl_latent_cache *c, int32_t dtype) {
    wl_status st;
    if (!c) return fail(WL_ERR_INVALID_ARG, "cache is NULL");
    if (c->format != WL_CACHE_BF16 && c->format != WL_CACHE_F32 && c->format != WL_CACHE_E4M3)
        return fail(WL_ERR_UNSUPPORTED, "cache format=%d is none of a latent cache", c->format);
    if ((c->format == WL_CACHE_F32) != (dtype == WL_DTYPE_F32))
        return fail(WL_ERR_UNSUPPORTED, "dtype=%d does not go with cache format=%d", dtype, c->format);
    if (c->n_pages < 1 || c->n_seq < 1 || c->max_pages < 1)
        return fail(WL_ERR_INVALID_ARG, "cache: n_pages=%d n_seq=%d max_pages=%d must be >= 1", c->n_pages, c->n_seq, c->max_pages);
    if ((st = check_page(c->page)) != WL_OK) return st;
    if (c->latent < 1 || c->rot < 1) return fail(WL_ERR_INVALID_ARG, "cache: latent=%d and rot=%d must be positive", c->latent, c->rot);
    if (c->latent != 128 && c->latent != 256 && c->latent != 512)
        return fail(WL_ERR_UNSUPPORTED, "cache: latent=%d is none of 128, 256, 512", c->latent);
    if (c->rot != 32 && c->rot != 64) return fail(WL_ERR_UNSUPPORTED, "cache: rot=%d is neither 32 nor 64", c->rot);
    if ((st = need(c->rows, 16, "cache rows")) != WL_OK || (st = need(c->table, 4, "cache table")) != WL_OK) return st;
    if (c->format == WL_CACHE_E4M3 && (st = need(c->scale, 16, "cache scale")) != WL_OK) return st;
    return WL_OK;
}

size_t pool_rows(const wl_latent_cache *c) { return (size_t)c->n_pages * c->page; }
Named pool(const wl_latent_cache *c) {
    const size_t row = c->format == WL_CACHE_E4M3 ? (size_t)c->latent + 2 * c->rot
                                                  : (size_t)(c->latent + c->rot) * (c->format == WL_CACHE_F32 ? 4 : 2);
    return {flat(c->rows, pool_rows(c) * row), "cache rows"};
}
Named scales(const wl_latent_cache *c) {
    return {flat(c->format == WL_CACHE_E4M3 ? c->scale : nullptr, pool_rows(c) * 4), "cache scale"};
}
Named table(const wl_latent_cache *c) { return array(c->table, (size_t)c->n_seq * c->max_pages, "cache table"); }

wl::LatentRef latent_ref(const wl_latent_cache *c) {
    return {c->rows, c->scale, c->table, c->n_pages, shift_of(c->page), c->latent, c->rot, c->n_seq, c->max_pages};
}

wl_status check_heads(int32_t nope) {
    if (nope < 0 || nope % 8 || nope > 256) return fail(WL_ERR_INVALID_ARG, "nope=%d is not a multiple of 8 from 0 to 256", nope);
    return WL_OK;
}

constexpr int32_t kMaxHeads = 1 << 12;

// Everything of an attention call but its workspace. T == 0 is accepted.
wl_status check_latent_attention(const wl_latent_attention_args *a, wl::LatentJob *job, int *form) {
    wl_status st;
    if (!a) return fail(WL_ERR_INVALID_ARG, "arguments are NULL");
    if ((st = check_dtype(a->dtype)) != WL_OK || (st = check_latent_cache(a->cache, a->dtype)) != WL_OK) return st;
    const wl_latent_cache *c = a->cache;
    if (a->T < 0 || a->max_q < 0 || a->max_kv < 0)
        return fail(WL_ERR_INVALID_ARG, "T=%d, max_q=%d or max_kv=%d is negative", a->T, a->max_q, a->max_kv);
    if (a->max_kv > kMaxKeys) return fail(WL_ERR_UNSUPPORTED, "max_kv=%d exceeds %d", a->max_kv, kMaxKeys);
    if (a->n_q < 1) return fail(WL_ERR_INVALID_ARG, "n_q=%d must be >= 1", a->n_q);
    if (a->n_q > kMaxHeads) return fail(WL_ERR_UNSUPPORTED, "n_q=%d exceeds %d", a->n_q, kMaxHeads);
    if (a->w) {
        if (a->nope < 32 || a->nope % 32 || a->value < 32 || a->value % 32)
            return fail(WL_ERR_INVALID_ARG, "nope=%d and value=%d must be positive multiples of 32", a->nope, a->value);
        if (a->nope > 256 || a->value > 256) return fail(WL_ERR_UNSUPPORTED, "nope=%d or value=%d exceeds 256", a->nope, a->value);
    } else if (a->nope != c->latent || a->value != c->latent) {
        return fail(WL_ERR_INVALID_ARG, "without w, nope=%d and value=%d must be latent=%d", a->nope, a->value, c->latent);
    }
    if (a->mask < WL_ATTN_CAUSAL || a->mask > WL_ATTN_FULL) return fail(WL_ERR_INVALID_ARG, "mask=%d is unknown", a->mask);
    if (a->window < 0 || (a->window && a->mask == WL_ATTN_FULL))
        return fail(WL_ERR_INVALID_ARG, "window=%d is negative, or given with WL_ATTN_FULL", a->window);
    if (a->mask == WL_ATTN_TREE) {
        if (a->tree_words < 1) return fail(WL_ERR_INVALID_ARG, "tree_words=%d must be >= 1", a->tree_words);
        if ((int64_t)a->T * a->tree_words >= kMaxElems) return fail(WL_ERR_INVALID_ARG, "tree has 2^31 or more words");
    }
    if (a->form < WL_LATENT_AUTO || a->form > WL_LATENT_EXPANDED) return fail(WL_ERR_INVALID_ARG, "form=%d is unknown", a->form);
    if (!std::isfinite(a->scale)) return fail(WL_ERR_INVALID_ARG, "scale is not finite");
    wl::LatentJob j{};
    j.a.c = {c->rows, c->rows, c->scale, c->scale, c->table, c->n_pages, shift_of(c->page), 1, c->latent, c->n_seq, c->max_pages};
    j.a.q = a->q, j.a.o = a->o;
    j.a.q_start = a->q_start, j.a.kv_len = a->kv_len, j.a.q_pos = a->q_pos, j.a.tree = a->tree;
    j.a.T = a->T, j.a.n_q = j.a.group = a->n_q, j.a.ldq = a->ldq, j.a.ldo = a->ldo;
    j.a.max_q = a->max_q < a->T ? a->max_q : a->T;
    j.a.max_kv = a->max_kv, j.a.mask = a->mask, j.a.window = a->window, j.a.tree_words = a->tree_words;
    j.a.scale2 = (float)(a->scale * 1.4426950408889634);   // log2(e)
    j.q = a->q, j.w = a->w, j.o = a->o;
    j.rot = c->rot, j.nope = a->nope, j.value = a->value, j.ldq = a->ldq, j.ldo = a->ldo;
    j.scale = a->scale;
    const bool f32 = a->dtype == WL_DTYPE_F32;
    if (a->form == WL_LATENT_EXPANDED && !wl::latent_can_expand(j, c->format))
        return fail(WL_ERR_UNSUPPORTED, "WL_LATENT_EXPANDED needs w, a bf16 cache, and nope=%d and value=%d both 64 or both 128", a->nope, a->value);
    *form = a->form;
    if (a->T == 0) return WL_OK;
    const int64_t wq = (int64_t)a->n_q * (a->nope + c->rot), wo = (int64_t)a->n_q * a->value;
    const size_t weights = (size_t)a->n_q * (a->nope + a->value) * c->latent * bytes_of(a->dtype);
    if ((st = check_rows(a->q, a->T, wq, a->ldq, "q")) != WL_OK || (st = check_rows(a->o, a->T, wo, a->ldo, "o")) != WL_OK ||
        (st = need(a->q_start, 4, "q_start")) != WL_OK || (st = need(a->kv_len, 4, "kv_len")) != WL_OK)
        return st;
    if (a->w && (st = need(a->w, 16, "w")) != WL_OK) return st;
    const bool tree = a->mask == WL_ATTN_TREE;
    if (tree) {
        if ((st = need(a->tree, 4, "tree")) != WL_OK) return st;
        if (a->q_pos && (st = need(a->q_pos, 4, "q_pos")) != WL_OK) return st;
    }
    st = check_out(row_set(a->o, a->T, wo, a->ldo, a->dtype, "o"),
                   {row_set(a->q, a->T, wq, a->ldq, a->dtype, "q"), {flat(a->w, weights), "w"}, pool(c), scales(c), table(c),
                    array(a->q_start, (size_t)c->n_seq + 1, "q_start"), array(a->kv_len, c->n_seq, "kv_len"),
                    array(tree ? a->tree : nullptr, (size_t)a->T * (tree ? a->tree_words : 0), "tree"),
                    array(tree ? a->q_pos : nullptr, a->T, "q_pos")});
    if (st != WL_OK) return st;
    const wl::LatentNeeds n = wl::latent_needs(j, c->format, f32, a->form);
    if (n.workgroups > kMaxWorkgroups)
        return fail(WL_ERR_UNSUPPORTED, "n_seq=%d, n_q=%d, T=%d and max_q=%d ask for %lld workgroups, more than %lld", c->n_seq, a->n_q, a->T,
                    a->max_q, (long long)n.workgroups, (long long)kMaxWorkgroups);
    *job = j;
    return WL_OK;
}

// ---- drafted tokens ---------------------------------------------------------------

constexpr int32_t kMaxVocab = 1 << 30;

// Everything of a verification but its workspace. T == 0 is accepted.
wl_status check_verify(const wl_verify_args *a, wl::VerifyJob *job) {
    wl_status st;
    if (!a) return fail(WL_ERR_INVALID_ARG, "arguments are NULL");
    if ((st = check_dtype(a->dtype)) != WL_OK) return st;
    if (a->T < 0) return fail(WL_ERR_INVALID_ARG, "T=%d is negative", a->T);
    if (a->n_seq < 1 || a->vocab < 1) return fail(WL_ERR_INVALID_ARG, "n_seq=%d and vocab=%d must be >= 1", a->n_seq, a->vocab);
    if (a->vocab > kMaxVocab) return fail(WL_ERR_UNSUPPORTED, "vocab=%d exceeds %d", a->vocab, kMaxVocab);
    if (a->max_q < 1 || a->max_q > wl::kVerifyRows)
        return fail(WL_ERR_INVALID_ARG, "max_q=%d is outside [1, %d]", a->max_q, wl::kVerifyRows);
    if (a->kind != WL_VERIFY_LOGITS && a->kind != WL_VERIFY_PROBABILITIES)
        return fail(WL_ERR_INVALID_ARG, "kind=%d is neither WL_VERIFY_LOGITS nor WL_VERIFY_PROBABILITIES", a->kind);
    if (a->draft && a->parent) return fail(WL_ERR_INVALID_ARG, "parent (trees) does not go with a draft's distribution");
    if (a->T == 0) {   // n_out is all there is to write
        if (!a->n_out) return WL_OK;
        if ((st = need(a->n_out, 4, "n_out")) != WL_OK) return st;
        const size_t n = a->n_seq;
        if ((st = check_out(array(a->n_out, n, "n_out"), {array(a->q_start, n + 1, "q_start"), array(a->temperature, n, "temperature"),
                                                         array(a->len, n, "len")})) != WL_OK)
            return st;
        job->n_out = a->n_out, job->n_seq = a->n_seq;
        return WL_OK;
    }
    if (a->T > kMaxTokens) return fail(WL_ERR_UNSUPPORTED, "T=%d exceeds %d", a->T, kMaxTokens);
    if ((st = need(a->target, 16, "target")) != WL_OK || (st = need(a->token, 4, "token")) != WL_OK ||
        (st = need(a->q_start, 4, "q_start")) != WL_OK || (st = need(a->u, 8, "u")) != WL_OK ||
        (st = need(a->out, 4, "out")) != WL_OK || (st = need(a->n_out, 4, "n_out")) != WL_OK)
        return st;
    if (a->draft && (st = need(a->draft, 16, "draft")) != WL_OK) return st;
    if (a->parent && (st = need(a->parent, 4, "parent")) != WL_OK) return st;
    if (a->temperature && (st = need(a->temperature, 4, "temperature")) != WL_OK) return st;
    if (a->path && (st = need(a->path, 4, "path")) != WL_OK) return st;
    if (a->len && (st = need(a->len, 4, "len")) != WL_OK) return st;
    if (a->ld_target < a->vocab || (a->draft && a->ld_draft < a->vocab))
        return fail(WL_ERR_INVALID_ARG, "ld_target=%d or ld_draft=%d is below vocab=%d", a->ld_target, a->ld_draft, a->vocab);
    if ((int64_t)a->T * a->ld_target >= kMaxElems || (a->draft && (int64_t)a->T * a->ld_draft >= kMaxElems))
        return fail(WL_ERR_INVALID_ARG, "target or draft spans 2^31 or more elements");
    const size_t T = a->T, n = a->n_seq;
    const Named target = row_set(a->target, a->T, a->vocab, a->ld_target, a->dtype, "target");
    const Named draft = a->draft ? row_set(a->draft, a->T, a->vocab, a->ld_draft, a->dtype, "draft") : Named{flat(nullptr, 0), "draft"};
    const Named token = array(a->token, T, "token"), start = array(a->q_start, n + 1, "q_start"), parent = array(a->parent, T, "parent");
    const Named u = array(a->u, 2 * T, "u"), temperature = array(a->temperature, n, "temperature");
    const Named outs[4] = {array(a->out, T, "out"), array(a->path, T, "path"), array(a->n_out, n, "n_out"), array(a->len, n, "len")};
    for (int i = 0; i < 4; ++i) {
        if (!outs[i].r.p) continue;
        if ((st = check_out(outs[i], {target, draft, token, start, parent, u, temperature})) != WL_OK) return st;
        for (int l = 0; l < i; ++l)
            if (outs[l].r.p && (st = check_out(outs[i], {outs[l]})) != WL_OK) return st;
    }
    wl::VerifyJob j{};
    j.target = a->target, j.draft = a->draft, j.token = a->token, j.q_start = a->q_start, j.parent = a->parent;
    j.u = reinterpret_cast<const float2 *>(a->u), j.temperature = a->temperature;
    j.out = a->out, j.path = a->path, j.n_out = a->n_out, j.len = a->len;
    j.T = a->T, j.n_seq = a->n_seq, j.vocab = a->vocab, j.ld_target = a->ld_target, j.ld_draft = a->ld_draft;
    j.max_q = a->max_q, j.logits = a->kind == WL_VERIFY_LOGITS;
    const int64_t blocks = wl::verify_workgroups(j, a->dtype == WL_DTYPE_F32);
    if (blocks > kMaxWorkgroups)
        return fail(WL_ERR_UNSUPPORTED, "T=%d and n_seq=%d ask for %lld workgroups, more than %lld", a->T, a->n_seq, (long long)blocks,
                    (long long)kMaxWorkgroups);
    *job = j;
    return WL_OK;
}

}  // namespace

extern "C" {

size_t wl_batch_plan_workspace_bytes(const wl_batch_plan_args *a) {
    wl::PlanJob j{};
    return check_plan(a, &j, nullptr, 0) == WL_OK ? ws_of(wl::plan_scratch(j)) : 0;
}

wl_status wl_batch_plan(const wl_batch_plan_args *a, void *ws, size_t ws_bytes, void *hip_stream) {
    wl::PlanJob j{};
    wl_status st = check_plan(a, &j, nullptr, 0);
    if (st != WL_OK) return st;
    const size_t scratch = wl::plan_scratch(j);
    void *at;
    if ((st = check_scratch(ws, ws_bytes, scratch, &at)) != WL_OK) return st;
    if (at && (st = check_plan(a, &j, at, scratch)) != WL_OK) return st;
    return launched(wl::launch_plan(j, at, static_cast<hipStream_t>(hip_stream)), "batch plan");
}

wl_status wl_latent_write(const wl_latent_write_args *a, void *hip_stream) {
    wl_status st;
    if (!a) return fail(WL_ERR_INVALID_ARG, "arguments are NULL");
    if ((st = check_dtype(a->dtype)) != WL_OK || (st = check_latent_cache(a->cache, a->dtype)) != WL_OK) return st;
    if (a->T < 0) return fail(WL_ERR_INVALID_ARG, "T=%d is negative", a->T);
    if (a->n_q < 0 || a->n_q > kMaxHeads) return fail(WL_ERR_INVALID_ARG, "n_q=%d is out of range", a->n_q);
    if (a->n_q && (st = check_heads(a->nope)) != WL_OK) return st;
    if (a->T == 0) return ok();
    const wl_latent_cache *c = a->cache;
    const int32_t T = a->T;
    if (T > kMaxWorkgroups) return fail(WL_ERR_UNSUPPORTED, "T=%d exceeds %lld", T, (long long)kMaxWorkgroups);
    const int64_t wc = c->latent + c->rot, wq = (int64_t)a->n_q * (a->nope + c->rot);
    const size_t e = bytes_of(a->dtype);
    const wl_rotary *r = a->rotary;
    if ((st = check_rotary(r, c->rot, false)) != WL_OK) return st;
    if (r && r->rot != c->rot) return fail(WL_ERR_INVALID_ARG, "rot=%d is not the cache's %d", r->rot, c->rot);
    if ((st = check_rows(a->c, T, wc, a->ldc, "c")) != WL_OK || (st = need(a->seq, 4, "seq")) != WL_OK ||
        (st = need(a->slot, 4, "slot")) != WL_OK)
        return st;
    if (a->norm && (st = need(a->norm, 16, "norm")) != WL_OK) return st;
    if (a->n_q && ((st = check_rows(a->q, T, wq, a->ldq, "q")) != WL_OK || (st = check_rows(a->q_out, T, wq, a->ldq_out, "q_out")) != WL_OK))
        return st;
    const Named none{flat(nullptr, 0), ""};
    const Named in = row_set(a->c, T, wc, a->ldc, a->dtype, "c"), norm{flat(a->norm, c->latent * e), "norm"};
    const Named q = a->n_q ? row_set(a->q, T, wq, a->ldq, a->dtype, "q") : none;
    const Named fr{flat(r ? r->freq : nullptr, r ? (size_t)r->rot * 4 : 0), "freq"}, ps = array(r ? r->pos : nullptr, T, "pos");
    const Named sq = array(a->seq, T, "seq"), sl = array(a->slot, T, "slot");
    const Named qo = a->n_q ? row_set(a->q_out, T, wq, a->ldq_out, a->dtype, "q_out") : none;
    if (a->n_q && (st = check_out(qo, {q, in, norm, fr, ps, sq, sl, table(c)}, {a->q})) != WL_OK) return st;
    if ((st = check_out(pool(c), {q, in, norm, fr, ps, sq, sl, table(c), qo, scales(c)})) != WL_OK) return st;
    if (c->format == WL_CACHE_E4M3 && (st = check_out(scales(c), {q, in, norm, fr, ps, sq, sl, table(c), qo})) != WL_OK) return st;
    wl::LatentWriteJob j{};
    j.c = latent_ref(c);
    j.in = a->c, j.norm = a->norm, j.q = a->q, j.q_out = a->q_out, j.seq = a->seq, j.slot = a->slot;
    if (r) j.freq = r->freq, j.pos = r->pos, j.interleaved = r->style == WL_ROPE_INTERLEAVED, j.turn_scale = r->scale;
    j.T = T, j.n_q = a->n_q, j.nope = a->n_q ? a->nope : 0, j.ldc = a->ldc, j.ldq = a->ldq, j.ldq_out = a->ldq_out;
    j.eps = a->eps, j.offset = a->offset;
    return launched(wl::launch_latent_write(j, c->format, static_cast<hipStream_t>(hip_stream)), "latent write");
}

wl_status wl_latent_read(const wl_latent_read_args *a, void *hip_stream) {
    wl_status st;
    if (!a) return fail(WL_ERR_INVALID_ARG, "arguments are NULL");
    if ((st = check_dtype(a->dtype)) != WL_OK || (st = check_latent_cache(a->cache, a->dtype)) != WL_OK) return st;
    if (a->T < 0) return fail(WL_ERR_INVALID_ARG, "T=%d is negative", a->T);
    if (a->T == 0) return ok();
    const wl_latent_cache *c = a->cache;
    const int32_t T = a->T;
    const int64_t w = c->latent + c->rot;
    if ((st = check_rows(a->out, T, w, a->ld, "out")) != WL_OK || (st = need(a->seq, 4, "seq")) != WL_OK ||
        (st = need(a->slot, 4, "slot")) != WL_OK)
        return st;
    st = check_out(row_set(a->out, T, w, a->ld, a->dtype, "out"),
                   {pool(c), scales(c), table(c), array(a->seq, T, "seq"), array(a->slot, T, "slot")});
    if (st != WL_OK) return st;
    return launched(wl::launch_latent_read({latent_ref(c), a->seq, a->slot, a->out, T, a->ld}, c->format, static_cast<hipStream_t>(hip_stream)),
                    "latent read");
}

size_t wl_latent_attention_workspace_bytes(const wl_latent_attention_args *a) {
    wl::LatentJob j{};
    int form;
    if (check_latent_attention(a, &j, &form) != WL_OK || a->T == 0) return 0;
    return ws_of(wl::latent_needs(j, a->cache->format, a->dtype == WL_DTYPE_F32, form).scratch);
}

wl_status wl_latent_attention(const wl_latent_attention_args *a, void *ws, size_t ws_bytes, void *hip_stream) {
    wl::LatentJob j{};
    int form;
    wl_status st = check_latent_attention(a, &j, &form);
    if (st != WL_OK) return st;
    if (a->T == 0 || j.a.max_q == 0) return ok();
    const wl_latent_cache *c = a->cache;
    const bool f32 = a->dtype == WL_DTYPE_F32;
    const size_t scratch = wl::latent_needs(j, c->format, f32, form).scratch;
    void *at;
    if ((st = check_scratch(ws, ws_bytes, scratch, &at)) != WL_OK) return st;
    if (at) {
        const int64_t wq = (int64_t)a->n_q * (a->nope + c->rot), wo = (int64_t)a->n_q * a->value;
        const bool tree = a->mask == WL_ATTN_TREE;
        st = check_out({flat(at, scratch), "workspace"},
                       {row_set(a->q, a->T, wq, a->ldq, a->dtype, "q"), row_set(a->o, a->T, wo, a->ldo, a->dtype, "o"),
                        {flat(a->w, (size_t)a->n_q * (a->nope + a->value) * c->latent * bytes_of(a->dtype)), "w"}, pool(c), scales(c), table(c),
                        array(a->q_start, (size_t)c->n_seq + 1, "q_start"), array(a->kv_len, c->n_seq, "kv_len"),
                        array(tree ? a->tree : nullptr, (size_t)a->T * (tree ? a->tree_words : 0), "tree"),
                        array(tree ? a->q_pos : nullptr, a->T, "q_pos")});
        if (st != WL_OK) return st;
    }
    return launched(wl::launch_latent(j, c->format, f32, form, at, static_cast<hipStream_t>(hip_stream)), "latent attention");
}

size_t wl_verify_drafts_workspace_bytes(const wl_verify_args *a) {
    wl::VerifyJob j{};
    if (check_verify(a, &j) != WL_OK || a->T == 0) return 0;
    return ws_of(wl::verify_scratch(j, a->dtype == WL_DTYPE_F32));
}

wl_status wl_verify_drafts(const wl_verify_args *a, void *ws, size_t ws_bytes, void *hip_stream) {
    wl::VerifyJob j{};
    wl_status st = check_verify(a, &j);
    if (st != WL_OK) return st;
    if (a->T == 0) return a->n_out ? launched(wl::launch_verify_no_rows(j, static_cast<hipStream_t>(hip_stream)), "verification") : ok();
    const bool f32 = a->dtype == WL_DTYPE_F32;
    const size_t scratch = wl::verify_scratch(j, f32), T = a->T, n = a->n_seq;
    void *at;
    if ((st = check_scratch(ws, ws_bytes, scratch, &at)) != WL_OK) return st;
    st = check_out({flat(at, scratch), "workspace"},
                   {row_set(a->target, a->T, a->vocab, a->ld_target, a->dtype, "target"),
                    a->draft ? row_set(a->draft, a->T, a->vocab, a->ld_draft, a->dtype, "draft") : Named{flat(nullptr, 0), "draft"},
                    array(a->token, T, "token"), array(a->q_start, n + 1, "q_start"), array(a->parent, T, "parent"), array(a->u, 2 * T, "u"),
                    array(a->temperature, n, "temperature"), array(a->out, T, "out"), array(a->path, T, "path"), array(a->n_out, n, "n_out"),
                    array(a->len, n, "len")});
    if (st != WL_OK) return st;
    return launched(wl::launch_verify(j, f32, at, static_cast<hipStream_t>(hip_stream)), "verification");
}

}  // extern "C"
