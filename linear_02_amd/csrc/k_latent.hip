// Attention over the latent cache: which form and kernels run, and the join of divided keys.
#include "wl_latent.h"

namespace wl {

namespace {

size_t pad(size_t b) { return (b + 255) & ~(size_t)255; }

// Fewest keys of a piece (whole calls, replayed from a graph). Waves with keys of their own (calls of at most 16
// rows a sequence) read a piece in 128-key steps: one token of 16 heads over 1000 keys takes 26.8 us with 128 and
// 28.2 with 256, over 4000 33.9 and 31.3, 8 streams over up to 4096 41.8 and 37.2. In fp32, 4 streams of 3
// tokens and 16 heads over 1024 keys take 63 us with 64 and 83 with 128. Elsewhere 256: 2 streams of 128 heads
// over up to 2000 keys 46.5 us, 58.8 with 512, 42.5 with 128, which costs where pieces are many (32 heads of
// 8 streams over up to 4096 keys 42.1 and 46.0).
constexpr int kMinChunk = 256, kMinChunkOwn = 128, kMinChunkF32 = 64;

struct Plan {
    CoreKind kind;
    Split sp;
    int64_t items;   // as in sp, which holds them if they are within a launch's limits
};

// Which kernel a bf16 or e4m3 call takes, and how its keys are divided, as plan_of in
// k_attn.hip does it.
Plan plan_of(const LatentJob &job, int fmt) {
    const bool f32 = fmt == kFmtF32;
    const AttnJob &a = job.a;
    Plan p{};
    const int64_t rows = a.max_q > 0 ? (int64_t)a.max_q * a.group : 1;
    int64_t span = a.max_kv;
    if (a.mask == kMaskCausal && a.window && (int64_t)a.window + a.max_q < span) span = (int64_t)a.window + a.max_q;
    span += 31;
    // Waves over keys instead of rows where rows are few: 64 streams of 32 heads over up to 4096 e4m3 keys 74 us with
    // two pairs, 94 with four waves of rows; of 16 heads 61 us with four waves that have keys of their own, 69 with
    // pairs (one token over 1000 bf16 keys 26.8 and 30.3).
    p.kind.row_waves = rows > (f32 ? 16 : 32) ? 4 : rows > 16 ? 2 : 1;
    p.kind.exact = job.w && !f32;
    p.sp.tile_rows = 16 * p.kind.row_waves;
    p.sp.rows = (int)(rows < p.sp.tile_rows ? rows : p.sp.tile_rows);
    p.sp.tiles = (int)((rows + p.sp.tile_rows - 1) / p.sp.tile_rows);
    const int64_t tiles = (int64_t)a.c.n_seq * p.sp.tiles;
    const int64_t places = kWorkgroups / 2 * (f32 ? 1 : workgroups_per_cu(fmt, a.c.d, p.kind.row_waves, p.kind.exact));
    const int64_t want = 2 * tiles > places ? 2 * places : places;
    int64_t chunk = (span * tiles + want - 1) / want;
    p.sp.least = f32 ? kMinChunkF32 : p.kind.row_waves == 1 ? kMinChunkOwn : kMinChunk;
    if (chunk < p.sp.least) chunk = p.sp.least;
    if (chunk < (span + kMaxSplit - 1) / kMaxSplit) chunk = (span + kMaxSplit - 1) / kMaxSplit;
    p.sp.step = 128 / p.kind.row_waves;
    chunk = (chunk + p.sp.step - 1) / p.sp.step * p.sp.step;
    p.sp.chunk = (int)(chunk < (1 << 30) ? chunk : (1 << 30));
    p.sp.n_split = (int)((span + chunk - 1) / chunk);
    p.items = tiles * p.sp.n_split;
    p.sp.want = (int)want, p.sp.places = (int)places;
    if (p.sp.n_split > 1 && a.c.n_seq <= 64) {
        p.sp.planned = 1;
        const int64_t most = (span + p.sp.least - 1) / p.sp.least;
        p.sp.n_split = (int)(most < kMaxSplit ? most : kMaxSplit);
        p.items = tiles * p.sp.n_split;
        if (want + tiles < p.items) p.items = want + tiles;
    }
    p.sp.all_fit = p.items <= places;
    p.sp.items = (int)(p.items < (1 << 30) ? p.items : (1 << 30));
    return p;
}

// The workspace: queries in the latent space, outputs there, divided outputs and their statistics.
struct Places {
    size_t q, o, part, ml, bytes;
};
Places places_of(const LatentJob &a, const Plan &p) {
    const size_t rows = (size_t)a.a.T * a.a.n_q, L = a.a.c.d;
    const bool split = p.sp.n_split > 1;
    Places w{};
    size_t at = 0;
    auto take = [&](size_t bytes) {
        const size_t here = at;
        at += pad(bytes);
        return here;
    };
    if (a.w) {
        w.q = take(rows * (L + a.rot) * 4);
        if (!split) w.o = take(rows * L * 4);
    }
    if (split) {
        w.part = take((size_t)p.items * p.sp.rows * L * 4);
        w.ml = take((size_t)p.items * p.sp.rows * 8);
    }
    w.bytes = at;
    return w;
}

// Expanded keys and values of a call at once, at most; heads are taken in groups that fit.
constexpr size_t kExpandedBytes = (size_t)8 << 30;

struct Expanded {
    int heads;         // of a group
    int keys, blocks, tiles;
    size_t bytes;      // of the keys, and of the values
    size_t all;        // with their scales
};
Expanded expanded_of(const LatentJob &job) {
    const AttnJob &a = job.a;
    Expanded e{};
    const int64_t room = (int64_t)a.c.max_pages << a.c.page_shift;
    const int64_t keys = a.max_kv < room ? a.max_kv : room;
    e.blocks = (int)((keys + 127) / 128);
    e.keys = 128 * e.blocks;
    e.tiles = (a.max_q + 127) / 128;
    const size_t rows = (size_t)a.c.n_seq * e.keys, one = rows * job.nope * 2;   // of a head
    const size_t fit = one ? kExpandedBytes / (2 * one + 8 * rows) : a.n_q;
    e.heads = fit < 1 ? 1 : fit > (size_t)a.n_q ? a.n_q : (int)fit;
    e.bytes = pad(one * e.heads);
    e.all = 2 * e.bytes + pad(8 * rows * e.heads);
    return e;
}

// Which form AUTO takes. The expanded one forms all keys and values once, and multiplies less per
// query and key then; 128 queries of a head are one workgroup that walks all of their keys, so it wants
// many of those, or few keys. Both times are estimated in us from constants fitted to measurements
// (absorbed, expanded; n_seq x queries over up to so many keys, heads; latent 512, heads of 128 + 64):
//   1 x 128 over 4096, 32   109, 216     1 x 512 over 4096, 32   289, 214     1 x 512 over 8192, 16   275, 357
//   1 x 192 over 192, 128    95, 36      1 x 512 over 512, 32     92, 47      1 x 2048 over 2048, 8   176, 101
//   1 x 256 over 4096, 128  549, 422     8 x 192 over 4096, 32   578, 495     8 x 256 over 2048, 32   499, 305
// and, of 1 x 512 over 4096 and 8 x 256 over 2048, 32 heads, at a latent of 256 with heads of 128: 150, 199 and 243, 246;
// 256 with 64: 139, 153 and 229, 142; 128 with 64: 102, 148 and 143, 128. The one taken is the faster or within 3 %,
// but for 8 x 192 over 4096 and the last, absorbed at 1.16 and 1.12 times the other: of 8 sequences of uneven lengths
// the host knows the longest.
// Calls of fewer queries than a tile has stay absorbed: the first constant is of many rows.
bool expands(const LatentJob &job, int fmt, int form) {
    const AttnJob &a = job.a;
    if (form != kFormAuto) return form == kFormExpanded;
    if (!latent_can_expand(job, fmt) || a.max_q < 128) return false;
    const Expanded e = expanded_of(job);
    // Never where the other form's workspace or launch would be beyond what calls may have.
    if (e.all > kExpandedBytes + 1024 || (int64_t)a.c.n_seq * (e.blocks > e.tiles ? e.blocks : e.tiles) * e.heads >= 1 << 23) return false;
    const double keys = e.keys, L = a.c.d, H = a.n_q;
    const double seen = a.mask == kMaskCausal && a.window && (double)a.window + a.max_q < keys ? (double)a.window + a.max_q : keys;
    const double tiles = (double)a.c.n_seq * e.tiles * H;
    const double absorbed = 50 + (L == 512 ? 1.6e-9 : 1.15e-9) * 2 * a.T * H * seen * (2 * L + job.rot);   // two workgroups a CU below 512
    const double expanded = 10 + 2e-9 * 2 * a.c.n_seq * keys * H * (job.nope + job.value) * L +
                            0.0327 * seen * (tiles < 394 ? 1.0 : tiles * (0.65 / 256));
    return expanded < absorbed;
}

}  // namespace

bool latent_can_expand(const LatentJob &a, int fmt) { return a.w && fmt == kFmtBf16 && a.nope == a.value && (a.nope == 64 || a.nope == 128); }

LatentNeeds latent_needs(const LatentJob &a, int fmt, bool f32, int form) {
    if (expands(a, fmt, form)) {
        const Expanded e = expanded_of(a);
        const int64_t wide = e.blocks > e.tiles ? e.blocks : e.tiles;
        return {e.all, (int64_t)a.a.c.n_seq * wide * e.heads};
    }
    const int64_t rows = (int64_t)a.a.T * a.a.n_q;
    const Plan p = plan_of(a, fmt);
    LatentNeeds n{places_of(a, p).bytes, p.items};
    // the products around it, of tokens and heads
    const int64_t around = (f32 ? rows : (rows + 15) / 16 * 8) + 8 * a.a.n_q;
    if (around > n.workgroups) n.workgroups = around;
    return n;
}

hipError_t launch_latent(const LatentJob &job, int fmt, bool f32, int form, void *ws, hipStream_t s) {
    LatentJob a = job;
    if (expands(a, fmt, form)) {
        const Expanded e = expanded_of(a);
        char *at = static_cast<char *>(ws);
        ExpandArgs x{a.a, a.w, reinterpret_cast<uint16_t *>(at), reinterpret_cast<uint16_t *>(at + e.bytes), reinterpret_cast<float *>(at + 2 * e.bytes),
                     a.rot, 0, 0, e.keys, e.blocks, e.tiles};
        x.a.group = 1;
        for (x.first = 0; x.first < a.a.n_q; x.first += e.heads) {
            x.heads = a.a.n_q - x.first < e.heads ? a.a.n_q - x.first : e.heads;
            launch_expanded(x, a.nope, s);
            const hipError_t err = hipGetLastError();
            if (err != hipSuccess) return err;
        }
        return hipSuccess;
    }
    const Plan p = plan_of(a, fmt);
    const Places w = places_of(a, p);
    char *at = static_cast<char *>(ws);
    CoreArgs x{a.a, p.sp, a.rot, a.w || f32};
    hipError_t e;
    if (a.w) {
        if (f32)
            launch_absorb_f32(a, reinterpret_cast<float *>(at + w.q), s);
        else
            launch_absorb(a, reinterpret_cast<float *>(at + w.q), s);
        if ((e = hipGetLastError()) != hipSuccess) return e;
        x.a.q = at + w.q, x.a.ldq = x.a.n_q * (x.a.c.d + a.rot);
        x.a.o = at + w.o, x.a.ldo = x.a.n_q * x.a.c.d;
    }
    if (p.sp.n_split > 1) {
        x.sp.part = reinterpret_cast<float *>(at + w.part);
        x.sp.ml = reinterpret_cast<float2 *>(at + w.ml);
    }
    if (f32)
        launch_latent_f32(x, p.kind, (unsigned)p.sp.items, s);
    else
        launch_latent_tile(x, fmt, p.kind, (unsigned)p.sp.items, s);
    if ((e = hipGetLastError()) != hipSuccess) return e;
    if (a.w)
        launch_up(a, x, f32, s);
    else if (p.sp.n_split > 1)
        launch_join(x, f32, s);
    return hipGetLastError();
}

}  // namespace wl
