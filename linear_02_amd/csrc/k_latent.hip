// Attention over the latent cache: which form and kernels run, and the join of divided keys.
#include <type_traits>

#include "wl_latent.h"

namespace wl {

namespace {

// Every query row of an fp32 call by a wave of its own, key by key.
template <class E, int F>
__global__ __launch_bounds__(256) void rows_kernel(CoreArgs x) {
    const AttnJob &a = x.a;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    const int64_t w = (int64_t)blockIdx.x * 4 + wave, per = (int64_t)a.max_q * a.group;
    const int s = (int)(w / per), r = (int)(w - (int64_t)s * per);
    if (s >= a.c.n_seq) return;
    const Seq q = seq_of(a, s);
    if (r >= q.rows * a.group) return;
    const int i = r / a.group, h = r - i * a.group;
    float acc[8], m, l;
    latent_row<E, F>(a, x.rot, q, i, h, 0, q.kv, acc, m, l);
    if (8 * lane >= a.c.d) return;
#pragma unroll
    for (int e = 0; e < 8; ++e) acc[e] = l == 0.0f ? 0.0f : acc[e] / l;
    E *o = static_cast<E *>(a.o) + (size_t)(q.q0 + i) * a.ldo + (size_t)h * a.c.d + 8 * lane;
    put4(o, acc);
    put4(o + 4, acc + 4);
}

// q' = W^K^T q of every token and head, its rotated part beside it.
template <class E>
__global__ __launch_bounds__(256) void absorb_kernel(LatentJob a, E *out) {
    __shared__ float qs[256];
    const int t = blockIdx.x / a.a.n_q, h = blockIdx.x - t * a.a.n_q, L = a.a.c.d, N = a.nope, R = a.rot;
    const E *q = static_cast<const E *>(a.q) + (size_t)t * a.ldq + (size_t)h * (N + R);
    E *o = out + ((size_t)t * a.a.n_q + h) * (L + R);
    if ((int)threadIdx.x < N) qs[threadIdx.x] = element(q + threadIdx.x);
    if ((int)threadIdx.x < R) o[L + threadIdx.x] = q[N + threadIdx.x];
    __syncthreads();
    const E *w = static_cast<const E *>(a.w) + (size_t)h * (N + a.value) * L;
    for (int l = threadIdx.x; l < L; l += 256) {
        float s = 0.0f;
        for (int n = 0; n < N; ++n) s += qs[n] * element(w + (size_t)n * L + l);
        o[l] = std::is_same<E, float>::value ? (E)s : (E)f_bf16(s);
    }
}

// o = W^V o' of every token and head that has a result: of a sequence's first max_q rows.
template <class E>
__global__ __launch_bounds__(256) void up_kernel(LatentJob a, const E *in) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int t = blockIdx.x / a.a.n_q, h = blockIdx.x - t * a.a.n_q, L = a.a.c.d, N = a.nope, V = a.value;
    if (!has_result(a.a, t)) return;
    const E *x = in + ((size_t)t * a.a.n_q + h) * L;
    const E *w = static_cast<const E *>(a.w) + ((size_t)h * (N + V) + N) * L;
    E *o = static_cast<E *>(a.o) + (size_t)t * a.ldo + (size_t)h * V;
    for (int v = wave; v < V; v += 4) {
        float s = 0.0f;
        for (int l = lane; l < L; l += 64) s += element(x + l) * element(w + (size_t)v * L + l);
        s = wave_sum(s);
        if (lane == 0) o[v] = std::is_same<E, float>::value ? (E)s : (E)f_bf16(s);
    }
}

size_t pad(size_t b) { return (b + 255) & ~(size_t)255; }

// Fewest keys of a piece.
constexpr int kMinChunk = 256;

struct Plan {
    CoreKind kind;
    Split sp;
    int64_t items;   // as in sp, which holds them if they are within a launch's limits
};

// Which kernel a bf16 or e4m3 call takes, and how its keys are divided, as plan_of in
// k_attn.hip does it.
Plan plan_of(const LatentJob &job, int fmt) {
    const AttnJob &a = job.a;
    Plan p{};
    const int64_t rows = a.max_q > 0 ? (int64_t)a.max_q * a.group : 1;
    p.kind.tiles = rows > 64 ? 2 : 1;
    p.kind.row_waves = rows > 32 ? 4 : rows > 16 ? 2 : 1;
    p.kind.exact = p.kind.row_waves == 1 && job.w;
    p.sp.tile_rows = 16 * p.kind.tiles * p.kind.row_waves;
    p.sp.rows = (int)(rows < p.sp.tile_rows ? rows : p.sp.tile_rows);
    p.sp.tiles = (int)((rows + p.sp.tile_rows - 1) / p.sp.tile_rows);
    int64_t span = a.max_kv;
    if (a.mask == kMaskCausal && a.window && (int64_t)a.window + a.max_q < span) span = (int64_t)a.window + a.max_q;
    span += 31;
    const int64_t tiles = (int64_t)a.c.n_seq * p.sp.tiles;
    const int64_t places = kWorkgroups / 2 * workgroups_per_cu(fmt, a.c.d, p.kind.tiles, p.kind.row_waves);
    const int64_t want = 2 * tiles > places ? 2 * places : places;
    int64_t chunk = (span * tiles + want - 1) / want;
    p.sp.least = kMinChunk;
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
Places places_of(const LatentJob &a, const Plan &p, bool f32) {
    const size_t rows = (size_t)a.a.T * a.a.n_q, L = a.a.c.d;
    const bool split = !f32 && p.sp.n_split > 1;
    Places w{};
    size_t at = 0;
    auto take = [&](size_t bytes) {
        const size_t here = at;
        at += pad(bytes);
        return here;
    };
    if (a.w) {
        w.q = take(rows * (L + a.rot) * (f32 || p.kind.exact ? 4 : 2));
        if (!split) w.o = take(rows * L * (f32 ? 4 : 2));
    }
    if (split) {
        w.part = take((size_t)p.items * p.sp.rows * L * 2);
        w.ml = take((size_t)p.items * p.sp.rows * 8);
    }
    w.bytes = at;
    return w;
}

hipError_t launch_f32(LatentJob a, const Places &w, char *ws, hipStream_t s) {
    const size_t rows = (size_t)a.a.T * a.a.n_q;
    float *q = reinterpret_cast<float *>(ws + w.q), *o = reinterpret_cast<float *>(ws + w.o);
    hipError_t e;
    if (a.w) {
        hipLaunchKernelGGL((absorb_kernel<float>), dim3((unsigned)rows), dim3(256), 0, s, a, q);
        if ((e = hipGetLastError()) != hipSuccess) return e;
        a.a.q = q, a.a.ldq = a.a.n_q * (a.a.c.d + a.rot);
        a.a.o = o, a.a.ldo = a.a.n_q * a.a.c.d;
    }
    const int64_t waves = (int64_t)a.a.c.n_seq * a.a.max_q * a.a.group;
    hipLaunchKernelGGL((rows_kernel<float, kFmtF32>), dim3((unsigned)((waves + 3) / 4)), dim3(256), 0, s, CoreArgs{a.a, Split{}, a.rot});
    if ((e = hipGetLastError()) != hipSuccess || !a.w) return e;
    hipLaunchKernelGGL((up_kernel<float>), dim3((unsigned)rows), dim3(256), 0, s, a, o);
    return hipGetLastError();
}

}  // namespace

bool latent_can_expand(const LatentJob &, bool) { return false; }

LatentNeeds latent_needs(const LatentJob &a, int fmt, bool f32, int) {
    const int64_t rows = (int64_t)a.a.T * a.a.n_q;
    const Plan p = plan_of(a, fmt);
    LatentNeeds n{places_of(a, p, f32).bytes, p.items};
    if (f32) n.workgroups = ((int64_t)a.a.c.n_seq * a.a.max_q * a.a.group + 3) / 4;
    // the products around it, of tokens and heads
    const int64_t around = f32 ? rows : (rows + 15) / 16 * 8 + 8 * a.a.n_q;
    if (around > n.workgroups) n.workgroups = around;
    return n;
}

hipError_t launch_latent(const LatentJob &job, int fmt, bool f32, int, void *ws, hipStream_t s) {
    LatentJob a = job;
    const Plan p = plan_of(a, fmt);
    const Places w = places_of(a, p, f32);
    char *at = static_cast<char *>(ws);
    if (f32) return launch_f32(a, w, at, s);
    CoreArgs x{a.a, p.sp, a.rot};
    hipError_t e;
    if (a.w) {
        launch_absorb(a, at + w.q, p.kind.exact, s);
        if ((e = hipGetLastError()) != hipSuccess) return e;
        x.a.q = at + w.q, x.a.ldq = x.a.n_q * (x.a.c.d + a.rot);
        x.a.o = at + w.o, x.a.ldo = x.a.n_q * x.a.c.d;
    }
    if (p.sp.n_split > 1) {
        x.sp.part = reinterpret_cast<float *>(at + w.part);
        x.sp.ml = reinterpret_cast<float2 *>(at + w.ml);
    }
    launch_latent_tile(x, fmt, p.kind, (unsigned)p.sp.items, s);
    if ((e = hipGetLastError()) != hipSuccess) return e;
    if (a.w)
        launch_up(a, x, s);
    else if (p.sp.n_split > 1)
        launch_join(x, s);
    return hipGetLastError();
}

}  // namespace wl
