// Attention over the paged cache: which kernel runs, how a long sequence's keys
// are divided, and the join of the parts.
#include "wl_attn_mfma.h"

namespace wl {

namespace {

// Joins the parts of every row: a wave per row, lane p weighs part p.
template <class E>
__global__ __launch_bounds__(256) void join_kernel(AttnJob a, Split sp) {
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    const int64_t w = (int64_t)blockIdx.x * 4 + wave;
    const int64_t per = (int64_t)a.max_q * a.group, unit = w / per;
    const int r = (int)(w - unit * per), s = (int)(unit / a.c.n_kv), kvh = (int)(unit % a.c.n_kv);
    if (s >= a.c.n_seq) return;
    const Seq q = seq_of(a, s);
    if (r >= q.rows * a.group) return;
    const int tile = r / sp.tile_rows;
    const Parts parts = parts_of(a, sp, s, tile);
    const int64_t first = part_row(a, sp, parts.first, kvh, tile, r), next = (int64_t)a.c.n_kv * sp.rows;
    float2 v = make_float2(kNegInf, 0.0f);
    if (lane < parts.n) v = sp.ml[first + lane * next];
    float m = v.x;
#pragma unroll
    for (int x = 1; x < 64; x <<= 1) m = fmaxf(m, __shfl_xor(m, x));
    // A piece without visible keys weighs nothing. One whose sum is NaN (a visible key's
    // score is) makes the row NaN, however far its maximum is below the others': a
    // piece of nothing but NaN has none at all.
    const float up = v.x == kNegInf && v.y == 0.0f ? 0.0f : v.y != v.y ? v.y : __builtin_amdgcn_exp2f(v.x - m);
    const float l = wave_sum(up * v.y);
    const int at = 4 * lane;
    f32x4 sum{0, 0, 0, 0};
    for (int p = 0; p < parts.n; ++p) {
        const float u = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(up), p));
        if (u == 0.0f) continue;
        if (at < a.c.d) sum += *reinterpret_cast<const f32x4 *>(sp.part + (first + p * next) * a.c.d + at) * u;
    }
    if (at >= a.c.d) return;
    const int i = r / a.group;
    const float o[4] = {sum.x, sum.y, sum.z, sum.w};
    float e[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) e[k] = l == 0.0f ? 0.0f : o[k] / l;
    put4(static_cast<E *>(a.o) + (size_t)(q.q0 + i) * a.ldo + (size_t)(kvh * a.group + r - i * a.group) * a.c.d + at, e);
}

enum Kind { kFew, kTile, kF32 };

struct Plan {
    Kind kind;
    int waves, tiles;   // per workgroup, tiles of query rows per wave
    bool exact;         // of the tile kernel: weights with their remainder
    int64_t items;      // as in Split, which holds it if it is within a launch's limits
    Split sp;
};

// Fewest keys of a piece. In us for 128, 256, 512 (bf16, 256 wide): one token of 4
// heads over 4096 keys 23.5, 21.5, 22.8; 128 tokens of 4 heads over 4096 keys 38.3,
// 34.3, 41.0; 512 tokens of 4 heads alone 25.8, 28.2, 36.6.
// In fp32, where a step of 16 keys is long, for 32, 64, 128, 256: one token of 4 heads
// over 1000 keys 27, 30, 40, 63; 8 tokens of 32 heads over up to 1024 keys 42, 42, 46, 67.
constexpr int kMinChunk = 256, kMinChunkF32 = 64;

// Most query rows per key/value head of the few-row kernel. Above 16 it takes two
// row tiles a wave, which at heads over 128 fill or pass its registers: 8 trees of 8
// tokens and 4 heads over up to 8192 keys of 256 took 189 us so in bf16 and 92 in
// int8, 97 and 77 us in the tile kernel; at 128 wide 57 and 58 us, 45 and 55 us.
int few_rows(const AttnJob &a) { return a.c.d > 128 ? 16 : 32; }

// Tiles of query rows per wave, and what the weights keep. Which of the two precisions a
// call has follows from its rows alone, not from max_kv: the remainder is kept for up to
// 64 rows per head, and up to this many tiles of 64 rows over all sequences and key/value
// heads, where the card has time for it (one tile a wave). In us, one tile with remainders
// against two without, heads of 256: 8 tiles over 512, 4096, 16384 keys in bf16 21, 29, 51
// and 26, 33, 50; 32 over 512, 4096 in int8 27, 43 and 34, 49; 24 over 2048, 16384 in int8
// 32, 83 and 42, 68; 64 over 128, 1024, 8192 in bf16 13, 30, 72 and 19, 34, 62; 256 over
// 512, 2048, 8192 38, 69, 206 and 40, 59, 139.
constexpr int kExactTiles = 32;
// Beyond, one tile a wave without remainders where the tiles of 64 rows in pieces of
// kMinChunk keys fit the card about twice, since with two much of it would be idle: 256
// tiles over 512 keys as above 36 us with one, 40 with two; 64 over 1024 29 and 34.
constexpr int kOneTilePieces = 2 * kWorkgroups;

Plan plan_of(const AttnJob &a, int fmt, bool f32) {
    Plan p{};
    p.kind = f32 ? kF32 : (int64_t)a.max_q * a.group > few_rows(a) ? kTile : kFew;
    const int64_t rows = a.max_q > 0 ? (int64_t)a.max_q * a.group : 1;
    // Most keys that the queries of one sequence see between them; pieces start at a multiple of 32.
    int64_t span = a.max_kv;
    if (a.mask == kMaskCausal && a.window && (int64_t)a.window + a.max_q < span) span = (int64_t)a.window + a.max_q;
    span += 31;
    const int64_t small = (int64_t)a.c.n_seq * a.c.n_kv * ((rows + 4 * kTileRows - 1) / (4 * kTileRows));   // tiles of 64 rows
    p.exact = rows <= 4 * kTileRows || small <= kExactTiles;
    p.tiles = !p.exact && (double)small * ((span + kMinChunk - 1) / kMinChunk) > kOneTilePieces ? 2 : 1;
    // Codes are widened once per workgroup: eight waves where they hold all rows.
    p.waves = p.tiles == 2 && fmt != kFmtBf16 && rows > 8 * kTileRows && rows <= 16 * kTileRows && p.kind == kTile ? 8 : 4;
    p.sp.tile_rows = p.kind == kTile ? p.waves * p.tiles * kTileRows : p.kind == kF32 ? kF32Rows : (int)rows;
    p.sp.rows = (int)(rows < p.sp.tile_rows ? rows : p.sp.tile_rows);
    p.sp.tiles = (int)((rows + p.sp.tile_rows - 1) / p.sp.tile_rows);
    const int64_t all_tiles = (int64_t)a.c.n_seq * p.sp.tiles, units = all_tiles * a.c.n_kv;
    // Enough pieces for every place on the card, one or two workgroups per CU; twice
    // as many where the sequences alone take more than half of the places, since
    // their lengths may be uneven.
    const bool one_per_cu = p.waves == 8 || (p.kind == kFew && fmt == kFmtBf16 && a.c.d > 128);
    const int64_t places = one_per_cu ? kWorkgroups / 2 : kWorkgroups;
    const int64_t want = p.kind == kFew && 2 * units > places ? 2 * places : places;
    int64_t chunk = (span * units + want - 1) / want;
    p.sp.least = p.kind == kF32 ? kMinChunkF32 : kMinChunk;
    if (chunk < p.sp.least) chunk = p.sp.least;
    if (chunk < (span + kMaxSplit - 1) / kMaxSplit) chunk = (span + kMaxSplit - 1) / kMaxSplit;
    p.sp.step = p.kind == kFew ? 128 : 32;   // whole 32s, for each of four waves if they divide a piece
    chunk = (chunk + p.sp.step - 1) / p.sp.step * p.sp.step;
    p.sp.chunk = (int)(chunk < (1 << 30) ? chunk : (1 << 30));
    p.sp.n_split = (int)((span + chunk - 1) / chunk);
    p.items = all_tiles * p.sp.n_split;
    p.sp.want = (int)want, p.sp.places = (int)places;
    // Sequences differ in length, and max_kv is often what they may reach one day:
    // the device divides them by their lengths, up to 64, a lane each. 8 sequences of
    // 2048 keys, one token, 32 and 8 heads of 256: 28 us whether max_kv is 2048 or
    // 131072 (in pieces of max_kv: 27 and 47 us); one of 4096 keys, 4 heads: 20 us (20
    // and 45). 64 sequences of up to 2048 keys, 4 heads over 1: 37 us under either; 65,
    // which are divided by max_kv, 45 and 70.
    if (p.sp.n_split > 1 && a.c.n_seq <= 64) {
        p.sp.planned = 1;
        const int64_t most = (span + p.sp.least - 1) / p.sp.least;
        p.sp.n_split = (int)(most < kMaxSplit ? most : kMaxSplit);
        p.items = all_tiles * p.sp.n_split;
        if (want / a.c.n_kv + all_tiles < p.items) p.items = want / a.c.n_kv + all_tiles;
    }
    p.sp.all_fit = p.items * a.c.n_kv <= kWorkgroups;
    p.sp.items = (int)(p.items < (1 << 30) ? p.items : (1 << 30));
    return p;
}

size_t part_rows(const AttnJob &a, const Plan &p) { return (size_t)p.items * a.c.n_kv * p.sp.rows; }

}  // namespace

int64_t attention_workgroups(const AttnJob &a, int fmt, bool f32) {
    const Plan p = plan_of(a, fmt, f32);
    return p.items * a.c.n_kv;
}

size_t attention_scratch(const AttnJob &a, int fmt, bool f32) {
    const Plan p = plan_of(a, fmt, f32);
    return p.sp.n_split > 1 ? part_rows(a, p) * (a.c.d + 2) * 4 : 0;
}

hipError_t launch_attention(const AttnJob &a, int fmt, bool f32, void *ws, hipStream_t s) {
    Plan p = plan_of(a, fmt, f32);
    if (p.sp.n_split > 1) {
        p.sp.part = static_cast<float *>(ws);
        p.sp.ml = reinterpret_cast<float2 *>(p.sp.part + part_rows(a, p) * a.c.d);
    }
    switch (p.kind) {
        case kFew: launch_few(a, fmt, p.sp, s); break;
        case kTile: launch_tile(a, fmt, p.sp, p.waves, p.tiles, p.exact, s); break;
        default: launch_f32(a, fmt, p.sp, s);
    }
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || p.sp.n_split == 1) return e;
    const dim3 grid((unsigned)(((int64_t)a.c.n_seq * a.c.n_kv * a.max_q * a.group + 3) / 4));
    if (f32)
        hipLaunchKernelGGL((join_kernel<float>), grid, dim3(256), 0, s, a, p.sp);
    else
        hipLaunchKernelGGL((join_kernel<uint16_t>), grid, dim3(256), 0, s, a, p.sp);
    return hipGetLastError();
}

}  // namespace wl
