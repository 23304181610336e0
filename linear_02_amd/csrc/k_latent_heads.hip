// Around latent attention: every head's queries into the latent space and outputs out of it, and
// the join of divided keys.
//
// q'[t][h] = W_h^K^T q[t][h] and o[t][h] = W_h^V o'[t][h]: per head a product with T columns
// and a weight of its own, so both are bound by reading the weights where tokens are few.
// In bf16 both are formed transposed on the matrix cores (rows of the weight times tokens): 16
// tokens are the columns of a product, and a lane gets four neighbouring outputs of one token.
//   into   a workgroup takes 128 columns of one head's W^K, which LDS's transposing reads turn
//   out    a workgroup takes 16 tokens of one head: it joins their pieces' outputs, which are fp32, into
//          LDS, as a bf16 head and a bf16 remainder (so o' is not rounded), and its four waves
//          share the latent axis of the product, whose partial sums meet in LDS
// 32 tokens of 128 heads: 10 us into (16.8 MB of weights), 19 out of it, with up to 42 MB of partial outputs.
#include "wl_latent.h"

namespace wl {

namespace {

constexpr int kColumns = 128;        // of the latent axis, a workgroup of the product into it
constexpr int kTokens = 64;          // tokens of a workgroup there

__global__ __launch_bounds__(256) void absorb_kernel(LatentJob a, float *out) {
    extern __shared__ __align__(16) char lds[];   // [nope][kColumns] bf16: piece c of row r at c ^ 2 (r & 7)
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), n = lane & 15, g = lane >> 4;
    const int L = a.a.c.d, N = a.nope, R = a.rot, H = a.a.n_q;
    const int parts = L / kColumns, unit = blockIdx.x / parts, l0 = (blockIdx.x - unit * parts) * kColumns;
    const int block = unit / H, h = unit - block * H, t0 = block * kTokens, t1 = min(t0 + kTokens, a.a.T);
    const char *w = static_cast<const char *>(a.w) + ((size_t)h * (N + a.value) * L + l0) * 2;
    for (int i = wave; i < N / 4; i += 4) {      // 4 rows of 16 pieces a load
        const int r = 4 * i + g;
        load_to_lds(scalar(w), r * L * 2 + ((n ^ (r & 7) << 1) << 4), lds_byte(lds) + i * 1024);
    }
    const int width = N + R;
    // The rotated part, once.
    if (l0 == 0) {
        const int pieces = R / 8;
        for (int i = threadIdx.x; i < (t1 - t0) * pieces; i += 256) {
            const int t = t0 + i / pieces, c = i % pieces;
            const u32x4 v = ldg(reinterpret_cast<const u32x4 *>(static_cast<const uint16_t *>(a.q) + (size_t)t * a.ldq + (size_t)h * width + N + 8 * c));
            float *to = out + ((size_t)t * H + h) * (L + R) + L + 8 * c;
            *reinterpret_cast<f32x4 *>(to) = f32x4{bf16_f(v.x & 0xFFFFu), __uint_as_float(v.x & 0xFFFF0000u), bf16_f(v.y & 0xFFFFu), __uint_as_float(v.y & 0xFFFF0000u)};
            *reinterpret_cast<f32x4 *>(to + 4) = f32x4{bf16_f(v.z & 0xFFFFu), __uint_as_float(v.z & 0xFFFF0000u), bf16_f(v.w & 0xFFFFu), __uint_as_float(v.w & 0xFFFF0000u)};
        }
    }
    auto row = [&](int t) { return static_cast<const uint16_t *>(a.q) + (size_t)min(t + n, t1 - 1) * a.ldq + (size_t)h * width + 8 * g; };
    u32x4 qf[8];   // the widest head has 256 elements
    auto read = [&](int t) {
#pragma unroll
        for (int k = 0; k < 8; ++k)
            if (k < N / 32) qf[k] = ldg(reinterpret_cast<const u32x4 *>(row(t) + 32 * k));
    };
    read(t0);
    wait_loads();
    __syncthreads();
    for (int t = t0; t < t1; t += 16) {
        const bool on = t + n < t1;
        f32x4 o[2] = {{0, 0, 0, 0}, {0, 0, 0, 0}};
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            if (k >= N / 32) break;
            // Slot (g, e) of the product over 32 rows stands for row 8 g + e in both operands.
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                const int c = 2 * (2 * wave + b) + (n >> 1 & 1), r = 32 * k + 8 * g + (n >> 2);
                auto at = [&](int r) { return lds + r * kColumns * 2 + ((c ^ (r & 7) << 1) << 4) + 8 * (n & 1); };
                const u32x2 x = read_tr16(at(r)), y = read_tr16(at(r + 4));
                o[b] = mfma16(u32x4{x.x, x.y, y.x, y.y}, qf[k], o[b]);
            }
        }
        if (t + 16 < t1) read(t + 16);
        if (!on) continue;
        float *to = out + ((size_t)(t + n) * H + h) * (L + R) + l0 + 32 * wave + 4 * g;
#pragma unroll
        for (int b = 0; b < 2; ++b) {
            const float v[4] = {o[b].x, o[b].y, o[b].z, o[b].w};
            put4(to + 16 * b, v);
        }
    }

}

// Which pieces the rows of a sequence have, worked out once per wave.
struct Pieces {
    int first, n, tiles;     // of this lane's sequence (planned)
    int q_start;             // of this lane's sequence
};
__device__ __forceinline__ Pieces pieces_of_call(const AttnJob &a, const Split &sp) {
    const int lane = threadIdx.x & 63;
    Pieces p{0, 0, 0, 0};
    p.q_start = a.q_start[min(lane, a.c.n_seq - 1)];
    if (!sp.planned || sp.n_split == 1) return p;
    const Lengths v = lengths_of(a, sp, lane);
    p.n = pieces_of(v, chunk_of(a, sp, v, lane));
    p.tiles = v.tiles;
    int before = 0, all = p.n * p.tiles;
    for (int j = 0; j < a.c.n_seq; ++j) {
        if (j == lane) p.first = before;
        before += __builtin_amdgcn_readlane(all, j);
    }
    return p;
}

// Row t's sequence; t and it are the same in the 16 lanes of a group.
__device__ __forceinline__ int sequence_of(const AttnJob &a, const Pieces &p, int t) {
    const int lane = threadIdx.x & 63;
    if (a.c.n_seq <= 64) {
        int s = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int tj = __builtin_amdgcn_readlane(t, 16 * j);
            const uint64_t before = __ballot(lane < a.c.n_seq && p.q_start <= tj);
            s = lane >> 4 == j && before ? 63 - __clzll((long long)before) : s;
        }
        return s;
    }
    int lo = 0, hi = a.c.n_seq;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (a.q_start[mid] <= t)
            lo = mid;
        else
            hi = mid;
    }
    return lo;
}

// The joined output of row t, head h, the same in the 16 lanes of a group: lane n of it gets
// elements 128 c + 8 n .. + 7. false: the row has no result. A wave joins four rows at once with
// several pieces of each on their way: a row after the other, a piece after the other, it waited
// for each (31 us instead of 18 for 32 tokens of 128 heads with about 8 pieces each).
template <int L>
__device__ __forceinline__ bool joined(const CoreArgs &x, const Pieces &pieces, int t, int h, float (&o)[L / 128][8]) {
    constexpr int kParts = L / 128, kAtOnce = 2;
    const AttnJob &a = x.a;
    const Split &sp = x.sp;
    const int lane = threadIdx.x & 63, n = lane & 15;
#pragma unroll
    for (int c = 0; c < kParts; ++c)
#pragma unroll
        for (int e = 0; e < 8; ++e) o[c][e] = 0.0f;
    const int s = sequence_of(a, pieces, t);
    const Seq q = seq_of(a, s);
    const bool on = t < a.T && t >= q.q0 && t < q.q0 + q.rows;
    if (sp.n_split == 1) {
        const float *p = static_cast<const float *>(a.o) + (on ? (size_t)t * a.ldo + (size_t)h * L : 0) + 8 * n;
#pragma unroll
        for (int c = 0; c < kParts; ++c) {
            query4(p + 128 * c, o[c]);
            query4(p + 128 * c + 4, o[c] + 4);
        }
        return on;
    }
    const int r = on ? (t - q.q0) * a.group + h : 0, tile = r / sp.tile_rows;
    const int per = __shfl(pieces.n, s), before = __shfl(pieces.first, s);
    const int first = !on ? 0 : sp.planned ? before + tile * per : (s * sp.tiles + tile) * sp.n_split;
    const int have = !on ? 0 : sp.planned ? per : sp.n_split;
    const int64_t at = part_row(a, sp, first, 0, tile, r), next = sp.rows;
    static_assert(kMaxSplit <= 64, "four pieces a lane");
    float2 v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = n + 16 * i < have ? sp.ml[at + (n + 16 * i) * next] : make_float2(kNegInf, 0.0f);
    float m = fmaxf(fmaxf(v[0].x, v[1].x), fmaxf(v[2].x, v[3].x));
#pragma unroll
    for (int y = 1; y < 16; y <<= 1) m = fmaxf(m, __shfl_xor(m, y));
    // A piece without visible keys weighs nothing; one whose sum is NaN makes the row NaN.
    float up[4], l = 0.0f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        up[i] = v[i].x == kNegInf && v[i].y == 0.0f ? 0.0f : v[i].y != v[i].y ? v[i].y : __builtin_amdgcn_exp2f(v[i].x - m) * v[i].y;
        l += up[i];
    }
    int most = have;
#pragma unroll
    for (int y = 1; y < 16; y <<= 1) l += __shfl_xor(l, y);
#pragma unroll
    for (int y = 16; y < 64; y <<= 1) most = max(most, __shfl_xor(most, y));
    most = __builtin_amdgcn_readfirstlane(most);
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
    const float *part = sp.part + at * L + 8 * n;
    for (int p0 = 0; p0 < most; p0 += kAtOnce) {
        f32x4 raw[kAtOnce][kParts][2];
#pragma unroll
        for (int j = 0; j < kAtOnce; ++j)
#pragma unroll
            for (int c = 0; c < kParts; ++c)
#pragma unroll
                for (int i = 0; i < 2; ++i)   // behind a row's pieces: its first one again, which weighs nothing then
                    raw[j][c][i] = ldg(reinterpret_cast<const f32x4 *>(part + (p0 + j < have ? p0 + j : 0) * next * L + 128 * c) + i);
        const int turn = p0 >> 4;
        const float mine = turn == 0 ? up[0] : turn == 1 ? up[1] : turn == 2 ? up[2] : up[3];
#pragma unroll
        for (int j = 0; j < kAtOnce; ++j) {
            const float got = __shfl(mine, (lane & 48) | ((p0 + j) & 15)) * inv, w = p0 + j < have ? got : 0.0f;
#pragma unroll
            for (int c = 0; c < kParts; ++c)
#pragma unroll
                for (int e = 0; e < 8; ++e) o[c][e] = w == 0.0f ? o[c][e] : __builtin_fmaf(raw[j][c][e >> 2][e & 3], w, o[c][e]);
        }
    }
    return on;
}

// On its own (without weights): 16 lanes a row.
template <class E, int L>
__global__ __launch_bounds__(256) void join_kernel(CoreArgs x) {
    const int n = threadIdx.x & 15;
    const int64_t w = (int64_t)blockIdx.x * 16 + (threadIdx.x >> 4);
    const int t = (int)(w / x.a.n_q), h = (int)(w - (int64_t)t * x.a.n_q);
    float o[L / 128][8];
    if (!joined<L>(x, pieces_of_call(x.a, x.sp), t, h, o)) return;
    E *to = static_cast<E *>(x.a.o) + (size_t)t * x.a.ldo + (size_t)h * L + 8 * n;
#pragma unroll
    for (int c = 0; c < L / 128; ++c) {
        put4(to + 128 * c, o[c]);
        put4(to + 128 * c + 4, o[c] + 4);
    }
}

struct UpArgs {
    LatentJob a;
    CoreArgs x;
    int splits;   // of `value`, a workgroup each
};

template <int L>
__global__ __launch_bounds__(256) void up_kernel(UpArgs u) {
    constexpr int kPitch = L + 8;   // elements of an LDS row of outputs
    constexpr int kOwn = L / 4;     // a wave's part of the latent axis
    __shared__ __align__(16) uint16_t head[16][kPitch], rest[16][kPitch];
    __shared__ f32x4 part[2][4][2][64];
    __shared__ int live[16];
    const LatentJob &a = u.a;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), n = lane & 15, g = lane >> 4;
    const int N = a.nope, V = a.value, H = a.a.n_q;
    const int unit = blockIdx.x / u.splits, split = blockIdx.x - unit * u.splits, block = unit / H, h = unit - block * H;
    const int t0 = 16 * block;
    const int per = V / u.splits, v_from = split * per, v_to = v_from + per;
    const uint16_t *w = static_cast<const uint16_t *>(a.w) + ((size_t)h * (N + V) + N + n) * L + wave * kOwn + 8 * g;
    u32x4 ahead[2][kOwn / 32];
    auto read = [&](int v0) {
#pragma unroll
        for (int b = 0; b < 2; ++b)
#pragma unroll
            for (int k = 0; k < kOwn / 32; ++k) ahead[b][k] = ldg(reinterpret_cast<const u32x4 *>(w + (size_t)(v0 + 16 * b) * L + 32 * k));
    };
    read(v_from);   // come in while the pieces are joined
    {
        const int i = 4 * wave + g;
        float o[L / 128][8];
        const bool on = joined<L>(u.x, pieces_of_call(u.x.a, u.x.sp), t0 + i, h, o);
        if (n == 0) live[i] = on;
#pragma unroll
        for (int c = 0; c < L / 128; ++c) {
            uint32_t hi[4], lo[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                hi[e] = pack2(o[c][2 * e], o[c][2 * e + 1]);
                lo[e] = pack2(o[c][2 * e] - bf16_f(hi[e] & 0xFFFFu), o[c][2 * e + 1] - __uint_as_float(hi[e] & 0xFFFF0000u));
            }
            *reinterpret_cast<u32x4 *>(&head[i][128 * c + 8 * n]) = u32x4{hi[0], hi[1], hi[2], hi[3]};
            *reinterpret_cast<u32x4 *>(&rest[i][128 * c + 8 * n]) = u32x4{lo[0], lo[1], lo[2], lo[3]};
        }
    }
    __syncthreads();
    u32x4 x[kOwn / 32], y[kOwn / 32];
#pragma unroll
    for (int k = 0; k < kOwn / 32; ++k) {
        x[k] = *reinterpret_cast<const u32x4 *>(&head[n][wave * kOwn + 32 * k + 8 * g]);
        y[k] = *reinterpret_cast<const u32x4 *>(&rest[n][wave * kOwn + 32 * k + 8 * g]);
    }
    int turn = 0;
    for (int v0 = v_from; v0 < v_to; v0 += 32, turn ^= 1) {
        u32x4 now[2][kOwn / 32];
#pragma unroll
        for (int b = 0; b < 2; ++b)
#pragma unroll
            for (int k = 0; k < kOwn / 32; ++k) now[b][k] = ahead[b][k];
        if (v0 + 32 < v_to) read(v0 + 32);
#pragma unroll
        for (int b = 0; b < 2; ++b) {
            f32x4 o{0, 0, 0, 0};
#pragma unroll
            for (int k = 0; k < kOwn / 32; ++k) {
                o = mfma16(now[b][k], x[k], o);
                o = mfma16(now[b][k], y[k], o);
            }
            part[turn][wave][b][lane] = o;
        }
        __syncthreads();
        if (wave < 2 && live[n]) {   // wave b: rows v0 + 16 b + 4 g .. + 3 of token n
            const f32x4 s = part[turn][0][wave][lane] + part[turn][1][wave][lane] + part[turn][2][wave][lane] + part[turn][3][wave][lane];
            const float v[4] = {s.x, s.y, s.z, s.w};
            put4(static_cast<uint16_t *>(a.o) + (size_t)(t0 + n) * a.ldo + (size_t)h * V + v0 + 16 * wave + 4 * g, v);
        }
    }
}

constexpr int kTokensF32 = 8;   // of a workgroup of the product into the latent space in fp32

// q' = W^K^T q in fp32: 64 columns of one head's latent axis, each wave a quarter of the sum's rows.
__global__ __launch_bounds__(256) void absorb_f32_kernel(LatentJob a, float *out) {
    __shared__ float qs[256][kTokensF32], part[4][kTokensF32][64];
    const int H = a.a.n_q, L = a.a.c.d, N = a.nope, R = a.rot;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int parts = L / 64, unit = blockIdx.x / parts, l0 = (blockIdx.x - unit * parts) * 64;
    const int block = unit / H, h = unit - block * H, t0 = block * kTokensF32, n_t = min(kTokensF32, a.a.T - t0);
    const float *q = static_cast<const float *>(a.q) + (size_t)t0 * a.ldq + (size_t)h * (N + R);
    for (int i = threadIdx.x; i < kTokensF32 * (N + R); i += 256) {
        const int t = i / (N + R), e = i - t * (N + R);
        const float v = t < n_t ? q[(size_t)t * a.ldq + e] : 0.0f;
        if (e < N)
            qs[e][t] = v;
        else if (l0 == 0 && t < n_t)
            out[((size_t)(t0 + t) * H + h) * (L + R) + L + e - N] = v;
    }
    __syncthreads();
    const int own = N / 4;
    const float *w = static_cast<const float *>(a.w) + ((size_t)h * (N + a.value) + wave * own) * L + l0 + lane;
    float s[kTokensF32] = {};
#pragma unroll 8
    for (int n = 0; n < own; ++n) {
        const float x = ldg(w + (size_t)n * L);
#pragma unroll
        for (int t = 0; t < kTokensF32; ++t) s[t] += qs[wave * own + n][t] * x;
    }
#pragma unroll
    for (int t = 0; t < kTokensF32; ++t) part[wave][t][lane] = s[t];
    __syncthreads();
    for (int t = wave; t < n_t; t += 4)
        out[((size_t)(t0 + t) * H + h) * (L + R) + l0 + lane] = part[0][t][lane] + part[1][t][lane] + part[2][t][lane] + part[3][t][lane];
}

// o = W^V o' in fp32: 16 tokens of one head, 16 rows of the weight at a time with 16 lanes each.
template <int L>
__global__ __launch_bounds__(256) void up_f32_kernel(UpArgs u) {
    __shared__ __align__(16) float xs[16][L];
    __shared__ int live[16];
    const LatentJob &a = u.a;
    const int n = threadIdx.x & 15, i = threadIdx.x >> 4;
    const int N = a.nope, V = a.value, H = a.a.n_q;
    const int unit = blockIdx.x / u.splits, split = blockIdx.x - unit * u.splits, block = unit / H, h = unit - block * H;
    const int t0 = 16 * block, per = V / u.splits, v_from = split * per, v_to = v_from + per;
    {
        float o[L / 128][8];
        const bool on = joined<L>(u.x, pieces_of_call(u.x.a, u.x.sp), t0 + i, h, o);
        if (n == 0) live[i] = on;
#pragma unroll
        for (int c = 0; c < L / 128; ++c) {
            *reinterpret_cast<f32x4 *>(&xs[i][128 * c + 8 * n]) = f32x4{o[c][0], o[c][1], o[c][2], o[c][3]};
            *reinterpret_cast<f32x4 *>(&xs[i][128 * c + 8 * n + 4]) = f32x4{o[c][4], o[c][5], o[c][6], o[c][7]};
        }
    }
    __syncthreads();
    for (int v0 = v_from; v0 < v_to; v0 += 16) {
        asm volatile("" ::: "memory");   // outputs are read from LDS again: they would not fit the registers
        const float *w = static_cast<const float *>(a.w) + ((size_t)h * (N + V) + N + v0 + i) * L + 4 * n;
        f32x4 x[L / 64];
#pragma unroll
        for (int k = 0; k < L / 64; ++k) x[k] = ldg(reinterpret_cast<const f32x4 *>(w + 64 * k));
        float s[16];
#pragma unroll
        for (int t = 0; t < 16; ++t) {
            s[t] = 0.0f;
#pragma unroll
            for (int k = 0; k < L / 64; ++k) {
                const f32x4 y = *reinterpret_cast<const f32x4 *>(&xs[t][64 * k + 4 * n]);
                s[t] += x[k].x * y.x + x[k].y * y.y + x[k].z * y.z + x[k].w * y.w;
            }
        }
        // Summed over the 16 lanes, token n's in lane n.
#pragma unroll
        for (int y = 8; y; y >>= 1)
#pragma unroll
            for (int t = 0; t < y; ++t) {
                const float keep = n & y ? s[t + y] : s[t], give = n & y ? s[t] : s[t + y];
                s[t] = keep + __shfl_xor(give, y);
            }
        if (live[n]) static_cast<float *>(a.o)[(size_t)(t0 + n) * a.ldo + (size_t)h * V + v0 + i] = s[0];
    }
}

}  // namespace

void launch_absorb(const LatentJob &a, float *out, hipStream_t s) {
    const dim3 g((unsigned)((int64_t)(a.a.T + kTokens - 1) / kTokens * a.a.n_q * (a.a.c.d / kColumns))), b(256);
    const size_t lds = (size_t)a.nope * kColumns * 2;
    hipLaunchKernelGGL(absorb_kernel, g, b, lds, s, a, out);
}

// Fewer units of 16 tokens and a head than this are divided over `value`, and every part joins
// their pieces again: 16 units divided and not, the whole call, 24.9 and 27.6 us (one token of 16
// heads), 37.0 and 48.7 us in fp32; 224 units of about 10 pieces, this kernel, 28 and 15 us.
constexpr int64_t kUnits = 128;

void launch_up(const LatentJob &a, const CoreArgs &x, bool f32, hipStream_t s) {
    const int64_t units = (int64_t)(a.a.T + 15) / 16 * a.a.n_q;
    const int splits = units >= kUnits ? 1 : a.value / (f32 ? 16 : 32);
    const dim3 g((unsigned)(units * splits)), b(256);
    const UpArgs u{a, x, splits};
    if (f32) {
        switch (a.a.c.d) {
            case 128: hipLaunchKernelGGL((up_f32_kernel<128>), g, b, 0, s, u); break;
            case 256: hipLaunchKernelGGL((up_f32_kernel<256>), g, b, 0, s, u); break;
            default: hipLaunchKernelGGL((up_f32_kernel<512>), g, b, 0, s, u);
        }
        return;
    }
    switch (a.a.c.d) {
        case 128: hipLaunchKernelGGL((up_kernel<128>), g, b, 0, s, u); break;
        case 256: hipLaunchKernelGGL((up_kernel<256>), g, b, 0, s, u); break;
        default: hipLaunchKernelGGL((up_kernel<512>), g, b, 0, s, u);
    }
}

void launch_absorb_f32(const LatentJob &a, float *out, hipStream_t s) {
    const dim3 g((unsigned)((int64_t)(a.a.T + kTokensF32 - 1) / kTokensF32 * a.a.n_q * (a.a.c.d / 64)));
    hipLaunchKernelGGL(absorb_f32_kernel, g, dim3(256), 0, s, a, out);
}

template <class E>
static void join(const CoreArgs &x, hipStream_t s) {
    const dim3 g((unsigned)(((int64_t)x.a.T * x.a.n_q + 15) / 16)), b(256);
    switch (x.a.c.d) {
        case 128: hipLaunchKernelGGL((join_kernel<E, 128>), g, b, 0, s, x); break;
        case 256: hipLaunchKernelGGL((join_kernel<E, 256>), g, b, 0, s, x); break;
        default: hipLaunchKernelGGL((join_kernel<E, 512>), g, b, 0, s, x);
    }
}

void launch_join(const CoreArgs &x, bool f32, hipStream_t s) {
    if (f32)
        join<float>(x, s);
    else
        join<uint16_t>(x, s);
}

}  // namespace wl
