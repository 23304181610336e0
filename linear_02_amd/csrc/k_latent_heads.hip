// Around latent attention: every head's queries into the latent space and outputs out of it in
// bf16, and the join of divided keys.
//
// q'[t][h] = W_h^K^T q[t][h] and o[t][h] = W_h^V o'[t][h]: per head a product with T columns
// and a weight of its own, so both are bound by reading the weights where tokens are few.
// Both are formed transposed on the matrix cores (rows of the weight times tokens): 16
// tokens are the columns of a product, and a lane gets four neighbouring outputs of one token.
//   into   a workgroup takes 128 columns of one head's W^K, which LDS's transposing reads turn
//   out    a workgroup takes 16 tokens of one head: it joins their pieces' outputs into LDS, as
//          a bf16 head and a bf16 remainder (so o' is not rounded), and its four waves share
//          the latent axis of the product, whose partial sums meet in LDS
#include "wl_latent.h"

namespace wl {

namespace {

constexpr int kColumns = 128;        // of the latent axis, a workgroup of the product into it
constexpr int kTokens = 64;          // tokens of a workgroup there

template <class E>
__global__ __launch_bounds__(256) void absorb_kernel(LatentJob a, E *out) {
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
            E *to = out + ((size_t)t * H + h) * (L + R) + L + 8 * c;
            if (sizeof(E) == 2) {
                *reinterpret_cast<u32x4 *>(to) = v;
            } else {
                *reinterpret_cast<f32x4 *>(to) = f32x4{bf16_f(v.x & 0xFFFFu), __uint_as_float(v.x & 0xFFFF0000u), bf16_f(v.y & 0xFFFFu), __uint_as_float(v.y & 0xFFFF0000u)};
                *reinterpret_cast<f32x4 *>(to + 4) = f32x4{bf16_f(v.z & 0xFFFFu), __uint_as_float(v.z & 0xFFFF0000u), bf16_f(v.w & 0xFFFFu), __uint_as_float(v.w & 0xFFFF0000u)};
            }
        }
    }
    wait_loads();
    __syncthreads();
    for (int t = t0; t < t1; t += 16) {
        const bool on = t + n < t1;
        const uint16_t *q = static_cast<const uint16_t *>(a.q) + (size_t)(on ? t + n : t) * a.ldq + (size_t)h * width + 8 * g;
        f32x4 o[2] = {{0, 0, 0, 0}, {0, 0, 0, 0}};
        for (int k = 0; k < N / 32; ++k) {
            const u32x4 qf = ldg(reinterpret_cast<const u32x4 *>(q + 32 * k));
            // Slot (g, e) of the product over 32 rows stands for row 8 g + e in both operands.
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                const int c = 2 * (2 * wave + b) + (n >> 1 & 1), r = 32 * k + 8 * g + (n >> 2);
                auto at = [&](int r) { return lds + r * kColumns * 2 + ((c ^ (r & 7) << 1) << 4) + 8 * (n & 1); };
                const u32x2 x = read_tr16(at(r)), y = read_tr16(at(r + 4));
                o[b] = mfma16(u32x4{x.x, x.y, y.x, y.y}, qf, o[b]);
            }
        }
        if (!on) continue;
        E *to = out + ((size_t)(t + n) * H + h) * (L + R) + l0 + 32 * wave + 4 * g;
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

// Row t's sequence, -1: it has no result. The same in all lanes.
__device__ __forceinline__ int sequence_of(const AttnJob &a, const Pieces &p, int t) {
    int s;
    if (a.c.n_seq <= 64) {
        const uint64_t before = __ballot((int)(threadIdx.x & 63) < a.c.n_seq && p.q_start <= t);
        s = before ? 63 - __clzll((long long)before) : 0;
    } else {
        int lo = 0, hi = a.c.n_seq;
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (a.q_start[mid] <= t)
                lo = mid;
            else
                hi = mid;
        }
        s = lo;
    }
    return __builtin_amdgcn_readfirstlane(s);
}

// The joined output of row t, head h, elements 8 lane .. + 7; false: the row has no result.
// E: of the pieces' outputs.
template <class E>
__device__ __forceinline__ bool joined(const CoreArgs &x, const Pieces &pieces, int t, int h, float (&o)[8]) {
    const AttnJob &a = x.a;
    const Split &sp = x.sp;
    const int lane = threadIdx.x & 63, L = a.c.d;
#pragma unroll
    for (int e = 0; e < 8; ++e) o[e] = 0.0f;
    if (t >= a.T) return false;
    const int s = sequence_of(a, pieces, t);
    const Seq q = seq_of(a, s);
    if (t < q.q0 || t >= q.q0 + q.rows) return false;
    const bool on = 8 * lane < L;
    auto add = [&](const E *p, float w) {
        float v[8];
        query4(p + 8 * lane, v);
        query4(p + 8 * lane + 4, v + 4);
#pragma unroll
        for (int e = 0; e < 8; ++e) o[e] += v[e] * w;
    };
    if (sp.n_split == 1) {
        if (on) add(static_cast<const E *>(a.o) + (size_t)t * a.ldo + (size_t)h * L, 1.0f);
        return true;
    }
    const int r = (t - q.q0) * a.group + h, tile = r / sp.tile_rows;
    int first, n;
    if (sp.planned) {
        n = __builtin_amdgcn_readlane(pieces.n, s);
        first = __builtin_amdgcn_readlane(pieces.first, s) + tile * n;
    } else {
        first = (s * sp.tiles + tile) * sp.n_split, n = sp.n_split;
    }
    const int64_t at = part_row(a, sp, first, 0, tile, r), next = sp.rows;
    float2 v = make_float2(kNegInf, 0.0f);
    if (lane < n) v = sp.ml[at + lane * next];
    float m = v.x;
#pragma unroll
    for (int y = 1; y < 64; y <<= 1) m = fmaxf(m, __shfl_xor(m, y));
    // A piece without visible keys weighs nothing; one whose sum is NaN makes the row NaN.
    const float up = v.x == kNegInf && v.y == 0.0f ? 0.0f : v.y != v.y ? v.y : __builtin_amdgcn_exp2f(v.x - m) * v.y;
    const float l = wave_sum(up), inv = l == 0.0f ? 0.0f : 1.0f / l;
    for (int p = 0; p < n; ++p) {
        const float w = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(up), p)) * inv;
        if (w != 0.0f && on) add(reinterpret_cast<const E *>(sp.part) + (at + p * next) * L, w);
    }
    return true;
}

// On its own (without weights, and in fp32): a wave a row.
template <class E>
__global__ __launch_bounds__(256) void join_kernel(CoreArgs x) {
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    const int64_t w = (int64_t)blockIdx.x * 4 + wave;
    const int t = (int)(w / x.a.n_q), h = (int)(w - (int64_t)t * x.a.n_q);
    if (t >= x.a.T) return;
    float o[8];
    if (!joined<E>(x, pieces_of_call(x.a, x.sp), t, h, o) || 8 * lane >= x.a.c.d) return;
    E *to = static_cast<E *>(x.a.o) + (size_t)t * x.a.ldo + (size_t)h * x.a.c.d + 8 * lane;
    put4(to, o);
    put4(to + 4, o + 4);
}

constexpr int kPitch = kMaxLatent + 8;   // elements of an LDS row of outputs

struct UpArgs {
    LatentJob a;
    CoreArgs x;
    int splits;   // of `value`, a workgroup each
};

__global__ __launch_bounds__(256) void up_kernel(UpArgs u) {
    __shared__ __align__(16) uint16_t head[16][kPitch], rest[16][kPitch];
    __shared__ f32x4 part[4][2][64];
    __shared__ int live[16];
    const LatentJob &a = u.a;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), n = lane & 15, g = lane >> 4;
    const int L = a.a.c.d, N = a.nope, V = a.value, H = a.a.n_q;
    const int unit = blockIdx.x / u.splits, split = blockIdx.x - unit * u.splits, block = unit / H, h = unit - block * H;
    const int t0 = 16 * block;
    const Pieces pieces = pieces_of_call(u.x.a, u.x.sp);
#pragma unroll 1
    for (int i = wave; i < 16; i += 4) {
        float o[8];
        const bool on = joined<uint16_t>(u.x, pieces, t0 + i, h, o);
        if (lane == 0) live[i] = on;
        if (8 * lane >= L) continue;
        uint32_t hi[4], lo[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            hi[e] = pack2(o[2 * e], o[2 * e + 1]);
            lo[e] = pack2(o[2 * e] - bf16_f(hi[e] & 0xFFFFu), o[2 * e + 1] - __uint_as_float(hi[e] & 0xFFFF0000u));
        }
        *reinterpret_cast<u32x4 *>(&head[i][8 * lane]) = u32x4{hi[0], hi[1], hi[2], hi[3]};
        *reinterpret_cast<u32x4 *>(&rest[i][8 * lane]) = u32x4{lo[0], lo[1], lo[2], lo[3]};
    }
    __syncthreads();
    const int per = V / u.splits, mine = L / 4;   // a wave's part of the latent axis
    for (int v0 = split * per; v0 < (split + 1) * per; v0 += 32) {
        const uint16_t *w = static_cast<const uint16_t *>(a.w) + ((size_t)h * (N + V) + N + v0 + n) * L + wave * mine + 8 * g;
        f32x4 o[2] = {{0, 0, 0, 0}, {0, 0, 0, 0}};
#pragma unroll 4
        for (int k = 0; k < mine / 32; ++k) {
            const u32x4 w0 = ldg(reinterpret_cast<const u32x4 *>(w + 32 * k)), w1 = ldg(reinterpret_cast<const u32x4 *>(w + 16 * L + 32 * k));
            const int at = wave * mine + 32 * k + 8 * g;
            const u32x4 x = *reinterpret_cast<const u32x4 *>(&head[n][at]), y = *reinterpret_cast<const u32x4 *>(&rest[n][at]);
            o[0] = mfma16(w0, x, o[0]);
            o[1] = mfma16(w1, x, o[1]);
            o[0] = mfma16(w0, y, o[0]);
            o[1] = mfma16(w1, y, o[1]);
        }
        part[wave][0][lane] = o[0];
        part[wave][1][lane] = o[1];
        __syncthreads();
        if (wave < 2 && live[n]) {   // wave b: rows v0 + 16 b + 4 g .. + 3 of token n
            const f32x4 s = part[0][wave][lane] + part[1][wave][lane] + part[2][wave][lane] + part[3][wave][lane];
            const float v[4] = {s.x, s.y, s.z, s.w};
            put4(static_cast<uint16_t *>(a.o) + (size_t)(t0 + n) * a.ldo + (size_t)h * V + v0 + 16 * wave + 4 * g, v);
        }
        __syncthreads();
    }
}

}  // namespace

void launch_absorb(const LatentJob &a, void *out, bool f32_out, hipStream_t s) {
    const dim3 g((unsigned)((int64_t)(a.a.T + kTokens - 1) / kTokens * a.a.n_q * (a.a.c.d / kColumns))), b(256);
    const size_t lds = (size_t)a.nope * kColumns * 2;
    if (f32_out)
        hipLaunchKernelGGL((absorb_kernel<float>), g, b, lds, s, a, static_cast<float *>(out));
    else
        hipLaunchKernelGGL((absorb_kernel<uint16_t>), g, b, lds, s, a, static_cast<uint16_t *>(out));
}

void launch_up(const LatentJob &a, const CoreArgs &x, hipStream_t s) {
    const int64_t units = (int64_t)(a.a.T + 15) / 16 * a.a.n_q;
    const int splits = units >= 256 ? 1 : a.value / 32;
    hipLaunchKernelGGL(up_kernel, dim3((unsigned)(units * splits)), dim3(256), 0, s, UpArgs{a, x, splits});
}

void launch_join(const CoreArgs &x, bool f32, hipStream_t s) {
    const dim3 g((unsigned)(((int64_t)x.a.T * x.a.n_q + 3) / 4)), b(256);
    if (f32)
        hipLaunchKernelGGL((join_kernel<float>), g, b, 0, s, x);
    else
        hipLaunchKernelGGL((join_kernel<uint16_t>), g, b, 0, s, x);
}

}  // namespace wl
