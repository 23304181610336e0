// Verification of drafted tokens against the target's distribution.
//
// p = softmax(x / t) or the given weights. With a draft's distribution, row r + 1 stays
// if u draft(d) < p(d), and behind the last that stays a token is drawn from
// max(p - draft, 0) (speculative sampling: the answer is distributed as p); without one, a
// token is drawn at every row and followed where it was drafted. A draw is the first x
// whose running sum passes u times the whole.
//
// The answers are whole numbers that a rounding must not decide: powers and sums are
// fp64 throughout (off by about 1e-15 of the whole, where neighbouring borders lie 1e-5
// apart), and the test u draft < p has no division in it.
//
// Bound by memory: every row is read once, in chunks, for its largest entry and the sum
// of its powers relative to that; a chunk of a row (of two, with a draft) is then read
// again to find the token in it. A row has at most 64 chunks, a lane each, so that every
// later step joins them in one wave. Rows start anywhere (an odd vocabulary): they are
// read in aligned groups of 16 bytes, the first and last element by element.
#include "wl_device.h"
#include "wl_serve.h"

namespace wl {

namespace {

constexpr int kThreads = 256, kWaves = kThreads / 64;
constexpr float kNegInf = -__builtin_inff();

struct Stat {
    double sum;   // of the powers relative to `top` (logits), of the weights
    float top;    // largest entry
    int at;       // its first place
};

// e^x for x <= 0: x = n ln 2 + r (ln 2 in two parts), the Taylor series of e^r up to r^12 for
// |r| <= ln 2 / 2 (the next term is below 2^-54), times 2^n.
__device__ __forceinline__ double exp_neg(double x) {
    const double n = rint(x * 1.4426950408889634074);
    const double r = __builtin_fma(-n, 1.9082149292705877000e-10, __builtin_fma(-n, 6.93147180369123816490e-1, x));
    double p = 1.0 / 479001600;
    p = __builtin_fma(p, r, 1.0 / 39916800);
    p = __builtin_fma(p, r, 1.0 / 3628800);
    p = __builtin_fma(p, r, 1.0 / 362880);
    p = __builtin_fma(p, r, 1.0 / 40320);
    p = __builtin_fma(p, r, 1.0 / 5040);
    p = __builtin_fma(p, r, 1.0 / 720);
    p = __builtin_fma(p, r, 1.0 / 120);
    p = __builtin_fma(p, r, 1.0 / 24);
    p = __builtin_fma(p, r, 1.0 / 6);
    p = __builtin_fma(p, r, 0.5);
    p = __builtin_fma(p, r, 1.0);
    p = __builtin_fma(p, r, 1.0);
    return x < -745.0 ? 0.0 : __builtin_amdgcn_ldexp(p, (int)n);
}

// One sequence: rows [q0, q0 + m).
struct Rows {
    int s, q0, m;
};
__device__ __forceinline__ Rows rows_of(const VerifyJob &a, int s) {
    const int q0 = min(max(a.q_start[s], 0), a.T), end = min(max(a.q_start[s + 1], q0), a.T);
    return {s, q0, min(end - q0, a.max_q)};
}
// The sequence of a row; m == 0: none.
__device__ __forceinline__ Rows sequence_of(const VerifyJob &a, int row) {
    int lo = 0, hi = a.n_seq;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (a.q_start[mid] <= row)
            lo = mid;
        else
            hi = mid;
    }
    Rows r = rows_of(a, lo);
    if (row < r.q0 || row >= r.q0 + r.m) r.m = 0;
    return r;
}

__device__ __forceinline__ float temperature_of(const VerifyJob &a, int s) { return a.temperature ? a.temperature[s] : 1.0f; }

__device__ __forceinline__ float value(const uint16_t *p) { return bf16_f(*p); }
__device__ __forceinline__ float value(const float *p) { return *p; }

// A row in groups of 16 bytes: element `at` of group g is g G - shift + at.
template <class E>
struct Row {
    static constexpr int G = 16 / sizeof(E);
    const E *p;
    int shift, n;
    bool logits;
    __device__ __forceinline__ Row(const void *base, int64_t ld, int row, const VerifyJob &a)
        : p(static_cast<const E *>(base) + (int64_t)row * ld), n(a.vocab), logits(a.logits) {
        shift = (int)(((uintptr_t)p & 15) / sizeof(E));
    }
    // What an element counts as: NaN, and what is not there, as nothing.
    __device__ __forceinline__ float counted(float x) const { return logits ? (x == x ? x : kNegInf) : (x > 0.0f ? x : 0.0f); }
    __device__ __forceinline__ float one(int e) const {
        return e >= 0 && e < n ? counted(value(p + e)) : logits ? kNegInf : 0.0f;
    }
    // The group that starts at element e.
    __device__ __forceinline__ void get(int e, float (&v)[G]) const {
        if (e >= 0 && e + G <= n && ((e + shift) & (G - 1)) == 0) {
            const u32x4 w = ldg(reinterpret_cast<const u32x4 *>(p + e));
            const uint32_t c[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                if (sizeof(E) == 2) {
                    v[2 * k] = counted(bf16_f(c[k] & 0xFFFFu));
                    v[2 * k + 1] = counted(__uint_as_float(c[k] & 0xFFFF0000u));
                } else {
                    v[k] = counted(__uint_as_float(c[k]));
                }
            }
        } else {
#pragma unroll
            for (int k = 0; k < G; ++k) v[k] = one(e + k);
        }
    }
};

// e^((x - top) / t), inv = 1 / t; nothing where there is nothing.
__device__ __forceinline__ double power(float x, float top, double inv) {
    return x == kNegInf ? 0.0 : x == top ? 1.0 : exp_neg(((double)x - (double)top) * inv);
}

// 1 / sum; a row of nothing stays nothing.
__device__ __forceinline__ double over(double sum) { return sum > 0.0 ? 1.0 / sum : 0.0; }

// Joined over the lanes of a wave, in every lane.
__device__ __forceinline__ Stat join(Stat v, double inv, bool logits) {
    float top = v.top;
#pragma unroll
    for (int x = 1; x < 64; x <<= 1) top = fmaxf(top, __shfl_xor(top, x));
    int at = v.top == top ? v.at : 0x7FFFFFFF;
    double sum = !logits ? v.sum : v.sum == 0.0 ? 0.0 : v.sum * power(v.top, top, inv);
#pragma unroll
    for (int x = 1; x < 64; x <<= 1) {
        at = min(at, __shfl_xor(at, x));
        sum += __shfl_xor(sum, x);
    }
    return {sum, top, at};
}

constexpr Stat kNothing{0.0, kNegInf, 0x7FFFFFFF};

// The statistics of a row from its chunks': this lane's chunk in `mine`, as part of the whole
// (its sum relative to the row's largest entry).
__device__ __forceinline__ Stat row_stat(const VerifyJob &a, const Stat *stats, int row, double inv, double &mine) {
    const int lane = threadIdx.x & 63;
    const Stat v = lane < a.chunks ? stats[(int64_t)row * a.chunks + lane] : kNothing;
    const Stat r = join(v, inv, a.logits);
    mine = !a.logits ? v.sum : v.sum == 0.0 ? 0.0 : v.sum * power(v.top, r.top, inv);
    return r;
}

// One chunk of a row of the target, or behind them of the draft: its largest entry and its sum.
template <class E>
__global__ __launch_bounds__(kThreads) void stats_kernel(VerifyJob a, Stat *stats) {
    __shared__ Stat lds[kWaves];
    const int64_t unit = blockIdx.x / a.chunks;
    const int chunk = blockIdx.x - (int)unit * a.chunks, row = (int)(unit % a.T);
    const bool of_draft = unit >= a.T;
    const Rows q = sequence_of(a, row);
    if (q.m == 0) return;
    const float t = temperature_of(a, q.s);
    const bool greedy = !(t > 0.0f);
    if (of_draft && (greedy || row == q.q0 + q.m - 1)) return;
    if (!a.logits && a.draft && !greedy) return;   // given weights of single tokens decide
    const double inv = greedy ? 0.0 : 1.0 / (double)t;
    const Row<E> x = of_draft ? Row<E>(a.draft, a.ld_draft, row, a) : Row<E>(a.target, a.ld_target, row, a);
    constexpr int G = Row<E>::G;
    const int first = chunk * a.groups, last = min(first + a.groups, (a.vocab + x.shift + G - 1) / G);
    Stat r = kNothing;
    for (int g = first + threadIdx.x; g < last; g += kThreads) {
        float v[G];
        x.get(g * G - x.shift, v);
        float top = v[0];
#pragma unroll
        for (int k = 1; k < G; ++k) top = fmaxf(top, v[k]);
        if (top > r.top) {
            if (!greedy && a.logits && r.sum != 0.0) r.sum *= power(r.top, top, inv);
            r.top = top;
            int at = 0;
#pragma unroll
            for (int k = G - 1; k >= 0; --k) at = v[k] == top ? k : at;
            r.at = g * G - x.shift + at;
        }
        if (greedy) continue;
#pragma unroll
        for (int k = 0; k < G; ++k) r.sum += a.logits ? power(v[k], r.top, inv) : (double)v[k];
    }
    r = join(r, inv, a.logits);
    if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = r;
    __syncthreads();
    if (threadIdx.x >= 64) return;
    r = join(threadIdx.x < kWaves ? lds[threadIdx.x] : kNothing, inv, a.logits);
    if (threadIdx.x == 0) stats[(of_draft ? (int64_t)a.T * a.chunks : 0) + (int64_t)row * a.chunks + chunk] = r;
}

// p and draft of one row: w(x) = max(p - draft, 0), or p alone.
template <class E>
struct Weights {
    Row<E> p, d;
    float top_p, top_d;
    double inv, one_p, one_d;   // 1 / t; 1 / sum of the powers
    bool both;
    static constexpr int G = Row<E>::G;
    __device__ __forceinline__ double of(const Row<E> &r, float x, float top, double one) const {
        return r.logits ? power(x, top, inv) * one : (double)x;
    }
    __device__ __forceinline__ void get(int e, double (&w)[G]) const {
        float x[G], y[G];
        p.get(e, x);
        if (both) d.get(e, y);
#pragma unroll
        for (int k = 0; k < G; ++k) {
            w[k] = of(p, x[k], top_p, one_p);
            if (both) w[k] = fmax(w[k] - of(d, y[k], top_d, one_d), 0.0);
        }
    }
};

// With a draft's distribution: how far a sequence's rows stay, and for the row behind
// them the sums of a chunk of what a token is drawn from: max(p - draft, 0), and p.
template <class E>
__global__ __launch_bounds__(kThreads) void walk_kernel(VerifyJob a, const Stat *stats, double2 *sums) {
    __shared__ int stays[kVerifyRows];   // whether row i + 1 does
    __shared__ double lds[2][kWaves];
    const int s = blockIdx.x / a.chunks, chunk = blockIdx.x - s * a.chunks;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const Rows q = rows_of(a, s);
    if (q.m == 0) {
        if (chunk == 0 && threadIdx.x == 0) a.n_out[s] = 0;
        return;
    }
    const float t = temperature_of(a, s);
    const bool greedy = !(t > 0.0f);
    const double inv = greedy ? 0.0 : 1.0 / (double)t;
    const Stat *draft_stats = stats + (int64_t)a.T * a.chunks;
    for (int i = wave; i < q.m; i += kWaves) {
        const int row = q.q0 + i, next = i + 1 < q.m ? a.token[row + 1] : -1;
        double mine;
        bool stay = false;
        if (greedy) {
            const Stat r = row_stat(a, stats, row, inv, mine);
            stay = next >= 0 && r.at == next && r.top > (a.logits ? kNegInf : 0.0f);
        } else if (next >= 0 && next < a.vocab) {
            const Row<E> x(a.target, a.ld_target, row, a), y(a.draft, a.ld_draft, row, a);
            const float xp = x.one(next), xd = y.one(next);
            double p = xp, d = xd;
            if (a.logits) {
                const Stat rp = row_stat(a, stats, row, inv, mine), rd = row_stat(a, draft_stats, row, inv, mine);
                p = power(xp, rp.top, inv) * over(rp.sum);
                d = power(xd, rd.top, inv) * over(rd.sum);
            }
            stay = (double)a.u[row].x * d < p;
        }
        if (lane == 0) stays[i] = stay;
    }
    __syncthreads();
    int stop = q.m - 1;
    for (int i = lane; i < q.m; i += 64) {
        const uint64_t no = __ballot(!stays[i]);
        if (no) {
            stop = min(q.m - 1, (i & ~63) + __ffsll((unsigned long long)no) - 1);
            break;
        }
    }
    stop = __builtin_amdgcn_readfirstlane(stop);
    const int row = q.q0 + stop;
    if (chunk == 0) {
        for (int i = threadIdx.x; i < q.m; i += kThreads) {
            if (i != stop) a.out[q.q0 + i] = i < stop ? a.token[q.q0 + i + 1] : -1;
            if (a.path) a.path[q.q0 + i] = i <= stop ? i : -1;
        }
        if (greedy && wave == 0) {
            double mine;
            const Stat r = row_stat(a, stats, row, inv, mine);
            if (lane == 0) a.out[row] = r.top > (a.logits ? kNegInf : 0.0f) ? r.at : -1;
        }
        if (threadIdx.x == 0) {
            a.n_out[s] = stop + 1;
            if (a.len) a.len[s] += stop + 1;
        }
    }
    if (greedy) return;
    Weights<E> w{Row<E>(a.target, a.ld_target, row, a), Row<E>(a.draft, a.ld_draft, row, a), 0, 0, inv, 1, 1, stop + 1 < q.m};
    if (a.logits) {
        double mine;
        const Stat rp = row_stat(a, stats, row, inv, mine);
        w.top_p = rp.top, w.one_p = over(rp.sum);
        if (w.both) {
            const Stat rd = row_stat(a, draft_stats, row, inv, mine);
            w.top_d = rd.top, w.one_d = over(rd.sum);
        }
    }
    constexpr int G = Row<E>::G;
    const int shift = w.p.shift, first = chunk * a.groups, last = min(first + a.groups, (a.vocab + shift + G - 1) / G);
    double left = 0.0, whole = 0.0;
    for (int g = first + threadIdx.x; g < last; g += kThreads) {
        float x[G], y[G];
        w.p.get(g * G - shift, x);
        if (w.both) w.d.get(g * G - shift, y);
#pragma unroll
        for (int k = 0; k < G; ++k) {
            const double p = w.of(w.p, x[k], w.top_p, w.one_p);
            whole += p;
            if (w.both) left += fmax(p - w.of(w.d, y[k], w.top_d, w.one_d), 0.0);
        }
    }
#pragma unroll
    for (int x = 1; x < 64; x <<= 1) left += __shfl_xor(left, x), whole += __shfl_xor(whole, x);
    if (lane == 0) lds[0][wave] = left, lds[1][wave] = whole;
    __syncthreads();
    if (threadIdx.x == 0) {
        left = whole = 0.0;
        for (int i = 0; i < kWaves; ++i) left += lds[0][i], whole += lds[1][i];
        sums[(int64_t)s * a.chunks + chunk] = make_double2(left, whole);
    }
}

// Inclusive running sum over a wave.
__device__ __forceinline__ double wave_scan(double v) {
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int x = 1; x < 64; x <<= 1) {
        const double o = __shfl_up(v, x);
        if (lane >= x) v += o;
    }
    return v;
}

// The first token at which the running sum of weights passes u times the whole, -1 if
// there is none: `mine` is the lane's chunk's part. By a whole workgroup.
template <class E>
__device__ __forceinline__ int draw(const VerifyJob &a, const Weights<E> &w, double mine, float u) {
    __shared__ double part[kWaves];
    __shared__ int found, lasts[kWaves];
    constexpr int G = Row<E>::G;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const double run = wave_scan(mine), whole = __shfl(run, 63), aim = (double)u * whole;
    const uint64_t some = __ballot(mine > 0.0), past = __ballot(run > aim) & some;
    if (!some) return -1;   // the same in every wave
    const int chunk = past ? __ffsll((unsigned long long)past) - 1 : 63 - __clzll((long long)some);
    double base = __shfl(run, chunk > 0 ? chunk - 1 : 0);
    if (chunk == 0) base = 0.0;
    if (threadIdx.x == 0) found = -1;
    const int shift = w.p.shift, first = chunk * a.groups, last = min(first + a.groups, (a.vocab + shift + G - 1) / G);
    int late = -1;   // the last token with any weight
    for (int g0 = first; g0 < last; g0 += kThreads) {
        const int g = g0 + threadIdx.x;
        double v[G], sum = 0.0;
        if (g < last) {
            w.get(g * G - shift, v);
        } else {
#pragma unroll
            for (int k = 0; k < G; ++k) v[k] = 0.0;
        }
#pragma unroll
        for (int k = 0; k < G; ++k) {
            sum += v[k];
            if (v[k] > 0.0) late = g * G - shift + k;
        }
        const double in_wave = wave_scan(sum);
        __syncthreads();   // what the last round wrote has been read
        if (lane == 63) part[wave] = in_wave;
        __syncthreads();
        double before = base, all = base;
        for (int i = 0; i < kWaves; ++i) {
            if (i == wave) before = all;
            all += part[i];
        }
        // The first thread whose sum passes: those behind it see that the one before them has.
        const double up = before + in_wave, ahead = before + (in_wave - sum);
        const uint64_t hits = __ballot(up > aim);
        const bool mine_first = hits && (__ffsll((unsigned long long)hits) - 1) == lane && !(before > aim);
        if (mine_first) {
            double r = ahead;
            int x = -1;
#pragma unroll
            for (int k = 0; k < G; ++k) {
                r += v[k];
                if (x < 0 && r > aim) x = g * G - shift + k;
            }
            found = x >= 0 ? x : late;   // `late` is in this group: its sum is not 0
        }
        __syncthreads();
        if (found >= 0) return found;
        base = all;
    }
    // The chunk's sum passed, in another order of adding, but not the running one.
#pragma unroll
    for (int x = 1; x < 64; x <<= 1) late = max(late, __shfl_xor(late, x));
    if (lane == 0) lasts[wave] = late;
    __syncthreads();
    late = lasts[0];
    for (int i = 1; i < kWaves; ++i) late = max(late, lasts[i]);
    return late;
}

// With a draft's distribution: the token behind those that stay.
template <class E>
__global__ __launch_bounds__(kThreads) void last_kernel(VerifyJob a, const Stat *stats, const double2 *sums) {
    const int s = blockIdx.x, lane = threadIdx.x & 63;
    const Rows q = rows_of(a, s);
    if (q.m == 0) return;
    const float t = temperature_of(a, s);
    if (!(t > 0.0f)) return;
    const double inv = 1.0 / (double)t;
    const int stop = a.n_out[s] - 1, row = q.q0 + stop;
    const double2 v = lane < a.chunks ? sums[(int64_t)s * a.chunks + lane] : make_double2(0.0, 0.0);
    const bool both = stop + 1 < q.m && __ballot(v.x > 0.0) != 0;
    Weights<E> w{Row<E>(a.target, a.ld_target, row, a), Row<E>(a.draft, a.ld_draft, row, a), 0, 0, inv, 1, 1, both};
    if (a.logits) {
        double mine;
        const Stat rp = row_stat(a, stats, row, inv, mine);
        w.top_p = rp.top, w.one_p = over(rp.sum);
        if (both) {
            const Stat rd = row_stat(a, stats + (int64_t)a.T * a.chunks, row, inv, mine);
            w.top_d = rd.top, w.one_d = over(rd.sum);
        }
    }
    const int x = draw(a, w, both ? v.x : v.y, a.u[row].y);
    if (threadIdx.x == 0) a.out[row] = x;
}

// Without: the token of every row.
template <class E>
__global__ __launch_bounds__(kThreads) void tokens_kernel(VerifyJob a, const Stat *stats, int32_t *tokens) {
    const int row = blockIdx.x;
    const Rows q = sequence_of(a, row);
    if (q.m == 0) return;
    const float t = temperature_of(a, q.s);
    const bool greedy = !(t > 0.0f);
    const double inv = greedy ? 0.0 : 1.0 / (double)t;
    double mine;
    const Stat r = row_stat(a, stats, row, inv, mine);
    int x;
    if (greedy) {
        x = r.top > (a.logits ? kNegInf : 0.0f) ? r.at : -1;
    } else {
        const Row<E> p(a.target, a.ld_target, row, a);
        x = draw(a, Weights<E>{p, p, r.top, 0, inv, 1, 1, false}, mine, a.u[row].y);
    }
    if (threadIdx.x == 0) tokens[row] = x;
}

// Without: the rows whose tokens were drawn, one after the other. A wave a sequence.
__global__ __launch_bounds__(64) void follow_kernel(VerifyJob a, const int32_t *tokens) {
    __shared__ int drawn[kVerifyRows], held[kVerifyRows], up[kVerifyRows];
    const int lane = threadIdx.x;
    const Rows q = rows_of(a, blockIdx.x);
    for (int i = lane; i < q.m; i += 64) {
        drawn[i] = tokens[q.q0 + i];
        held[i] = a.token[q.q0 + i];
        up[i] = a.parent ? a.parent[q.q0 + i] : i - 1;
    }
    __syncthreads();
    int at = 0, n = 0;
    while (n < q.m) {
        const int x = drawn[at];
        if (lane == 0) {
            a.out[q.q0 + n] = x;
            if (a.path) a.path[q.q0 + n] = at;
        }
        ++n;
        int next = -1;
        for (int i0 = (at + 1) & ~63; x >= 0 && i0 < q.m; i0 += 64) {
            const int i = i0 + lane;
            const uint64_t hit = __ballot(i > at && i < q.m && held[i] == x && up[i] == at);
            if (hit) {
                next = i0 + __ffsll((unsigned long long)hit) - 1;
                break;
            }
        }
        if (next < 0) break;
        at = next;
    }
    for (int i = n + lane; i < q.m; i += 64) {
        a.out[q.q0 + i] = -1;
        if (a.path) a.path[q.q0 + i] = -1;
    }
    if (lane == 0) {
        a.n_out[blockIdx.x] = n;
        if (a.len) a.len[blockIdx.x] += n;
    }
}

// Workgroups wanted of the launch that reads the rows, and the fewest 16-byte groups of a chunk.
constexpr int64_t kWanted = 4096;
constexpr int kMinGroups = 2 * kThreads;

VerifyJob divided(VerifyJob a, bool f32) {
    const int G = f32 ? 4 : 8;
    const int64_t groups = ((int64_t)a.vocab + 2 * G - 2) / G, rows = (int64_t)a.T * (a.draft ? 2 : 1);
    int64_t chunks = (kWanted + rows - 1) / rows, most = (groups + kMinGroups - 1) / kMinGroups;
    chunks = chunks < most ? chunks : most;
    chunks = chunks > kVerifyChunks ? kVerifyChunks : chunks;
    a.groups = (int)((groups + chunks - 1) / chunks);
    a.chunks = (int)((groups + a.groups - 1) / a.groups);
    return a;
}

size_t stats_bytes(const VerifyJob &a) { return (size_t)a.T * (a.draft ? 2 : 1) * a.chunks * sizeof(Stat); }

template <class E>
hipError_t run(const VerifyJob &a, void *ws, hipStream_t s) {
    Stat *stats = static_cast<Stat *>(ws);
    void *behind = static_cast<char *>(ws) + stats_bytes(a);
    const int64_t rows = (int64_t)a.T * (a.draft ? 2 : 1);
    hipError_t e;
    if (a.logits || !a.draft || a.temperature) {
        hipLaunchKernelGGL((stats_kernel<E>), dim3((unsigned)(rows * a.chunks)), dim3(kThreads), 0, s, a, stats);
        if ((e = hipGetLastError()) != hipSuccess) return e;
    }
    if (a.draft) {
        double2 *sums = static_cast<double2 *>(behind);
        hipLaunchKernelGGL((walk_kernel<E>), dim3((unsigned)(a.n_seq * a.chunks)), dim3(kThreads), 0, s, a, stats, sums);
        if ((e = hipGetLastError()) != hipSuccess) return e;
        hipLaunchKernelGGL((last_kernel<E>), dim3((unsigned)a.n_seq), dim3(kThreads), 0, s, a, stats, sums);
        return hipGetLastError();
    }
    int32_t *tokens = static_cast<int32_t *>(behind);
    hipLaunchKernelGGL((tokens_kernel<E>), dim3((unsigned)a.T), dim3(kThreads), 0, s, a, stats, tokens);
    if ((e = hipGetLastError()) != hipSuccess) return e;
    hipLaunchKernelGGL(follow_kernel, dim3((unsigned)a.n_seq), dim3(64), 0, s, a, tokens);
    return hipGetLastError();
}

}  // namespace

int64_t verify_workgroups(const VerifyJob &a, bool f32) {
    const VerifyJob j = divided(a, f32);
    const int64_t rows = (int64_t)a.T * (a.draft ? 2 : 1) * j.chunks, walks = (int64_t)a.n_seq * j.chunks;
    return rows > walks ? rows : walks;
}

size_t verify_scratch(const VerifyJob &a, bool f32) {
    const VerifyJob j = divided(a, f32);
    return stats_bytes(j) + (a.draft ? (size_t)a.n_seq * j.chunks * sizeof(double2) : (size_t)a.T * 4);
}

hipError_t launch_verify(VerifyJob a, bool f32, void *ws, hipStream_t s) {
    a = divided(a, f32);
    return f32 ? run<float>(a, ws, s) : run<uint16_t>(a, ws, s);
}

}  // namespace wl
