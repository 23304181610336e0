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
// Bound by the vector units, which take 35 us for the powers of 288 rows of 131072 bf16 logits, 2.2 TB/s:
// every row is read once, in up to 64 chunks of a wave each, for a chunk's largest entry and the sum of its powers relative to that; a chunk
// of a row (of two, with a draft) is then read again to find the token in it. All later steps
// join a row's chunks in one wave, a lane each. Rows start anywhere (an odd vocabulary):
// they are read in aligned groups of 16 bytes, the first and last element by element.
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

// 2^y for y <= 0: y = k / 32 + r with |r| <= 1/64, 2^(k % 32 / 32) from a table, the Taylor series
// of 2^r up to r^5 (the next term is below 2^-48), and k / 32 added to the exponent. k is read
// off the low bits of y + 1.5 2^47, where the step is 1/32.
constexpr double kLog2e = 1.4426950408889634074;
constexpr int kTable = 32;
__device__ __forceinline__ void fill_table(double *table) {
    if (threadIdx.x < kTable) table[threadIdx.x] = exp2((double)threadIdx.x * (1.0 / kTable));
}
// kZero: whether far below 1 it is exactly 0 (else it may be 2^-1000).
template <bool kZero>
__device__ __forceinline__ double power_of_two(double y, const double *table) {
    constexpr double kRound = 0x1.8p47, l = 0.69314718055994530942;   // ln 2
    if (!kZero) y = fmax(y, -1000.0);
    const double t = y + kRound, r = y - (t - kRound);
    const uint32_t k = (uint32_t)__double_as_longlong(t);
    double p = __builtin_fma(l * l * l * l * l / 120, r, l * l * l * l / 24);
    p = __builtin_fma(p, r, l * l * l / 6);
    p = __builtin_fma(p, r, l * l / 2);
    p = __builtin_fma(p, r, l);
    p = __builtin_fma(p, r, 1.0);
    const u32x2 w = __builtin_bit_cast(u32x2, *reinterpret_cast<const double *>(reinterpret_cast<const char *>(table) + (k << 3 & 8 * (kTable - 1))));
    const double v = __builtin_bit_cast(double, u32x2{w.x, w.y + ((k & ~31u) << 15)}) * p;
    return kZero && y < -1000.0 ? 0.0 : v;
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
template <class E, bool kLogits>
struct Row {
    static constexpr int G = 16 / sizeof(E);
    const E *p;
    int shift, n;
    float least;
    __device__ __forceinline__ Row(const void *base, int64_t ld, int row, const VerifyJob &a)
        : p(static_cast<const E *>(base) + (int64_t)row * ld), n(a.vocab) {
        shift = (int)(((uintptr_t)p & 15) / sizeof(E));
        least = kLogits ? kNegInf : 0.0f;
        asm("" : "+s"(least));
    }
    // What an element counts as: NaN, and what is not there, as nothing; infinity as the largest number.
    // (The median of three gives the least of the others for a NaN; the compiler, if it knew that
    // one of them is -inf, would take the minimum with the last instead.)
    __device__ __forceinline__ float counted(float x) const { return __builtin_amdgcn_fmed3f(x, least, 0x1.fffffep127f); }
    __device__ __forceinline__ float one(int e) const {
        return e >= 0 && e < n ? counted(value(p + e)) : kLogits ? kNegInf : 0.0f;
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

// e^((x - top) / t), inv = log2(e) / t, for x <= top and top not -inf. Without branches: a group
// of them is worked on at once, which hides the table's latency.
template <bool kZero>
__device__ __forceinline__ double power(float x, float top, double inv, const double *table) {
    return power_of_two<kZero>(((double)x - (double)top) * inv, table);
}
// log2(e) / t; never 0, so that -inf stays that.
__device__ __forceinline__ double inverse(float t) { return fmax(kLog2e / (double)t, 1e-300); }

// 1 / sum; a row of nothing stays nothing.
__device__ __forceinline__ double over(double sum) { return sum > 0.0 ? 1.0 / sum : 0.0; }

// One step of a join over the 64 lanes: v with that of another lane. 0 .. 3: within 16 lanes.
template <int kStep>
__device__ __forceinline__ uint32_t other(uint32_t v) {
    constexpr int kCtrl = kStep == 0 ? 0xB1 : kStep == 1 ? 0x4E : kStep == 2 ? 0x141 : 0x140;
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, kCtrl, 0xF, 0xF, true);
}
// The two values that a lane and its partner in another row of 16 (step 4), or half (5), hold.
template <int kStep>
__device__ __forceinline__ u32x2 both(uint32_t v) {
    return kStep == 4 ? __builtin_bit_cast(u32x2, __builtin_amdgcn_permlane16_swap(v, v, false, false))
                      : __builtin_bit_cast(u32x2, __builtin_amdgcn_permlane32_swap(v, v, false, false));
}
__device__ __forceinline__ double of_words(uint32_t lo, uint32_t hi) { return __longlong_as_double((long long)((uint64_t)hi << 32 | lo)); }
__device__ __forceinline__ uint32_t low(double v) { return (uint32_t)__double_as_longlong(v); }
__device__ __forceinline__ uint32_t high(double v) { return (uint32_t)((uint64_t)__double_as_longlong(v) >> 32); }

// Sum, maximum and minimum over the lanes of a wave, in every lane.
__device__ __forceinline__ double all_sum(double v) {
    v += of_words(other<0>(low(v)), other<0>(high(v)));
    v += of_words(other<1>(low(v)), other<1>(high(v)));
    v += of_words(other<2>(low(v)), other<2>(high(v)));
    v += of_words(other<3>(low(v)), other<3>(high(v)));
    u32x2 a = both<4>(low(v)), b = both<4>(high(v));
    v = of_words(a.x, b.x) + of_words(a.y, b.y);
    a = both<5>(low(v)), b = both<5>(high(v));
    return of_words(a.x, b.x) + of_words(a.y, b.y);
}
__device__ __forceinline__ float all_max(float v) {
    v = fmaxf(v, __uint_as_float(other<0>(__float_as_uint(v))));
    v = fmaxf(v, __uint_as_float(other<1>(__float_as_uint(v))));
    v = fmaxf(v, __uint_as_float(other<2>(__float_as_uint(v))));
    v = fmaxf(v, __uint_as_float(other<3>(__float_as_uint(v))));
    u32x2 a = both<4>(__float_as_uint(v));
    v = fmaxf(__uint_as_float(a.x), __uint_as_float(a.y));
    a = both<5>(__float_as_uint(v));
    return fmaxf(__uint_as_float(a.x), __uint_as_float(a.y));
}
__device__ __forceinline__ int all_min(int v) {
    v = min(v, (int)other<0>((uint32_t)v));
    v = min(v, (int)other<1>((uint32_t)v));
    v = min(v, (int)other<2>((uint32_t)v));
    v = min(v, (int)other<3>((uint32_t)v));
    u32x2 a = both<4>((uint32_t)v);
    v = min((int)a.x, (int)a.y);
    a = both<5>((uint32_t)v);
    return min((int)a.x, (int)a.y);
}

// Joined over the lanes of a wave, in every lane; part: the lane's own as part of the whole (its
// sum relative to the largest entry of all).
template <bool kLogits>
__device__ __forceinline__ Stat join(Stat v, double inv, const double *table, double &part) {
    const float top = all_max(v.top);
    part = !kLogits ? v.sum : v.sum == 0.0 ? 0.0 : v.sum * power<true>(v.top, top, inv, table);
    return {all_sum(part), top, all_min(v.top == top ? v.at : 0x7FFFFFFF)};
}

constexpr Stat kNothing{0.0, kNegInf, 0x7FFFFFFF};

// The statistics of a row from its chunks': this lane's chunk's part in `mine`.
template <bool kLogits>
__device__ __forceinline__ Stat row_stat(const VerifyJob &a, const Stat *stats, int row, double inv, const double *table, double &mine) {
    const int lane = threadIdx.x & 63;
    return join<kLogits>(lane < a.chunks ? stats[(int64_t)row * a.chunks + lane] : kNothing, inv, table, mine);
}

// A wave a chunk of a row of the target, or behind them of the draft: its largest entry and its sum.
template <class E, bool kLogits>
__global__ __launch_bounds__(kThreads) void stats_kernel(VerifyJob a, Stat *stats) {
    __shared__ double table[kTable];
    const int per = (a.chunks + kWaves - 1) / kWaves, lane = threadIdx.x & 63;
    const int64_t unit = blockIdx.x / per;
    const int chunk = ((int)blockIdx.x - (int)unit * per) * kWaves + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int row = (int)(unit % a.T);
    const bool of_draft = unit >= a.T;
    const Rows q = sequence_of(a, row);
    if (q.m == 0) return;
    const float t = temperature_of(a, q.s);
    const bool greedy = !(t > 0.0f);
    if (of_draft && (greedy || row == q.q0 + q.m - 1)) return;
    if (!kLogits && a.draft && !greedy) return;   // given weights of single tokens decide
    fill_table(table);
    __syncthreads();
    if (chunk >= a.chunks) return;
    const double inv = greedy ? 0.0 : inverse(t);
    const Row<E, kLogits> x = of_draft ? Row<E, kLogits>(a.draft, a.ld_draft, row, a) : Row<E, kLogits>(a.target, a.ld_target, row, a);
    constexpr int G = Row<E, kLogits>::G;
    const int first = chunk * a.groups, last = min(first + a.groups, (a.vocab + x.shift + G - 1) / G);
    Stat r = kNothing;
    for (int g = first + lane; g < last; g += 64) {
        float v[G];
        x.get(g * G - x.shift, v);
        float top = v[0];
#pragma unroll
        for (int k = 1; k < G; ++k) top = fmaxf(top, v[k]);
        if (top > r.top) {
            if (!greedy && kLogits && r.sum != 0.0) r.sum *= power<false>(r.top, top, inv, table);
            r.top = top;
            int at = 0;
#pragma unroll
            for (int k = G - 1; k >= 0; --k) at = v[k] == top ? k : at;
            r.at = g * G - x.shift + at;
        }
        if (greedy || r.top == kNegInf) continue;
        double w[G];
#pragma unroll
        for (int k = 0; k < G; ++k) w[k] = kLogits ? power<false>(v[k], r.top, inv, table) : (double)v[k];
#pragma unroll
        for (int x = 1; x < G; x <<= 1)
#pragma unroll
            for (int k = 0; k < G; k += 2 * x) w[k] += w[k + x];
        r.sum += w[0];
    }
    double part;
    r = join<kLogits>(r, inv, table, part);
    if (lane == 0) stats[(of_draft ? (int64_t)a.T * a.chunks : 0) + (int64_t)row * a.chunks + chunk] = r;
}

// p and draft of one row: w(x) = max(p - draft, 0), or p alone.
template <class E, bool kLogits>
struct Weights {
    Row<E, kLogits> p, d;
    float top_p, top_d;
    double inv, one_p, one_d;   // log2(e) / t; 1 / sum of the powers
    bool both;
    const double *table;
    static constexpr int G = Row<E, kLogits>::G;
    __device__ __forceinline__ double of(const Row<E, kLogits> &r, float x, float top, double one) const {
        return kLogits ? power<true>(x, top, inv, table) * one : (double)x;
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
template <class E, bool kLogits>
__global__ __launch_bounds__(kThreads) void walk_kernel(VerifyJob a, const Stat *stats, double2 *sums) {
    __shared__ int stays[kVerifyRows];   // whether row i + 1 does
    __shared__ double table[kTable];
    const int per = (a.chunks + kWaves - 1) / kWaves, s = blockIdx.x / per, block = blockIdx.x - s * per;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), chunk = block * kWaves + wave;
    const Rows q = rows_of(a, s);
    if (q.m == 0) {
        if (block == 0 && threadIdx.x == 0) a.n_out[s] = 0;
        return;
    }
    const float t = temperature_of(a, s);
    const bool greedy = !(t > 0.0f);
    const double inv = greedy ? 0.0 : inverse(t);
    const Stat *draft_stats = stats + (int64_t)a.T * a.chunks;
    fill_table(table);
    __syncthreads();
    for (int i = wave; i < q.m; i += kWaves) {
        const int row = q.q0 + i, next = i + 1 < q.m ? a.token[row + 1] : -1;
        double mine;
        bool stay = false;
        if (greedy) {
            const Stat r = row_stat<kLogits>(a, stats, row, inv, table, mine);
            stay = next >= 0 && r.at == next && r.top > (kLogits ? kNegInf : 0.0f);
        } else if (next >= 0 && next < a.vocab) {
            const Row<E, kLogits> x(a.target, a.ld_target, row, a), y(a.draft, a.ld_draft, row, a);
            const float xp = x.one(next), xd = y.one(next);
            double p = xp, d = xd;
            if (kLogits) {
                const Stat rp = row_stat<kLogits>(a, stats, row, inv, table, mine), rd = row_stat<kLogits>(a, draft_stats, row, inv, table, mine);
                p = rp.sum > 0.0 ? power<true>(xp, rp.top, inv, table) / rp.sum : 0.0;   // a row of nothing stays nothing
                d = rd.sum > 0.0 ? power<true>(xd, rd.top, inv, table) / rd.sum : 0.0;
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
    if (block == 0) {
        for (int i = threadIdx.x; i < q.m; i += kThreads) {
            if (i != stop) a.out[q.q0 + i] = i < stop ? a.token[q.q0 + i + 1] : -1;
            if (a.path) a.path[q.q0 + i] = i <= stop ? i : -1;
        }
        if (greedy && wave == 0) {
            double mine;
            const Stat r = row_stat<kLogits>(a, stats, row, inv, table, mine);
            if (lane == 0) a.out[row] = r.top > (kLogits ? kNegInf : 0.0f) ? r.at : -1;
        }
        if (threadIdx.x == 0) {
            a.n_out[s] = stop + 1;
            if (a.len) a.len[s] += stop + 1;
        }
    }
    if (greedy || chunk >= a.chunks) return;
    Weights<E, kLogits> w{Row<E, kLogits>(a.target, a.ld_target, row, a), Row<E, kLogits>(a.draft, a.ld_draft, row, a), 0, 0, inv, 1, 1, stop + 1 < q.m, table};
    if (kLogits) {
        double mine;
        const Stat rp = row_stat<kLogits>(a, stats, row, inv, table, mine);
        w.top_p = rp.top, w.one_p = over(rp.sum);
        if (w.both) {
            const Stat rd = row_stat<kLogits>(a, draft_stats, row, inv, table, mine);
            w.top_d = rd.top, w.one_d = over(rd.sum);
        }
    }
    constexpr int G = Row<E, kLogits>::G;
    const int shift = w.p.shift, first = chunk * a.groups, last = min(first + a.groups, (a.vocab + shift + G - 1) / G);
    double left = 0.0, whole = 0.0;
    for (int g = first + lane; g < last; g += 64) {
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
    left = all_sum(left), whole = all_sum(whole);
    if (lane == 0) sums[(int64_t)s * a.chunks + chunk] = make_double2(left, whole);
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
// A scan over lanes adds up every lane's sum in another order, so that a running sum may fall, or pass the
// border at a lane without weight, by a rounding. Only lanes with weight are asked, and the first that passes
// is taken, whatever the ones behind it say.
template <class E, bool kLogits>
__device__ __forceinline__ int draw(const VerifyJob &a, const Weights<E, kLogits> &w, double mine, float u) {
    __shared__ double part[kWaves];
    __shared__ int found[kWaves], lasts[kWaves];
    constexpr int G = Row<E, kLogits>::G;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const double run = wave_scan(mine), whole = __shfl(run, 63), aim = (double)u * whole;
    const uint64_t some = __ballot(mine > 0.0), past = __ballot(run > aim) & some;
    if (!some) return -1;   // the same in every wave
    const int chunk = past ? __ffsll((unsigned long long)past) - 1 : 63 - __clzll((long long)some);
    double base = __shfl(run, chunk > 0 ? chunk - 1 : 0);
    if (chunk == 0) base = 0.0;
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
        const uint64_t hits = __ballot(sum > 0.0 && before + in_wave > aim);
        int x = -1;
        if (hits && lane == __ffsll((unsigned long long)hits) - 1) {
            double r = before + (in_wave - sum);
#pragma unroll
            for (int k = 0; k < G; ++k) {
                r += v[k];
                if (x < 0 && v[k] > 0.0 && r > aim) x = g * G - shift + k;
            }
            if (x < 0) x = late;   // in this group, which has weight
        }
        if (lane == (hits ? __ffsll((unsigned long long)hits) - 1 : 0)) found[wave] = x;
        __syncthreads();
        for (int i = 0; i < kWaves; ++i)
            if (found[i] >= 0) return found[i];
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
template <class E, bool kLogits>
__global__ __launch_bounds__(kThreads) void last_kernel(VerifyJob a, const Stat *stats, const double2 *sums) {
    __shared__ double table[kTable];
    const int s = blockIdx.x, lane = threadIdx.x & 63;
    const Rows q = rows_of(a, s);
    if (q.m == 0) return;
    fill_table(table);
    __syncthreads();
    const float t = temperature_of(a, s);
    if (!(t > 0.0f)) return;
    const double inv = inverse(t);
    const int stop = a.n_out[s] - 1, row = q.q0 + stop;
    const double2 v = lane < a.chunks ? sums[(int64_t)s * a.chunks + lane] : make_double2(0.0, 0.0);
    const bool both = stop + 1 < q.m && __ballot(v.x > 0.0) != 0;
    Weights<E, kLogits> w{Row<E, kLogits>(a.target, a.ld_target, row, a), Row<E, kLogits>(a.draft, a.ld_draft, row, a), 0, 0, inv, 1, 1, both, table};
    if (kLogits) {
        double mine;
        const Stat rp = row_stat<kLogits>(a, stats, row, inv, table, mine);
        w.top_p = rp.top, w.one_p = over(rp.sum);
        if (both) {
            const Stat rd = row_stat<kLogits>(a, stats + (int64_t)a.T * a.chunks, row, inv, table, mine);
            w.top_d = rd.top, w.one_d = over(rd.sum);
        }
    }
    const int x = draw(a, w, both ? v.x : v.y, a.u[row].y);
    if (threadIdx.x == 0) a.out[row] = x;
}

// Without: the token of every row.
template <class E, bool kLogits>
__global__ __launch_bounds__(kThreads) void tokens_kernel(VerifyJob a, const Stat *stats, int32_t *tokens) {
    __shared__ double table[kTable];
    const int row = blockIdx.x;
    const Rows q = sequence_of(a, row);
    if (q.m == 0) return;
    fill_table(table);
    __syncthreads();
    const float t = temperature_of(a, q.s);
    const bool greedy = !(t > 0.0f);
    const double inv = greedy ? 0.0 : inverse(t);
    double mine;
    const Stat r = row_stat<kLogits>(a, stats, row, inv, table, mine);
    int x;
    if (greedy) {
        x = r.top > (kLogits ? kNegInf : 0.0f) ? r.at : -1;
    } else {
        const Row<E, kLogits> p(a.target, a.ld_target, row, a);
        x = draw(a, Weights<E, kLogits>{p, p, r.top, 0, inv, 1, 1, false, table}, mine, a.u[row].y);
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

__global__ __launch_bounds__(kThreads) void no_rows_kernel(VerifyJob a) {
    const int64_t s = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    if (s < a.n_seq) a.n_out[s] = 0;
}

// A row's chunks: a wave each, as many as kWavesWanted of all rows give, with 64 groups of 16 bytes or
// more each (32 chains of 5 rows of 131072 logits, with the draft's, replayed from a graph: 66 us so, 88
// with 4096 waves).
constexpr int64_t kWavesWanted = 16384;
VerifyJob divided(VerifyJob a, bool f32) {
    const int G = f32 ? 4 : 8;
    const int64_t groups = ((int64_t)a.vocab + 2 * G - 2) / G, most = (groups + 63) / 64, rows = (int64_t)a.T * (a.draft ? 2 : 1);
    int64_t chunks = (kWavesWanted + rows - 1) / rows;
    chunks = chunks < 16 ? 16 : chunks > kVerifyChunks ? kVerifyChunks : chunks;   // the fewest keep the second reading short
    if (chunks > most) chunks = most;
    a.groups = (int)((groups + chunks - 1) / chunks);
    a.chunks = (int)((groups + a.groups - 1) / a.groups);
    return a;
}
int workgroups_of_row(const VerifyJob &a) { return (a.chunks + kWaves - 1) / kWaves; }

size_t stats_bytes(const VerifyJob &a) { return (size_t)a.T * (a.draft ? 2 : 1) * a.chunks * sizeof(Stat); }

template <class E, bool kLogits>
hipError_t run(const VerifyJob &a, void *ws, hipStream_t s) {
    Stat *stats = static_cast<Stat *>(ws);
    void *behind = static_cast<char *>(ws) + stats_bytes(a);
    const int64_t rows = (int64_t)a.T * (a.draft ? 2 : 1);
    hipError_t e;
    if (kLogits || !a.draft || a.temperature) {
        hipLaunchKernelGGL((stats_kernel<E, kLogits>), dim3((unsigned)(rows * workgroups_of_row(a))), dim3(kThreads), 0, s, a, stats);
        if ((e = hipGetLastError()) != hipSuccess) return e;
    }
    if (a.draft) {
        double2 *sums = static_cast<double2 *>(behind);
        hipLaunchKernelGGL((walk_kernel<E, kLogits>), dim3((unsigned)(a.n_seq * workgroups_of_row(a))), dim3(kThreads), 0, s, a, stats, sums);
        if ((e = hipGetLastError()) != hipSuccess) return e;
        hipLaunchKernelGGL((last_kernel<E, kLogits>), dim3((unsigned)a.n_seq), dim3(kThreads), 0, s, a, stats, sums);
        return hipGetLastError();
    }
    int32_t *tokens = static_cast<int32_t *>(behind);
    hipLaunchKernelGGL((tokens_kernel<E, kLogits>), dim3((unsigned)a.T), dim3(kThreads), 0, s, a, stats, tokens);
    if ((e = hipGetLastError()) != hipSuccess) return e;
    hipLaunchKernelGGL(follow_kernel, dim3((unsigned)a.n_seq), dim3(64), 0, s, a, tokens);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_verify_no_rows(const VerifyJob &a, hipStream_t s) {
    hipLaunchKernelGGL(no_rows_kernel, dim3((unsigned)(((int64_t)a.n_seq + kThreads - 1) / kThreads)), dim3(kThreads), 0, s, a);
    return hipGetLastError();
}

int64_t verify_workgroups(const VerifyJob &a, bool f32) {
    const VerifyJob j = divided(a, f32);
    const int64_t rows = (int64_t)a.T * (a.draft ? 2 : 1) * workgroups_of_row(j), walks = (int64_t)a.n_seq * workgroups_of_row(j);
    return rows > walks ? rows : walks;
}

size_t verify_scratch(const VerifyJob &a, bool f32) {
    const VerifyJob j = divided(a, f32);
    return stats_bytes(j) + (a.draft ? (size_t)a.n_seq * j.chunks * sizeof(double2) : (size_t)a.T * 4);
}

hipError_t launch_verify(VerifyJob a, bool f32, void *ws, hipStream_t s) {
    a = divided(a, f32);
    if (a.logits) return f32 ? run<float, true>(a, ws, s) : run<uint16_t, true>(a, ws, s);
    return f32 ? run<float, false>(a, ws, s) : run<uint16_t, false>(a, ws, s);
}

}  // namespace wl
