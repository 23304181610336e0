// The batch of a serving step, planned on the device: pages given and taken back
// over a stack of free ones, rows mapped to sequences and slots.
//
// Everything follows from three running sums over the sequences, each over what the
// one before left in: pages lacking (against the stack's height), rows asked for
// (against T), and, of the sequences served, rows, pages taken and pages given back.
// The k-th page taken is the k-th from the top, and those given back lie on top of
// what is left, so that entry j above the new bottom (n_free - taken + j) is popped
// and pushed by one thread, which reads it before it writes it; a sequence either
// takes or gives, so no table entry has two threads either.
//
// Bound by latency: a workgroup of 1024 threads sums over 1024 sequences at a time,
// with every load issued before the first sum. A small batch is filled by the same
// workgroup out of LDS; a larger one by a second launch out of the workspace.
#include "wl_device.h"
#include "wl_serve.h"

namespace wl {

namespace {

constexpr int kThreads = 1024, kWaves = kThreads / 64;

// Inclusive sum over the workgroup of N values a thread; `all`: the whole. One slot of
// LDS per wave and value; the caller's barrier comes before the next use.
template <int N, class V>
__device__ __forceinline__ void block_scan(V (&v)[N], V (&all)[N], V (*lds)[kWaves]) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
    for (int x = 1; x < 64; x <<= 1)
#pragma unroll
        for (int n = 0; n < N; ++n) {
            const V o = __shfl_up(v[n], x);
            if (lane >= x) v[n] += o;
        }
    if (lane == 63)
#pragma unroll
        for (int n = 0; n < N; ++n) lds[n][wave] = v[n];
    __syncthreads();
#pragma unroll
    for (int n = 0; n < N; ++n) {
        V before = 0, sum = 0;
        for (int w = 0; w < kWaves; ++w) {
            if (w == wave) before = sum;
            sum += lds[n][w];
        }
        v[n] += before;
        all[n] = sum;
    }
}

// The last s of [0, n) with start[s] <= x, where start[0] <= x: the one whose run
// [start[s], start[s + 1]) holds x.
template <class P>
__device__ __forceinline__ int run_of(P start, int n, int x) {
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (start[mid] <= x)
            lo = mid;
        else
            hi = mid;
    }
    return lo;
}

struct Moves {
    int taken, given, n_free;   // n_free: before the call
};

// Entries i, i + step, .. of the rows and of the moved pages. rows, take, give: running
// sums [n_seq + 1]; held: pages of the sequences after the call.
template <class P>
__device__ __forceinline__ void fill(const PlanJob &a, P rows, P take, P give, P held, const Moves &m, int i, int step) {
    const int n_rows = rows[a.n_seq];
    for (int t = i; t < a.T; t += step) {
        int s = -1, slot = -1;
        if (t < n_rows) {
            s = run_of(rows, a.n_seq, t);
            slot = max(a.past[s], 0) + t - rows[s];
        }
        a.seq[t] = s;
        a.slot[t] = slot;
    }
    for (int j = i; j < max(m.taken, m.given); j += step) {
        const int at = m.n_free - m.taken + j;
        const int popped = j < m.taken ? a.free_pages[at] : -1;
        int pushed = -1;
        if (j < m.given) {
            const int s = run_of(give, a.n_seq, j);
            int32_t *entry = a.table + (int64_t)s * a.max_pages + held[s] + j - give[s];
            pushed = *entry;
            *entry = -1;
        }
        if (at < a.n_pages) a.free_pages[at] = pushed;
        if (j < m.taken) {
            const int k = m.taken - 1 - j, s = run_of(take, a.n_seq, k);
            a.table[(int64_t)s * a.max_pages + held[s] - take[s + 1] + k] = popped;
        }
    }
}

// kFill: the whole plan by one workgroup, at most kThreads sequences; else the sums go
// to scratch, [rows unused][take][give] of n_seq + 1 and the moves.
template <bool kFill>
__global__ __launch_bounds__(kThreads) void plan_kernel(PlanJob a, int32_t *scratch) {
    __shared__ int64_t lds64[2][kWaves];
    __shared__ int lds32[3][kWaves];
    constexpr int kKept = kFill ? kThreads + 1 : 1;
    __shared__ int lds_rows[kKept], lds_take[kKept], lds_give[kKept], lds_held[kKept];
    int32_t *take_to = scratch, *give_to = scratch + a.n_seq + 1;
    const int n_free = min(max(*a.n_free, 0), a.n_pages);
    const int64_t page = (int64_t)1 << a.page_shift;
    int64_t lack_sum = 0, ask_sum = 0;
    int sum[3] = {0, 0, 0};
    for (int base = 0; base < a.n_seq; base += kThreads) {
        const int s = base + threadIdx.x;
        const bool on = s < a.n_seq;
        const int64_t past = on ? max(a.past[s], 0) : 0, fresh = on ? max(a.n_new[s], 0) : 0;
        const int held = on ? min(max(a.held[s], 0), a.max_pages) : 0;
        const int64_t want = (past + fresh + page - 1) >> a.page_shift;
        bool ok = on && want <= a.max_pages;
        const int lack = ok ? max((int)want - held, 0) : 0;
        int64_t v[1] = {lack}, all[1];
        block_scan<1>(v, all, lds64);
        ok = ok && (lack == 0 || lack_sum + v[0] <= n_free);
        lack_sum += all[0];
        v[0] = ok ? fresh : 0;
        block_scan<1>(v, all, lds64 + 1);
        ok = ok && (fresh == 0 || ask_sum + v[0] <= a.T);
        ask_sum += all[0];
        const int keys = (int)(ok ? past + fresh : past);
        const int keep = (int)min(((int64_t)keys + page - 1) >> a.page_shift, (int64_t)a.max_pages);
        const int rows = ok ? (int)fresh : 0, take = ok ? lack : 0, give = max(held - keep, 0);
        int w[3] = {rows, take, give}, whole[3];
        block_scan<3>(w, whole, lds32);
        if (on) {
            a.q_start[s + 1] = sum[0] + w[0];
            a.kv_len[s] = keys;
            a.held[s] = held + take - give;
            if (kFill) {
                lds_rows[s + 1] = w[0], lds_take[s + 1] = w[1], lds_give[s + 1] = w[2];
                lds_held[s] = held + take - give;
            } else {
                take_to[s + 1] = sum[1] + w[1], give_to[s + 1] = sum[2] + w[2];
            }
        }
#pragma unroll
        for (int n = 0; n < 3; ++n) sum[n] += whole[n];
        __syncthreads();   // the slots are free again
    }
    const Moves m{sum[1], sum[2], n_free};
    if (threadIdx.x == 0) {
        a.q_start[0] = 0;
        *a.n_free = min(n_free - m.taken + m.given, a.n_pages);
        if (kFill) {
            lds_rows[0] = lds_take[0] = lds_give[0] = 0;
        } else {
            take_to[0] = give_to[0] = 0;
            int32_t *to = scratch + 2 * (a.n_seq + 1);
            to[0] = m.taken, to[1] = m.given, to[2] = n_free;
        }
    }
    if (!kFill) return;
    __syncthreads();
    fill(a, lds_rows, lds_take, lds_give, lds_held, m, threadIdx.x, kThreads);
}

__global__ __launch_bounds__(256) void fill_kernel(PlanJob a, const int32_t *scratch) {
    const int32_t *to = scratch + 2 * (a.n_seq + 1);
    const Moves m{to[0], to[1], to[2]};
    fill(a, (const int32_t *)a.q_start, scratch, scratch + a.n_seq + 1, (const int32_t *)a.held, m,
         (int)(blockIdx.x * 256 + threadIdx.x), (int)(gridDim.x * 256));
}

// Rows of a batch that the planning workgroup fills by itself. 256 sequences, in one launch and in
// two, replayed from a graph: 1024 rows 5.9 and 8.1 us, 4096 rows 8.1 and 8.3 us, 8192 rows 10.9 and
// 8.4 us. (Pages given back may be more, and are not known here: 9000 of 1000 sequences in a call of
// one row take 17 us.)
constexpr int kOneLaunchRows = 4096;

bool one_launch(const PlanJob &a) { return a.n_seq <= kThreads && a.T <= kOneLaunchRows; }

}  // namespace

size_t plan_scratch(const PlanJob &a) { return one_launch(a) ? 0 : ((size_t)2 * (a.n_seq + 1) + 3) * 4; }

hipError_t launch_plan(const PlanJob &a, void *ws, hipStream_t s) {
    if (one_launch(a)) {
        hipLaunchKernelGGL((plan_kernel<true>), dim3(1), dim3(kThreads), 0, s, a, nullptr);
        return hipGetLastError();
    }
    int32_t *scratch = static_cast<int32_t *>(ws);
    hipLaunchKernelGGL((plan_kernel<false>), dim3(1), dim3(kThreads), 0, s, a, scratch);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    // A row a thread: 1000 sequences and 130000 rows 12.7 us with four, 7 us with one.
    const int blocks = a.T / 256 < 64 ? 64 : a.T / 256 > 2048 ? 2048 : a.T / 256;
    hipLaunchKernelGGL(fill_kernel, dim3(blocks), dim3(256), 0, s, a, scratch);
    return hipGetLastError();
}

}  // namespace wl
