// Attention over the paged cache:
//   o = sum_j w_j v_j,  w = softmax_j(scale q . k_j) over the keys j a query sees.
#include "wl_attn.h"

namespace wl {

namespace {

// A wave per query row and head.
template <class E, int F>
__global__ __launch_bounds__(256) void attn_rows_kernel(AttnJob a) {
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    const int64_t unit = (int64_t)blockIdx.x * 4 + wave;
    const int t = (int)(unit / a.n_q), h = (int)(unit % a.n_q);
    if (t >= a.T) return;
    int s = -1;
    for (int c = 0; c < a.c.n_seq; ++c)
        if (t >= a.q_start[c] && t < a.q_start[c + 1]) {
            s = c;
            break;
        }
    if (s < 0) return;
    const Seq q = seq_of(a, s);
    const int i = t - q.q0;
    if (i >= q.rows) return;
    float acc[4], m, l;
    one_row<E, F>(a, q, i, h, 0, q.kv, acc, m, l);
    if (4 * lane >= a.c.d) return;
#pragma unroll
    for (int e = 0; e < 4; ++e) acc[e] = l == 0.0f ? 0.0f : acc[e] / l;
    put4(static_cast<E *>(a.o) + (size_t)t * a.ldo + (size_t)h * a.c.d + 4 * lane, acc);
}

template <class E, int F>
void run(const AttnJob &a, hipStream_t s) {
    const int64_t units = (int64_t)a.T * a.n_q;
    hipLaunchKernelGGL((attn_rows_kernel<E, F>), dim3((unsigned)((units + 3) / 4)), dim3(256), 0, s, a);
}

}  // namespace

size_t attention_scratch(const AttnJob &a, int fmt, bool f32) { return 0; }

hipError_t launch_attention(const AttnJob &a, int fmt, bool f32, void *ws, hipStream_t s) {
    switch (fmt) {
        case kFmtBf16: run<uint16_t, kFmtBf16>(a, s); break;
        case kFmtF32: run<float, kFmtF32>(a, s); break;
        case kFmtInt8: f32 ? run<float, kFmtInt8>(a, s) : run<uint16_t, kFmtInt8>(a, s); break;
        default: f32 ? run<float, kFmtE4m3>(a, s) : run<uint16_t, kFmtE4m3>(a, s);
    }
    return hipGetLastError();
}

}  // namespace wl
