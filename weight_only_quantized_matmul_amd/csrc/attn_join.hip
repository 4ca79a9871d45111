// Attention rows whose positions were split among blocks: the partial results
// become one. Bound by latency: one wave a row reads its splits' references,
// then its partial rows, all in flight together.
#include "attn_common.h"

namespace wq {
namespace {

// Rows whose positions were split: one wave a row joins its splits.
template <typename T, int D>
__global__ __launch_bounds__(256) void attn_join_kernel(const AttnArgs a, const Partials pt, const int R, const int step) {
    const int lane = threadIdx.x & 63;
    const long row = (long)blockIdx.x * 4 + (threadIdx.x >> 6);
    if (row >= (long)a.b.T * a.H) return;
    const int G = a.H / a.c.heads;
    const int tok = (int)(row / a.H), h = (int)(row % a.H);
    const int b = sequence_of<64>(a.b.q_start, a.b.B, tok, lane);
    if (b >= a.b.B) return;
    const int s0 = min(max(a.b.q_start[b], 0), a.b.T), s1 = min(max(a.b.q_start[b + 1], 0), a.b.T);
    if (tok < s0 || tok >= s1) return;
    // the tile that this row was in
    Tile t;
    const int r = (tok - s0) * G + h % G;
    t.n = s1 - s0;
    t.row0 = r / R * R;
    t.rows = min(R, t.n * G - t.row0);
    const int kv = max(a.b.kv_len[b], 0);
    const long held = (long)a.b.width * a.c.page;
    t.past = kv - t.n;
    t.kv = kv < held ? kv : (int)held;
    int lo, hi, x;
    seen_range(t, t.row0 / G, a.causal, a.window, &lo, &x);
    seen_range(t, (t.row0 + t.rows - 1) / G, a.causal, a.window, &x, &hi);
    const Span sp = find_span(step, lo, hi, pt.least, pt.nsplit);
    if (sp.splits <= 1) return;
    const float *ml = pt.ml + row * pt.nsplit * 2;
    float M = -INFINITY;
    for (int s = lane; s < sp.splits; s += 64) M = fmaxf(M, ml[2 * s]);
#pragma unroll
    for (int k = 32; k > 0; k >>= 1) M = fmaxf(M, __shfl_xor(M, k));
    const float base = M == -INFINITY ? 0.f : M;
    float L = 0.f, o[D / 64] = {};
    const float *part = pt.part + row * pt.nsplit * D + lane * (D / 64);
    for (int s = 0; s < sp.splits; ++s) {
        const float f = __builtin_amdgcn_exp2f(ml[2 * s] - base);
        L += ml[2 * s + 1] * f;
        float v[D / 64];
        load_vec<float, D / 64>(part + (long)s * D, v);
#pragma unroll
        for (int k = 0; k < D / 64; ++k) o[k] = fmaf(v[k], f, o[k]);
    }
    const bool none = M == -INFINITY && L == 0.f;
    const float inv = none ? 0.f : 1.0f / L;
    T *dst = (T *)a.o + (long)tok * a.ot + (long)h * a.oh + lane * (D / 64);
#pragma unroll
    for (int k = 0; k < D / 64; ++k) dst[k] = (T)(none ? 0.f : o[k] * inv);
    if (a.lse && lane == 0) a.lse[row] = none ? -INFINITY : (M + __builtin_amdgcn_logf(L)) * kLn2;
}

template <typename T>
hipError_t launch_t(const AttnArgs &a, const AttnPlan &p, const Partials &pt, int dim, hipStream_t st) {
    const long rows = (long)a.b.T * a.H;
    const dim3 grid((unsigned)((rows + 3) / 4)), block(256);
    switch (dim) {
    case 64: hipLaunchKernelGGL((attn_join_kernel<T, 64>), grid, block, 0, st, a, pt, p.rows, p.step); break;
    case 128: hipLaunchKernelGGL((attn_join_kernel<T, 128>), grid, block, 0, st, a, pt, p.rows, p.step); break;
    default: hipLaunchKernelGGL((attn_join_kernel<T, 256>), grid, block, 0, st, a, pt, p.rows, p.step); break;
    }
    return hipGetLastError();
}

} // namespace

hipError_t launch_attn_join(const AttnArgs &a, const AttnPlan &p, const Partials &pt, int dim, int dtype, hipStream_t st) {
    switch (dtype) {
    case WQ_DT_F32: return launch_t<float>(a, p, pt, dim, st);
    case WQ_DT_BF16: return launch_t<bf16>(a, p, pt, dim, st);
    default: return launch_t<f16>(a, p, pt, dim, st);
    }
}

} // namespace wq
