// Attention rows whose positions were split among blocks: the partial results
// become one.
//
// Bound by latency, so nothing waits for what it does not need: four waves take
// a row, each every fourth split (one wave where there are rows for every CU
// and few splits), and the first partial rows are read before it is known how many there are (their places depend on the
// row alone) beside the lengths from which that follows. With the lengths read
// one after another and one wave a row the join of 32 splits took 17 us, now 5 us.
#include "attn_common.h"

namespace wq {
namespace {

// AT: partial rows a wave has in flight; WPR: waves a row (1 or 4)
template <typename T, int D, int AT, int WPR>
__global__ __launch_bounds__(256) void attn_join_kernel(const AttnArgs a, const Partials pt, const int R, const int step) {
    constexpr int E = D / 64; // elements a lane
    __shared__ float sh_o[3][D], sh_l[3];
    const int lane = threadIdx.x & 63, at_wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wave = WPR == 1 ? 0 : at_wave;
    const long row = WPR == 1 ? (long)blockIdx.x * 4 + at_wave : blockIdx.x;
    if (row >= (long)a.b.T * a.H) return;
    const int G = a.H / a.c.heads;
    const int tok = (int)(row / a.H), h = (int)(row % a.H);
    const float *ml = pt.ml + row * pt.nsplit * 2, *part = pt.part + row * pt.nsplit * D + lane * E;
    // splits lane, lane + 64, ... for the references; splits wave, wave + WPR, ... for the rows
    float ref = lane < pt.nsplit ? ml[2 * lane] : -INFINITY;
    float v[AT][E], r[AT], l[AT];
    auto read = [&](int s0) {
#pragma unroll
        for (int k = 0; k < AT; ++k) {
            const int s = min(s0 + WPR * k, pt.nsplit - 1);
            load_vec<float, E>(part + (long)s * D, v[k]);
            r[k] = ml[2 * s];
            l[k] = ml[2 * s + 1];
        }
    };
    read(wave);
    // the tile that this row was in, and how its positions were split
    int seq = -1, s0 = 0, s1 = 0, kv = 0;
    for (int i0 = 0; i0 < a.b.B && seq < 0; i0 += 64) {
        const int i = i0 + lane;
        int x0 = 0, x1 = 0, n = 0;
        if (i < a.b.B) {
            x0 = min(max(a.b.q_start[i], 0), a.b.T);
            x1 = min(max(a.b.q_start[i + 1], 0), a.b.T);
            n = a.b.kv_len[i];
        }
        const uint64_t m = __ballot(x0 <= tok && tok < x1);
        if (m) {
            const int hit = __builtin_ctzll(m);
            seq = i0 + hit;
            s0 = __builtin_amdgcn_readlane(x0, hit);
            s1 = __builtin_amdgcn_readlane(x1, hit);
            kv = max(__builtin_amdgcn_readlane(n, hit), 0);
        }
    }
    if (seq < 0) return;
    Tile t;
    t.n = s1 - s0;
    const int at = (tok - s0) * G + h % G;
    t.row0 = at / R * R;
    t.rows = (int)min((long)R, (long)t.n * G - t.row0);
    const long held = (long)a.b.width * a.c.page;
    t.past = kv - t.n;
    t.kv = kv < held ? kv : (int)held;
    int lo, hi, x;
    seen_range(t, t.row0 / G, a.causal, a.window, &lo, &x);
    seen_range(t, (t.row0 + t.rows - 1) / G, a.causal, a.window, &x, &hi);
    const Span sp = find_span(step, lo, hi, pt.least, pt.nsplit);
    if (sp.splits <= 1) return;
    float M = lane < sp.splits ? ref : -INFINITY;
    for (int s = lane + 64; s < sp.splits; s += 64) M = fmaxf(M, ml[2 * s]);
#pragma unroll
    for (int k = 32; k > 0; k >>= 1) M = fmaxf(M, __shfl_xor(M, k));
    const float base = M == -INFINITY ? 0.f : M;
    float L = 0.f, o[E] = {};
    for (int first = wave; first < sp.splits; first += WPR * AT) {
        if (first != wave) read(first);
#pragma unroll
        for (int k = 0; k < AT; ++k) {
            const bool on = first + WPR * k < sp.splits; // what stands past the splits is not looked at
            const float f = on ? half_way(r[k] - base) : 0.f;
            L = on ? fmaf(l[k] * f, f, L) : L;
#pragma unroll
            for (int e = 0; e < E; ++e) o[e] = on ? fmaf(v[k][e], f * f, o[e]) : o[e];
        }
    }
    if constexpr (WPR > 1) {
        if (wave > 0) {
#pragma unroll
            for (int e = 0; e < E; ++e) sh_o[wave - 1][lane * E + e] = o[e];
            if (lane == 0) sh_l[wave - 1] = L;
        }
        __syncthreads();
        if (wave > 0) return;
#pragma unroll
        for (int w = 0; w < 3; ++w) {
            L += sh_l[w];
#pragma unroll
            for (int e = 0; e < E; ++e) o[e] += sh_o[w][lane * E + e];
        }
    }
    const bool none = M == -INFINITY && L == 0.f;
    const float inv = none ? 0.f : 1.0f / L;
    T *dst = (T *)a.o + (long)tok * a.ot + (long)h * a.oh + lane * E;
#pragma unroll
    for (int e = 0; e < E; ++e) dst[e] = (T)(none ? 0.f : o[e] * inv);
    if (a.lse && lane == 0) a.lse[row] = none ? -INFINITY : (M + __builtin_amdgcn_logf(L)) * kLn2;
}

template <typename T, int D>
hipError_t launch_d(const AttnArgs &a, const AttnPlan &p, const Partials &pt, hipStream_t st) {
    const long rows = (long)a.b.T * a.H;
    if (rows > kMaxThreads / 256) return hipErrorNotSupported;
    const dim3 block(256);
    const JoinPlan j = plan_join(rows, pt.nsplit);
    if (j.waves == 1)
        hipLaunchKernelGGL((attn_join_kernel<T, D, 4, 1>), dim3((unsigned)((rows + 3) / 4)), block, 0, st, a, pt, p.rows, p.step);
    else if (j.at == 2)
        hipLaunchKernelGGL((attn_join_kernel<T, D, 2, 4>), dim3((unsigned)rows), block, 0, st, a, pt, p.rows, p.step);
    else
        hipLaunchKernelGGL((attn_join_kernel<T, D, 8, 4>), dim3((unsigned)rows), block, 0, st, a, pt, p.rows, p.step);
    return hipGetLastError();
}

template <typename T>
hipError_t launch_t(const AttnArgs &a, const AttnPlan &p, const Partials &pt, int dim, hipStream_t st) {
    switch (dim) {
    case 64: return launch_d<T, 64>(a, p, pt, st);
    case 128: return launch_d<T, 128>(a, p, pt, st);
    default: return launch_d<T, 256>(a, p, pt, st);
    }
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
