// Attention of new tokens over a paged, quantised cache.
//
// One wave takes one (token, query head): a lane scores one position of a
// 64-position tile, the wave keeps the running maximum and sum of the softmax,
// then every lane gathers D/64 elements of the output over the tile.
#include "decoder.h"

namespace wq {
namespace {

template <int KIND>
__device__ __forceinline__ float code_at(const uint8_t *row, int d) {
    if constexpr (KIND == WQ_KV_F16) return (float)((const f16 *)row)[d];
    if constexpr (KIND == WQ_KV_I8) return (float)((const int8_t *)row)[d];
    return (float)((row[d >> 1] >> (4 * (d & 1)) & 15) - 8);
}

template <typename T, int KIND, int D>
__global__ __launch_bounds__(64) void attn_row_kernel(const AttnArgs a) {
    __shared__ float q[D];
    __shared__ float ps[64];
    __shared__ const uint8_t *vrow[64];
    const int lane = threadIdx.x, tok = blockIdx.x, h = blockIdx.y;
    const int kvh = h / (a.H / a.c.heads);
    const int b = sequence_of<64>(a.b.q_start, a.b.B, tok, lane);
    long lo = 0, hi = 0;
    if (b < a.b.B) {
        const int first = a.b.q_start[b], next = a.b.q_start[b + 1];
        if (first <= tok && tok < next) {
            const long kv = a.b.kv_len[b], p = kv - next + tok;
            hi = a.causal && p + 1 < kv ? p + 1 : kv;
            if (a.window > 0 && p + 1 > a.window) lo = p + 1 - a.window;
        }
    }
    for (int d = lane; d < D; d += 64) q[d] = (float)((const T *)a.q)[(long)tok * a.qt + (long)h * a.qh + d] * a.scale;
    __syncthreads();
    float m = -INFINITY, l = 0.f, o[D / 64] = {};
    for (long t0 = lo; t0 < hi; t0 += 64) {
        const long t = t0 + lane;
        int page, slot;
        const bool seen = t < hi && find_row(a.c, a.b, b, t, &page, &slot);
        float s = -INFINITY, vs = 0.f;
        const uint8_t *vr = nullptr;
        if (seen) {
            const long r = page * a.c.rp + kvh * a.c.rh + slot * a.c.rs, f = page * a.c.sp + kvh * a.c.sh + slot * a.c.ss;
            float acc = 0.f;
            for (int d = 0; d < D; ++d) acc = fmaf(q[d], code_at<KIND>(a.c.k + r, d), acc);
            s = acc * a.c.ks[f];
            vs = a.c.vs[f];
            vr = a.c.v + r;
        }
        float top = s;
        for (int x = 32; x > 0; x >>= 1) top = fmaxf(top, __shfl_xor(top, x));
        const float mn = fmaxf(m, top);
        const float base = mn == -INFINITY ? 0.f : mn;
        const float grow = expf(m - base);
        const float p = seen ? expf(s - base) : 0.f;
        float sum = p;
        for (int x = 32; x > 0; x >>= 1) sum += __shfl_xor(sum, x);
        l = l * grow + sum;
        m = mn;
        __syncthreads();
        ps[lane] = p * vs;
        vrow[lane] = vr;
        __syncthreads();
        for (int i = 0; i < D / 64; ++i) {
            float acc = o[i] * grow;
            for (int j = 0; j < 64; ++j)
                if (vrow[j]) acc = fmaf(ps[j], code_at<KIND>(vrow[j], lane + 64 * i), acc);
            o[i] = acc;
        }
    }
    const float inv = l == 0.f ? 0.f : 1.0f / l;
    for (int i = 0; i < D / 64; ++i)
        ((T *)a.o)[(long)tok * a.ot + (long)h * a.oh + lane + 64 * i] = (T)(l == 0.f ? 0.f : o[i] * inv);
    if (a.lse && lane == 0) a.lse[(long)tok * a.H + h] = l == 0.f ? -INFINITY : m + logf(l);
}

template <typename T, int KIND>
hipError_t launch_kind(const AttnArgs &a, int dim, hipStream_t st) {
    const dim3 grid((unsigned)a.b.T, (unsigned)a.H), block(64);
    switch (dim) {
    case 64: hipLaunchKernelGGL((attn_row_kernel<T, KIND, 64>), grid, block, 0, st, a); break;
    case 128: hipLaunchKernelGGL((attn_row_kernel<T, KIND, 128>), grid, block, 0, st, a); break;
    default: hipLaunchKernelGGL((attn_row_kernel<T, KIND, 256>), grid, block, 0, st, a); break;
    }
    return hipGetLastError();
}

template <typename T>
hipError_t launch_t(const AttnArgs &a, int kind, int dim, hipStream_t st) {
    switch (kind) {
    case WQ_KV_F16: return launch_kind<T, WQ_KV_F16>(a, dim, st);
    case WQ_KV_I8: return launch_kind<T, WQ_KV_I8>(a, dim, st);
    default: return launch_kind<T, WQ_KV_I4>(a, dim, st);
    }
}

} // namespace

hipError_t launch_attn(const AttnArgs &a, int kind, int dim, int dtype, hipStream_t st) {
    switch (dtype) {
    case WQ_DT_F32: return launch_t<float>(a, kind, dim, st);
    case WQ_DT_BF16: return launch_t<bf16>(a, kind, dim, st);
    default: return launch_t<f16>(a, kind, dim, st);
    }
}

} // namespace wq
