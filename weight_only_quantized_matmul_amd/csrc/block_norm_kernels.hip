// The norms after a block and before the next one, with the block's gate and
// the residual between them:
//
//     z = x / sqrt(mean(x^2) + eps) * w_post,   r = residual + alpha * gate * z,
//     y = r / sqrt(mean(r^2) + eps) * w_pre.
//
// One block takes one row and holds it in registers as fp32 from the only read
// of x, gate and residual to the only write of r and y; two block-wide sums.
// Memory bounds it: 8191 rows of 6144 in bf16, 503 MB, 93.6 us, 5.4 TB/s (a
// large copy: 4.8, an elementwise sum 6.2; part of 503 MB stays in the 256 MB
// cache behind the L2 from pass to pass); one row is latency, 3.9 us with two barriers in a row.
#include "rows.h"

namespace wq {
namespace {

// The sum of v over the block's threads. Between two calls with the same `red` stands another barrier.
__device__ __forceinline__ float block_sum(float v, float *red) {
#pragma unroll
    for (int m = 32; m > 0; m >>= 1) v += __shfl_xor(v, m);
    if (blockDim.x > 64) {
        if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
        __syncthreads();
        v = 0.f;
        for (int i = 0; i < (int)blockDim.x >> 6; ++i) v += red[i];
    }
    return v;
}

// What the row's elements are multiplied by, in two factors: 1 / sqrt(mean(v^2) + eps). Squares overflow from elements
// of about 2^56 on and lose those below 2^-63: rows whose sum shows either are summed again after a power of two, the
// first factor, is taken off.
template <int NV, int VEC>
__device__ __forceinline__ float2 norm_factors(const float (&v)[NV][VEC], int n, float eps, float *red, float *red_far) {
    float sq = 0.f;
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int i = 0; i < VEC; ++i) sq = fmaf(v[j][i], v[j][i], sq);
    sq = block_sum(sq, red);
    float ms = sq / (float)n + eps, up = 1.f;
    if (__builtin_amdgcn_readfirstlane(!(ms < INFINITY) || (sq < 0x1p-80f && eps < 0x1p-60f))) { // all threads see the same sum
        up = ms < INFINITY ? 0x1p90f : 0x1p-75f;
        sq = 0.f;
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
            for (int i = 0; i < VEC; ++i) sq = fmaf(v[j][i] * up, v[j][i] * up, sq);
        ms = block_sum(sq, red_far) / (float)n + eps * up * up;
    }
    return make_float2(up, 1.0f / sqrtf(ms));
}

template <typename TX, typename TY, int VEC, int NV, bool ANY>
__global__ __launch_bounds__(1024) void block_norm_kernel(const BlockNormArgs a) {
    __shared__ float red[4][16];
    const int tid = threadIdx.x, nt = blockDim.x, n = a.n;
    const long row = blockIdx.x;
    float v[NV][VEC], r[NV][VEC], f[NV][VEC];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int e = (j * nt + tid) * VEC;
        const auto x = load_row<TX, VEC, ANY>((const TX *)a.x + row * a.xs + e, n - e);
        const auto s = load_row<TX, VEC, ANY>((const TX *)a.res + row * a.rs + e, n - e);
        typename Vec<TX, VEC>::type g;
        if (a.gate) g = load_row<TX, VEC, ANY>((const TX *)a.gate + row * a.gs + e, n - e);
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
            v[j][i] = (float)x[i];
            r[j][i] = (float)s[i];
            f[j][i] = a.gate ? (float)g[i] : 1.f;
        }
    }
    if (a.w_post) {
        const float2 by = norm_factors<NV, VEC>(v, n, a.eps, red[0], red[1]);
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const auto w = load_row<float, VEC, ANY>(a.w_post + (j * nt + tid) * VEC, n - (j * nt + tid) * VEC);
#pragma unroll
            for (int i = 0; i < VEC; ++i) v[j][i] = v[j][i] * by.x * by.y * w[i];
        }
    }
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
            const float z = a.gate ? v[j][i] * f[j][i] : v[j][i];
            v[j][i] = fmaf(a.alpha, z, r[j][i]);
        }
    if (a.sum) {
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int e = (j * nt + tid) * VEC;
            store_row<TX, VEC, ANY>((TX *)a.sum + row * a.ss + e, n - e, v[j]);
        }
    }
    if (!a.y) return;
    const float2 by = norm_factors<NV, VEC>(v, n, a.eps, red[2], red[3]);
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int e = (j * nt + tid) * VEC;
        const auto w = load_row<float, VEC, ANY>(a.w_pre + e, n - e);
        float o[VEC];
#pragma unroll
        for (int i = 0; i < VEC; ++i) o[i] = v[j][i] * by.x * by.y * w[i];
        store_row<TY, VEC, ANY>((TY *)a.y + row * a.ys + e, n - e, o);
    }
}

template <typename TX, typename TY, int VEC, bool ANY>
hipError_t launch_nv(const BlockNormArgs &a, int cus, hipStream_t st) {
    const int chunks = (a.n + VEC - 1) / VEC;
    constexpr int LAST = 32768 / 1024 / VEC; // loads a thread at the longest row
    int nv = 0;
    for (int want = a.rows >= 2 * cus ? 256 : 1024; want <= 1024 && nv == 0; want *= 2)
        for (int k = 1; k <= 4 && nv == 0; ++k)
            if ((chunks + k - 1) / k <= want) nv = k;
    if (nv == 0) nv = LAST;
    const int nt = ((chunks + nv - 1) / nv + 63) / 64 * 64;
    if (nt > 1024) return hipErrorInvalidValue;
    const int piece = (int)(kMaxThreads / nt); // rows a launch
    for (long done = 0; done < a.rows; done += piece) {
        BlockNormArgs b = a;
        b.x = (const TX *)a.x + done * a.xs;
        b.res = (const TX *)a.res + done * a.rs;
        b.gate = a.gate ? (const TX *)a.gate + done * a.gs : nullptr;
        b.y = a.y ? (TY *)a.y + done * a.ys : nullptr;
        b.sum = a.sum ? (TX *)a.sum + done * a.ss : nullptr;
        b.rows = (int)(a.rows - done < piece ? a.rows - done : piece);
        const dim3 grid((unsigned)b.rows), block((unsigned)nt);
        switch (nv) {
#define WQ_NV(N)                                                                                                       \
    case N:                                                                                                            \
        if constexpr (N <= LAST) hipLaunchKernelGGL((block_norm_kernel<TX, TY, VEC, N, ANY>), grid, block, 0, st, b);  \
        break;
            WQ_NV(1) WQ_NV(2) WQ_NV(3) WQ_NV(4) WQ_NV(8)
#undef WQ_NV
        default: return hipErrorInvalidValue;
        }
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

template <typename TX>
hipError_t launch_x(const BlockNormArgs &a, int y_dtype, bool vec, int cus, hipStream_t st) {
    constexpr int V = sizeof(TX) == 4 ? 4 : 8;
    switch (y_dtype) {
    case WQ_DT_F32: return vec ? launch_nv<TX, float, V, false>(a, cus, st) : launch_nv<TX, float, V, true>(a, cus, st);
    case WQ_DT_BF16: return vec ? launch_nv<TX, bf16, V, false>(a, cus, st) : launch_nv<TX, bf16, V, true>(a, cus, st);
    default: return vec ? launch_nv<TX, f16, V, false>(a, cus, st) : launch_nv<TX, f16, V, true>(a, cus, st);
    }
}

} // namespace

hipError_t launch_block_norm(const BlockNormArgs &a, int x_dtype, int y_dtype, bool vec, int cus, hipStream_t st) {
    switch (x_dtype) {
    case WQ_DT_F32: return launch_x<float>(a, y_dtype, vec, cus, st);
    case WQ_DT_BF16: return launch_x<bf16>(a, y_dtype, vec, cus, st);
    default: return launch_x<f16>(a, y_dtype, vec, cus, st);
    }
}

} // namespace wq
