// Root-mean-square norm with the residual's addition, out in a float type or
// in int8 codes with a scale per row.
//
// One block takes one row and holds it in registers as fp32 from the only
// read of x and residual to the only write of y and the sum, so the row
// crosses HBM once in each direction; the block-wide reductions (the sum of
// squares, and for int8 max|r*w|) share one barrier.
#include "decoder.h"

namespace wq {
namespace {

template <typename TY>
struct IsCode {
    static constexpr bool value = false;
};
template <>
struct IsCode<int8_t> {
    static constexpr bool value = true;
};

// The larger of two non-negative doubles across lanes m apart.
__device__ __forceinline__ double max_across(double t, int m) { return fmax(t, __shfl_xor(t, m)); }

// VEC elements from p. ANY: p is aligned to its element only and the row may end
// before them (`left` elements are there; the rest are zeros). The hardware
// takes wide loads and stores at any address, so odd rows keep them too: only
// a row's last elements go one by one.
template <typename T, int VEC, bool ANY>
__device__ __forceinline__ void load_row(const T *p, int left, float *v) {
    if constexpr (!ANY) {
        load_vec<T, VEC>(p, v);
    } else {
        typedef T vt __attribute__((ext_vector_type(VEC), aligned(sizeof(T))));
        if (left >= VEC) {
            const vt r = *reinterpret_cast<const vt *>(p);
#pragma unroll
            for (int i = 0; i < VEC; ++i) v[i] = (float)r[i];
        } else {
#pragma unroll
            for (int i = 0; i < VEC; ++i) v[i] = i < left ? (float)p[i] : 0.f;
        }
    }
}

template <typename T, int VEC, bool ANY>
__device__ __forceinline__ void store_row(T *p, int left, const float *v) {
    if constexpr (!ANY) {
        store_vec<T, VEC>(p, v);
    } else {
        typedef T vt __attribute__((ext_vector_type(VEC), aligned(sizeof(T))));
        if (left >= VEC) {
            vt r;
#pragma unroll
            for (int i = 0; i < VEC; ++i) r[i] = (T)v[i];
            *reinterpret_cast<vt *>(p) = r;
        } else {
#pragma unroll
            for (int i = 0; i < VEC; ++i)
                if (i < left) p[i] = (T)v[i];
        }
    }
}

// VEC elements a load, NV loads a thread: n <= blockDim * NV * VEC. w is read
// twice (from L2) rather than held: fewer registers, more rows in flight.
template <typename TX, typename TY, int VEC, int NV, bool ANY>
__global__ __launch_bounds__(1024) void rmsnorm_kernel(const NormArgs a) {
    constexpr bool CODE = IsCode<TY>::value;
    __shared__ float red[16];
    __shared__ double red64[16];
    const long row = blockIdx.x;
    const int tid = threadIdx.x, nt = blockDim.x, n = a.n;
    const TX *x = (const TX *)a.x + row * a.xs;
    const TX *res = a.res ? (const TX *)a.res + row * a.rs : nullptr;
    float v[NV][VEC];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int e = (j * nt + tid) * VEC;
#pragma unroll
        for (int i = 0; i < VEC; ++i) v[j][i] = 0.f;
        if (e < n) load_row<TX, VEC, ANY>(x + e, n - e, v[j]);
    }
    if (res) {
        float r[NV][VEC];
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int e = (j * nt + tid) * VEC;
#pragma unroll
            for (int i = 0; i < VEC; ++i) r[j][i] = 0.f;
            if (e < n) load_row<TX, VEC, ANY>(res + e, n - e, r[j]);
        }
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
            for (int i = 0; i < VEC; ++i) v[j][i] += r[j][i];
    }
    float sq = 0.f;
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int i = 0; i < VEC; ++i) sq = fmaf(v[j][i], v[j][i], sq);
    double top = 0.0; // max |r * w|, in fp64, where the products are exact
    if constexpr (CODE) {
        // rounding to fp32 keeps the order, so a thread's largest is among its products at its fp32 maximum
        float t = 0.f, w[NV][VEC];
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int e = (j * nt + tid) * VEC;
#pragma unroll
            for (int i = 0; i < VEC; ++i) w[j][i] = 0.f;
            if (e < n) load_row<float, VEC, ANY>(a.w + e, n - e, w[j]);
        }
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
            for (int i = 0; i < VEC; ++i) t = fmaxf(t, fabsf(v[j][i] * w[j][i]));
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
            for (int i = 0; i < VEC; ++i)
                if (fabsf(v[j][i] * w[j][i]) == t) top = fmax(top, fabs((double)v[j][i] * (double)w[j][i]));
    }
#pragma unroll
    for (int m = 32; m > 0; m >>= 1) {
        sq += __shfl_xor(sq, m);
        if (CODE) top = max_across(top, m);
    }
    if (nt > 64) {
        if ((tid & 63) == 0) {
            red[tid >> 6] = sq;
            if (CODE) red64[tid >> 6] = top;
        }
        __syncthreads();
        sq = 0.f;
        for (int i = 0; i < nt >> 6; ++i) {
            sq += red[i];
            if (CODE) top = fmax(top, red64[i]);
        }
    }
    const float rstd = 1.0f / sqrtf(sq / (float)n + a.eps);
    if (a.sum) {
        TX *s = (TX *)a.sum + row * a.ss;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int e = (j * nt + tid) * VEC;
            if (e < n) store_row<TX, VEC, ANY>(s + e, n - e, v[j]);
        }
    }
    TY *y = (TY *)a.y + row * a.ys;
    if constexpr (!CODE) {
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int e = (j * nt + tid) * VEC;
            if (e < n) {
                float o[VEC], w[VEC];
                load_row<float, VEC, ANY>(a.w + e, n - e, w);
#pragma unroll
                for (int i = 0; i < VEC; ++i) o[i] = v[j][i] * rstd * w[i];
                store_row<TY, VEC, ANY>(y + e, n - e, o);
            }
        }
    } else {
        const float scale = (float)(top * (double)rstd / 127.0);
        if (tid == 0) a.y_scale[row] = scale;
        // top = 0: a row of zeros. A NaN scale: an infinity or a NaN in the row.
        const bool ok = top > 0.0 && scale == scale;
        const float inv = 127.0f / (float)top;
        const bool range = top > 1e-30 && top < 1e30; // fp32 holds the products and inv
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int e = (j * nt + tid) * VEC;
            if (e < n) {
                float o[VEC], w[VEC];
                load_row<float, VEC, ANY>(a.w + e, n - e, w);
#pragma unroll
                for (int i = 0; i < VEC; ++i) {
                    const float f = v[j][i] * w[i] * inv; // within 127 * 4 * 2^-24 of the quotient
                    float c = rintf(f);
                    if (!range || fabsf(f - c) > 0.4999f) // next to a border: decide in fp64
                        c = (float)rint((double)v[j][i] * (double)w[i] * 127.0 / top);
                    o[i] = ok ? c : 0.f;
                }
                store_row<TY, VEC, ANY>(y + e, n - e, o);
            }
        }
    }
}

template <typename TX, typename TY, int VEC, bool ANY>
hipError_t launch_nv(const NormArgs &a, int cus, hipStream_t st) {
    const int chunks = (a.n + VEC - 1) / VEC;
    // With rows for every CU, blocks of 256 threads (several a CU, a long row
    // in more registers); with few rows, more threads a row: the latency of
    // one row is what counts then.
    const int want = a.rows >= 2 * cus ? 256 : 1024;
    constexpr int LAST = 32768 / 1024 / VEC; // loads a thread at the longest row
    const int sizes[] = {1, 2, 3, 4, 8};
    int nv = 1;
    for (int i = 0; i < 5 && sizes[i] <= LAST; ++i) {
        nv = sizes[i];
        if ((chunks + nv - 1) / nv <= want) break;
    }
    int nt = ((chunks + nv - 1) / nv + 63) / 64 * 64;
    if (nt > 1024) return hipErrorInvalidValue;
    const dim3 grid((unsigned)a.rows), block((unsigned)nt);
    switch (nv) {
#define WQ_NV(N)                                                                                         \
    case N:                                                                                              \
        if constexpr (N <= LAST) hipLaunchKernelGGL((rmsnorm_kernel<TX, TY, VEC, N, ANY>), grid, block, 0, st, a); \
        break;
        WQ_NV(1) WQ_NV(2) WQ_NV(3) WQ_NV(4) WQ_NV(8)
#undef WQ_NV
    default: return hipErrorInvalidValue;
    }
    return hipGetLastError();
}

template <typename TX>
hipError_t launch_x(const NormArgs &a, int y_dtype, bool vec, int cus, hipStream_t st) {
    constexpr int V = sizeof(TX) == 4 ? 4 : 8;
    switch (y_dtype) {
    case WQ_DT_F32: return vec ? launch_nv<TX, float, V, false>(a, cus, st) : launch_nv<TX, float, V, true>(a, cus, st);
    case WQ_DT_BF16: return vec ? launch_nv<TX, bf16, V, false>(a, cus, st) : launch_nv<TX, bf16, V, true>(a, cus, st);
    case WQ_DT_F16: return vec ? launch_nv<TX, f16, V, false>(a, cus, st) : launch_nv<TX, f16, V, true>(a, cus, st);
    default: return vec ? launch_nv<TX, int8_t, V, false>(a, cus, st) : launch_nv<TX, int8_t, V, true>(a, cus, st);
    }
}

} // namespace

hipError_t launch_rmsnorm(const NormArgs &a, int x_dtype, int y_dtype, bool vec, int cus, hipStream_t st) {
    switch (x_dtype) {
    case WQ_DT_F32: return launch_x<float>(a, y_dtype, vec, cus, st);
    case WQ_DT_BF16: return launch_x<bf16>(a, y_dtype, vec, cus, st);
    default: return launch_x<f16>(a, y_dtype, vec, cus, st);
    }
}

} // namespace wq
