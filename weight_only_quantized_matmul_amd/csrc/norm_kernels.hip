// Root-mean-square norm with the residual's addition, out in a float type or
// in int8 codes with a scale per row.
//
// One block takes one row and holds it in registers as fp32 from the only
// read of x and residual to the only write of y and the sum, so the row
// crosses HBM once in each direction; the block-wide reductions (the sum of
// squares, and for int8 max|r*w|) share one barrier.
//
// Bound by HBM at many rows: 8191 x 6144, bf16 and residual in, sum and int8
// out, 352 MB in 77 us (4.6 TB/s; a device copy reaches 5.46). A block there
// walks rows (one row a block, w read again for each: 94 us). One row of 6144
// in f32 takes 3.4 us, latency. Rows that leave fp32's range when squared pay a
// second reduction.
#include "rows.h"

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

// VEC elements a load, NV loads a thread: n <= blockDim * NV * VEC. LOOP: a
// block takes every gridDim-th row, with w in registers and the next row's
// loads in flight while it reduces and writes one.
template <typename TX, typename TY, int VEC, int NV, bool ANY, bool LOOP>
__global__ __launch_bounds__(LOOP ? 512 : 1024) void rmsnorm_kernel(const NormArgs a) {
    constexpr bool CODE = IsCode<TY>::value;
    __shared__ float red[2][16], red_far[16]; // red: of odd and even rows, one barrier a row
    __shared__ double red64[2][16];
    const int tid = threadIdx.x, nt = blockDim.x, n = a.n;
    typename Vec<TX, VEC>::type nx[NV], nr[NV];
    auto fetch = [&](long row) {
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int e = (j * nt + tid) * VEC;
            nx[j] = load_row<TX, VEC, ANY>((const TX *)a.x + row * a.xs + e, n - e);
            if (a.res) nr[j] = load_row<TX, VEC, ANY>((const TX *)a.res + row * a.rs + e, n - e);
        }
    };
    fetch(blockIdx.x);
    float w[NV][VEC];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const auto x = load_row<float, VEC, ANY>(a.w + (j * nt + tid) * VEC, n - (j * nt + tid) * VEC);
#pragma unroll
        for (int i = 0; i < VEC; ++i) w[j][i] = x[i];
    }
    int buf = 0;
    for (long row = blockIdx.x; row < a.rows; row += gridDim.x, buf ^= 1) {
        float v[NV][VEC];
        // w is the same in every round, but its fp64 forms are not to be kept: they would take twice its registers
        if (CODE && LOOP) {
#pragma unroll
            for (int j = 0; j < NV; ++j)
#pragma unroll
                for (int i = 0; i < VEC; ++i) asm volatile("" : "+v"(w[j][i]));
        }
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
            for (int i = 0; i < VEC; ++i) v[j][i] = a.res ? (float)nx[j][i] + (float)nr[j][i] : (float)nx[j][i];
        if (LOOP && row + gridDim.x < a.rows) fetch(row + gridDim.x);
        float sq = 0.f, t = 0.f;
        double top = 0.0; // max |r * w|, in fp64, where the products are exact
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                sq = fmaf(v[j][i], v[j][i], sq);
                if (CODE) t = fmaxf(t, fabsf(v[j][i] * w[j][i]));
            }
        if constexpr (CODE) {
            // rounding to fp32 keeps the order, so a thread's largest is among its products at its fp32 maximum
#pragma unroll
            for (int j = 0; j < NV; ++j)
#pragma unroll
                for (int i = 0; i < VEC; ++i)
                    if (fabsf(v[j][i] * w[j][i]) == t) top = fmax(top, fabs((double)v[j][i] * (double)w[j][i]));
        }
#pragma unroll
        for (int m = 32; m > 0; m >>= 1) {
            sq += __shfl_xor(sq, m);
            if (CODE) top = fmax(top, __shfl_xor(top, m));
        }
        if (nt > 64) {
            if ((tid & 63) == 0) {
                red[buf][tid >> 6] = sq;
                if (CODE) red64[buf][tid >> 6] = top;
            }
            __syncthreads();
            sq = 0.f;
            for (int i = 0; i < nt >> 6; ++i) {
                sq += red[buf][i];
                if (CODE) top = fmax(top, red64[buf][i]);
            }
        }
        // Squares overflow from elements of about 2^56 on and lose those below 2^-63. Rows whose sum shows either (all
        // threads see the same sum) are taken up or down by a power of two first, and eps with them: the products stay
        // exact, and every fp32 row then has its squares between 2^-118 and 2^121.
        float ms = sq / (float)n + a.eps, up = 1.f;
        if (__builtin_amdgcn_readfirstlane(!(ms < INFINITY) || (sq < 0x1p-80f && a.eps < 0x1p-60f))) {
            up = ms < INFINITY ? 0x1p90f : 0x1p-75f;
            sq = 0.f;
#pragma unroll
            for (int j = 0; j < NV; ++j)
#pragma unroll
                for (int i = 0; i < VEC; ++i) sq = fmaf(v[j][i] * up, v[j][i] * up, sq);
#pragma unroll
            for (int m = 32; m > 0; m >>= 1) sq += __shfl_xor(sq, m);
            if (nt > 64) {
                if ((tid & 63) == 0) red_far[tid >> 6] = sq;
                __syncthreads(); // between these reads and the next row's writes stands that row's first barrier
                sq = 0.f;
                for (int i = 0; i < nt >> 6; ++i) sq += red_far[i];
            }
            ms = sq / (float)n + a.eps * up * up;
        }
        const float rstd = 1.0f / sqrtf(ms); // of the row times `up`
        // Products and fp64 forms made for the maximum are made again below where they would spill: 8 loads of 20000 bf16
        // to int8 31.5 us, kept 35.7. The row-walking form does best with most of them (74 us for 8191 x 6144, made again 81),
        // but for the last load's of its longest rows (5000 x 8192: 61 us, two registers spilled 67).
        if (CODE && (!LOOP || NV * VEC >= 32)) {
#pragma unroll
            for (int j = LOOP ? NV - 1 : 0; j < NV; ++j)
#pragma unroll
                for (int i = 0; i < VEC; ++i) asm volatile("" : "+v"(v[j][i]), "+v"(w[j][i]));
        }
        if (a.sum) {
            TX *s = (TX *)a.sum + row * a.ss;
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                const int e = (j * nt + tid) * VEC;
                store_row<TX, VEC, ANY>(s + e, n - e, v[j]);
            }
        }
        TY *y = (TY *)a.y + row * a.ys;
        if constexpr (!CODE) {
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                const int e = (j * nt + tid) * VEC;
                float o[VEC];
#pragma unroll
                for (int i = 0; i < VEC; ++i) o[i] = v[j][i] * up * rstd * w[j][i];
                store_row<TY, VEC, ANY>(y + e, n - e, o);
            }
        } else {
            // sq is finite where the row is, whatever its weights hide; a row of zeros without eps has an infinite rstd
            const float scale = !(sq < INFINITY) ? NAN : top == 0.0 ? 0.f : (float)(top * (double)up * (double)rstd / 127.0);
            if (tid == 0) a.y_scale[row] = scale;
            const bool ok = top > 0.0 && scale == scale;
            const bool range = top > 1e-30 && top < 1e30; // fp32 holds the products and the quotient's factor
            const double inv64 = 127.0 / top;
            const float inv = (float)inv64;
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                const int e = (j * nt + tid) * VEC;
                float o[VEC];
#pragma unroll
                for (int i = 0; i < VEC; ++i) {
                    // within 127 * 4 * 2^-24 of the quotient
                    const float f = range ? v[j][i] * w[j][i] * inv : (float)((double)v[j][i] * (double)w[j][i] * inv64);
                    float c = rintf(f);
                    if (fabsf(f - c) > 0.4999f) { // next to a border: on which side, in fp64 and without a division
                        const float k = floorf(f);
                        const double d = fma(-(double)(k + 0.5f), top, (double)v[j][i] * (double)w[j][i] * 127.0);
                        c = d > 0.0 ? k + 1.f : d < 0.0 ? k : 2.f * rintf(0.5f * (k + 0.5f)); // a tie: the even one
                    }
                    o[i] = ok ? c : 0.f;
                }
                store_row<TY, VEC, ANY>(y + e, n - e, o);
            }
        }
        if (!LOOP) break;
    }
}

template <typename TX, typename TY, int VEC, bool ANY>
hipError_t launch_nv(const NormArgs &a, int cus, hipStream_t st) {
    const int chunks = (a.n + VEC - 1) / VEC;
    // With rows for every CU, the smallest block whose threads hold at most four
    // loads (several blocks a CU; with eight, the row-walking form of 6144 fp32
    // elements to int8 spilled: 331 us for 8138 rows, now 118); with few rows, up to
    // 1024 threads: the latency of one row is what counts then.
    constexpr int LAST = 32768 / 1024 / VEC; // loads a thread at the longest row
    int nv = 0;
    for (int want = a.rows >= 2 * cus ? 256 : 1024; want <= 1024 && nv == 0; want *= 2)
        for (int k = 1; k <= 4 && nv == 0; ++k)
            if ((chunks + k - 1) / k <= want) nv = k;
    if (nv == 0) nv = LAST;
    int nt = ((chunks + nv - 1) / nv + 63) / 64 * 64;
    if (nt > 1024) return hipErrorInvalidValue;
    // 16 waves a CU then hold a row each and the next one's loads
    const long most = (long)cus * (1024 / nt);
    const bool loop = nt <= 512 && a.rows > most;
    const int piece = (int)(kMaxThreads / nt); // rows a launch where a block takes one row
    for (long done = 0; done < a.rows; done += piece) {
        NormArgs b = a;
        if (!loop && a.rows > piece) {
            b.x = (const TX *)a.x + done * a.xs;
            b.res = a.res ? (const TX *)a.res + done * a.rs : nullptr;
            b.y = (TY *)a.y + done * a.ys;
            b.sum = a.sum ? (TX *)a.sum + done * a.ss : nullptr;
            b.y_scale = a.y_scale ? a.y_scale + done : nullptr;
            b.rows = (int)(a.rows - done < piece ? a.rows - done : piece);
        }
        const dim3 grid((unsigned)(loop ? most : b.rows)), block((unsigned)nt);
        switch (nv) {
#define WQ_NV(N)                                                                                                       \
    case N:                                                                                                            \
        if constexpr (N <= LAST) {                                                                                     \
            if (!loop) {                                                                                               \
                hipLaunchKernelGGL((rmsnorm_kernel<TX, TY, VEC, N, ANY, false>), grid, block, 0, st, b);               \
            } else if constexpr (N <= 4) { /* eight loads a thread only where 512 threads do not hold the row */       \
                hipLaunchKernelGGL((rmsnorm_kernel<TX, TY, VEC, N, ANY, true>), grid, block, 0, st, b);                \
            }                                                                                                          \
        }                                                                                                              \
        break;
            WQ_NV(1) WQ_NV(2) WQ_NV(3) WQ_NV(4) WQ_NV(8)
#undef WQ_NV
        default: return hipErrorInvalidValue;
        }
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess || loop) return e;
    }
    return hipSuccess;
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
