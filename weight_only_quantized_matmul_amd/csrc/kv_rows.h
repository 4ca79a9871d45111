// Rows of the paged cache: 8 elements a lane, quantised or moved.
#pragma once

#include "decoder.h"

namespace wq {
namespace {

constexpr float kTiny = 0x1p-100f;

template <int KIND>
struct Codes { // 8 codes
    static constexpr int bytes = KIND == WQ_KV_F16 ? 16 : KIND == WQ_KV_I8 ? 8 : 4;
};

template <typename T, bool VEC>
__device__ __forceinline__ void load8(const T *p, float *v) {
    if (VEC) {
        load_vec<T, 8>(p, v);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = (float)p[i];
    }
}

template <typename T, bool VEC>
__device__ __forceinline__ void store8(T *p, const float *v) {
    if (VEC) {
        store_vec<T, 8>(p, v);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) p[i] = (T)v[i];
    }
}

// The largest over a group of LANES lanes.
template <int LANES>
__device__ __forceinline__ float group_max(float v) {
#pragma unroll
    for (int m = LANES / 2; m > 0; m >>= 1) v = fmaxf(v, __shfl_xor(v, m));
    return v;
}

// Largest magnitude of a row whose lanes hold v each; infinite where the row is not finite.
template <int LANES>
__device__ __forceinline__ float row_top(const float (&v)[8]) {
    float top = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) top = fmaxf(top, fabsf(v[i]));
    // a NaN is not seen by the maximum: its lane hands on an infinity
    bool nan = false;
#pragma unroll
    for (int i = 0; i < 8; ++i) nan = nan || v[i] != v[i];
    return group_max<LANES>(nan ? INFINITY : top);
}

// This lane's 8 codes of a row with that largest magnitude, to `row`; the row's scale.
template <int KIND>
__device__ __forceinline__ float store_codes(uint8_t *row, const float (&v)[8], float top) {
    const bool bad = !(top < INFINITY), zero = bad || top < kTiny;
    float scale;
    if constexpr (KIND == WQ_KV_F16) {
        typedef f16 f16x8 __attribute__((ext_vector_type(8)));
        const int e = ilogbf(top) - 14;
        scale = ldexpf(1.0f, e);
        f16x8 c;
#pragma unroll
        for (int i = 0; i < 8; ++i) c[i] = zero ? (f16)0.f : (f16)ldexpf(v[i], -e); // exact but for the half's own rounding
        *reinterpret_cast<f16x8 *>(row) = c;
    } else {
        constexpr int N = KIND == WQ_KV_I8 ? 127 : 7;
        scale = (float)((double)top / N);
        const float inv = 1.0f / scale;
        int c[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float f = v[i] * inv; // within N * 3 * 2^-24 of the quotient
            float q = rintf(f);
            if (fabsf(f - q) > 0.4999f) q = (float)rint((double)v[i] / (double)scale); // next to a border
            c[i] = zero ? 0 : (int)q;
        }
        if constexpr (KIND == WQ_KV_I8) {
            uint32_t u[2];
#pragma unroll
            for (int k = 0; k < 2; ++k)
                u[k] = (c[4 * k] & 255) | (c[4 * k + 1] & 255) << 8 | (c[4 * k + 2] & 255) << 16 | (uint32_t)c[4 * k + 3] << 24;
            *reinterpret_cast<uint2 *>(row) = make_uint2(u[0], u[1]);
        } else {
            uint32_t u = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) u |= (uint32_t)(c[i] + 8) << (4 * i);
            *reinterpret_cast<uint32_t *>(row) = u;
        }
    }
    return bad ? NAN : zero ? 0.f : scale;
}

} // namespace
} // namespace wq
