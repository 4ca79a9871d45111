// Quantising a key/value cache as it is written, and reading it back.
//
// D / 8 lanes take one row of one token, head and pool side, 8 elements a
// lane: a wide load, the row's maximum over the lane group, 8 codes back in
// one store. Both directions move every byte once and are bound by HBM (few
// tokens: by the chain q_start -> kv_len -> table -> store).
#include "decoder.h"

namespace wq {
namespace {

constexpr int kThreads = 256;
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

// What a lane group works on: token, side (0 keys, 1 values), head.
struct Where {
    int tok, side, head;
    bool any, there; // a row of the tokens' side; one of the cache too
    long row, scale; // offsets in the pools (bytes, floats)
};

template <int LANES>
__device__ __forceinline__ Where locate(const KvCopyArgs &a, int lane) {
    Where w;
    const long r = ((long)blockIdx.x * kThreads + threadIdx.x) / LANES;
    const int per = 2 * a.c.heads;
    w.any = r < (long)a.b.T * per;
    const long tok = w.any ? r / per : 0;
    const int s = w.any ? (int)(r - tok * per) : 0;
    w.tok = (int)tok;
    w.side = s >= a.c.heads;
    w.head = s - w.side * a.c.heads;
    const int b = sequence_of<LANES>(a.b.q_start, a.b.B, w.tok, lane);
    w.there = false;
    w.row = w.scale = 0;
    if (w.any && b < a.b.B) {
        const int first = a.b.q_start[b], next = a.b.q_start[b + 1];
        if (first <= w.tok && w.tok < next) {
            const long t = (long)a.b.kv_len[b] - next + w.tok;
            int page, slot;
            if (find_row(a.c, a.b, b, t, &page, &slot)) {
                w.there = true;
                w.row = page * a.c.rp + w.head * a.c.rh + slot * a.c.rs;
                w.scale = page * a.c.sp + w.head * a.c.sh + slot * a.c.ss;
            }
        }
    }
    return w;
}

template <typename T, int KIND, int D, bool VEC>
__global__ __launch_bounds__(kThreads) void kv_append_kernel(const KvCopyArgs a) {
    constexpr int LANES = D / 8;
    const int lane = threadIdx.x & (LANES - 1);
    const Where w = locate<LANES>(a, lane);
    float v[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    if (w.there) load8<T, VEC>((const T *)(w.side ? a.v : a.k) + (long)w.tok * a.tok + (long)w.head * a.head + 8 * lane, v);
    float top = 0.f;
    bool bad = false;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        top = fmaxf(top, fabsf(v[i]));
        bad = bad || !(fabsf(v[i]) < INFINITY);
    }
    int nb = bad ? 1 : 0;
#pragma unroll
    for (int m = LANES / 2; m > 0; m >>= 1) {
        top = fmaxf(top, __shfl_xor(top, m));
        nb |= __shfl_xor(nb, m);
    }
    if (!w.there) return;
    uint8_t *row = const_cast<uint8_t *>(w.side ? a.c.v : a.c.k) + w.row + (long)lane * Codes<KIND>::bytes;
    float scale;
    const bool zero = nb || top < kTiny;
    if constexpr (KIND == WQ_KV_F16) {
        const int e = ilogbf(top) - 14;
        scale = ldexpf(1.0f, e);
        typedef f16 f16x8 __attribute__((ext_vector_type(8)));
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
            for (int j = 0; j < 2; ++j)
                u[j] = (c[4 * j] & 255) | (c[4 * j + 1] & 255) << 8 | (c[4 * j + 2] & 255) << 16 | (uint32_t)c[4 * j + 3] << 24;
            *reinterpret_cast<uint2 *>(row) = make_uint2(u[0], u[1]);
        } else {
            uint32_t u = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) u |= (uint32_t)(c[i] + 8) << (4 * i);
            *reinterpret_cast<uint32_t *>(row) = u;
        }
    }
    if (lane == 0) const_cast<float *>(w.side ? a.c.vs : a.c.ks)[w.scale] = nb ? NAN : zero ? 0.f : scale;
}

template <typename T, int KIND, int D, bool VEC>
__global__ __launch_bounds__(kThreads) void kv_read_kernel(const KvCopyArgs a) {
    constexpr int LANES = D / 8;
    const int lane = threadIdx.x & (LANES - 1);
    const Where w = locate<LANES>(a, lane);
    if (!w.any) return;
    float v[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    if (w.there) {
        const uint8_t *row = (w.side ? a.c.v : a.c.k) + w.row + (long)lane * Codes<KIND>::bytes;
        const float scale = (w.side ? a.c.vs : a.c.ks)[w.scale];
        if constexpr (KIND == WQ_KV_F16) {
            load_vec<f16, 8>((const f16 *)row, v);
        } else if constexpr (KIND == WQ_KV_I8) {
            load_vec<int8_t, 8>((const int8_t *)row, v);
        } else {
            const uint32_t u = *reinterpret_cast<const uint32_t *>(row);
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = (float)((int)(u >> (4 * i) & 15) - 8);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] *= scale;
    }
    store8<T, VEC>((T *)(w.side ? a.v : a.k) + (long)w.tok * a.tok + (long)w.head * a.head + 8 * lane, v);
}

template <typename T, int KIND, int D>
hipError_t launch_d(const KvCopyArgs &a, bool write, bool vec, hipStream_t st) {
    const long rows = (long)a.b.T * 2 * a.c.heads;
    const long blocks = (rows * (D / 8) + kThreads - 1) / kThreads;
    if (blocks > 0x7fffffffL) return hipErrorInvalidValue;
    const dim3 grid((unsigned)blocks), block(kThreads);
    if (write) {
        if (vec)
            hipLaunchKernelGGL((kv_append_kernel<T, KIND, D, true>), grid, block, 0, st, a);
        else
            hipLaunchKernelGGL((kv_append_kernel<T, KIND, D, false>), grid, block, 0, st, a);
    } else {
        if (vec)
            hipLaunchKernelGGL((kv_read_kernel<T, KIND, D, true>), grid, block, 0, st, a);
        else
            hipLaunchKernelGGL((kv_read_kernel<T, KIND, D, false>), grid, block, 0, st, a);
    }
    return hipGetLastError();
}

template <typename T, int KIND>
hipError_t launch_kind(const KvCopyArgs &a, int dim, bool write, bool vec, hipStream_t st) {
    switch (dim) {
    case 64: return launch_d<T, KIND, 64>(a, write, vec, st);
    case 128: return launch_d<T, KIND, 128>(a, write, vec, st);
    default: return launch_d<T, KIND, 256>(a, write, vec, st);
    }
}

template <typename T>
hipError_t launch_t(const KvCopyArgs &a, int kind, int dim, bool write, bool vec, hipStream_t st) {
    switch (kind) {
    case WQ_KV_F16: return launch_kind<T, WQ_KV_F16>(a, dim, write, vec, st);
    case WQ_KV_I8: return launch_kind<T, WQ_KV_I8>(a, dim, write, vec, st);
    default: return launch_kind<T, WQ_KV_I4>(a, dim, write, vec, st);
    }
}

hipError_t launch_kv(const KvCopyArgs &a, int kind, int dim, int dtype, bool write, bool vec, hipStream_t st) {
    switch (dtype) {
    case WQ_DT_F32: return launch_t<float>(a, kind, dim, write, vec, st);
    case WQ_DT_BF16: return launch_t<bf16>(a, kind, dim, write, vec, st);
    default: return launch_t<f16>(a, kind, dim, write, vec, st);
    }
}

} // namespace

hipError_t launch_kv_append(const KvCopyArgs &a, int kind, int dim, int dtype, bool vec, hipStream_t st) {
    return launch_kv(a, kind, dim, dtype, true, vec, st);
}

hipError_t launch_kv_read(const KvCopyArgs &a, int kind, int dim, int dtype, bool vec, hipStream_t st) {
    return launch_kv(a, kind, dim, dtype, false, vec, st);
}

} // namespace wq
