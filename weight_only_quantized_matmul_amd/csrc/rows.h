// Rows of any length and alignment in wide loads and stores.
#pragma once

#include "decoder.h"

namespace wq {
namespace {

template <typename T, int VEC>
struct Vec {
    typedef T type __attribute__((ext_vector_type(VEC), aligned(VEC * sizeof(T) < 16 ? VEC * sizeof(T) : 16)));
    typedef T any __attribute__((ext_vector_type(VEC), aligned(sizeof(T))));
};

// VEC elements from p. ANY: p is aligned to its element only and the row may end
// before them (`left` elements are there; the rest are zeros). The hardware
// takes wide loads and stores at any address, so odd rows keep them too: only
// a row's last elements go one by one.
template <typename T, int VEC, bool ANY>
__device__ __forceinline__ typename Vec<T, VEC>::type load_row(const T *p, int left) {
    typename Vec<T, VEC>::type v;
#pragma unroll
    for (int i = 0; i < VEC; ++i) v[i] = (T)0.f;
    if (left >= VEC) {
        if constexpr (ANY)
            v = *reinterpret_cast<const typename Vec<T, VEC>::any *>(p);
        else
            v = *reinterpret_cast<const typename Vec<T, VEC>::type *>(p);
    } else if (ANY) {
#pragma unroll
        for (int i = 0; i < VEC; ++i)
            if (i < left) v[i] = p[i];
    }
    return v;
}

template <typename T, int VEC, bool ANY>
__device__ __forceinline__ void store_row(T *p, int left, const float *v) {
    if constexpr (!ANY) {
        if (left >= VEC) store_vec<T, VEC>(p, v);
    } else if (left >= VEC) {
        typename Vec<T, VEC>::any r;
#pragma unroll
        for (int i = 0; i < VEC; ++i) r[i] = (T)v[i];
        *reinterpret_cast<typename Vec<T, VEC>::any *>(p) = r;
    } else {
#pragma unroll
        for (int i = 0; i < VEC; ++i)
            if (i < left) p[i] = (T)v[i];
    }
}

} // namespace
} // namespace wq
