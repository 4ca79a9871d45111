// Activations as the expert layer's products take them: 31-bit integers in four signed base-256 digits, their parts.
#pragma once

#include "moe.h"

namespace wq {
namespace {

typedef unsigned int u32x2 __attribute__((ext_vector_type(2)));
typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));
typedef int i32x4 __attribute__((ext_vector_type(4)));

template <int FMT>
struct Fmt {
    static constexpr int EPB = FMT == WQ_I8 ? 1 : FMT == WQ_I4 ? 2 : 4;
    static constexpr int POS = 128 * EPB; // positions of a step
    // Units take off what the codes are multiplied by, and 2^16 that the sums give back (kBack): a step's activations times codes
    // can be 2^14 times the largest activation, and their sum stays finite like it.
    static constexpr float UNSCALE = (FMT == WQ_I8 ? 1.0f : FMT == WQ_I4 ? 0x1p-4f : 0x1p-6f) * 0x1p-16f;
};
constexpr float kBack = 0x1p16f;

// Bytes of b where sel's are 0..3, of a where 4..7.
__device__ __forceinline__ uint32_t bytes(uint32_t a, uint32_t b, uint32_t sel) { return __builtin_amdgcn_perm(a, b, sel); }

constexpr int kPiece = kMoePiece;

// The parts of 16 neighbouring positions' activations x, in the order in which the codes come out of their words, and the unit
// of the step that they belong to, of all of whose pieces the lanes come here together.
template <int FMT>
__device__ __forceinline__ float make_parts(const float (&x)[16], u32x4 (&part)[4]) {
    using F = Fmt<FMT>;
    // the step's largest magnitude; NaN and infinities order above all numbers as bits
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 16; ++i) top = max(top, __float_as_uint(x[i]) & 0x7FFFFFFFu);
#pragma unroll
    for (int m = F::POS / kPiece / 2; m > 0; m >>= 1) top = max(top, (uint32_t)__shfl_xor((int)top, m));
    // 2^(e + 1) is above it; 2^(e - 29) and its inverse are normal numbers, and the unit, at least 2^-147, is exact
    const int e = min(max((int)(top >> 23) - 127, -96), 127);
    const bool bad = top >= 0x7F800000u;
    const float up = __uint_as_float((uint32_t)(127 + 29 - e) << 23); // 2^(29 - e)
    uint32_t d[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        // balanced digits: the carries of adding 128 to each byte, and 128 off again
        const int v = bad ? 0 : (int)rintf(x[i] * up);
        d[i] = ((uint32_t)v + 0x80808080u) ^ 0x80808080u;
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const int s = FMT == WQ_I8 ? 4 * k : FMT == WQ_I4 ? 8 * (k >> 1) + (k & 1) : k, t = FMT == WQ_I8 ? 1 : FMT == WQ_I4 ? 2 : 4;
        const uint32_t e0 = d[s], e1 = d[s + t], e2 = d[s + 2 * t], e3 = d[s + 3 * t];
        const uint32_t l01 = bytes(e1, e0, 0x05010400u), h01 = bytes(e1, e0, 0x07030602u);
        const uint32_t l23 = bytes(e3, e2, 0x05010400u), h23 = bytes(e3, e2, 0x07030602u);
        part[0][k] = bytes(l23, l01, 0x05040100u);
        part[1][k] = bytes(l23, l01, 0x07060302u);
        part[2][k] = bytes(h23, h01, 0x05040100u);
        part[3][k] = bytes(h23, h01, 0x07060302u);
    }
    return bad ? NAN : __uint_as_float((uint32_t)(127 - 29 + e) << 23) * F::UNSCALE;
}

// A row's positions first .. first + 15 (threads of a wave: neighbouring pieces) to the prepared parts of row `row`: four
// planes of a step's positions a step, and a unit.
template <int FMT, typename T>
__device__ __forceinline__ void prepare_piece(const T *x, int n, const MoeShape &sh, long row, int first, uint8_t *parts, float *units) {
    using F = Fmt<FMT>;
    float v[16];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        const int e = (int)elem_of_pos4(FMT, first + 4 * q, sh.nfull);
#pragma unroll
        for (int j = 0; j < 4; ++j) v[4 * q + j] = e + j < n ? (float)x[e + j] : 0.f;
    }
    u32x4 part[4];
    const float unit = make_parts<FMT>(v, part);
    const long step = row * sh.steps + first / F::POS;
    uint8_t *to = parts + step * 4 * F::POS + first % F::POS;
#pragma unroll
    for (int p = 0; p < 4; ++p) *reinterpret_cast<u32x4 *>(to + p * F::POS) = part[p];
    if (first % F::POS == 0) units[step] = unit;
}

} // namespace
} // namespace wq
