// What the attention kernels share: the rows of a tile and the positions they
// see, how cache codes become f16 operands, and partial results.
#pragma once

#include <type_traits>

#include "decoder.h"

namespace wq {

typedef f16 f16x2 __attribute__((ext_vector_type(2)));
typedef f16 f16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef bf16 bf16x8 __attribute__((ext_vector_type(8)));

constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.69314718055994530942f;

// A tile: up to R rows of one sequence and key/value head, row r standing for
// new token r / G and query head kvh * G + r % G.
//
// Sequence b owns the tile numbers floor(q_start[b] G / R) + b up to
// floor(q_start[b+1] G / R) + b, at least as many as its rows need, so a
// block finds its sequence by comparing every lane's sequence with the tile's
// number, without a prefix sum and without knowing the lengths on the host.
struct Tile {
    int b, tok0, n, row0, rows; // sequence, its first token and token count, first row, rows here (0: no tile)
    int kv;                     // positions, those past the table left out
    int past;                   // kv_len - n: position of new token 0
};

__host__ __device__ inline long tile_count(long T, long G, long R, long B) { return T * G / R + B; }

template <int R>
__device__ __forceinline__ Tile find_tile(const BatchView &b, int page, int G, long id, int lane) {
    Tile t;
    t.rows = 0;
    t.b = t.tok0 = t.n = t.row0 = t.kv = t.past = 0;
    for (int i0 = 0; i0 < b.B; i0 += 64) {
        const int i = i0 + lane;
        bool mine = false;
        int s0 = 0, s1 = 0, kv = 0;
        if (i < b.B) {
            s0 = b.q_start[i];
            s1 = b.q_start[i + 1];
            kv = b.kv_len[i]; // with the others, not after them: the chain of loads is what a short call waits for
            s0 = min(max(s0, 0), b.T);
            s1 = min(max(s1, 0), b.T);
            mine = s1 > s0 && id >= (long)s0 * G / R + i && id <= (long)s1 * G / R + i;
        }
        const uint64_t m = __ballot(mine);
        if (!m) continue;
        const int hit = __builtin_ctzll(m);
        t.b = i0 + hit;
        t.tok0 = __builtin_amdgcn_readlane(s0, hit);
        t.n = __builtin_amdgcn_readlane(s1, hit) - t.tok0;
        kv = max(__builtin_amdgcn_readlane(kv, hit), 0);
        // a sequence's last tile comes first: under a causal mask it sees the most
        const long all = (long)t.n * G, row0 = ((all + R - 1) / R - 1 - (id - ((long)t.tok0 * G / R + t.b))) * R;
        t.row0 = (int)max(row0, 0L);
        t.rows = row0 >= 0 ? (int)min((long)R, all - row0) : 0;
        const long held = (long)b.width * page;
        t.past = kv - t.n;
        t.kv = kv < held ? kv : (int)held;
        return t;
    }
    return t;
}

// Position `lane` of block i. Past 2^31 - 1 it wraps to a negative number, which no row sees.
__device__ __forceinline__ int position(int base, int i, int step, int lane) {
    return (int)((unsigned)base + (unsigned)i * (unsigned)step + (unsigned)lane);
}

// Positions [lo, hi) that new token i sees.
__device__ __forceinline__ void seen_range(const Tile &t, int i, int causal, int window, int *lo, int *hi) {
    const long p = (long)t.past + i;
    long h = t.kv, l = 0;
    if (causal && p + 1 < h) h = p + 1;
    if (window > 0 && p + 1 > window) l = p + 1 - window;
    *hi = (int)(h < 0 ? 0 : h);
    *lo = (int)(l > *hi ? *hi : l);
}

// Bits `from` .. `to` - 1 of `keys` (a lane's keys of a step that are there), the others cleared.
__device__ __forceinline__ uint64_t seen_bits(uint64_t keys, int from, int to) {
    from = min(max(from, 0), 64);
    to = min(max(to, 0), 64);
    const uint64_t below = to == 64 ? ~0ull : (1ull << to) - 1, first = from == 64 ? ~0ull : (1ull << from) - 1;
    return keys & below & ~first;
}

// x where bit k is set, else `other`: a bit extract and a bitwise select, no branch.
__device__ __forceinline__ float where_seen(uint64_t bits, int k, float x, float other) {
    const uint32_t m = (uint32_t)__builtin_amdgcn_sbfe((int)(uint32_t)(k < 32 ? bits : bits >> 32), k & 31, 1);
    return __uint_as_float((m & __float_as_uint(x)) | (~m & __float_as_uint(other)));
}

// Blocks of `step` positions that the rows of a tile see, and their split: `per`
// blocks each, at least `least` where there are as many and at most nsplit splits.
struct Span {
    int base, blocks, per, splits;
};

__device__ __forceinline__ Span find_span(int step, int lo, int hi, int least, int nsplit) {
    Span s;
    s.base = lo & -step;
    s.blocks = hi > lo ? (int)(((unsigned)(hi - s.base) + (unsigned)step - 1) / (unsigned)step) : 0; // hi up to 2^31 - 1
    const int most = max(least, (s.blocks + nsplit - 1) / nsplit);
    s.splits = max(1, (s.blocks + most - 1) / most);
    s.per = (s.blocks + s.splits - 1) / s.splits; // splits of equal length
    s.splits = max(1, s.per == 0 ? 1 : (s.blocks + s.per - 1) / s.per);
    return s;
}

// ---------------------------------------------------------------------------
// Codes to matrix operands, exactly.
//
// To f16: a half 0x6400 + u is 1024 + u for u < 1024, so one and-or puts two
// codes into halves and one packed add takes the offset off. The constants are
// opaque registers, one scalar: with literals the and and the or are two
// instructions (an instruction takes one scalar register and no literal here).
struct OpenConst {
    uint32_t m0, m1, magic;
    __device__ __forceinline__ OpenConst() : m0(0x000f000fu), m1(0x00f000f0u), magic(0x64006400u) {
        asm volatile("" : "+s"(m0));
        asm volatile("" : "+s"(m1));
        asm volatile("" : "+v"(magic));
    }
};

__device__ __forceinline__ uint32_t pk_add(uint32_t a, float c) {
    const f16x2 r = __builtin_bit_cast(f16x2, a) + f16x2{(f16)c, (f16)c};
    return __builtin_bit_cast(uint32_t, r);
}

__device__ __forceinline__ uint32_t pk_fma(uint32_t a, float m, float c) {
    const f16x2 r = __builtin_elementwise_fma(__builtin_bit_cast(f16x2, a), f16x2{(f16)m, (f16)m}, f16x2{(f16)c, (f16)c});
    return __builtin_bit_cast(uint32_t, r);
}

// Four int8 codes, in order: two registers of two halves.
__device__ __forceinline__ void open_i8(uint32_t w, uint32_t *o) {
    const uint32_t x = w ^ 0x80808080u; // code + 128
    o[0] = pk_add(__builtin_amdgcn_perm(0x64646464u, x, 0x04010400u), -1152.f);
    o[1] = pk_add(__builtin_amdgcn_perm(0x64646464u, x, 0x04030402u), -1152.f);
}

// The nibbles of two 16-bit halves: registers with nibble 0, 1, 2, 3 of both.
__device__ __forceinline__ void open_i4(const OpenConst &k, uint32_t w, uint32_t *o) {
    const uint32_t v = w >> 8;
    o[0] = pk_add((w & k.m0) | k.magic, -1032.f);
    o[1] = pk_fma((w & k.m1) | k.magic, 0.0625f, -72.f);
    o[2] = pk_add((v & k.m0) | k.magic, -1032.f);
    o[3] = pk_fma((v & k.m1) | k.magic, 0.0625f, -72.f);
}

// To bf16: a code in fp32 has its low 16 bits clear, so the upper halves of two
// are the two bf16 values.
__device__ __forceinline__ uint32_t high_halves(float a, float b) {
    return __builtin_amdgcn_perm(__float_as_uint(b), __float_as_uint(a), 0x07060302u);
}

// Byte k of w as a signed number (one conversion with its byte select).
__device__ __forceinline__ float byte_i8(uint32_t w, int k) {
    return (float)(int8_t)(w >> (8 * k));
}

// The low nibble of byte k of w, two's complement, times 1/16.
__device__ __forceinline__ float nibble_i4(uint32_t w, int k) { return __builtin_amdgcn_cvt_off_f32_i4((int)(w >> (8 * k) & 0xffu)); }

// Element order of eight consecutive codes in a K operand.
template <int KIND>
__device__ __forceinline__ constexpr int k_order(int e) {
    return KIND == WQ_KV_I4 ? (e >> 1) + 4 * (e & 1) : e;
}

__device__ __forceinline__ f16x8 join4(const uint32_t *r) {
    const u32x4 v = {r[0], r[1], r[2], r[3]};
    return __builtin_bit_cast(f16x8, v);
}

// Power of two that brings |x| <= top to below 2^14 (top itself into [2^13, 2^14)), as its exponent.
__device__ __forceinline__ int head_room(float top) {
    if (!(top < INFINITY)) return 0; // a row with an infinity or a NaN has no result
    const int e = (int)(__float_as_uint(top) >> 23) - 127;
    return 13 - max(e, -100);
}

// The exponent that brings a value scale of up to `big` below 2^room.
__device__ __forceinline__ float scale_room(float big, int room) {
    return (float)(room - 1 - max((int)(__float_as_uint(big) >> 23) - 127, -90));
}

// Maxima and sums across lanes 32 or 16 apart, both lanes with the same bits.
__device__ __forceinline__ u32x2 swap32(float x) {
    return __builtin_bit_cast(u32x2, __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false));
}
__device__ __forceinline__ u32x2 swap16(float x) {
    return __builtin_bit_cast(u32x2, __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false));
}
template <int NG> // lanes that share a row: 2 (32 apart) or 4 (16 and 32 apart)
__device__ __forceinline__ float row_max(float x) {
    if (NG == 4) {
        const u32x2 r = swap16(x);
        x = fmaxf(__uint_as_float(r.x), __uint_as_float(r.y));
    }
    const u32x2 r = swap32(x);
    return fmaxf(__uint_as_float(r.x), __uint_as_float(r.y));
}
template <int NG>
__device__ __forceinline__ float row_sum(float x) {
    if (NG == 4) {
        const u32x2 r = swap16(x);
        x = __uint_as_float(r.x) + __uint_as_float(r.y);
    }
    const u32x2 r = swap32(x);
    return __uint_as_float(r.x) + __uint_as_float(r.y);
}

// The maximum over the wave, in every lane (x >= 0).
__device__ __forceinline__ float wave_max(float x) {
    x = row_max<4>(x);
#define WQ_ROR(n) x = fmaxf(x, __uint_as_float(__builtin_amdgcn_update_dpp(0, (int)__float_as_uint(x), 0x120 + n, 0xf, 0xf, true)))
    WQ_ROR(8); // row_ror: lanes of a row of 16, rotated
    WQ_ROR(4);
    WQ_ROR(2);
    WQ_ROR(1);
#undef WQ_ROR
    return x;
}

__device__ __forceinline__ float pow2(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

// A pair of floats as three bf16 pairs that sum to them exactly (24 bits).
__device__ __forceinline__ void split3(float a, float b, uint32_t *o) {
    o[0] = high_halves(a, b);
    a -= __uint_as_float(__float_as_uint(a) & 0xffff0000u);
    b -= __uint_as_float(__float_as_uint(b) & 0xffff0000u);
    o[1] = high_halves(a, b);
    a -= __uint_as_float(__float_as_uint(a) & 0xffff0000u);
    b -= __uint_as_float(__float_as_uint(b) & 0xffff0000u);
    o[2] = high_halves(a, b);
}

// 2^(x/2): sums of probabilities are rescaled by 2^x in two steps. Exponents of partial sums differ by up to 217 (values'
// scales from 2^-90 to 2^127), and 2^x alone is 0 below 2^-126, where the sum still counts. The values' sums do not need it:
// what they lose then is below 2^-126 of the largest scale.
__device__ __forceinline__ float half_way(float x) { return __builtin_amdgcn_exp2f(0.5f * x); }

// Two floats rounded to halves (to nearest), in one register.
__device__ __forceinline__ uint32_t pack_half(float a, float b) {
    const f32x2 v = {a, b};
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, f16x2));
}

// words of `bytes` (1, 2, 4, 8, 16, 32) at p
template <int BYTES>
__device__ __forceinline__ void load_words(const uint8_t *p, uint32_t *w) {
    if constexpr (BYTES == 1) {
        w[0] = *p;
    } else if constexpr (BYTES == 2) {
        w[0] = *reinterpret_cast<const uint16_t *>(p);
    } else if constexpr (BYTES == 4) {
        w[0] = *reinterpret_cast<const uint32_t *>(p);
    } else if constexpr (BYTES == 8) {
        const u32x2 v = *reinterpret_cast<const u32x2 *>(p);
        w[0] = v.x;
        w[1] = v.y;
    } else {
#pragma unroll
        for (int i = 0; i < BYTES / 16; ++i) {
            const u32x4 v = *reinterpret_cast<const u32x4 *>(p + 16 * i);
            w[4 * i] = v.x;
            w[4 * i + 1] = v.y;
            w[4 * i + 2] = v.z;
            w[4 * i + 3] = v.w;
        }
    }
}

// ---------------------------------------------------------------------------
// Rows a wave of the tiled kernel takes: 16 where 32 rows' operands and sums do not fit its registers.
constexpr int tiled_rows(int dim, bool f32) { return dim == 256 || (dim == 128 && f32) ? 16 : 32; }

struct AttnPlan {
    bool few;       // few-rows kernel, else the tiled one
    int waves;      // waves a block (tiled kernel)
    int rows;       // rows a tile
    int step;       // positions a step
    int nsplit;     // most splits of a tile's positions
    int least;      // fewest steps a split takes
    size_t ws_bytes;
};

// How the join reads `rows` rows of nsplit splits: one wave a row once that gives every CU four rows and there are few
// splits, else four; enough partial rows in flight for all splits, at most eight a wave.
struct JoinPlan {
    int waves, at;
};
inline JoinPlan plan_join(long rows, int nsplit) {
    if (rows >= 1024 && nsplit <= 16) return {1, 4};
    return {4, nsplit <= 8 ? 2 : 8};
}

// Partial results of a split: row (token, head) and split s at part[(row * nsplit + s) * D], the exponent they
// are scaled by (2^-ref) and their sum of probabilities at ml[(row * nsplit + s) * 2].
struct Partials {
    float *part, *ml;
    int nsplit, least;
};

} // namespace wq
