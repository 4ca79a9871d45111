// The products of the expert layer (moe_kernels.hip), included once a format of weights.
//
// They run on v_mfma_i32_16x16x64_i8. Codes become int8 with a shift and a mask for four of them (int8 ones as they are; int4
// as 16 * q, int2 as 64 * q), where bf16 ones took two instructions each and bound the vector units. An activation becomes a
// 31-bit integer, in units of a power of two that the activations of a step (the 128 bytes of a row of weights that they
// meet: 128, 256 or 512 of them) share, and that as four signed base-256 digits, its parts: x = unit * sum_p d_p 256^p within
// 2^-30 of the step's largest magnitude. The integer sums are exact; each step's goes to the fp32 sum with its unit.
//
// With a few rows an expert the weights' stream bounds them, read once: one token on 8 experts of 2048 x 6144 in int4, 151 MB,
// 20.4 us (gate and up: 4.9 TB/s) and 11.2 us (down: 4.5 TB/s; a large copy 4.8), 34.5 us with all launches; in int8 57 us, in
// int2 26 us. Loads of the next two steps are always in flight, across tiles too. With more rows reading the operands from LDS
// bounds them, 16 stacked rows a KiB: 64 tokens on 8 experts of the same shape in int8, 302 MB, 62.4 and 40.3 us (3.2 and 2.5
// TB/s), 119 us with all launches.
#pragma once

#include <type_traits>

#include "moe_parts.h"

namespace wq {
namespace {

// (How a block's waves share its work: moe_plan.h.) A block makes a tile of outputs at a time; it takes several tiles of one
// expert one after another.
constexpr int kWaves = kMoeWaves;
constexpr int NT = kMoeTiles;
// Pointers read from the experts' table are of no known address space otherwise, and their loads would count as LDS loads too.
#define GLOBAL __attribute__((address_space(1)))

// GS: 0 one scale a row, 1 a group covers whole 64-byte halves of a step, 2 groups of any multiple of 64 positions (int4 and
// int2: the operands are then turned so that each product takes 64 neighbouring positions). M: operands of 16 stacked rows,
// four parts of four activations each.
template <int FMT, bool GATED, int GS, int M, int WK>
struct Products {
    using F = Fmt<FMT>;
    static constexpr int WR = kWaves / WK;
    static constexpr int OUT = moe_outputs(GATED, WK);      // outputs of a block
    static constexpr int UNITS = F::EPB;                    // products of 64 positions in 64 bytes
    static constexpr bool TURN = GS == 2 && F::EPB > 1;
    static constexpr int RED = kWaves * NT * 64 * 4;        // bytes of the waves' sums
    // Many rows: activations whose parts stand prepared in memory, where every block would make them again (8 experts of
    // 2048 x 6144 in int8 with 16 rows each: 190 us instead of 126).
    static constexpr bool BIG = moe_big(M);
    static constexpr int LDS = moe_lds(M), ROWS = moe_rows(M, WK, F::POS);
    static_assert(ROWS >= 1, "a phase holds two steps of every wave");
    static constexpr int PIECE = kPiece;                    // positions that a thread stages at a time
    static constexpr int PRE = moe_ahead(M);

    const MoeArgs &a;
    const MoeShape &sh;
    const MoeMatrix m0, m1;
    const int wr, wk, lane, li, g;
    uint8_t *lds;
    float *red;

    __device__ __forceinline__ const MoeMatrix &matrix(int b) const { return GATED && b ? m1 : m0; }
    // first output row of this wave's weight tile b, in a block's tile
    __device__ __forceinline__ int row0(int b) const { return GATED ? 16 * wr : 16 * (NT * wr + b); }

    // Sixteen activations as memory holds them: four runs of four, of 16 bytes (f32) or 8.
    struct Piece {
        u32x4 v[4];
    };

    // The activations of positions pos .. pos + 15 of a slot; BIG: their parts.
    __device__ __forceinline__ void fetch(int slot, int pos, Piece &p) const {
        if constexpr (BIG) {
            const int step = pos / F::POS;
            const uint8_t *from = (GATED ? a.xp : a.hp) + ((long)(GATED ? slot / a.k : slot) * sh.steps + step) * (4 * F::POS) + pos % F::POS;
#pragma unroll
            for (int q = 0; q < 4; ++q) p.v[q] = step < sh.steps ? *reinterpret_cast<const u32x4 *>(from + q * F::POS) : u32x4{0, 0, 0, 0};
            return;
        }
        const bool wide = !GATED || a.x_size == 4;
        const uint8_t *row = GATED ? (const uint8_t *)a.xe + (long)(slot / a.k) * a.xes * a.x_size : (const uint8_t *)(a.h + (long)slot * a.ldh);
        const int end = GATED ? a.xe_n : a.ldh; // elements of a row, a multiple of four
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const int e = (int)elem_of_pos4(FMT, pos + 4 * q, sh.nfull);
            p.v[q] = u32x4{0, 0, 0, 0};
            if (e < end) {
                if (wide)
                    p.v[q] = *reinterpret_cast<const u32x4 *>(row + 4L * e);
                else
                    p.v[q].xy = *reinterpret_cast<const u32x2 *>(row + 2L * e);
            }
        }
    }

    // Puts the parts of a piece to `to` (the parts' rows `pitch` bytes apart) and the step's unit to `unit`.
    __device__ __forceinline__ void put(const Piece &p, int slot, int pos, uint8_t *to, int pitch, float *unit) const {
        u32x4 part[4];
        if constexpr (BIG) {
#pragma unroll
            for (int q = 0; q < 4; ++q) part[q] = p.v[q];
            const int step = pos / F::POS;
            if (pos % F::POS == 0)
                *unit = step < sh.steps ? (GATED ? a.xunit : a.hunit)[(long)(GATED ? slot / a.k : slot) * sh.steps + step] : 0.f;
        } else {
            float x[16];
#pragma unroll
            for (int q = 0; q < 4; ++q)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const uint16_t half = (uint16_t)(p.v[q][j >> 1] >> (16 * (j & 1)));
                    x[4 * q + j] = !GATED || a.x_size == 4 ? __uint_as_float(p.v[q][j])
                                   : a.x_bf16              ? __uint_as_float((uint32_t)half << 16)
                                                           : (float)__builtin_bit_cast(f16, half);
                }
            *unit = make_parts<FMT>(x, part);
        }
#pragma unroll
        for (int q = 0; q < 4; ++q) *reinterpret_cast<u32x4 *>(to + q * pitch) = part[q];
    }

    // Output tiles [t0, t1) of n rows, the expert's slots; n <= ROWS.
    __device__ __forceinline__ void rows(const int *slots, int n, int t0, int t1) {
        const int all = moe_steps(sh.steps, WK), per = moe_phase(M, WK, F::POS, n, all), phases = (all + per - 1) / per;
        const int span = per * WK * F::POS, pitch = span + 16;         // positions; bytes of a part's row, 16 apart in the banks
        float *units = reinterpret_cast<float *>(lds + n * 4 * pitch); // [n][per * WK]
        // pieces of a phase: `row` of each slot (the last phase: `rest`); i / row for i, row < 2^16 by its reciprocal
        const int whole = span / PIECE, rest = (all * WK * F::POS - (phases - 1) * span) / PIECE;
        const uint32_t by_whole = 0xFFFFFFFFu / whole + 1, by_rest = 0xFFFFFFFFu / rest + 1;
        auto piece = [&](int i, int ph, Piece &p) __attribute__((always_inline)) {
            const bool last = ph == phases - 1;
            const int row = last ? rest : whole;
            if (i >= n * row) return;
            const int s = (int)__umulhi((uint32_t)i, last ? by_rest : by_whole);
            fetch(slots[s], ph * span + PIECE * (i - s * row), p);
        };
        auto away = [&](int i, int ph, const Piece &p) __attribute__((always_inline)) {
            const bool last = ph == phases - 1;
            const int row = last ? rest : whole;
            if (i >= n * row) return;
            const int s = (int)__umulhi((uint32_t)i, last ? by_rest : by_whole), c = PIECE * (i - s * row);
            put(p, slots[s], ph * span + c, lds + s * 4 * pitch + c, pitch, units + s * per * WK + c / F::POS);
        };
        auto stage = [&](int ph, int from) __attribute__((always_inline)) {
            const int row = ph == phases - 1 ? rest : whole;
#pragma unroll 1
            for (int i = threadIdx.x + from * 64 * kWaves; i < n * row; i += 64 * kWaves) {
                Piece p;
                piece(i, ph, p);
                away(i, ph, p);
            }
        };
        // weights: half of a tile's rows a load, 128 bytes each
        uint32_t woff[NT][2], real = ~0u;
        const uint32_t lane_byte = 16 * (g + 4 * (li >> 3)), last16 = sh.stride - 16;
        // Rows past the matrix read its last row. Behind the last tile every lane reads the matrix's first bytes: the loads stay,
        // for the counts of those in flight are what the waits go by, and cost next to nothing.
        auto aim = [&](int tile) __attribute__((always_inline)) {
            real = tile < t1 ? ~0u : 0u;
#pragma unroll
            for (int b = 0; b < NT; ++b)
#pragma unroll
                for (int u = 0; u < 2; ++u) woff[b][u] = real & (uint32_t)min(tile * OUT + row0(b) + 8 * u + (li & 7), sh.O - 1) * (uint32_t)sh.stride;
        };
        u32x4 w[2][NT][2];
        auto load_w = [&](u32x4(&to)[NT][2], int i) __attribute__((always_inline)) {
            const uint32_t byte = real & min(128u * (wk + WK * i) + lane_byte, last16);
#pragma unroll
            for (int b = 0; b < NT; ++b)
#pragma unroll
                for (int u = 0; u < 2; ++u)
                    to[b][u] = __builtin_nontemporal_load((const GLOBAL u32x4 *)((const GLOBAL uint8_t *)matrix(b).w + (woff[b][u] + byte)));
        };
        // Group scales of a step's halves (units), asked for a step ahead and before the weights that follow: the waits go by the
        // order of the loads. (Where the registers for them would spill, each when it is needed.)
        constexpr int SC = GS == 0 ? 1 : TURN ? 2 * UNITS : 2;
        constexpr bool EARLY = GS != 0 && !BIG && SC <= 4;
        float sc[2][SC][NT];
        auto load_sc = [&](float(&to)[SC][NT], int tile, int i) __attribute__((always_inline)) {
            if constexpr (EARLY) {
#pragma unroll
                for (int k = 0; k < SC; ++k) {
                    const int grp = min(((wk + WK * i) * F::POS + k * (F::POS / SC)) / sh.gs, sh.ng - 1);
#pragma unroll
                    for (int b = 0; b < NT; ++b)
                        to[k][b] = ((const GLOBAL float *)matrix(b).scales)[(long)grp * sh.O + min(tile * OUT + row0(b) + li, sh.O - 1)];
                }
            }
        };
        // the first phase's activations are asked for ahead of the weights: behind them they would wait for all of those
        Piece ahead[PRE > 0 ? PRE : 1];
#pragma unroll
        for (int q = 0; q < PRE; ++q) piece(threadIdx.x + q * 64 * kWaves, 0, ahead[q]);
        __builtin_amdgcn_sched_barrier(0);
        aim(t0);
        load_w(w[0], 0);
        load_sc(sc[0], t0, 0);
        load_w(w[1], 1);
        __builtin_amdgcn_sched_barrier(0);
        __syncthreads(); // the buffer's last readers are done
#pragma unroll
        for (int q = 0; q < PRE; ++q) away(threadIdx.x + q * 64 * kWaves, 0, ahead[q]);
        stage(0, PRE);
        __syncthreads();
        // this lane's stacked row (part li & 3 of activation li / 4 of each four), and the unit of its column of sums
        uint32_t xrow[M], xunit[M];
#pragma unroll
        for (int m = 0; m < M; ++m) {
            xrow[m] = (uint32_t)((min(4 * m + (li >> 2), n - 1) * 4 + (li & 3)) * pitch) + (TURN ? 4 * F::EPB : 16 * F::EPB) * g;
            xunit[m] = min(4 * m + g, n - 1) * per * WK;
        }
        float acc[NT][M];
        int tile = t0;
        auto body = [&](auto slot_c, int i, int at) __attribute__((always_inline)) { // at: the step's number in the phase
            constexpr int SLOT = decltype(slot_c)::value;
            // the two loads' rows to the operands' lanes: h[0] holds the step's first 64 bytes of row li, h[1] the others
            u32x4 h[2][NT];
#pragma unroll
            for (int b = 0; b < NT; ++b)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int v0 = w[SLOT][b][0][j], v1 = w[SLOT][b][1][j];
                    h[0][b][j] = __builtin_amdgcn_update_dpp(v0, v1, 0x128, 0xF, 0xC, false);
                    h[1][b][j] = __builtin_amdgcn_update_dpp(v1, v0, 0x128, 0xF, 0x3, false);
                }
            load_sc(sc[SLOT ^ 1], i + 1 < all ? tile : tile + 1, i + 1 < all ? i + 1 : 0);
            if (i + 2 == all) aim(tile + 1); // the next tile's first steps follow
            load_w(w[SLOT], i + 2 < all ? i + 2 : i + 2 - all);
            i32x4 part[NT][M];
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                if constexpr (TURN) { // word j of a half to the four 16-byte pieces number j of its rows
#pragma unroll
                    for (int b = 0; b < NT; ++b) {
                        u32x4 &t = h[half][b];
                        const auto p = __builtin_amdgcn_permlane32_swap(t[0], t[2], false, false), q = __builtin_amdgcn_permlane32_swap(t[1], t[3], false, false);
                        const auto r = __builtin_amdgcn_permlane16_swap(p[0], q[0], false, false), s = __builtin_amdgcn_permlane16_swap(p[1], q[1], false, false);
                        t = u32x4{r[0], r[1], s[0], s[1]};
                    }
                }
#pragma unroll
                for (int u = 0; u < UNITS; ++u) {
                    const uint32_t off = (uint32_t)at * F::POS + half * (F::POS / 2) + (TURN ? 64 : 16) * u;
                    const bool fresh = GS == 0 ? half + u == 0 : TURN || u == 0, last = GS == 0 ? half == 1 && u == UNITS - 1 : TURN || u == UNITS - 1;
                    if (BIG) __builtin_amdgcn_sched_barrier(0); // (the scheduler would read a whole step's operands at once, and spill)
                    i32x4 x[M];
#pragma unroll
                    for (int m = 0; m < M; ++m) {
                        const uint8_t *p = lds + xrow[m] + off;
                        if constexpr (TURN && FMT == WQ_I4) { // eight positions of each of two pieces
                            const u32x2 lo = *reinterpret_cast<const u32x2 *>(p), hi = *reinterpret_cast<const u32x2 *>(p + 32);
                            x[m] = i32x4{(int)lo.x, (int)lo.y, (int)hi.x, (int)hi.y};
                        } else {
                            x[m] = *reinterpret_cast<const i32x4 *>(p);
                        }
                    }
#pragma unroll
                    for (int b = 0; b < NT; ++b) {
                        const u32x4 &c = h[half][b];
                        i32x4 q;
                        if constexpr (FMT == WQ_I8) {
                            q = __builtin_bit_cast(i32x4, c);
                        } else if constexpr (FMT == WQ_I4) { // a nibble's bits in a byte's upper half: 16 times the signed code
                            const uint32_t t0_ = c[2 * u] ^ 0x88888888u, t1_ = c[2 * u + 1] ^ 0x88888888u;
                            q = i32x4{(int)(t0_ << 4 & 0xF0F0F0F0u), (int)(t0_ & 0xF0F0F0F0u), (int)(t1_ << 4 & 0xF0F0F0F0u), (int)(t1_ & 0xF0F0F0F0u)};
                        } else { // two bits in a byte's uppermost: 64 times
                            const uint32_t t = c[u] ^ 0xAAAAAAAAu;
                            q = i32x4{(int)(t << 6 & 0xC0C0C0C0u), (int)(t << 4 & 0xC0C0C0C0u), (int)(t << 2 & 0xC0C0C0C0u), (int)(t & 0xC0C0C0C0u)};
                        }
#pragma unroll
                        for (int m = 0; m < M; ++m)
                            part[b][m] = __builtin_amdgcn_mfma_i32_16x16x64_i8(x[m], q, fresh ? i32x4{0, 0, 0, 0} : part[b][m], 0, 0, 0);
                    }
                    if (last) {
                        float unit[M];
#pragma unroll
                        for (int m = 0; m < M; ++m) unit[m] = units[xunit[m] + at];
                        constexpr int NOW = EARLY ? SLOT : 0;
                        const int k = TURN ? half * UNITS + u : half;
                        if constexpr (GS != 0 && !EARLY) {
                            const int grp = min(((wk + WK * i) * F::POS + k * (F::POS / SC)) / sh.gs, sh.ng - 1);
#pragma unroll
                            for (int b = 0; b < NT; ++b)
                                sc[0][k][b] = ((const GLOBAL float *)matrix(b).scales)[(long)grp * sh.O + min(tile * OUT + row0(b) + li, sh.O - 1)];
                        }
                        // The parts' sums are below 2^24, exact in fp32. A step's sum meets its unit first and a group's scale
                        // after: a unit times a scale could be too small to keep its bits where the product of all three is not.
#pragma unroll
                        for (int b = 0; b < NT; ++b)
#pragma unroll
                            for (int m = 0; m < M; ++m) {
                                const i32x4 &d = part[b][m];
                                const float v = fmaf(fmaf(fmaf((float)d[3], 256.f, (float)d[2]), 256.f, (float)d[1]), 256.f, (float)d[0]);
                                acc[b][m] = GS ? fmaf(v * unit[m], sc[NOW][k][b], acc[b][m]) : fmaf(v, unit[m], acc[b][m]);
                            }
                        if (BIG) __builtin_amdgcn_sched_barrier(0);
                    }
                }
            }
        };
        for (; tile < t1; ++tile) {
#pragma unroll
            for (int b = 0; b < NT; ++b)
#pragma unroll
                for (int m = 0; m < M; ++m) acc[b][m] = 0.f;
            for (int ph = 0; ph < phases; ++ph) {
                if (phases > 1) {
                    if (ph > 0 || tile > t0) {
                        __syncthreads();
                        if (BIG)
#pragma unroll
                            for (int q = 0; q < PRE; ++q) away(threadIdx.x + q * 64 * kWaves, ph, ahead[q]);
                        stage(ph, BIG ? PRE : 0);
                        __syncthreads();
                    }
                    // the next phase's activations are on their way while this one's meet the weights
                    if (BIG)
#pragma unroll
                        for (int q = 0; q < PRE; ++q) piece(threadIdx.x + q * 64 * kWaves, ph + 1 < phases ? ph + 1 : 0, ahead[q]);
                }
                const int end = min((ph + 1) * per, all);
                for (int i = ph * per; i < end; i += 2) {
                    const int at = (i - ph * per) * WK + wk;
                    body(std::integral_constant<int, 0>{}, i, at);
                    body(std::integral_constant<int, 1>{}, i + 1, at + WK);
                }
            }
            finish(acc, slots, n, tile);
        }
    }

    // Adds the waves' sums in order; what becomes of the outputs.
    __device__ __forceinline__ void finish(float (&acc)[NT][M], const int *slots, int n, int tile) {
        const int wave = wr * WK + wk, o0 = tile * OUT;
#pragma unroll 1
        for (int m = 0; 4 * m < n; ++m) { // four rows at a time
            __syncthreads(); // (the sums' last readers are done)
#pragma unroll
            for (int b = 0; b < NT; ++b) {
                red[(wave * NT + b) * 64 + lane] = acc[b][0];
#pragma unroll
                for (int r = 0; r + 1 < M; ++r) acc[b][r] = acc[b][r + 1];
            }
            __syncthreads();
            const int rows_m = min(4, n - 4 * m);
#pragma unroll 1
            for (int i = threadIdx.x; i < rows_m * OUT; i += 64 * kWaves) {
                const int s = i / OUT, c = i % OUT, o = o0 + c;
                if (o >= sh.O) continue;
                auto sum = [&](int grp, int b) {
                    float v = 0.f;
#pragma unroll
                    for (int q = 0; q < WK; ++q) v += red[((grp * WK + q) * NT + b) * 64 + 16 * s + (c & 15)];
                    if constexpr (GS) return v * kBack; // (what was lost below the smallest number is below 2^-133 here)
                    const float s_ = ((const GLOBAL float *)matrix(b).scales)[o];
                    return fabsf(v) < 1.f ? v * kBack * s_ : v * (s_ * kBack);
                };
                const int slot = slots[4 * m + s];
                if constexpr (GATED) {
                    const float z = sum(c >> 4, 0), u = sum(c >> 4, 1);
                    a.h[(long)slot * a.ldh + o] = z / (1.0f + expf(-z)) * u;
                } else {
                    a.d[(long)slot * sh.O + o] = sum(c / (16 * NT), c >> 4 & (NT - 1));
                }
            }
        }
        if (GATED && o0 + OUT >= sh.O) { // zeros up to a multiple of four
            const int pad = a.ldh - sh.O;
            for (int i = threadIdx.x; i < n * pad; i += 64 * kWaves) a.h[(long)slots[i / pad] * a.ldh + sh.O + i % pad] = 0.f;
        }
    }
};

template <int FMT, bool GATED, int GS, int M, int WK, bool INLINE>
__global__ __launch_bounds__(64 * kWaves, M >= 3 ? 2 : 3) void moe_products_kernel(const MoeArgs a) {
    using P = Products<FMT, GATED, GS, M, WK>;
    __shared__ __align__(16) uint8_t lds[P::LDS];
    __shared__ __align__(16) float red[P::RED / 4];
    __shared__ int here[INLINE ? kInlineSlots : 64];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const MoeShape &sh = GATED ? a.in : a.out;
    const int tiles = (sh.O + P::OUT - 1) / P::OUT, per = GATED ? a.form_in.tiles : a.form_out.tiles;
    const int t0 = blockIdx.x * per, t1 = min(t0 + per, tiles);
    auto work = [&](const MoeMatrix &m0, const MoeMatrix &m1) {
        return P{a, sh, m0, m1, wave / WK, wave % WK, lane, lane & 15, lane >> 4, lds, red};
    };
    if constexpr (INLINE) {
        // a few slots: a block a slot, of which the first of an expert works for all of that expert's
        const int N = a.T * a.k;
        int id[kInlineSlots / 64];
#pragma unroll
        for (int q = 0; q < kInlineSlots / 64; ++q) id[q] = 64 * q + lane < N ? a.ids[64 * q + lane] : -1;
        int mine = id[0];
#pragma unroll
        for (int q = 1; q < kInlineSlots / 64; ++q) mine = (int)blockIdx.y >= 64 * q ? id[q] : mine;
        const int e = __builtin_amdgcn_readlane(mine, blockIdx.y & 63);
        if (e < 0 || e >= a.E) return;
        int n = 0, first = -1;
#pragma unroll
        for (int q = 0; q < kInlineSlots / 64; ++q) {
            const uint64_t same = __ballot(id[q] == e);
            if (wave == 0 && id[q] == e) here[n + __popcll(same & ((1ull << lane) - 1))] = 64 * q + lane;
            if (first < 0 && same) first = 64 * q + __builtin_ctzll(same);
            n += __popcll(same);
        }
        if (first != (int)blockIdx.y) return;
        const MoeExpert &ex = a.experts[e];
        P w = work(GATED ? ex.gate : ex.down, GATED ? ex.up : ex.down);
        __syncthreads();
        for (int s = 0; s < n; s += P::ROWS) w.rows(here + s, min(P::ROWS, n - s), t0, t1);
    } else {
        // every wave reads the plan, for its expert's matrices; the rows are those that the first one read
        __shared__ int span[2];
        const int N = a.T * a.k;
        MoeWork raw = a.plan[blockIdx.y];
        asm("" : "+s"(raw.expert), "+s"(raw.rows), "+s"(raw.first)); // (read once: what is checked is what is used)
        const MoeWork k = bounded(raw, a.E, N);
        const MoeExpert &ex = a.experts[k.expert];
        const MoeMatrix m0 = GATED ? ex.gate : ex.down, m1 = GATED ? ex.up : ex.down; // (scalar loads, ahead of the barrier)
        if (threadIdx.x == 0) {
            span[0] = k.rows;
            span[1] = k.first;
        }
        __syncthreads();
        const int n = __builtin_amdgcn_readfirstlane(span[0]);
        if (n == 0) return;
        P w = work(m0, m1);
        const int *slots = a.order + __builtin_amdgcn_readfirstlane(span[1]);
        for (int s = 0; s < n; s += P::ROWS) {
            const int some = min(P::ROWS, n - s);
            if (s > 0) __syncthreads(); // the last rows' readers are done
            if (threadIdx.x < some) here[threadIdx.x] = bounded_slot(slots[s + threadIdx.x], N);
            __syncthreads();
            w.rows(here, some, t0, t1);
        }
    }
}

template <int FMT, bool GATED, int GS, int M, int WK>
hipError_t launch_products(MoeArgs &a, hipStream_t st) {
    const MoeShape &sh = GATED ? a.in : a.out;
    const long N = (long)a.T * a.k;
    using P = Products<FMT, GATED, GS, M, WK>;
    const int tiles = (sh.O + P::OUT - 1) / P::OUT, per = GATED ? a.form_in.tiles : a.form_out.tiles;
    const dim3 grid((unsigned)((tiles + per - 1) / per), (unsigned)(a.plan == nullptr ? N : N < a.E ? N : a.E));
    if constexpr (!P::BIG) {
        if (a.plan == nullptr) {
            hipLaunchKernelGGL((moe_products_kernel<FMT, GATED, GS, M, WK, true>), grid, dim3(64 * kWaves), 0, st, a);
            return hipGetLastError();
        }
    }
    if (a.plan != nullptr)
        hipLaunchKernelGGL((moe_products_kernel<FMT, GATED, GS, M, WK, false>), grid, dim3(64 * kWaves), 0, st, a);
    return hipGetLastError();
}

template <int FMT, bool GATED, int GS, int M>
hipError_t launch_wk(MoeArgs &a, hipStream_t st) {
    switch (GATED ? a.form_in.wk : a.form_out.wk) {
    case 1: return launch_products<FMT, GATED, GS, M, 1>(a, st);
    case 2: return launch_products<FMT, GATED, GS, M, 2>(a, st);
    default: return launch_products<FMT, GATED, GS, M, 4>(a, st);
    }
}

template <int FMT, bool GATED, int GS>
hipError_t launch_m(MoeArgs &a, hipStream_t st) {
    switch (GATED ? a.form_in.m : a.form_out.m) {
    case 1: return launch_wk<FMT, GATED, GS, 1>(a, st);
    case 2: return launch_wk<FMT, GATED, GS, 2>(a, st);
    case 3:
        if constexpr (GS == 2) return launch_wk<FMT, GATED, GS, 3>(a, st);
        return hipErrorInvalidValue;
    case 4:
        if constexpr (GS != 2) return launch_wk<FMT, GATED, GS, 4>(a, st);
        return hipErrorInvalidValue;
    default:
        if constexpr (GS != 2) return launch_wk<FMT, GATED, GS, 8>(a, st);
        return hipErrorInvalidValue;
    }
}

template <int FMT, bool GATED>
hipError_t launch_gs(MoeArgs &a, hipStream_t st) {
    const int gs = GATED ? a.in.gs : a.out.gs;
    if (gs == 0) return launch_m<FMT, GATED, 0>(a, st);
    if (gs % (64 * Fmt<FMT>::EPB) == 0) return launch_m<FMT, GATED, 1>(a, st);
    if constexpr (FMT != WQ_I8) return launch_m<FMT, GATED, 2>(a, st);
    return hipErrorInvalidValue;
}

// h in parts, for many rows. Rows of empty slots hold anything, and their parts are not read.
template <int FMT>
__global__ __launch_bounds__(256) void moe_parts_kernel(const MoeArgs a) {
    const int per_row = a.out.kp / kPiece;
    const long i = (long)blockIdx.x * 256 + threadIdx.x;
    const long row = i / per_row;
    if (row >= (long)a.T * a.k) return;
    prepare_piece<FMT>(a.h + row * a.ldh, a.in.O, a.out, row, (int)(i - row * per_row) * kPiece, a.hp, a.hunit);
}

template <int FMT>
hipError_t launch_both(MoeArgs &a, hipStream_t st) {
    hipError_t e = launch_gs<FMT, true>(a, st);
    if (e == hipSuccess && a.operands >= 4) {
        const long pieces = (long)a.T * a.k * (a.out.kp / kPiece);
        hipLaunchKernelGGL((moe_parts_kernel<FMT>), dim3((unsigned)((pieces + 255) / 256)), dim3(256), 0, st, a);
        e = hipGetLastError();
    }
    return e == hipSuccess ? launch_gs<FMT, false>(a, st) : e;
}

} // namespace
} // namespace wq
