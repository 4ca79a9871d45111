// The gated feed-forward layer of chosen experts, for a few tokens.
//
//     y[t] = add[t] + sum_j weights[t,j] * down_e . (silu(gate_e . x[t]) * (up_e . x[t])),  e = ids[t,j]
//
// Which expert works on which rows is known on the device only. A first
// kernel sorts the slots t * k + j by expert and lays the activations out; then
// the products of gate and up, with the activation as their epilogue, write h;
// the products of down write one row a slot; and the last kernel adds each
// token's rows in the order of its slots, so results do not depend on what
// else the batch holds.
//
// The products run on v_mfma_f32_16x16x32_bf16 with exact operands, as in the
// few-rows matmul: every activation is split into bf16 parts (three of an fp32
// value, two of an f16 one, one of a bf16 one), every code is its exact value.
#include "moe.h"

namespace wq {
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

constexpr int kPrepThreads = 512;
constexpr int kWaves = 8; // waves a block of the products, each with every eighth step of the rows

template <int FMT>
struct Fmt {
    static constexpr int EPB = FMT == WQ_I8 ? 1 : FMT == WQ_I4 ? 2 : 4;
    static constexpr int KS = 4 * EPB;      // 32-position MFMA steps in 128 bytes
    static constexpr int QUADS = KS / 4;    // the step's parts of four MFMA steps
    static constexpr int POS = 128 * EPB;   // positions of a step
    static constexpr float UNSCALE = FMT == WQ_I8 ? 1.0f : FMT == WQ_I4 ? 0.0625f : 0.015625f;
};

// Bytes [lo.2, lo.3, hi.2, hi.3]: two fp32 values that bf16 holds exactly.
__device__ __forceinline__ uint32_t pack_hi(uint32_t lo_bits, uint32_t hi_bits) {
    return __builtin_amdgcn_perm(hi_bits, lo_bits, 0x07060302u);
}
__device__ __forceinline__ uint32_t sbyte_f32(uint32_t w, int b) {
    return __float_as_uint((float)(int)(int8_t)(w >> (8 * b)));
}
__device__ __forceinline__ uint32_t reg(uint32_t v) { // keeps the compiler from folding masks into each extraction
    asm("" : "+v"(v));
    return v;
}

// The codes of 8 consecutive positions as bf16: int4 16 * q, int8 q, int2 64 * q.
__device__ __forceinline__ u32x4 frag_i4(uint32_t w) {
    const uint32_t t = w ^ 0x88888888u;
    const uint32_t ev = reg((t << 4) & 0xF0F0F0F0u), od = reg(t & 0xF0F0F0F0u);
    u32x4 r;
#pragma unroll
    for (int i = 0; i < 4; ++i) r[i] = pack_hi(sbyte_f32(ev, i), sbyte_f32(od, i));
    return r;
}
__device__ __forceinline__ u32x4 frag_i8(uint32_t w0, uint32_t w1) {
    u32x4 r;
    r[0] = pack_hi(sbyte_f32(w0, 0), sbyte_f32(w0, 1));
    r[1] = pack_hi(sbyte_f32(w0, 2), sbyte_f32(w0, 3));
    r[2] = pack_hi(sbyte_f32(w1, 0), sbyte_f32(w1, 1));
    r[3] = pack_hi(sbyte_f32(w1, 2), sbyte_f32(w1, 3));
    return r;
}
// half 0 or 1: the dword's positions 0..7 or 8..15
__device__ __forceinline__ u32x4 frag_i2(uint32_t w, int half) {
    const uint32_t t = w ^ 0xAAAAAAAAu;
    const uint32_t m0 = reg((t << 6) & 0xC0C0C0C0u), m1 = reg((t << 4) & 0xC0C0C0C0u);
    const uint32_t m2 = reg((t << 2) & 0xC0C0C0C0u), m3 = reg(t & 0xC0C0C0C0u);
    u32x4 r;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        r[2 * i] = pack_hi(sbyte_f32(m0, 2 * half + i), sbyte_f32(m1, 2 * half + i));
        r[2 * i + 1] = pack_hi(sbyte_f32(m2, 2 * half + i), sbyte_f32(m3, 2 * half + i));
    }
    return r;
}

// Position of element e of a row (the inverse of elem_of_pos4 for single elements).
template <int FMT>
__device__ __forceinline__ int pos_of_elem(int e, int nfull) {
    constexpr int PER = kBlockBytes * Fmt<FMT>::EPB, G = 16 * Fmt<FMT>::EPB;
    const int b = e / PER;
    if (b >= nfull) return e;
    const int r = e - b * PER;
    return b * PER + (r & 255) / 4 * G + 4 * (r >> 8) + (r & 3);
}

// x in bf16 parts by truncation: x = b[0] + b[1] + b[2] exactly (each part's upper half is the bf16).
__device__ __forceinline__ void split3(float x, uint32_t *b) {
    b[0] = __float_as_uint(x) & 0xFFFF0000u;
    const float r = x - __uint_as_float(b[0]);
    b[1] = __float_as_uint(r) & 0xFFFF0000u;
    b[2] = __float_as_uint(r - __uint_as_float(b[1]));
}

// ---------------------------------------------------------------------------
// Block 0 makes the plan; the others lay out the activations, eight positions a thread.
template <int FMT, typename T>
__global__ __launch_bounds__(kPrepThreads) void moe_prepare_kernel(const MoeArgs a) {
    __shared__ int cnt[WQ_MOE_MAX_EXPERTS], at[WQ_MOE_MAX_EXPERTS];
    __shared__ uint32_t part[kPrepThreads / 64];
    constexpr int P = sizeof(T) == 4 ? 3 : __is_same(T, bf16) ? 1 : 2;
    const int tid = threadIdx.x, lane = tid & 63, N = a.T * a.k;
    if (blockIdx.x == 0) {
        for (int e = tid; e < WQ_MOE_MAX_EXPERTS; e += kPrepThreads) cnt[e] = 0;
        __syncthreads();
        for (int i = tid; i < N; i += kPrepThreads) {
            const int e = a.ids[i];
            if (e >= 0 && e < a.E) atomicAdd(&cnt[e], 1);
        }
        __syncthreads();
        // rows (at most 2^14) in the low half, experts in the high half: one sum for both
        constexpr int PER = WQ_MOE_MAX_EXPERTS / kPrepThreads;
        uint32_t v = 0;
        for (int i = 0; i < PER; ++i) v += cnt[tid * PER + i] ? 0x10000u + cnt[tid * PER + i] : 0;
        uint32_t sum = v;
        for (int m = 1; m < 64; m <<= 1) {
            const uint32_t o = __shfl_up((int)sum, m);
            if (lane >= m) sum += o;
        }
        if (lane == 63) part[tid >> 6] = sum;
        __syncthreads();
        uint32_t all = 0;
        for (int i = 0; i < kPrepThreads / 64; ++i) {
            if (i == tid >> 6) sum += all;
            all += part[i];
        }
        uint32_t run = sum - v;
        for (int i = 0; i < PER; ++i) {
            const int e = tid * PER + i, n = cnt[e];
            at[e] = run & 0xFFFF;
            if (n) {
                int *p = a.plan + 4 + 3 * (run >> 16);
                p[0] = e;
                p[1] = run & 0xFFFF;
                p[2] = n;
                run += 0x10000u + n;
            }
        }
        if (tid == 0) a.plan[0] = all >> 16;
        __syncthreads();
        // (the order of an expert's rows may differ from run to run: no result depends on it)
        int *order = a.plan + 4 + 3 * a.E;
        for (int i = tid; i < N; i += kPrepThreads) {
            const int e = a.ids[i];
            if (e >= 0 && e < a.E) order[atomicAdd(&at[e], 1)] = i;
        }
        return;
    }
    const int per_row = a.in.kp / 8;
    const long items = (long)a.T * per_row;
    for (long i = (long)(blockIdx.x - 1) * kPrepThreads + tid; i < items; i += (long)(gridDim.x - 1) * kPrepThreads) {
        const int t = (int)(i / per_row), pos = (int)(i - (long)t * per_row) * 8;
        const T *x = (const T *)a.x + t * a.xs;
        uint32_t b[8][3];
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            const int e = (int)elem_of_pos4(FMT, pos + 4 * q, a.in.nfull);
#pragma unroll
            for (int j = 0; j < 4; ++j) split3(e + j < a.in.I ? (float)x[e + j] : 0.f, b[4 * q + j]);
        }
#pragma unroll
        for (int p = 0; p < P; ++p) {
            u32x4 v;
#pragma unroll
            for (int j = 0; j < 4; ++j) v[j] = pack_hi(b[2 * j][p], b[2 * j + 1][p]);
            *reinterpret_cast<u32x4 *>(a.xp + ((long)t * P + p) * a.in.kp + pos) = v;
        }
    }
}

// ---------------------------------------------------------------------------
// GATED: gate and up, writing h; else down, writing a row a slot. NBO: 16-row tiles of outputs a block. GS: 0 one scale
// a row, 1 a group covers whole 64-byte halves of a step, 2 groups of any multiple of 64 positions.
template <int FMT, bool GATED, int GS, int NBO>
struct Products {
    using F = Fmt<FMT>;
    static constexpr int NB = GATED ? 2 * NBO : NBO; // 16-row tiles of weights
    static constexpr int RP = F::KS / 2;             // MFMA steps in a half
    static constexpr int SUBS = GS == 2 ? F::EPB : 1; // groups that a half may hold

    const MoeArgs &a;
    const MoeShape &sh;
    const MoeMatrix m0, m1;
    const int o0, wave, lane, li, g;
    float *red; // [kWaves][NB][64][4]

    __device__ __forceinline__ const MoeMatrix &matrix(int b) const { return GATED && (b & 1) ? m1 : m0; }
    // first output row of weight tile b
    __device__ __forceinline__ int row0(int b) const { return o0 + 16 * (GATED ? b >> 1 : b); }

    // Rows [s0, s0 + n) of the expert's slots, n <= 16 M / pitch.
    template <int M>
    __device__ __forceinline__ void rows(const int *slots, int n) {
        const int planes = GATED ? a.planes : 3, sh2 = planes == 3 ? 2 : planes - 1; // log2 of the pitch: stacked row s << sh2 | part
        // this lane's stacked rows
        const uint16_t *xr[M];
#pragma unroll
        for (int m = 0; m < M; ++m) {
            const int rho = li + 16 * m, s = min(rho >> sh2, n - 1), p = min(rho & ((1 << sh2) - 1), planes - 1);
            const int slot = slots[s];
            const long row = GATED ? (long)(slot / a.k) * planes + p : (long)slot * 3 + p;
            xr[m] = (GATED ? a.xp : a.hp) + row * sh.kp + 16 * F::EPB * g;
        }
        // and rows of weights: half of a tile's rows a load, 128 bytes each
        uint32_t woff[NB][2];
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int u = 0; u < 2; ++u) woff[b][u] = (uint32_t)min(row0(b) + 8 * u + (li & 7), sh.O - 1) * (uint32_t)sh.stride;
        const uint32_t lane_byte = 16 * (g + 4 * (li >> 3)), last16 = sh.stride - 16;
        const int steps = (sh.steps - wave + kWaves - 1) / kWaves; // this wave's, at least 0
        auto step_of = [&](int i) { return min(wave + kWaves * i, sh.steps - 1); };
        auto load_w = [&](u32x4(&w)[NB][2], int step) {
            const uint32_t byte = min(128u * step + lane_byte, last16);
#pragma unroll
            for (int b = 0; b < NB; ++b)
#pragma unroll
                for (int u = 0; u < 2; ++u)
                    w[b][u] = __builtin_nontemporal_load(reinterpret_cast<const u32x4 *>(matrix(b).w + (woff[b][u] + byte)));
        };
        auto load_x = [&](bf16x8(&x)[4][M], int step, int quad) {
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int ks = 4 * quad + q, off = step * F::POS + ks / RP * (F::POS / 2) + ks % RP * 8;
#pragma unroll
                for (int m = 0; m < M; ++m) x[q][m] = *reinterpret_cast<const bf16x8 *>(xr[m] + off);
            }
        };
        f32x4 acc[NB][M];
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int m = 0; m < M; ++m) acc[b][m] = f32x4{0.f, 0.f, 0.f, 0.f};
        u32x4 w[2][NB][2];
        bf16x8 x[2][4][M];
        load_w(w[0], step_of(0));
        load_x(x[0], step_of(0), 0);
        load_w(w[1], step_of(1));
        auto body = [&](auto odd_c, int i) __attribute__((always_inline)) {
            constexpr int ODD = decltype(odd_c)::value;
            // the two loads' rows to the operands' lanes: lo holds the step's first 64 bytes of row li, hi the others
            u32x4 h[2][NB];
#pragma unroll
            for (int b = 0; b < NB; ++b)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int v0 = w[ODD][b][0][j], v1 = w[ODD][b][1][j];
                    h[0][b][j] = __builtin_amdgcn_update_dpp(v0, v1, 0x128, 0xF, 0xC, false);
                    h[1][b][j] = __builtin_amdgcn_update_dpp(v1, v0, 0x128, 0xF, 0x3, false);
                }
            const int step = step_of(i);
            load_w(w[ODD], step_of(i + 2));
            f32x4 part[NB][M][SUBS];
#pragma unroll
            for (int quad = 0; quad < F::QUADS; ++quad) {
                constexpr int Q = F::QUADS;
                const int par = (ODD * Q + quad) & 1;
                if (quad + 1 < Q)
                    load_x(x[par ^ 1], step, quad + 1);
                else
                    load_x(x[par ^ 1], step_of(i + 1), 0);
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const int ks = 4 * quad + q, half = ks / RP, j = ks % RP;
#pragma unroll
                    for (int b = 0; b < NB; ++b) {
                        const u32x4 &c = h[half][b];
                        const u32x4 f = FMT == WQ_I4 ? frag_i4(c[j & 3]) : FMT == WQ_I8 ? frag_i8(c[2 * j & 3], c[(2 * j & 3) + 1]) : frag_i2(c[j >> 1 & 3], j & 1);
                        const bf16x8 bw = __builtin_bit_cast(bf16x8, f);
#pragma unroll
                        for (int m = 0; m < M; ++m) {
                            if constexpr (GS == 0) {
                                acc[b][m] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(x[par][q][m], bw, acc[b][m], 0, 0, 0);
                            } else {
#pragma unroll
                                for (int u = 0; u < SUBS; ++u) {
                                    // positions of other groups are zeros in this product
                                    u32x4 xv = __builtin_bit_cast(u32x4, x[par][q][m]);
                                    if (SUBS > 1 && g * SUBS / 4 != u) xv = u32x4{0, 0, 0, 0};
                                    part[b][m][u] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                                        __builtin_bit_cast(bf16x8, xv), bw, j == 0 ? f32x4{0.f, 0.f, 0.f, 0.f} : part[b][m][u], 0, 0, 0);
                                }
                            }
                        }
                    }
                    if (GS != 0 && j == RP - 1) {
#pragma unroll
                        for (int u = 0; u < SUBS; ++u) {
                            const int grp = min((step * F::POS + half * (F::POS / 2) + u * (F::POS / 2 / SUBS)) / sh.gs, sh.ng - 1);
#pragma unroll
                            for (int b = 0; b < NB; ++b) {
                                const float sc = matrix(b).scales[(long)grp * sh.O + min(row0(b) + li, sh.O - 1)];
#pragma unroll
                                for (int m = 0; m < M; ++m)
#pragma unroll
                                    for (int r = 0; r < 4; ++r) acc[b][m][r] = fmaf(sc, part[b][m][u][r], acc[b][m][r]);
                            }
                        }
                    }
                }
            }
        };
        for (int i = 0; i < steps; i += 2) {
            body(std::integral_constant<int, 0>{}, i);
            if (i + 1 < steps) body(std::integral_constant<int, 1>{}, i + 1);
        }
        // add the parts of an activation (adjacent stacked rows, in one lane), then the waves' sums in order
        const int per_m = 16 >> sh2; // rows of 16 stacked ones
#pragma unroll
        for (int m = 0; m < M; ++m) {
            if (m * per_m >= n) break;
            __syncthreads();
#pragma unroll
            for (int b = 0; b < NB; ++b) {
                f32x4 v = acc[b][m];
                float *to = red + ((wave * NB + b) * 64 + lane) * 4;
                if (sh2 == 2)
                    to[0] = v[0] + v[1] + v[2];
                else if (sh2 == 1)
                    *reinterpret_cast<float2 *>(to) = make_float2(v[0] + v[1], v[2] + v[3]);
                else
                    *reinterpret_cast<f32x4 *>(to) = v;
            }
            __syncthreads();
            const int rows_m = min(per_m, n - m * per_m), cols = 16 * NBO;
            for (int i = threadIdx.x; i < rows_m * cols; i += 64 * kWaves) {
                const int s = i / cols, c = i - s * cols, o = o0 + c;
                if (o >= sh.O) continue;
                // row s of these 16: lane group and register
                const int from = (((s << sh2) >> 2) * 16 + (c & 15)) * 4 + ((s << sh2 & 3) >> sh2);
                auto sum = [&](int b) {
                    float v = 0.f;
#pragma unroll
                    for (int wv = 0; wv < kWaves; ++wv) v += red[(wv * NB + b) * 256 + from];
                    v *= F::UNSCALE;
                    return GS ? v : v * matrix(b).scales[o];
                };
                const int slot = slots[m * per_m + s];
                if constexpr (GATED) {
                    const float z = sum(2 * (c >> 4)), u = sum(2 * (c >> 4) + 1);
                    const float hv = z / (1.0f + expf(-z)) * u;
                    uint32_t b3[3];
                    split3(hv, b3);
                    const int pos = pos_of_elem<FMT>(o, a.out.nfull);
#pragma unroll
                    for (int p = 0; p < 3; ++p) a.hp[((long)slot * 3 + p) * a.out.kp + pos] = (uint16_t)(b3[p] >> 16);
                } else {
                    a.d[(long)slot * sh.O + o] = sum(c >> 4);
                }
            }
        }
        if (GATED && o0 + 16 * NBO >= sh.O) { // the positions past the row: zeros
            const int first = a.out.I, pad = a.out.kp - first;
            for (int i = threadIdx.x; i < n * 3 * pad; i += 64 * kWaves) {
                const int r = i / pad;
                a.hp[((long)slots[r / 3] * 3 + r % 3) * a.out.kp + first + (i - r * pad)] = 0;
            }
        }
    }
};

template <int FMT, bool GATED, int GS, int NBO, bool MANY>
__global__ __launch_bounds__(64 * kWaves) void moe_products_kernel(const MoeArgs a) {
    using P = Products<FMT, GATED, GS, NBO>;
    __shared__ __align__(16) float red[kWaves * P::NB * 256];
    if ((int)blockIdx.y >= a.plan[0]) return;
    const int *p = a.plan + 4 + 3 * blockIdx.y;
    const int e = p[0], n = p[2];
    const int *slots = a.plan + 4 + 3 * a.E + p[1];
    const MoeExpert &ex = a.experts[e];
    const int lane = threadIdx.x & 63;
    P w{a, GATED ? a.in : a.out, GATED ? ex.gate : ex.down, GATED ? ex.up : ex.down, (int)blockIdx.x * 16 * NBO,
        (int)__builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane, lane & 15, lane >> 4, red};
    const int planes = GATED ? a.planes : 3, unit = 16 >> (planes == 3 ? 2 : planes - 1); // rows of 16 stacked ones
    if constexpr (!MANY) {
        for (int s = 0; s < n; s += unit) w.template rows<1>(slots + s, min(unit, n - s));
    } else {
        for (int s = 0; s < n; s += 4 * unit) {
            const int left = min(4 * unit, n - s);
            if (left <= unit)
                w.template rows<1>(slots + s, left);
            else if (left <= 2 * unit)
                w.template rows<2>(slots + s, left);
            else
                w.template rows<4>(slots + s, left);
        }
    }
}

// ---------------------------------------------------------------------------
template <typename T>
__global__ __launch_bounds__(256) void moe_combine_kernel(const MoeArgs a) {
    const int t = blockIdx.y, o = blockIdx.x * 256 + threadIdx.x;
    if (o >= a.out.O) return;
    float v = a.add ? (float)((const T *)a.add)[t * a.as + o] : 0.f;
    for (int j = 0; j < a.k; ++j) {
        const int slot = t * a.k + j, e = a.ids[slot];
        if (e >= 0 && e < a.E) v = fmaf(a.weights[slot], a.d[(long)slot * a.out.O + o], v);
    }
    ((T *)a.y)[t * a.ys + o] = (T)v;
}

template <int FMT, bool GATED, int GS, bool MANY>
hipError_t launch_products(const MoeArgs &a, hipStream_t st) {
    constexpr int NBO = GATED ? 1 : 2;
    const MoeShape &sh = GATED ? a.in : a.out;
    const long N = (long)a.T * a.k;
    const dim3 grid((unsigned)((sh.O + 16 * NBO - 1) / (16 * NBO)), (unsigned)(N < a.E ? N : a.E));
    hipLaunchKernelGGL((moe_products_kernel<FMT, GATED, GS, NBO, MANY>), grid, dim3(64 * kWaves), 0, st, a);
    return hipGetLastError();
}

template <int FMT, bool GATED>
hipError_t launch_gs(const MoeArgs &a, hipStream_t st) {
    const int gs = GATED ? a.in.gs : a.out.gs, planes = GATED ? a.planes : 3;
    const bool many = a.T * a.k > (16 >> (planes == 3 ? 2 : planes - 1)); // an expert may have more rows than one operand holds
    if (gs == 0) return many ? launch_products<FMT, GATED, 0, true>(a, st) : launch_products<FMT, GATED, 0, false>(a, st);
    if (gs % (64 * Fmt<FMT>::EPB) == 0)
        return many ? launch_products<FMT, GATED, 1, true>(a, st) : launch_products<FMT, GATED, 1, false>(a, st);
    return many ? launch_products<FMT, GATED, 2, true>(a, st) : launch_products<FMT, GATED, 2, false>(a, st);
}

template <int FMT, typename T>
hipError_t launch_ft(const MoeArgs &a, hipStream_t st) {
    const long blocks = ((long)a.T * (a.in.kp / 8) + kPrepThreads - 1) / kPrepThreads;
    hipLaunchKernelGGL((moe_prepare_kernel<FMT, T>), dim3((unsigned)(1 + (blocks < 1024 ? blocks : 1024))), dim3(kPrepThreads), 0, st, a);
    hipError_t e = hipGetLastError();
    if (e == hipSuccess) e = launch_gs<FMT, true>(a, st);
    if (e == hipSuccess) e = launch_gs<FMT, false>(a, st);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL((moe_combine_kernel<T>), dim3((unsigned)((a.out.O + 255) / 256), (unsigned)a.T), dim3(256), 0, st, a);
    return hipGetLastError();
}

template <int FMT>
hipError_t launch_f(const MoeArgs &a, int dtype, hipStream_t st) {
    switch (dtype) {
    case WQ_DT_F32: return launch_ft<FMT, float>(a, st);
    case WQ_DT_BF16: return launch_ft<FMT, bf16>(a, st);
    default: return launch_ft<FMT, f16>(a, st);
    }
}

} // namespace

hipError_t launch_moe(const MoeArgs &a, int fmt, int dtype, hipStream_t st) {
    switch (fmt) {
    case WQ_I8: return launch_f<WQ_I8>(a, dtype, st);
    case WQ_I4: return launch_f<WQ_I4>(a, dtype, st);
    default: return launch_f<WQ_I2>(a, dtype, st);
    }
}

} // namespace wq
