// Attention of many rows a sequence and key/value head (prefill, chunks of new
// tokens): the cache's tiles are opened once into LDS and shared by the rows.
//
// A block of NW waves takes a tile of RW * NW rows and walks the positions in
// steps of TK. K goes to LDS as f16 rows, V transposed, so both are read back
// as whole 16-byte operands; the next step's codes are in flight from HBM or L2
// meanwhile, and two buffers leave one barrier a step. Per step a wave computes
// for its RW rows
//     S^T[key][row]  = sum_d K[key][d] Q[row][d]           (A = K, B = Q)
//     O^T[d][row]   += sum_key V^T[d][key] P^T[key][row]   (A = V^T, B = P^T)
// with v_mfma_f32_32x32x16 (RW = 32) or 16x16x32 (RW = 16: rows of 256
// elements, whose operands would not fit the registers otherwise). A lane
// holds quads of four consecutive keys of one row in S^T; V's columns stand in
// LDS in the order in which these quads form P^T operands, so probabilities
// never leave their lane. Parts and scales are as in the few-rows kernel, but
// for bf16 queries, whose probabilities enter as one f16 part (2^-11): the prompt
// below takes 202 us so, 245 and more with two, and rounding the output to bf16
// leaves eight times as much (error against 64 bits 1.672e-3 of the root mean
// square, with exact probabilities 1.658e-3). f16 outputs show it (2.98e-4
// against 2.08e-4), so f16 queries take two parts: that prompt in 259 us.
//
// Bound by the vector units and the matrix units in turn (the softmax costs six
// instructions and an exponential an element). With the clocks settled (after a
// hundred passes; the first 20 after idling take a quarter more): 4096 tokens,
// causal, 32 heads over 8, bf16 on an f16 cache, 137 GFLOP in 202 us
// (680 TFLOP/s); eight chunks of up to 511 tokens on up to 5000 positions, f32 on
// int8, 159 GFLOP, 2.5 times that in parts, in 450 us.
#include "attn_common.h"

namespace wq {
namespace {

typedef float f32x16 __attribute__((ext_vector_type(16)));

template <int RW>
struct Mma;
template <>
struct Mma<32> {
    typedef f32x16 acc;
    static __device__ __forceinline__ acc f16(f16x8 a, f16x8 b, acc c) { return __builtin_amdgcn_mfma_f32_32x32x16_f16(a, b, c, 0, 0, 0); }
    static __device__ __forceinline__ acc bf16(f16x8 a, f16x8 b, acc c) {
        return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
    }
};
template <>
struct Mma<16> {
    typedef f32x4 acc;
    static __device__ __forceinline__ acc f16(f16x8 a, f16x8 b, acc c) { return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0); }
    static __device__ __forceinline__ acc bf16(f16x8 a, f16x8 b, acc c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
    }
};

template <typename T, int KIND, int D, int NW>
struct Tiled {
    static constexpr int RW = tiled_rows(D, sizeof(T) == 4); // rows a wave
    // Positions a step. LDS holds 4 buffers of TK * D halves, 75 KiB for rows of 128 and 256: two four-wave blocks a CU. Of
    // eight waves a CU holds one block, whose 164 to 241 registers leave two waves a SIMD.
    static constexpr int TK = D == 256 ? 32 : 64;
    static constexpr int NT = 64 * NW, R = RW * NW;
    static constexpr int NG = 64 / RW;               // lanes that share a row
    static constexpr int CH = D / 8, CV = TK / 8;    // 16-byte chunks of a K row and of a V^T row in LDS
    static constexpr int KS = D / (8 * NG);          // steps of a K operand
    static constexpr int KBN = TK / RW, DB = D / RW; // blocks of S^T and of O^T
    static constexpr int QB = RW * RW / 256;         // quads a lane holds of a block
    static constexpr int NQ = KBN * QB;              // quads a lane holds of a step: keys 4 NG q + 4 g + 0..3
    static constexpr int ST = NQ / 2;                // steps of a V operand: quads 2s, 2s + 1
    static constexpr int HV = RW == 32 ? 2 : 1;      // a step is taken in so many parts (registers)
    static constexpr int KBH = KBN / HV, NQH = NQ / HV, STH = ST / HV;
    static constexpr int P = sizeof(T) == 4 ? 2 : 1; // f16 parts of q
    static constexpr bool BF = P == 2 && KIND != WQ_KV_F16;
    static constexpr int PP = BF ? 3 : sizeof(T) == 4 || std::is_same<T, f16>::value ? 2 : 1;            // parts of p
    static constexpr int KU = TK * CH / NT;          // 8-code units of K a thread brings
    static constexpr int KW = KIND == WQ_KV_F16 ? 4 : KIND == WQ_KV_I8 ? 2 : 1; // words of one
    static constexpr int DG = TK * 32 / NT >= 4 ? 32 : 64; // parts of a V row
    static constexpr int VK = TK * DG / NT;          // keys of V a thread brings, VE codes each
    static constexpr int VE = D / DG;
    // In LDS, rows end with 16 bytes of padding (lanes that read 16 bytes of consecutive rows meet no bank twice),
    // and V^T's row of element d is row d / VE of group d % VE, groups 256 / VE bytes apart besides: threads write
    // rows of one group, lanes read rows of all, both without conflicts. An operand is then a lane's base plus a
    // constant: no address arithmetic, one register.
    static constexpr int KROW = 16 * (CH + 1), KSIZE = TK * KROW;
    static constexpr int VROW = 16 * (CV + 1), VGROUP = DG * VROW + 256 / VE, VSIZE = VE * VGROUP;
    static constexpr int VB = KIND == WQ_KV_F16 ? 2 * VE : KIND == WQ_KV_I8 ? VE : VE / 2;
    static constexpr int VW = VB < 4 ? 1 : VB / 4;
};

template <typename T, int KIND, int D, int NW, typename OFF>
__global__ __launch_bounds__(64 * NW, 2) void attn_tiled_kernel(const AttnArgs a, const Partials pt, const int vec) {
    typedef Tiled<T, KIND, D, NW> F;
    constexpr int RW = F::RW, NG = F::NG, TK = F::TK, P = F::P;
    typedef typename Mma<RW>::acc acc;
    __shared__ __align__(16) uint8_t sk[2 * F::KSIZE];
    __shared__ __align__(16) uint8_t sv[2 * F::VSIZE];
    __shared__ OFF s_off[4][TK], s_sc[4][TK]; // rows (bytes) and scales (floats) of a step's positions
    __shared__ float s_ks[2][TK], s_vs[2][TK], s_big[2];
    __shared__ uint64_t s_mask[4];
    __shared__ int s_bad[3]; // of step i at i % 3: set a step before its use, cleared a step after

    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int n = lane & (RW - 1), g = lane / RW;
    const int G = a.H / a.c.heads;
    const int kvh = blockIdx.x % a.c.heads;
    // heads, then tiles, then splits: neighbours have equal work. Blocks go to the shader engines in turn, and where
    // every other one is short or empty half the engines would get all the work.
    const long rest = blockIdx.x / a.c.heads, tiles = tile_count(a.b.T, G, F::R, a.b.B);
    const int split = (int)(rest / tiles);
    const Tile t = find_tile<F::R>(a.b, a.c.page, G, rest % tiles, lane);
    if (t.rows == 0) return;
    int lo, hi, lo_max, hi_min;
    seen_range(t, t.row0 / G, a.causal, a.window, &lo, &hi_min);
    seen_range(t, (t.row0 + t.rows - 1) / G, a.causal, a.window, &lo_max, &hi);
    const Span sp = find_span(TK, lo, hi, pt.least, pt.nsplit);
    if (split >= sp.splits) return;
    const int blk0 = split * sp.per, blk1 = min(sp.blocks, blk0 + sp.per);

    // this lane's row and Q
    const int r_in = wave * RW + n;
    const bool live = r_in < t.rows;
    const int row = t.row0 + (live ? r_in : 0), tok = row / G, head = kvh * G + row % G;
    int row_lo, row_hi;
    seen_range(t, tok, a.causal, a.window, &row_lo, &row_hi);
    // what the wave's rows see: nothing outside [w_lo, w_hi), all of [w_lo_max, w_hi_min)
    int w_lo = 0, w_hi = 0, w_lo_max = 0, w_hi_min = 0;
    const bool working = wave * RW < t.rows;
    if (working) {
        seen_range(t, (t.row0 + wave * RW) / G, a.causal, a.window, &w_lo, &w_hi_min);
        seen_range(t, (t.row0 + min(wave * RW + RW, t.rows) - 1) / G, a.causal, a.window, &w_lo_max, &w_hi);
    }
    float rs;
    f16x8 q[F::KS][P];
    {
        const T *src = (const T *)a.q + (long)(t.tok0 + tok) * a.qt + (long)head * a.qh;
        float top = 0.f;
#pragma unroll
        for (int pass = 0; pass < 2; ++pass) {
            float up = 1.f;
            if (pass == 1) {
                const int e = head_room(row_max<NG>(top));
                // the scale's sign goes to q, and a scale of zero too, so that rs > 0 and -inf * rs stays -inf
                up = a.scale < 0.f ? -pow2(e) : a.scale == 0.f ? 0.f : pow2(e);
                rs = fmaxf(fabsf(a.scale) * kLog2e * pow2(-e), 0x1p-126f);
            }
#pragma unroll
            for (int s = 0; s < F::KS; ++s) {
                const int d0 = (s * NG + g) * 8;
                float u[8], v[8];
                if (vec) {
                    load_vec<T, 8>(src + d0, u);
                } else {
#pragma unroll
                    for (int e = 0; e < 8; ++e) u[e] = (float)src[d0 + e];
                }
#pragma unroll
                for (int e = 0; e < 8; ++e) v[e] = live ? u[k_order<KIND>(e)] : 0.f;
                if (pass == 0) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) top = fmaxf(top, fabsf(v[e]));
                } else {
                    uint32_t h[4], l[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const float x0 = v[2 * k] * up, x1 = v[2 * k + 1] * up;
                        h[k] = pack_half(x0, x1);
                        if (P == 2) {
                            const f16x2 y = __builtin_bit_cast(f16x2, h[k]);
                            l[k] = pack_half(x0 - (float)y.x, x1 - (float)y.y);
                        }
                    }
                    q[s][0] = join4(h);
                    if (P == 2) q[s][P - 1] = join4(l);
                }
            }
        }
    }

    const OpenConst oc;
    const uint8_t *kp = a.c.k + (long)kvh * a.c.rh, *vp = a.c.v + (long)kvh * a.c.rh;
    const float *ksp = a.c.ks + (long)kvh * a.c.sh, *vsp = a.c.vs + (long)kvh * a.c.sh;
    const int *table = a.b.table + (long)t.b * a.b.table_stride;

    // Page and place of position `lane` of step i (wave 0); positions that are not there take row 0, which exists.
    struct Key {
        int page, slot;
        bool there;
    };
    auto look = [&](int i) {
        Key k;
        const int pos = position(sp.base, i, TK, lane);
        k.there = i < blk1 && (TK == 64 || lane < TK) && pos >= lo && pos < hi;
        const int idx = page_index(a.c, pos);
        k.slot = pos - idx * a.c.page;
        k.page = k.there ? table[idx] : -1;
        return k;
    };
    struct Place {
        OFF row, scale;
        bool ok;
        uint64_t mask;
    };
    auto place = [&](const Key &k) {
        Place p;
        p.ok = k.there && k.page >= 0 && k.page < a.c.pages;
        const OFF page = p.ok ? k.page : 0, slot = p.ok ? k.slot : 0;
        p.row = page * (OFF)a.c.rp + slot * (OFF)a.c.rs;
        p.scale = page * (OFF)a.c.sp + slot * (OFF)a.c.ss;
        p.mask = __ballot(p.ok);
        return p;
    };
    // Bringing a step's places and scales is spread over three waves (0: places, 1: keys' scales, 2: values' scales):
    // the others wait at the barrier for the slowest.
    auto put_place = [&](int slot, const Place &p) {
        if (TK == 64 || lane < TK) {
            s_off[slot][lane] = p.row;
            s_sc[slot][lane] = p.scale;
        }
        if (lane == 0) s_mask[slot] = p.mask;
    };
    auto get_scale = [&](int slot) {
        const OFF at = s_sc[slot][lane & (TK - 1)];
        return wave == 1 ? ksp[at] : vsp[at];
    };
    auto put_scale = [&](int buf, int slot, float x) {
        x = s_mask[slot] >> lane & 1 ? x : 0.f;
        if (TK == 64 || lane < TK) (wave == 1 ? s_ks : s_vs)[buf][lane] = x;
        if (!F::BF && wave == 2) {
            const float big = wave_max(fabsf(x));
            if (lane == 0) s_big[buf] = big;
        }
    };

    // A thread's share of a step: KU units of K, VK keys of V.
    uint32_t rk[F::KU][F::KW], rv[F::VK][F::VW];
    const int dg = tid & (F::DG - 1), hc = tid / F::DG;
    const int vc = F::VK == 8 ? hc : hc >> 1; // its chunk of V^T: keys v0 .. v0+3 and (VK = 8) v0 + 4 NG .. + 3
    const int v0 = (vc / NG) * 8 * NG + (vc % NG) * 4 + (F::VK == 8 ? 0 : (hc & 1) * 4 * NG);
    auto fetch_k = [&](const OFF *off) {
#pragma unroll
        for (int u = 0; u < F::KU; ++u) {
            const int x = u * F::NT + tid;
            load_words<4 * F::KW>(kp + (off[x / F::CH] + (OFF)((x % F::CH) * 4 * F::KW)), rk[u]);
        }
    };
    auto fetch_v = [&](const OFF *off) {
#pragma unroll
        for (int k = 0; k < F::VK; ++k)
            load_words<F::VB>(vp + (off[v0 + (k & 3) + (k >> 2) * 4 * NG] + (OFF)(dg * F::VB)), rv[k]);
    };
    // ... opened into LDS
    auto store_k = [&](int buf) {
#pragma unroll
        for (int u = 0; u < F::KU; ++u) {
            const int x = u * F::NT + tid;
            uint32_t w[4];
            if constexpr (KIND == WQ_KV_F16) {
#pragma unroll
                for (int k = 0; k < 4; ++k) w[k] = rk[u][k];
            } else if constexpr (KIND == WQ_KV_I8) {
                open_i8(rk[u][0], w);
                open_i8(rk[u][1], w + 2);
            } else {
                open_i4(oc, rk[u][0], w);
            }
            *reinterpret_cast<u32x4 *>(sk + buf * F::KSIZE + x / F::CH * F::KROW + x % F::CH * 16) = u32x4{w[0], w[1], w[2], w[3]};
        }
    };
    // `edge`: some rows see less than others or not every position is there.
    auto store_v = [&](int buf, int step, uint64_t mask, bool edge) {
        if constexpr (KIND == WQ_KV_F16) {
            // An infinity or a NaN among the codes must not reach rows that do not see it (0 * NaN):
            // where rows differ in what they see, such codes leave the operands and are looked up at the end.
            if (edge) {
                bool bad = false;
#pragma unroll
                for (int k = 0; k < F::VK; ++k) {
                    const bool gone = !(mask >> (v0 + (k & 3) + (k >> 2) * 4 * NG) & 1);
#pragma unroll
                    for (int w = 0; w < F::VW; ++w) {
                        uint32_t x = gone ? 0u : rv[k][w];
                        const bool b0 = (x & 0x7c00u) == 0x7c00u, b1 = (x & 0x7c000000u) == 0x7c000000u;
                        bad = bad || b0 || b1;
                        x = b0 ? x & 0xffff0000u : x;
                        rv[k][w] = b1 ? x & 0xffffu : x;
                    }
                }
                if (bad) s_bad[step % 3] = 1;
            }
        }
        uint32_t o[F::VE][F::VK / 2];
#pragma unroll
        for (int k = 0; k < F::VK / 2; ++k) {
            const uint32_t *x = rv[2 * k], *y = rv[2 * k + 1];
            if constexpr (KIND == WQ_KV_F16) {
#pragma unroll
                for (int e = 0; e < F::VE; ++e) o[e][k] = __builtin_amdgcn_perm(y[e / 2], x[e / 2], e & 1 ? 0x07060302u : 0x05040100u);
            } else if constexpr (KIND == WQ_KV_I8) {
#pragma unroll
                for (int e = 0; e < F::VE; ++e) {
                    const uint32_t sel = 0x0c000c00u | (uint32_t)(e & 3) | (uint32_t)(4 + (e & 3)) << 16;
                    o[e][k] = F::BF ? high_halves(byte_i8(x[e / 4], e & 3), byte_i8(y[e / 4], e & 3))
                                    : pk_add(__builtin_amdgcn_perm(y[e / 4], x[e / 4], sel) ^ 0x64806480u, -1152.f);
                }
            } else if constexpr (F::BF) {
                const uint32_t x0 = x[0] ^ 0x88888888u, y0 = y[0] ^ 0x88888888u, x1 = x0 >> 4, y1 = y0 >> 4;
#pragma unroll
                for (int e = 0; e < F::VE; ++e)
                    o[e][k] = e & 1 ? high_halves(nibble_i4(x1, e / 2), nibble_i4(y1, e / 2)) : high_halves(nibble_i4(x0, e / 2), nibble_i4(y0, e / 2));
            } else {
#pragma unroll
                for (int e = 0; e < F::VE; e += 4) {
                    uint32_t w[4];
                    open_i4(oc, __builtin_amdgcn_perm(y[0], x[0], e ? 0x07060302u : 0x05040100u), w);
#pragma unroll
                    for (int j = 0; j < 4 && e + j < F::VE; ++j) o[e + j][k] = w[j];
                }
            }
        }
#pragma unroll
        for (int e = 0; e < F::VE; ++e) {
            uint8_t *at = sv + buf * F::VSIZE + e * F::VGROUP + dg * F::VROW + vc * 16;
            if constexpr (F::VK == 8)
                *reinterpret_cast<u32x4 *>(at) = u32x4{o[e][0], o[e][1], o[e][2], o[e][3]};
            else
                *reinterpret_cast<u32x2 *>(at + (hc & 1) * 8) = u32x2{o[e][0], o[e][1]};
        }
    };
    constexpr uint64_t all = TK == 64 ? ~0ull : 0xffffffffull;
    auto is_edge = [&](int i, uint64_t mask) {
        const int t0 = position(sp.base, i, TK, 0);
        return mask != all || t0 < lo_max || t0 > hi_min - TK;
    };

    float ref = -INFINITY, m = -INFINITY, l = 0.f; // p = 2^(s - ref)
    // ref = m - e_min: 2^e_min brings the values' scales below 2^14. A row's sums are rescaled only when its maximum
    // has grown by more than SLACK powers of two since: all rows of a wave wait when one of them does, and among 32
    // rows one's maximum moves in most steps of a start. f16 parts leave little room for it above (2^16) or below.
    constexpr float SLACK = F::BF ? 8.f : F::PP == 1 ? 1.f : 0.f;
    float e_min = F::BF ? 0.f : 127.f;
    acc o[F::DB];
#pragma unroll
    for (int d = 0; d < F::DB; ++d)
#pragma unroll
        for (int k = 0; k < 4 * F::QB; ++k) o[d][k] = 0.f;

    // Operands are read from LDS a fixed number of matrix operations ahead and the order is pinned: left to
    // itself the scheduler puts every read right before its use, and each operation waits out the LDS's latency.
    constexpr int KN = F::KBH * F::KS, VN = F::STH * F::DB; // operands of a part
    constexpr int KWANT = P == 1 ? 6 : 4, VWANT = F::PP == 1 ? 6 : F::PP == 2 ? 4 : 3;
    constexpr int KAHEAD = KWANT < KN ? KWANT : KN, VAHEAD = VWANT < VN ? VWANT : VN;
    const int k_lane = n * F::KROW + g * 16, v_lane = n % F::VE * F::VGROUP + n / F::VE * F::VROW + g * 16;
    acc s[F::KBH];
    auto scores = [&](int kbuf, int h, auto beside) { // S^T of part h from K buffer kbuf; beside(0 .. NQH - 1) as reads end
        constexpr int N = KN;
        f16x8 fr[KAHEAD];
        const uint8_t *from = sk + kbuf * F::KSIZE + h * F::KBH * RW * F::KROW + k_lane;
        auto read = [&](int x) { return *reinterpret_cast<const f16x8 *>(from + x % F::KBH * RW * F::KROW + x / F::KBH * NG * 16); };
#pragma unroll
        for (int x = 0; x < KAHEAD; ++x) fr[x] = read(x);
#pragma unroll
        for (int kb = 0; kb < F::KBH; ++kb)
#pragma unroll
            for (int k = 0; k < 4 * F::QB; ++k) s[kb][k] = 0.f;
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int x = 0; x < N; ++x) {
#pragma unroll
            for (int k = 0; k < P; ++k) s[x % F::KBH] = Mma<RW>::f16(fr[x % KAHEAD], q[x / F::KBH][k], s[x % F::KBH]);
            if (x + KAHEAD < N) {
                fr[x % KAHEAD] = read(x + KAHEAD);
            } else {
                constexpr int PER = (F::NQH + KAHEAD - 1) / KAHEAD;
#pragma unroll
                for (int k = 0; k < PER; ++k)
                    if ((x + KAHEAD - N) * PER + k < F::NQH) beside((x + KAHEAD - N) * PER + k);
            }
            __builtin_amdgcn_sched_barrier(0);
        }
    };
    // does the wave work on step i?
    auto active = [&](int i) { return working && i < blk1 && sp.base + i * TK < w_hi && sp.base + i * TK > w_lo - TK; };

    // Step c of this split works on block blk0 + c. Before its barrier: its K, V and scales, places of it and the next.
    if (wave == 0) {
        const Key k0 = look(blk0), k1 = look(blk0 + 1);
        put_place(0, place(k0));
        put_place(1, place(k1));
        if (lane == 0) s_bad[0] = s_bad[1] = s_bad[2] = 0;
    }
    __syncthreads();
    if (wave == 1 || wave == 2) put_scale(0, 0, get_scale(0));
    if (blk1 > blk0) {
        fetch_k(s_off[0]);
        fetch_v(s_off[0]);
        store_k(0);
        store_v(0, 0, s_mask[0], is_edge(blk0, s_mask[0]));
    }
    __syncthreads();

    int bad_from = blk1, bad_to = blk0; // steps that codes were taken out of
    for (int i = blk0; i < blk1; ++i) {
        const int c = i - blk0, buf = c & 1, t0 = sp.base + i * TK;
        const uint64_t mask = s_mask[c & 3], mask_next = s_mask[(c + 1) & 3];
        const float big_all = F::BF ? 0.f : s_big[buf];
        if (KIND == WQ_KV_F16 && s_bad[c % 3]) {
            bad_from = min(bad_from, i);
            bad_to = i + 1;
        }
        fetch_k(s_off[(c + 1) & 3]); // past the last step: row 0 again, unused
        fetch_v(s_off[(c + 1) & 3]);
        Key key2;
        float scale1 = 0.f;
        if (wave == 0) key2 = look(i + 2);
        if (wave == 1 || wave == 2) scale1 = get_scale((c + 1) & 3);
        if (active(i)) {
#pragma unroll
        for (int h = 0; h < F::HV; ++h) {
            f32x4 ksq[F::NQH], vsq[F::NQH]; // scales of keys and values, read ahead of their use
            const float *ks_at = &s_ks[buf][h * (TK / F::HV) + 4 * g], *vs_at = &s_vs[buf][h * (TK / F::HV) + 4 * g];
            __builtin_amdgcn_s_setprio(1);
            scores(buf, h, [&](int j) { ksq[j] = *reinterpret_cast<const f32x4 *>(ks_at + 4 * NG * j); });
            __builtin_amdgcn_s_setprio(0);
#pragma unroll
            for (int j = 0; j < F::NQH; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) s[j / F::QB][4 * (j % F::QB) + e] *= ksq[j][e];
#pragma unroll
            for (int j = 0; j < F::NQH; ++j) vsq[j] = *reinterpret_cast<const f32x4 *>(vs_at + 4 * NG * j);
            __builtin_amdgcn_sched_barrier(0);
            float big = big_all;
            const bool edge = mask != all || t0 < w_lo_max || t0 > w_hi_min - TK;
            // the lane's row sees key 4 g + k of the part: bit k
            const uint64_t sees = seen_bits(mask >> (4 * g), row_lo - t0 - 4 * g, row_hi - t0 - 4 * g) >> (h * (TK / F::HV));
            if (edge) { // a key that a row does not see scores -inf there
                float most = 0.f;
#pragma unroll
                for (int j = 0; j < F::NQH; ++j) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        s[j / F::QB][4 * (j % F::QB) + e] = where_seen(sees, 4 * NG * j + e, s[j / F::QB][4 * (j % F::QB) + e], -INFINITY);
                        if (!F::BF) most = fmaxf(most, fabsf(where_seen(sees, 4 * NG * j + e, vsq[j][e], 0.f)));
                    }
                }
                if (!F::BF) big = row_max<NG>(most);
            }
            float top = -INFINITY;
#pragma unroll
            for (int j = 0; j < F::NQH; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) top = fmaxf(top, s[j / F::QB][4 * (j % F::QB) + e]);
            const float now = row_max<NG>(top) * rs;
            float grow = 1.f;
            const float room = F::BF ? 0.f : fminf(e_min, scale_room(big, 14));
            // rows that move: the maximum has left the slack, or a value's scale its room (or is not a number)
            const bool moves = !(now <= m + SLACK) || room < e_min;
            if (__ballot(moves)) {
                const float was = ref;
                m = moves ? fmaxf(m, now) : m;
                e_min = moves ? room : e_min;
                ref = m == -INFINITY ? -INFINITY : m - e_min;
                grow = half_way(was - (m == -INFINITY ? 0.f : ref));
#pragma unroll
                for (int d = 0; d < F::DB; ++d) o[d] *= grow * grow;
            }
            const float base = m == -INFINITY ? 0.f : ref;
            float sum = 0.f;
#pragma unroll
            for (int j = 0; j < F::NQH; ++j) {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float p = __builtin_amdgcn_exp2f(fmaf(s[j / F::QB][4 * (j % F::QB) + e], rs, -base));
                    sum += p;
                    s[j / F::QB][4 * (j % F::QB) + e] = p * vsq[j][e];
                }
            }
            if (edge) { // ... and takes no part of the value, whatever its scale (0 * NaN)
#pragma unroll
                for (int j = 0; j < F::NQH; ++j)
#pragma unroll
                    for (int e = 0; e < 4; ++e) s[j / F::QB][4 * (j % F::QB) + e] = where_seen(sees, 4 * NG * j + e, s[j / F::QB][4 * (j % F::QB) + e], 0.f);
            }
            l = l * grow * grow + sum;
            constexpr int N = VN;
            __builtin_amdgcn_s_setprio(1);
            f16x8 fr[VAHEAD];
            const uint8_t *from = sv + buf * F::VSIZE + h * F::STH * NG * 16 + v_lane;
            auto read = [&](int x) { return *reinterpret_cast<const f16x8 *>(from + x % F::DB * (RW / F::VE) * F::VROW + x / F::DB * NG * 16); };
#pragma unroll
            for (int x = 0; x < VAHEAD; ++x) fr[x] = read(x);
#pragma unroll
            for (int st = 0; st < F::STH; ++st) {
                uint32_t pb[F::PP][4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int j = 2 * st + (k >> 1), at = 4 * (j % F::QB) + 2 * (k & 1);
                    const float y0 = s[j / F::QB][at], y1 = s[j / F::QB][at + 1];
                    if constexpr (F::BF) {
                        uint32_t w[3];
                        split3(y0, y1, w);
                        pb[0][k] = w[0];
                        pb[1][k] = w[1];
                        pb[2][k] = w[2];
                    } else {
                        pb[0][k] = pack_half(y0, y1);
                        if constexpr (F::PP == 2) {
                            const f16x2 z = __builtin_bit_cast(f16x2, pb[0][k]);
                            pb[1][k] = pack_half(y0 - (float)z.x, y1 - (float)z.y);
                        }
                    }
                }
                __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                for (int d = 0; d < F::DB; ++d) {
                    const int x = st * F::DB + d;
#pragma unroll
                    for (int k = 0; k < F::PP; ++k)
                        o[d] = F::BF ? Mma<RW>::bf16(fr[x % VAHEAD], join4(pb[k]), o[d]) : Mma<RW>::f16(fr[x % VAHEAD], join4(pb[k]), o[d]);
                    if (x + VAHEAD < N) fr[x % VAHEAD] = read(x + VAHEAD);
                    __builtin_amdgcn_sched_barrier(0);
                }
            __builtin_amdgcn_s_setprio(0);
            }
        }
        }
        if (KIND == WQ_KV_F16 && tid == 0) s_bad[(c + 2) % 3] = 0;
        store_k(buf ^ 1);
        store_v(buf ^ 1, c + 1, mask_next, is_edge(i + 1, mask_next));
        if (wave == 0) put_place((c + 2) & 3, place(key2));
        if (wave == 1 || wave == 2) put_scale(buf ^ 1, (c + 1) & 3, scale1);
        __syncthreads();
    }

    if (!working) return;
    if constexpr (KIND == WQ_KV_F16) {
        // Codes that are not finite and were taken out: what sees one is not finite either, whatever else it sums. Here
        // and not in the step, where this loop's registers would add to all the others (8 spilled, 52 with two parts).
        const int last = (int)min((long)sp.base + (long)bad_to * TK, (long)w_hi);
        for (int pos = max(position(sp.base, bad_from, TK, 0), w_lo); bad_from < bad_to && pos < last; ++pos) {
            const int idx = page_index(a.c, pos), page = table[idx], slot = pos - idx * a.c.page;
            if (page < 0 || page >= a.c.pages) continue;
            const f16 *src = (const f16 *)(vp + ((OFF)page * (OFF)a.c.rp + (OFF)slot * (OFF)a.c.rs));
            const float scale = vsp[(OFF)page * (OFF)a.c.sp + (OFF)slot * (OFF)a.c.ss];
            if (pos >= row_lo && pos < row_hi) {
#pragma unroll
                for (int d = 0; d < F::DB; ++d)
#pragma unroll
                    for (int k = 0; k < 4 * F::QB; ++k) {
                        const float code = (float)src[d * RW + 4 * NG * (k >> 2) + 4 * g + (k & 3)];
                        if (!(fabsf(code) < INFINITY)) o[d][k] = fmaf(scale, code, o[d][k]);
                    }
            }
        }
    }
    l = row_sum<NG>(l);
    if (!live) return;
    const long at = (long)(t.tok0 + tok) * a.H + head;
    constexpr float unit = F::BF && KIND == WQ_KV_I4 ? 16.f : 1.f;
    if (sp.splits > 1) {
        float *dst = pt.part + (at * pt.nsplit + split) * D;
#pragma unroll
        for (int d = 0; d < F::DB; ++d)
#pragma unroll
            for (int j = 0; j < F::QB; ++j)
                *reinterpret_cast<f32x4 *>(dst + d * RW + 4 * NG * j + 4 * g) =
                    f32x4{o[d][4 * j] * unit, o[d][4 * j + 1] * unit, o[d][4 * j + 2] * unit, o[d][4 * j + 3] * unit};
        if (g == 0) {
            pt.ml[(at * pt.nsplit + split) * 2] = ref;
            pt.ml[(at * pt.nsplit + split) * 2 + 1] = l;
        }
        return;
    }
    const bool none = m == -INFINITY && l == 0.f;
    const float inv = none ? 0.f : unit / l;
    T *dst = (T *)a.o + (long)(t.tok0 + tok) * a.ot + (long)head * a.oh;
#pragma unroll
    for (int d = 0; d < F::DB; ++d)
#pragma unroll
        for (int j = 0; j < F::QB; ++j) {
            float y[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) y[e] = none ? 0.f : o[d][4 * j + e] * inv;
            T *p = dst + d * RW + 4 * NG * j + 4 * g;
            if (vec) {
                store_vec<T, 4>(p, y);
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e) p[e] = (T)y[e];
            }
        }
    if (a.lse && g == 0) a.lse[at] = none ? -INFINITY : (ref + __builtin_amdgcn_logf(l)) * kLn2;
}

template <typename T, int KIND, int D, int NW>
hipError_t launch_nw(const AttnArgs &a, const AttnPlan &p, const Partials &pt, bool vec, bool wide, hipStream_t st) {
    typedef Tiled<T, KIND, D, NW> F;
    const long blocks = tile_count(a.b.T, a.H / a.c.heads, F::R, a.b.B) * p.nsplit * a.c.heads;
    if (p.rows != F::R) return hipErrorInvalidValue;
    if (blocks > kMaxThreads / F::NT) return hipErrorNotSupported;
    const dim3 grid((unsigned)blocks), block(F::NT);
    if (wide)
        hipLaunchKernelGGL((attn_tiled_kernel<T, KIND, D, NW, uint64_t>), grid, block, 0, st, a, pt, vec ? 1 : 0);
    else
        hipLaunchKernelGGL((attn_tiled_kernel<T, KIND, D, NW, uint32_t>), grid, block, 0, st, a, pt, vec ? 1 : 0);
    return hipGetLastError();
}

template <typename T, int KIND, int D>
hipError_t launch_d(const AttnArgs &a, const AttnPlan &p, const Partials &pt, bool vec, bool wide, hipStream_t st) {
    if (p.waves == 4) return launch_nw<T, KIND, D, 4>(a, p, pt, vec, wide, st);
    if constexpr (D > 64) // rows of 64 always take four waves
        return launch_nw<T, KIND, D, 8>(a, p, pt, vec, wide, st);
    return hipErrorInvalidValue;
}

template <typename T, int KIND>
hipError_t launch_dim(const AttnArgs &a, const AttnPlan &p, const Partials &pt, int dim, bool vec, bool wide, hipStream_t st) {
    switch (dim) {
    case 64: return launch_d<T, KIND, 64>(a, p, pt, vec, wide, st);
    case 128: return launch_d<T, KIND, 128>(a, p, pt, vec, wide, st);
    default: return launch_d<T, KIND, 256>(a, p, pt, vec, wide, st);
    }
}

template <typename T>
hipError_t launch_t(const AttnArgs &a, const AttnPlan &p, const Partials &pt, int kind, int dim, bool vec, bool wide, hipStream_t st) {
    switch (kind) {
    case WQ_KV_F16: return launch_dim<T, WQ_KV_F16>(a, p, pt, dim, vec, wide, st);
    case WQ_KV_I8: return launch_dim<T, WQ_KV_I8>(a, p, pt, dim, vec, wide, st);
    default: return launch_dim<T, WQ_KV_I4>(a, p, pt, dim, vec, wide, st);
    }
}

} // namespace

hipError_t launch_attn_tiled(const AttnArgs &a, const AttnPlan &p, const Partials &pt, int kind, int dim, int dtype, bool vec,
                             bool wide, hipStream_t st) {
    switch (dtype) {
    case WQ_DT_F32: return launch_t<float>(a, p, pt, kind, dim, vec, wide, st);
    case WQ_DT_BF16: return launch_t<bf16>(a, p, pt, kind, dim, vec, wide, st);
    default: return launch_t<f16>(a, p, pt, kind, dim, vec, wide, st);
    }
}

} // namespace wq
