// Attention of a few rows a sequence and key/value head (decode): the cache
// streams once from HBM straight into matrix operands.
//
// A block takes one tile of 16 * MT rows and one split of its positions; its
// four waves take every fourth block of TK positions and join at the end. Per
// block of positions a wave computes, with v_mfma_f32_16x16x32_f16,
//     S^T[key][row]  = sum_d K[key][d] Q[row][d]      (A = K, B = Q)
//     O^T[d][row]   += sum_key V^T[d][key] P^T[key][row]  (A = V^T, B = P^T)
// Every lane holds four keys of one row of S^T in exactly the order in which
// it supplies P^T, so probabilities never cross lanes; the order of the
// elements d inside a K operand and of the keys inside a V operand is free as
// long as both sides agree, so K rows are loaded as whole 16-byte runs and V
// rows as D/16 consecutive elements a lane, and both become operands in
// registers (codes are exact in f16). Scales never touch the codes: a key's
// scale multiplies its score, a value's its probability.
//
// A query row is brought to [2^13, 2^14) by a power of two; f32 rows enter as
// two f16 parts (22 bits and more), 16-bit types exactly as one. A probability
// times its value's scale enters, for f32 and integer codes, as three bf16
// parts (all 24 bits, any magnitude; the codes are exact in bf16 too); else as
// two f16 parts (22 bits; with one, 2^-11, f16 outputs were 1.4 times as far
// from 64 bits and the batch below 1 us faster), the exponent of all of a row's
// probabilities shifted so that times its largest value scale so far they stay
// below 2^14.
//
// Next to the bytes the opening of codes is what costs: K's and V's of a step
// are about 370 of its 850 vector instructions in int4. 64 ragged sequences up to
// 8192 positions (48 heads over 8, int8, 672 MB) take 139 us (4.8 TB/s); four of
// 131072 in int4 (571 MB) 143 us (4.0 TB/s, vector units 69 % busy); one of 1500
// 8 us (medians of the kernel alone, clocks settled).
#include "attn_common.h"

namespace wq {
namespace {

template <typename T, int KIND, int D, int MT>
struct Few {
    static constexpr int RB = KIND == WQ_KV_F16 ? 2 * D : KIND == WQ_KV_I8 ? D : D / 2; // row bytes
    static constexpr int EPB2 = KIND == WQ_KV_F16 ? 1 : KIND == WQ_KV_I8 ? 2 : 4;       // codes per two bytes
    static constexpr int P = sizeof(T) == 4 ? 2 : 1;                                    // f16 parts of q
    static constexpr bool BF = P == 2 && KIND != WQ_KV_F16;                             // p and v in bf16
    static constexpr int PP = BF ? 3 : 2;                                               // parts of p
    static constexpr int TK = RB <= 64 ? 64 : 32;                                      // positions a block
    static constexpr int LB = RB / 4 < 16 ? RB / 4 : 16; // bytes of one K load
    static constexpr int KL = RB / 4 / LB;               // K loads a lane and key
    static constexpr int KW = LB / 4;                    // words of one
    static constexpr int VB = RB / 16;                   // bytes of a lane's part of a V row
    static constexpr int VW = VB < 4 ? 1 : VB / 4;       // words of it
    static constexpr int KB = TK / 16, VG = TK / 32, DT = D / 16, KS = D / 32;
};

template <typename T, int KIND, int D, int MT, typename OFF>
__global__ __launch_bounds__(256) void attn_few_kernel(const AttnArgs a, const Partials pt, const int vec) {
    typedef Few<T, KIND, D, MT> F;
    constexpr int R = 16 * MT, TK = F::TK, P = F::P;
    struct Meta {
        OFF off[2][TK];
        float ks[2][TK], vs[2][TK];
    };
    __shared__ union {
        Meta meta[4];
        float o[2][R][D + 4];
    } sh;
    __shared__ float sh_m[4][R], sh_l[4][R];

    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int n = lane & 15, g = lane >> 4;
    const int G = a.H / a.c.heads;
    const int kvh = blockIdx.x % a.c.heads;
    const long rest = blockIdx.x / a.c.heads;
    const int split = (int)(rest % pt.nsplit);
    const Tile t = find_tile<R>(a.b, a.c.page, G, rest / pt.nsplit, lane);
    if (t.rows == 0) return;
    int lo, hi, lo_max, hi_min;
    seen_range(t, t.row0 / G, a.causal, a.window, &lo, &hi_min);
    seen_range(t, (t.row0 + t.rows - 1) / G, a.causal, a.window, &lo_max, &hi);
    const Span sp = find_span(TK, lo, hi, pt.least, pt.nsplit);
    if (split >= sp.splits) return;
    const int blk0 = split * sp.per, blk1 = min(sp.blocks, blk0 + sp.per);

    // rows of this lane; Q as it comes
    int row_lo[MT], row_hi[MT];
    bool live[MT];
    float qv[MT][F::KS][8];
    auto load_q = [&]() {
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
            const int r = mt * 16 + n;
            live[mt] = r < t.rows;
            const int i = (t.row0 + (live[mt] ? r : 0)) / G, j = (t.row0 + (live[mt] ? r : 0)) % G;
            seen_range(t, i, a.causal, a.window, &row_lo[mt], &row_hi[mt]);
            const T *src = (const T *)a.q + (long)(t.tok0 + i) * a.qt + (long)(kvh * G + j) * a.qh;
#pragma unroll
            for (int s = 0; s < F::KS; ++s) {
                // step s: load s / spl of the K row, part s % spl of the lane's run
                constexpr int run = F::LB * F::EPB2 / 2, spl = run / 8;
                const int d0 = (s / spl) * 4 * run + g * run + (s % spl) * 8;
                if (vec) {
                    load_vec<T, 8>(src + d0, qv[mt][s]);
                } else {
#pragma unroll
                    for (int e = 0; e < 8; ++e) qv[mt][s][e] = (float)src[d0 + e];
                }
            }
        }
    };
    float rs[MT];
    f16x8 q[MT][F::KS][P];
    auto open_q = [&]() {
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
            float top = 0.f;
#pragma unroll
            for (int s = 0; s < F::KS; ++s)
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    qv[mt][s][e] = live[mt] ? qv[mt][s][e] : 0.f;
                    top = fmaxf(top, fabsf(qv[mt][s][e]));
                }
            const int e = head_room(row_max<4>(top));
            // the scale's sign goes to q, and a scale of zero too, so that rs > 0 and -inf * rs stays -inf
            const float up = a.scale < 0.f ? -pow2(e) : a.scale == 0.f ? 0.f : pow2(e);
            rs[mt] = fmaxf(fabsf(a.scale) * kLog2e * pow2(-e), 0x1p-126f);
#pragma unroll
            for (int s = 0; s < F::KS; ++s) {
                uint32_t h[4], l[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const float x0 = qv[mt][s][k_order<KIND>(2 * k)] * up, x1 = qv[mt][s][k_order<KIND>(2 * k + 1)] * up;
                    h[k] = pack_half(x0, x1);
                    if (P == 2) {
                        const f16x2 y = __builtin_bit_cast(f16x2, h[k]);
                        l[k] = pack_half(x0 - (float)y.x, x1 - (float)y.y);
                    }
                }
                q[mt][s][0] = join4(h);
                if (P == 2) q[mt][s][P - 1] = join4(l);
            }
        }
    };

    const OpenConst oc;
    Meta &meta = sh.meta[wave];
    const uint8_t *kp = a.c.k + (long)kvh * a.c.rh, *vp = a.c.v + (long)kvh * a.c.rh;
    const float *ksp = a.c.ks + (long)kvh * a.c.sh, *vsp = a.c.vs + (long)kvh * a.c.sh;
    const int *table = a.b.table + (long)t.b * a.b.table_stride;

    // Page and place of position `lane` of block i; positions that are not there take row 0, which exists, and scale 0.
    struct Key {
        int page, slot;
        bool there;
    };
    auto look = [&](int i) {
        Key k;
        const int pos = position(sp.base, i, TK, lane);
        k.there = i < blk1 && lane < TK && pos >= lo && pos < hi;
        const int idx = page_index(a.c, pos);
        k.slot = pos - idx * a.c.page;
        k.page = k.there ? table[idx] : -1;
        return k;
    };
    struct Place {
        OFF row, scale; // scale in floats
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
    auto fence = []() {
        asm volatile("" ::: "memory");
        __builtin_amdgcn_wave_barrier();
    };

    uint32_t kr[F::KB][F::KL][F::KW], vr[F::VG][8][F::VW];
    auto load_k = [&](int buf) {
#pragma unroll
        for (int kb = 0; kb < F::KB; ++kb) {
            const OFF off = meta.off[buf][kb * 16 + n] + (OFF)(g * F::LB);
#pragma unroll
            for (int j = 0; j < F::KL; ++j) load_words<F::LB>(kp + off + j * 4 * F::LB, kr[kb][j]);
        }
    };
    auto load_v = [&](int buf) {
#pragma unroll
        for (int kg = 0; kg < F::VG; ++kg)
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const OFF off = meta.off[buf][kg * 32 + (i >> 2) * 16 + 4 * g + (i & 3)] + (OFF)(n * F::VB);
                load_words<F::VB>(vp + off, vr[kg][i]);
            }
    };

    float m[MT], ref[MT], e_min[MT], l[MT]; // p = 2^(s - ref), ref = m - e_min: p times any value scale stays below 2^14
    f32x4 o[MT][F::DT];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
        m[mt] = ref[mt] = -INFINITY;
        e_min[mt] = F::BF ? 0.f : 127.f;
        l[mt] = 0.f;
#pragma unroll
        for (int d = 0; d < F::DT; ++d) o[mt][d] = f32x4{0, 0, 0, 0};
    }

    // the chain q_start -> table -> rows is what a short call waits for: q comes beside it and is opened last
    int i = blk0 + wave;
    uint64_t mask0 = 0, mask1 = 0;
    Place next;
    {
        const Key k0 = look(i), k1 = look(i + 4);
        load_q();
        const Place p0 = place(k0);
        next = place(k1);
        mask0 = p0.mask;
        mask1 = next.mask;
        if (lane < TK) {
            meta.off[0][lane] = p0.row;
            meta.off[1][lane] = next.row;
        }
        const float ks0 = ksp[p0.scale], vs0 = vsp[p0.scale];
        fence();
        load_k(0);
        load_v(0);
        open_q();
        if (lane < TK) {
            meta.ks[0][lane] = p0.ok ? ks0 : 0.f;
            meta.vs[0][lane] = p0.ok ? vs0 : 0.f;
        }
        fence();
    }
    for (int buf = 0; i < blk1; i += 4, buf ^= 1) {
        // in flight through this block: scales of the next, pages of the one after
        const float ks1 = ksp[next.scale], vs1 = vsp[next.scale];
        const Key after = look(i + 8);
        const int t0 = sp.base + i * TK;

        f32x4 s[MT][F::KB];
#pragma unroll
        for (int kb = 0; kb < F::KB; ++kb) {
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) s[mt][kb] = f32x4{0, 0, 0, 0};
#pragma unroll
            for (int st = 0; st < F::KS; ++st) {
                constexpr int spl = F::KS / F::KL; // steps a load
                uint32_t w[4];
                const uint32_t *raw = &kr[kb][st / spl][(st % spl) * (F::KW / spl)];
                if constexpr (KIND == WQ_KV_F16) {
#pragma unroll
                    for (int k = 0; k < 4; ++k) w[k] = raw[k];
                } else if constexpr (KIND == WQ_KV_I8) {
                    open_i8(raw[0], w);
                    open_i8(raw[1], w + 2);
                } else {
                    open_i4(oc, raw[0], w);
                }
                const f16x8 kf = join4(w);
#pragma unroll
                for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                    for (int pl = 0; pl < P; ++pl)
                        s[mt][kb] = __builtin_amdgcn_mfma_f32_16x16x32_f16(kf, q[mt][st][pl], s[mt][kb], 0, 0, 0);
            }
        }
        load_k(buf ^ 1); // past the last block: row 0 again, unused

        f32x4 vsc[MT][F::KB];
#pragma unroll
        for (int kb = 0; kb < F::KB; ++kb) {
            const f32x4 ksc = *reinterpret_cast<const f32x4 *>(&meta.ks[buf][kb * 16 + 4 * g]);
            const f32x4 v = *reinterpret_cast<const f32x4 *>(&meta.vs[buf][kb * 16 + 4 * g]);
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
                vsc[mt][kb] = v;
#pragma unroll
                for (int r = 0; r < 4; ++r) s[mt][kb][r] *= ksc[r];
            }
        }
        constexpr uint64_t all = TK == 64 ? ~0ull : 0xffffffffull;
        const bool edge = mask0 != all || t0 < lo_max || t0 > hi_min - TK;
        if (edge) { // a key that a row does not see scores -inf there and has scale 0, whatever it held
            const uint64_t own = mask0 >> (4 * g);
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
                const uint64_t sees = seen_bits(own, row_lo[mt] - t0 - 4 * g, row_hi[mt] - t0 - 4 * g);
#pragma unroll
                for (int kb = 0; kb < F::KB; ++kb)
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        s[mt][kb][r] = where_seen(sees, kb * 16 + r, s[mt][kb][r], -INFINITY);
                        vsc[mt][kb][r] = where_seen(sees, kb * 16 + r, vsc[mt][kb][r], 0.f);
                    }
            }
        }
        uint32_t ph[MT][F::KB][2][F::PP];
        float pf[MT][F::KB][4]; // f16 codes only: for codes that are not finite
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
            float top = -INFINITY, big = 0.f;
#pragma unroll
            for (int kb = 0; kb < F::KB; ++kb)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    top = fmaxf(top, s[mt][kb][r]);
                    if (!F::BF) big = fmaxf(big, fabsf(vsc[mt][kb][r]));
                }
            m[mt] = fmaxf(m[mt], row_max<4>(top) * rs[mt]);
            if (!F::BF) e_min[mt] = fminf(e_min[mt], scale_room(row_max<4>(big), 14));
            const float was = ref[mt];
            ref[mt] = m[mt] == -INFINITY ? -INFINITY : m[mt] - e_min[mt];
            const float base = m[mt] == -INFINITY ? 0.f : ref[mt];
            const float grow = half_way(was - base);
            float sum = 0.f;
#pragma unroll
            for (int kb = 0; kb < F::KB; ++kb) {
                float y[4];
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const float p = __builtin_amdgcn_exp2f(fmaf(s[mt][kb][r], rs[mt], -base));
                    sum += p;
                    y[r] = p * vsc[mt][kb][r];
                    if (KIND == WQ_KV_F16) pf[mt][kb][r] = y[r];
                }
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const float y0 = y[2 * k], y1 = y[2 * k + 1];
                    if constexpr (F::BF) {
                        split3(y0, y1, ph[mt][kb][k]);
                    } else {
                        ph[mt][kb][k][0] = pack_half(y0, y1);
                        if constexpr (F::PP == 2) {
                            const f16x2 z = __builtin_bit_cast(f16x2, ph[mt][kb][k][0]);
                            ph[mt][kb][k][1] = pack_half(y0 - (float)z.x, y1 - (float)z.y);
                        }
                    }
                }
            }
            l[mt] = l[mt] * grow * grow + sum;
            if (__ballot(grow != 1.f)) {
#pragma unroll
                for (int d = 0; d < F::DT; ++d) o[mt][d] *= grow * grow;
            }
        }

        if constexpr (KIND == WQ_KV_F16) {
            // Where some rows see less than others, an infinity or a NaN among the codes must not
            // reach those that do not see it (0 * NaN): such codes leave the operands, and rows
            // that see them take them by themselves.
            if (edge) {
                bool bad = false;
#pragma unroll
                for (int kg = 0; kg < F::VG; ++kg)
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        const bool gone = !(mask0 >> (kg * 32 + (k >> 2) * 16 + 4 * g + (k & 3)) & 1);
#pragma unroll
                        for (int w = 0; w < F::VW; ++w) {
                            uint32_t x = gone ? 0u : vr[kg][k][w];
                            const bool b0 = (x & 0x7c00u) == 0x7c00u, b1 = (x & 0x7c000000u) == 0x7c000000u;
                            bad = bad || b0 || b1;
                            x = b0 ? x & 0xffff0000u : x;
                            vr[kg][k][w] = b1 ? x & 0xffffu : x;
                        }
                    }
                if (__ballot(bad)) {
                    for (int key = 0; key < TK; ++key) {
                        if (!(mask0 >> key & 1)) continue;
                        const f16 *row = (const f16 *)(vp + meta.off[buf][key]);
                        const int from = (key >> 2 & 3) * 16 + n;
#pragma unroll
                        for (int mt = 0; mt < MT; ++mt) {
                            float y = 0.f;
#pragma unroll
                            for (int kb = 0; kb < F::KB; ++kb)
#pragma unroll
                                for (int r = 0; r < 4; ++r)
                                    if (kb == key >> 4 && r == (key & 3)) y = pf[mt][kb][r];
                            y = __shfl(y, from);
                            if (t0 + key >= row_lo[mt] && t0 + key < row_hi[mt]) {
#pragma unroll
                                for (int d = 0; d < F::DT; ++d)
#pragma unroll
                                    for (int r = 0; r < 4; ++r) {
                                        const float code = (float)row[(4 * g + r) * F::DT + d];
                                        if (!(fabsf(code) < INFINITY)) o[mt][d][r] = fmaf(y, code, o[mt][d][r]);
                                    }
                            }
                        }
                    }
                }
            }
        }
#pragma unroll
        for (int kg = 0; kg < F::VG; ++kg) {
            auto use = [&](int d, const uint32_t *w) {
#pragma unroll
                for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                    for (int k = 0; k < F::PP; ++k) {
                        const uint32_t u[4] = {ph[mt][2 * kg][0][k], ph[mt][2 * kg][1][k], ph[mt][2 * kg + 1][0][k], ph[mt][2 * kg + 1][1][k]};
                        if constexpr (F::BF)
                            o[mt][d] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, join4(w)), __builtin_bit_cast(bf16x8, join4(u)), o[mt][d], 0, 0, 0);
                        else
                            o[mt][d] = __builtin_amdgcn_mfma_f32_16x16x32_f16(join4(w), join4(u), o[mt][d], 0, 0, 0);
                    }
            };
            // operand d: element d of the lane's part of the eight rows
            if constexpr (KIND == WQ_KV_F16) {
#pragma unroll
                for (int d = 0; d < F::DT; ++d) {
                    uint32_t w[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        w[k] = __builtin_amdgcn_perm(vr[kg][2 * k + 1][d / 2], vr[kg][2 * k][d / 2], d & 1 ? 0x07060302u : 0x05040100u);
                    use(d, w);
                }
            } else if constexpr (KIND == WQ_KV_I8) {
#pragma unroll
                for (int d = 0; d < F::DT; ++d) {
                    uint32_t w[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const uint32_t x = vr[kg][2 * k][d / 4], y = vr[kg][2 * k + 1][d / 4];
                        const uint32_t sel = 0x0c000c00u | (uint32_t)(d & 3) | (uint32_t)(4 + (d & 3)) << 16;
                        if constexpr (F::BF)
                            w[k] = high_halves(byte_i8(x, d & 3), byte_i8(y, d & 3));
                        else
                            w[k] = pk_add(__builtin_amdgcn_perm(y, x, sel) ^ 0x64806480u, -1152.f);
                    }
                    use(d, w);
                }
            } else if constexpr (F::BF) { // codes / 16; the join multiplies by 16
#pragma unroll
                for (int d2 = 0; d2 < F::DT; d2 += 8) {
                    uint32_t e[8][2]; // even and odd elements of the eight rows, two's complement
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        e[k][0] = vr[kg][k][d2 / 8] ^ 0x88888888u;
                        e[k][1] = e[k][0] >> 4;
                    }
#pragma unroll
                    for (int d = 0; d < (F::DT < 8 ? F::DT : 8); ++d) {
                        uint32_t w[4];
#pragma unroll
                        for (int k = 0; k < 4; ++k) w[k] = high_halves(nibble_i4(e[2 * k][d & 1], d / 2), nibble_i4(e[2 * k + 1][d & 1], d / 2));
                        use(d2 + d, w);
                    }
                }
            } else {
#pragma unroll
                for (int d4 = 0; d4 < F::DT / 4; ++d4) {
                    uint32_t w[4][4];
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        open_i4(oc, __builtin_amdgcn_perm(vr[kg][2 * k + 1][d4 / 2], vr[kg][2 * k][d4 / 2], d4 & 1 ? 0x07060302u : 0x05040100u), w[k]);
#pragma unroll
                    for (int d = 0; d < 4; ++d) {
                        const uint32_t u[4] = {w[0][d], w[1][d], w[2][d], w[3][d]};
                        use(4 * d4 + d, u);
                    }
                }
            }
        }
        load_v(buf ^ 1);
        // what was in flight for the next blocks
        const Place p2 = place(after);
        fence();
        if (lane < TK) {
            meta.ks[buf ^ 1][lane] = next.ok ? ks1 : 0.f;
            meta.vs[buf ^ 1][lane] = next.ok ? vs1 : 0.f;
            meta.off[buf][lane] = p2.row;
        }
        fence();
        mask0 = mask1;
        mask1 = p2.mask;
        next = p2;
    }

    // join the four waves
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
        l[mt] = row_sum<4>(l[mt]);
        if (g == 0) {
            sh_m[wave][mt * 16 + n] = ref[mt];
            sh_l[wave][mt * 16 + n] = l[mt];
        }
    }
    __syncthreads();
    float M[MT], L[MT];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
        const int r = mt * 16 + n;
        M[mt] = fmaxf(fmaxf(sh_m[0][r], sh_m[1][r]), fmaxf(sh_m[2][r], sh_m[3][r]));
        const float base = M[mt] == -INFINITY ? 0.f : M[mt];
        L[mt] = 0.f;
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            const float h = half_way(sh_m[w][r] - base);
            L[mt] += sh_l[w][r] * h * h;
        }
        const float f = __builtin_amdgcn_exp2f(ref[mt] - base) * (F::BF && KIND == WQ_KV_I4 ? 16.f : 1.f);
#pragma unroll
        for (int d = 0; d < F::DT; ++d) o[mt][d] *= f;
    }
    for (int half = 2; half > 0; half >>= 1) {
        if (wave >= half && wave < 2 * half) {
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int r = 0; r < 4; ++r)
#pragma unroll
                    for (int d = 0; d < F::DT; d += 4)
                        *reinterpret_cast<f32x4 *>(&sh.o[wave - half][mt * 16 + n][(4 * g + r) * F::DT + d]) =
                            f32x4{o[mt][d][r], o[mt][d + 1][r], o[mt][d + 2][r], o[mt][d + 3][r]};
        }
        __syncthreads();
        if (wave < half) {
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int r = 0; r < 4; ++r)
#pragma unroll
                    for (int d = 0; d < F::DT; d += 4) {
                        const f32x4 v = *reinterpret_cast<const f32x4 *>(&sh.o[wave][mt * 16 + n][(4 * g + r) * F::DT + d]);
#pragma unroll
                        for (int k = 0; k < 4; ++k) o[mt][d + k][r] += v[k];
                    }
        }
        __syncthreads();
    }
    if (wave != 0) return;
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
        const int r = mt * 16 + n;
        if (r >= t.rows) continue;
        const int ti = (t.row0 + r) / G, j = (t.row0 + r) % G;
        const long row = (long)(t.tok0 + ti) * a.H + kvh * G + j;
        if (sp.splits > 1) {
            float *dst = pt.part + (row * pt.nsplit + split) * D;
#pragma unroll
            for (int k = 0; k < 4; ++k)
#pragma unroll
                for (int d = 0; d < F::DT; d += 4)
                    *reinterpret_cast<f32x4 *>(dst + (4 * g + k) * F::DT + d) =
                        f32x4{o[mt][d][k], o[mt][d + 1][k], o[mt][d + 2][k], o[mt][d + 3][k]};
            if (g == 0) {
                pt.ml[(row * pt.nsplit + split) * 2] = M[mt];
                pt.ml[(row * pt.nsplit + split) * 2 + 1] = L[mt];
            }
        } else {
            const bool none = M[mt] == -INFINITY && L[mt] == 0.f; // nothing seen
            const float inv = none ? 0.f : 1.0f / L[mt];
            T *dst = (T *)a.o + (long)(t.tok0 + ti) * a.ot + (long)(kvh * G + j) * a.oh;
#pragma unroll
            for (int k = 0; k < 4; ++k)
#pragma unroll
                for (int d = 0; d < F::DT; d += 4) {
                    float y[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) y[e] = none ? 0.f : o[mt][d + e][k] * inv;
                    T *p = dst + (4 * g + k) * F::DT + d;
                    if (vec) {
                        store_vec<T, 4>(p, y);
                    } else {
#pragma unroll
                        for (int e = 0; e < 4; ++e) p[e] = (T)y[e];
                    }
                }
            if (a.lse && g == 0) a.lse[row] = none ? -INFINITY : (M[mt] + __builtin_amdgcn_logf(L[mt])) * kLn2;
        }
    }
}

template <typename T, int KIND, int D, int MT>
hipError_t launch_few(const AttnArgs &a, const AttnPlan &p, const Partials &pt, bool vec, bool wide, hipStream_t st) {
    const long blocks = tile_count(a.b.T, a.H / a.c.heads, 16 * MT, a.b.B) * p.nsplit * a.c.heads;
    if (p.rows != 16 * MT || p.step != Few<T, KIND, D, MT>::TK) return hipErrorInvalidValue;
    if (blocks > kMaxThreads / 256) return hipErrorNotSupported;
    const dim3 grid((unsigned)blocks), block(256);
    if (wide)
        hipLaunchKernelGGL((attn_few_kernel<T, KIND, D, MT, uint64_t>), grid, block, 0, st, a, pt, vec ? 1 : 0);
    else
        hipLaunchKernelGGL((attn_few_kernel<T, KIND, D, MT, uint32_t>), grid, block, 0, st, a, pt, vec ? 1 : 0);
    return hipGetLastError();
}

template <typename T, int KIND, int D>
hipError_t launch_mt(const AttnArgs &a, const AttnPlan &p, const Partials &pt, bool vec, bool wide, hipStream_t st) {
    if constexpr (D <= 128) // two tiles of 256-element rows do not fit the registers
        if (p.rows == 32) return launch_few<T, KIND, D, 2>(a, p, pt, vec, wide, st);
    return launch_few<T, KIND, D, 1>(a, p, pt, vec, wide, st);
}

template <typename T, int KIND>
hipError_t launch_dim(const AttnArgs &a, const AttnPlan &p, const Partials &pt, int dim, bool vec, bool wide, hipStream_t st) {
    switch (dim) {
    case 64: return launch_mt<T, KIND, 64>(a, p, pt, vec, wide, st);
    case 128: return launch_mt<T, KIND, 128>(a, p, pt, vec, wide, st);
    default: return launch_mt<T, KIND, 256>(a, p, pt, vec, wide, st);
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

hipError_t launch_attn_few(const AttnArgs &a, const AttnPlan &p, const Partials &pt, int kind, int dim, int dtype, bool vec,
                           bool wide, hipStream_t st) {
    switch (dtype) {
    case WQ_DT_F32: return launch_t<float>(a, p, pt, kind, dim, vec, wide, st);
    case WQ_DT_BF16: return launch_t<bf16>(a, p, pt, kind, dim, vec, wide, st);
    default: return launch_t<f16>(a, p, pt, kind, dim, vec, wide, st);
    }
}

} // namespace wq
