// Rotary positions of queries and keys while keys and values go into the cache.
//
// A block takes one token (few tokens: some of its heads). It finds the
// token's place and turns every pair's angle once, in fp64, into a cosine and
// sine in LDS, of which each thread keeps the ones of its 8 elements for all
// the rows it takes. Rotated keys are rounded to fp32 and quantised from
// registers, so they never pass through memory.
//
// Sines and cosines in fp64 once a token and pair, then loads and stores bound
// it: 64 tokens of 48 query and 8 key/value heads of 128 in fp32 5.7 us (launch
// and latency), 2436 tokens of the same heads in bf16 into a 4-bit cache 22.0 us,
// 73 MB at 3.3 TB/s (with the queries' products in fp64 23.2).
#include <type_traits>

#include "kv_rows.h"

namespace wq {
namespace {

constexpr int kThreads = 256;

template <typename T, int KIND, int D, bool VEC>
__global__ __launch_bounds__(kThreads) void kv_append_rope_kernel(const KvRopeArgs a) {
    constexpr int LANES = D / 8;
    __shared__ double2 trig[WQ_ROPE_MAX_ROT / 2];
    __shared__ long found; // sequence << 32 | position, or -1
    const int tid = threadIdx.x, lane = tid & (LANES - 1), half = a.rot / 2;
    const int tok = a.first + (int)blockIdx.x;
    const int Hq = a.q ? a.H : 0, rows = Hq + 2 * a.c.heads;
    const int r0 = (int)((long)rows * blockIdx.y / gridDim.y), r1 = (int)((long)rows * (blockIdx.y + 1) / gridDim.y);
    // a row's 8 elements and those that they turn with (asked for a round ahead, 2436 tokens took 43 us, with the read, instead of 36)
    const int e0 = 8 * lane;
    auto load = [&](int r, float (&v)[8], float (&o)[8]) __attribute__((always_inline)) {
        const bool is_q = r < Hq, is_v = r >= Hq + a.c.heads;
        const int head = is_q ? r : is_v ? r - Hq - a.c.heads : r - Hq;
        const T *x = is_q ? (const T *)a.q + (long)tok * a.qt + (long)head * a.qh
                          : (const T *)(is_v ? a.v : a.k) + (long)tok * a.tok + (long)head * a.head;
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = o[i] = 0.f;
        if (r >= r1) return;
        load8<T, VEC>(x + e0, v);
        if (is_v || e0 >= a.rot || a.pairing == 1) return;
        if (VEC && half % 8 == 0) {
            load8<T, VEC>(x + (e0 < half ? e0 + half : e0 - half), o);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int e = e0 + i;
                o[i] = e < half ? (float)x[e + half] : e < a.rot ? (float)x[e - half] : 0.f;
            }
        }
    };
    if (tid == 0) found = -1;
    __syncthreads();
    for (int i = tid; i < a.b.B; i += kThreads) {
        const int first = a.b.q_start[i], next = a.b.q_start[i + 1], kv = a.b.kv_len[i];
        if (first <= tok && tok < next) found = (long)i << 32 | (uint32_t)(max(kv, 0) - next + tok);
    }
    __syncthreads();
    const long at = found;
    if (at < 0) return; // none of the sequences' tokens
    const int seq = (int)(at >> 32), t = (int)at;
    for (int f = tid; f < half; f += kThreads) {
        const int pos = a.pos ? a.pos[(long)a.axis[f] * a.pos_stride + tok] : t;
        const double turn = (double)pos * a.turns[f];
        double s, c;
        sincospi(2.0 * (turn - rint(turn)), &s, &c);
        trig[f] = make_double2(c, s);
    }
    int page = 0, slot = 0;
    const bool there = find_row(a.c, a.b, seq, t, &page, &slot);
    const long row_at = page * a.c.rp + slot * a.c.rs, scale_at = page * a.c.sp + slot * a.c.ss;
    __syncthreads();
    // What this thread's elements turn by: y[i] = x[i] * cs[i].x + (the pair's other element) * cs[i].y. Queries of 16 bits turn in
    // fp32, whose error is far below their own rounding; keys, whose codes may lie next to a border, and fp32 queries in fp64.
    constexpr bool HALF = sizeof(T) == 2;
    typedef typename std::conditional<HALF, float, double>::type Q;
    auto turn = [&](int i, double &c, double &s) __attribute__((always_inline)) {
        const int e = e0 + i, f = a.pairing == 0 ? (e < half ? e : e - half) : e / 2;
        const bool first = a.pairing == 0 ? e < half : (e & 1) == 0;
        const double2 w = e < a.rot ? trig[f] : make_double2(1.0, 0.0);
        c = w.x;
        s = first ? -w.y : w.y;
    };
    Q cs[8][2];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        double c, s;
        turn(i, c, s);
        cs[i][0] = (Q)c;
        cs[i][1] = (Q)s;
    }
    constexpr int STEP = kThreads / LANES;
    for (int base = r0; base < r1; base += STEP) { // (all lanes of a wave go round together)
        const int r = base + tid / LANES;
        const bool live = r < r1, is_q = r < Hq, is_v = r >= Hq + a.c.heads;
        const int head = is_q ? r : is_v ? r - Hq - a.c.heads : r - Hq;
        float v[8], o[8], y[8];
        load(r, v, o);
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = v[i];
        if (HALF && !is_q && !is_v) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                double c, s;
                turn(i, c, s);
                if (e0 + i < a.rot) y[i] = (float)((double)v[i] * c + (double)(a.pairing == 1 ? v[i ^ 1] : o[i]) * s);
            }
        } else if (!is_v) {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (e0 + i < a.rot) y[i] = (float)((Q)v[i] * cs[i][0] + (Q)(a.pairing == 1 ? v[i ^ 1] : o[i]) * cs[i][1]);
        }
        // (a query's row may be written over itself: its lanes are of one wave, whose loads are done)
        if (live && is_q) store8<T, VEC>((T *)a.q_out + (long)tok * a.ot + (long)head * a.oh + e0, y);
        if (base + STEP > Hq) { // rows of keys or values among the block's
            const float top = row_top<LANES>(y);
            if (live && !is_q && there) {
                uint8_t *row = const_cast<uint8_t *>(is_v ? a.c.v : a.c.k) + row_at + head * a.c.rh + (long)lane * Codes<KIND>::bytes;
                const float scale = store_codes<KIND>(row, y, top);
                if (lane == 0) const_cast<float *>(is_v ? a.c.vs : a.c.ks)[scale_at + head * a.c.sh] = scale;
            }
        }
    }
}

template <typename T, int KIND, int D>
hipError_t launch_d(const KvRopeArgs &a, bool vec, int cus, hipStream_t st) {
    const long rows = (a.q ? a.H : 0) + 2L * a.c.heads, most = (rows * (D / 8) + kThreads - 1) / kThreads;
    long gy = a.b.T >= 2 * cus ? 1 : (2 * cus + a.b.T - 1) / a.b.T;
    gy = gy < most ? gy : most;
    const long piece = kMaxThreads / kThreads / gy; // tokens a launch
    for (long done = 0; done < a.b.T; done += piece) {
        KvRopeArgs b = a;
        b.first = (int)done;
        const dim3 grid((unsigned)(a.b.T - done < piece ? a.b.T - done : piece), (unsigned)gy), block(kThreads);
        if (vec)
            hipLaunchKernelGGL((kv_append_rope_kernel<T, KIND, D, true>), grid, block, 0, st, b);
        else
            hipLaunchKernelGGL((kv_append_rope_kernel<T, KIND, D, false>), grid, block, 0, st, b);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

template <typename T, int KIND>
hipError_t launch_kind(const KvRopeArgs &a, int dim, bool vec, int cus, hipStream_t st) {
    switch (dim) {
    case 64: return launch_d<T, KIND, 64>(a, vec, cus, st);
    case 128: return launch_d<T, KIND, 128>(a, vec, cus, st);
    default: return launch_d<T, KIND, 256>(a, vec, cus, st);
    }
}

template <typename T>
hipError_t launch_t(const KvRopeArgs &a, int kind, int dim, bool vec, int cus, hipStream_t st) {
    switch (kind) {
    case WQ_KV_F16: return launch_kind<T, WQ_KV_F16>(a, dim, vec, cus, st);
    case WQ_KV_I8: return launch_kind<T, WQ_KV_I8>(a, dim, vec, cus, st);
    default: return launch_kind<T, WQ_KV_I4>(a, dim, vec, cus, st);
    }
}

} // namespace

hipError_t launch_kv_append_rope(const KvRopeArgs &a, int kind, int dim, int dtype, bool vec, int cus, hipStream_t st) {
    switch (dtype) {
    case WQ_DT_F32: return launch_t<float>(a, kind, dim, vec, cus, st);
    case WQ_DT_BF16: return launch_t<bf16>(a, kind, dim, vec, cus, st);
    default: return launch_t<f16>(a, kind, dim, vec, cus, st);
    }
}

} // namespace wq
