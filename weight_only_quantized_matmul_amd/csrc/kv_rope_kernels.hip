// Rotary positions of queries and keys while keys and values go into the cache.
//
// A block takes one token (few tokens: some of its heads). It finds the
// token's place and turns every pair's angle once, in fp64, into a cosine and
// sine in LDS, of which each thread keeps the ones of its 8 elements for all
// the rows it takes. Rotated keys are rounded to fp32 and quantised from
// registers, so they never pass through memory.
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
    const int tok = blockIdx.x;
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
    // what this thread's elements turn by: y[i] = x[i] * cs[i].x + (the pair's other element) * cs[i].y
    const int e0 = 8 * lane;
    double2 cs[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int e = e0 + i;
        cs[i] = make_double2(1.0, 0.0);
        if (e < a.rot) {
            const int f = a.pairing == 0 ? (e < half ? e : e - half) : e / 2;
            const bool first = a.pairing == 0 ? e < half : (e & 1) == 0;
            const double2 w = trig[f];
            cs[i] = make_double2(w.x, first ? -w.y : w.y);
        }
    }
    const int Hq = a.q ? a.H : 0, rows = Hq + 2 * a.c.heads;
    const int r0 = (int)((long)rows * blockIdx.y / gridDim.y), r1 = (int)((long)rows * (blockIdx.y + 1) / gridDim.y);
    for (int base = r0; base < r1; base += kThreads / LANES) { // (all lanes of a wave go round together)
        const int r = base + tid / LANES;
        const bool live = r < r1;
        const bool is_q = r < Hq, is_v = r >= Hq + a.c.heads;
        const int head = is_q ? r : is_v ? r - Hq - a.c.heads : r - Hq;
        const T *x = is_q ? (const T *)a.q + (long)tok * a.qt + (long)head * a.qh
                          : (const T *)(is_v ? a.v : a.k) + (long)tok * a.tok + (long)head * a.head;
        float v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = 0.f;
        if (live) {
            load8<T, VEC>(x + e0, v);
            if (!is_v && e0 < a.rot) {
                float o[8];
                if (a.pairing == 1) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) o[i] = v[i ^ 1];
                } else if (VEC && half % 8 == 0) {
                    load8<T, VEC>(x + (e0 < half ? e0 + half : e0 - half), o);
                } else {
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const int e = e0 + i;
                        o[i] = e < half ? (float)x[e + half] : e < a.rot ? (float)x[e - half] : 0.f;
                    }
                }
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (e0 + i < a.rot) v[i] = (float)((double)v[i] * cs[i].x + (double)o[i] * cs[i].y);
            }
            if (is_q) store8<T, VEC>((T *)a.q_out + (long)tok * a.ot + (long)head * a.oh + e0, v);
        }
        const float top = row_top<LANES>(v);
        if (!live || is_q || !there) continue;
        uint8_t *row = const_cast<uint8_t *>(is_v ? a.c.v : a.c.k) + row_at + head * a.c.rh + (long)lane * Codes<KIND>::bytes;
        const float scale = store_codes<KIND>(row, v, top);
        if (lane == 0) const_cast<float *>(is_v ? a.c.vs : a.c.ks)[scale_at + head * a.c.sh] = scale;
    }
}

template <typename T, int KIND, int D>
hipError_t launch_d(const KvRopeArgs &a, bool vec, int cus, hipStream_t st) {
    const long rows = (a.q ? a.H : 0) + 2L * a.c.heads, most = (rows * (D / 8) + kThreads - 1) / kThreads;
    long gy = a.b.T >= 2 * cus ? 1 : (2 * cus + a.b.T - 1) / a.b.T;
    gy = gy < most ? gy : most;
    const long piece = kMaxThreads / kThreads; // tokens a launch: all that an int counts fit in one
    if (a.b.T > piece) return hipErrorNotSupported;
    const dim3 grid((unsigned)a.b.T, (unsigned)gy), block(kThreads);
    if (vec)
        hipLaunchKernelGGL((kv_append_rope_kernel<T, KIND, D, true>), grid, block, 0, st, a);
    else
        hipLaunchKernelGGL((kv_append_rope_kernel<T, KIND, D, false>), grid, block, 0, st, a);
    return hipGetLastError();
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
