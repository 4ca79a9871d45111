// The gated feed-forward layer of chosen experts, for a few tokens.
//
//     y[t] = add[t] + sum_j weights[t,j] * down_e . (silu(gate_e . x[t]) * (up_e . x[t])),  e = ids[t,j]
//
// Which expert works on which rows is known on the device only. Up to
// kInlineSlots slots t * k + j the products' blocks find their expert's slots
// themselves. For more, and where the activations have to be laid out first, a
// kernel of its own sorts the slots by expert (a counting sort in one block)
// and makes the activations' parts, or a copy whose rows can be read four
// elements at a time. The products of gate and up, with the activation as their
// epilogue, write h; the products of down write one row a slot; and the last
// kernel adds each token's rows in the order of its slots, so results do not
// depend on what else the batch holds. (Products that add into y themselves
// would need atomics, whose order changes results.)
//
// What these two kernels take is mostly their launch and one pass through
// memory's latency: 4.0 us for the sum of one token's 8 rows of 6144, 5.8 us for
// the plan and parts of 64 tokens of 6144, 17 tokens on 64 experts without a
// plan 42.2 us, with one 43.4 us.
#include "moe_parts.h"

namespace wq {
namespace {

constexpr int kPrepThreads = 512;

// Block 0 makes the plan; the others make x's parts, or copy x where its rows cannot be read four elements at a time.
template <int FMT, typename T>
__global__ __launch_bounds__(kPrepThreads) void moe_prepare_kernel(const MoeArgs a) {
    __shared__ int cnt[WQ_MOE_MAX_EXPERTS], at[WQ_MOE_MAX_EXPERTS];
    __shared__ uint32_t part[kPrepThreads / 64];
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
                MoeWork &w = a.plan[run >> 16];
                w.expert = e;
                w.rows = n;
                w.first = run & 0xFFFF;
                run += 0x10000u + n;
            }
        }
        for (int i = (int)(all >> 16) + tid; i < min(a.E, N); i += kPrepThreads) a.plan[i].rows = 0;
        __syncthreads();
        // (the order of an expert's rows may differ from run to run: no result depends on it)
        for (int i = tid; i < N; i += kPrepThreads) {
            const int e = a.ids[i];
            if (e >= 0 && e < a.E) a.order[atomicAdd(&at[e], 1)] = i;
        }
        return;
    }
    if (a.xp != nullptr) {
        const int per_row = a.in.kp / kPiece;
        for (long i = (long)(blockIdx.x - 1) * kPrepThreads + tid; i < (long)a.T * per_row; i += (long)(gridDim.x - 1) * kPrepThreads) {
            const long row = i / per_row;
            prepare_piece<FMT>((const T *)a.x + row * a.xs, a.in.I, a.in, row, (int)(i - row * per_row) * kPiece, a.xp, a.xunit);
        }
        return;
    }
    const long items = (long)a.T * a.xe_n;
    for (long i = (long)(blockIdx.x - 1) * kPrepThreads + tid; i < items; i += (long)(gridDim.x - 1) * kPrepThreads) {
        const int t = (int)(i / a.xe_n), e = (int)(i - (long)t * a.xe_n);
        ((T *)a.copy)[i] = e < a.in.I ? ((const T *)a.x)[t * a.xs + e] : (T)0.f;
    }
}

// Eight slots' rows are read at a time; what an empty slot's row holds does not count.
template <typename T>
__global__ __launch_bounds__(256) void moe_combine_kernel(const MoeArgs a) {
    const int t = blockIdx.y, o = blockIdx.x * 256 + threadIdx.x;
    if (o >= a.out.O) return;
    float v = a.add ? (float)((const T *)a.add)[t * a.as + o] : 0.f;
    for (int j0 = 0; j0 < a.k; j0 += 8) {
        float w[8], d[8];
        bool there[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int slot = t * a.k + min(j0 + j, a.k - 1), e = a.ids[slot];
            there[j] = j0 + j < a.k && e >= 0 && e < a.E;
            w[j] = a.weights[slot];
            d[j] = a.d[(long)slot * a.out.O + o];
        }
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (there[j]) v = fmaf(w[j], d[j], v);
    }
    ((T *)a.y)[t * a.ys + o] = (T)v;
}

template <typename T>
hipError_t launch_t(MoeArgs &a, int fmt, hipStream_t st) {
    hipError_t e = hipSuccess;
    if (a.plan != nullptr) {
        const long items = a.xp ? (long)a.T * (a.in.kp / kPiece) : a.copy ? (long)a.T * a.xe_n : 0;
        const long blocks = (items + kPrepThreads - 1) / kPrepThreads;
        const dim3 grid((unsigned)(1 + (blocks < 1024 ? blocks : 1024)));
        if (fmt == WQ_I8)
            hipLaunchKernelGGL((moe_prepare_kernel<WQ_I8, T>), grid, dim3(kPrepThreads), 0, st, a);
        else if (fmt == WQ_I4)
            hipLaunchKernelGGL((moe_prepare_kernel<WQ_I4, T>), grid, dim3(kPrepThreads), 0, st, a);
        else
            hipLaunchKernelGGL((moe_prepare_kernel<WQ_I2, T>), grid, dim3(kPrepThreads), 0, st, a);
        e = hipGetLastError();
    }
    if (e == hipSuccess) e = fmt == WQ_I8 ? launch_moe_i8(a, st) : fmt == WQ_I4 ? launch_moe_i4(a, st) : launch_moe_i2(a, st);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL((moe_combine_kernel<T>), dim3((unsigned)((a.out.O + 255) / 256), (unsigned)a.T), dim3(256), 0, st, a);
    return hipGetLastError();
}

} // namespace

hipError_t launch_moe(MoeArgs &a, int fmt, int dtype, hipStream_t st) {
    switch (dtype) {
    case WQ_DT_F32: return launch_t<float>(a, fmt, st);
    case WQ_DT_BF16: return launch_t<bf16>(a, fmt, st);
    default: return launch_t<f16>(a, fmt, st);
    }
}

} // namespace wq
