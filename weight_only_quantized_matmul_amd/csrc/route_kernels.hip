// The choice of a token's experts from the router's scores.
//
// A wave takes one token; expert e is in lane e % 64. Probabilities and the
// values that decide the choice are fp64, so that the choice is the one the
// definition makes whatever the scores' type, and the weights are rounded
// once. Groups are valued by their two largest experts, lanes sharing a group;
// the k largest are then found one after another, the lowest expert first
// among equals: a maximum over the wave of order-preserving integers, in steps
// of DPP (shuffles through LDS: 7.8 us for one token, 6.6 so).
//
// One token (256 experts in 8 groups, 8 chosen) is latency: 6.6 us, a chain
// of fp64 exponentials and k maxima, each of which waits for the last. A prompt
// of 8191 tokens over 128 experts is bound by the fp64 and integer work of the
// vector units: 12.7 us, 2.6 MB at 0.2 TB/s.
#include "moe.h"

namespace wq {
namespace {

constexpr int kWaves = 4; // tokens a block

// Order-preserving code of a double (no NaN): larger values have larger codes, and every code is above 0.
__device__ __forceinline__ uint64_t order(double v) {
    const uint64_t u = __builtin_bit_cast(uint64_t, v + 0.0); // -0 counts as 0
    return u >> 63 ? ~u : u | 1ull << 63;
}

// The largest code of the wave's lanes, in all of them: within 16 lanes by rotations of rows, then across them.
template <int N>
__device__ __forceinline__ uint64_t max_rotated(uint64_t v) {
    const int lo = __builtin_amdgcn_update_dpp(0, (int)v, 0x120 + N, 0xF, 0xF, false);
    const int hi = __builtin_amdgcn_update_dpp(0, (int)(v >> 32), 0x120 + N, 0xF, 0xF, false);
    const uint64_t o = (uint64_t)(uint32_t)hi << 32 | (uint32_t)lo;
    return o > v ? o : v;
}
__device__ __forceinline__ uint64_t wave_max(uint64_t v) {
    v = max_rotated<8>(v);
    v = max_rotated<4>(v);
    v = max_rotated<2>(v);
    v = max_rotated<1>(v);
    uint64_t most = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint64_t o = (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(v >> 32), 16 * i) << 32 |
                           (uint32_t)__builtin_amdgcn_readlane((int)v, 16 * i);
        most = o > most ? o : most;
    }
    return most;
}

// NPL: experts a lane
template <typename T, int NPL>
__global__ __launch_bounds__(64 * kWaves) void route_kernel(const RouteArgs a) {
    extern __shared__ double lds[]; // with groups: E values a wave
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const long tok = (long)blockIdx.x * kWaves + wave;
    if (tok >= a.T) return; // (waves share nothing: no barrier below)
    const T *row = (const T *)a.scores + tok * a.stride;
    float x[NPL];
    float top = -INFINITY;
#pragma unroll
    for (int i = 0; i < NPL; ++i) {
        const int e = i * 64 + lane;
        x[i] = e < a.E ? (float)row[e] : -INFINITY;
        x[i] = x[i] != x[i] ? -INFINITY : fminf(x[i], 3.402823466e+38f);
        top = fmaxf(top, x[i]);
    }
    double p[NPL];
    if (a.sigmoid) {
#pragma unroll
        for (int i = 0; i < NPL; ++i) p[i] = 1.0 / (1.0 + exp(-(double)x[i]));
    } else {
#pragma unroll
        for (int m = 32; m > 0; m >>= 1) top = fmaxf(top, __shfl_xor(top, m));
        double sum = 0.0;
#pragma unroll
        for (int i = 0; i < NPL; ++i) {
            p[i] = top == -INFINITY ? 0.0 : exp((double)x[i] - (double)top); // no expert has a score: no probability
            sum += p[i];
        }
#pragma unroll
        for (int m = 32; m > 0; m >>= 1) sum += __shfl_xor(sum, m);
        if (sum == 0.0) sum = 1.0;
#pragma unroll
        for (int i = 0; i < NPL; ++i) p[i] /= sum;
    }
    uint64_t key[NPL]; // 0: not to be chosen
#pragma unroll
    for (int i = 0; i < NPL; ++i) {
        const int e = i * 64 + lane;
        double c = p[i] + (a.bias && e < a.E ? (double)a.bias[e] : 0.0);
        if (c != c) c = -INFINITY;
        key[i] = e < a.E ? order(c) : 0;
        if (a.groups > 1 && e < a.E) lds[wave * a.E + e] = c;
    }
    if (a.groups > 1) {
        __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
        __builtin_amdgcn_wave_barrier();
        const int n = a.E / a.groups;
        int L = 64; // lanes a group
        while (L * a.groups > 64) L >>= 1;
        const int grp = lane / L;
        double one = -INFINITY, two = -INFINITY; // the group's largest, and the next
        if (grp < a.groups)
            for (int i = lane & (L - 1); i < n; i += L) {
                const double c = lds[wave * a.E + grp * n + i];
                two = fmax(two, fmin(one, c));
                one = fmax(one, c);
            }
        for (int m = L >> 1; m > 0; m >>= 1) {
            const double o1 = __shfl_xor(one, m), o2 = __shfl_xor(two, m);
            two = fmax(fmin(one, o1), fmax(two, o2));
            one = fmax(one, o1);
        }
        double value = n > 1 ? one + two : one;
        if (value != value) value = -INFINITY;
        int before = 0; // groups that go before this one
        for (int g = 0; g < a.groups; ++g) {
            const double v = __shfl(value, g * L);
            before += v > value || (v == value && g < grp);
        }
        const uint64_t kept = __ballot(grp < a.groups && before < a.top_groups && (lane & (L - 1)) == 0);
#pragma unroll
        for (int i = 0; i < NPL; ++i) {
            const int e = i * 64 + lane;
            if (e < a.E && !(kept >> (e / n * L) & 1)) key[i] = 0;
        }
    }
    int id = 0;
    double w = 0.0;
    for (int j = 0; j < a.k; ++j) {
        uint64_t best = 0;
        int e = 1 << 30;
        double pe = 0.0;
#pragma unroll
        for (int i = 0; i < NPL; ++i)
            if (key[i] > best) {
                best = key[i];
                e = i * 64 + lane;
                pe = p[i];
            }
        const uint64_t most = wave_max(best);
        uint64_t ties = __ballot(best == most);
        int first = __builtin_amdgcn_readlane(e, __builtin_ctzll(ties));
        for (ties &= ties - 1; ties; ties &= ties - 1) first = min(first, __builtin_amdgcn_readlane(e, __builtin_ctzll(ties))); // the lowest expert
        const int from = first & 63;
        pe = __builtin_bit_cast(double, (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(__builtin_bit_cast(uint64_t, pe) >> 32), from) << 32 |
                                            (uint32_t)__builtin_amdgcn_readlane((int)__builtin_bit_cast(uint64_t, pe), from));
        if (lane == j) {
            id = first;
            w = pe;
        }
        if (lane == from) {
#pragma unroll
            for (int i = 0; i < NPL; ++i)
                if (i == first >> 6) key[i] = 0;
        }
    }
    if (a.normalise) {
        double sum = lane < a.k ? w : 0.0;
#pragma unroll
        for (int m = 32; m > 0; m >>= 1) sum += __shfl_xor(sum, m);
        w = sum > 0.0 ? w / sum : 0.0;
    }
    if (lane < a.k) {
        a.ids[tok * a.k + lane] = id;
        a.weights[tok * a.k + lane] = (float)(w * (double)a.scale);
    }
}

template <typename T>
hipError_t launch_t(const RouteArgs &a, hipStream_t st) {
    const dim3 block(64 * kWaves);
    const size_t lds = a.groups > 1 ? sizeof(double) * kWaves * a.E : 0;
    const int piece = (int)(kMaxThreads / 64) / kWaves * kWaves; // tokens a launch
    for (long done = 0; done < a.T; done += piece) {
        RouteArgs b = a;
        b.scores = (const T *)a.scores + done * a.stride;
        b.ids = a.ids + done * a.k;
        b.weights = a.weights + done * a.k;
        b.T = (int)(a.T - done < piece ? a.T - done : piece);
        const dim3 grid((unsigned)((b.T + kWaves - 1) / kWaves));
        if (a.E <= 64)
            hipLaunchKernelGGL((route_kernel<T, 1>), grid, block, lds, st, b);
        else if (a.E <= 128)
            hipLaunchKernelGGL((route_kernel<T, 2>), grid, block, lds, st, b);
        else if (a.E <= 256)
            hipLaunchKernelGGL((route_kernel<T, 4>), grid, block, lds, st, b);
        else if (a.E <= 512)
            hipLaunchKernelGGL((route_kernel<T, 8>), grid, block, lds, st, b);
        else
            hipLaunchKernelGGL((route_kernel<T, 16>), grid, block, lds, st, b);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

} // namespace

hipError_t launch_route(const RouteArgs &a, int dtype, hipStream_t st) {
    switch (dtype) {
    case WQ_DT_F32: return launch_t<float>(a, st);
    case WQ_DT_BF16: return launch_t<bf16>(a, st);
    default: return launch_t<f16>(a, st);
    }
}

} // namespace wq
