// Rotary positions with several axes.
//
// A block takes `tb` tokens: it first turns every (token, pair) angle once
// into a cosine and sine in LDS, which all heads of the token share, then
// streams the heads' pairs through. Angles are kept in turns: position times
// turns-per-position in fp64, whole quarter turns taken off exactly, and only
// the remaining eighth-turn either way goes through fp32, so a position of a
// million loses nothing.
//
// Bound by HBM: 8191 tokens x 40 heads x 128 in bf16, 168 MB, 28 us (inputs in
// the last-level cache) to 38 us (not); 64 tokens x 56 heads in f32 4 us.
#include "decoder.h"

namespace wq {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxTb = 16;

template <typename T, int VEC>
__global__ __launch_bounds__(kThreads) void rope_kernel(const RopeArgs a) {
    __shared__ float2 trig[kMaxTb * (WQ_ROPE_MAX_ROT / 2)];
    const int half = a.rot / 2, tid = threadIdx.x;
    const int t0 = blockIdx.x * a.tb, nt = min(a.tb, a.T - t0);
    for (int i = tid; i < nt * half; i += kThreads) {
        const int t = i / half, f = i - t * half;
        const double at = (double)a.pos[(long)a.axis[f] * a.pos_stride + t0 + t] * a.turns[f];
        const double q = 4.0 * (at - rint(at)); // quarter turns in [-2, 2]
        const double n = rint(q);
        float s, c;
        sincospif(0.5f * (float)(q - n), &s, &c);
        const int k = (int)n & 3;
        const float c2 = (k & 1) ? s : c, s2 = (k & 1) ? c : s;
        trig[i] = make_float2(k == 1 || k == 2 ? -c2 : c2, k >= 2 ? -s2 : s2);
    }
    __syncthreads();
    // items of a head: the vectors of rotated pairs, then those copied
    const int turned = a.pairing == 0 ? half / VEC : VEC == 1 ? half : a.rot / VEC;
    const int per_head = turned + (a.D - a.rot) / VEC;
    const int h0 = (int)((long)a.H * blockIdx.y / gridDim.y), h1 = (int)((long)a.H * (blockIdx.y + 1) / gridDim.y);
    const int items = nt * (h1 - h0) * per_head;
    for (int i = tid; i < items; i += kThreads) {
        const int r = i / per_head, c = i - r * per_head;
        const int t = r / (h1 - h0), h = h0 + r - t * (h1 - h0);
        const T *x = (const T *)a.x + (long)(t0 + t) * a.xt + (long)h * a.xh;
        T *y = (T *)a.y + (long)(t0 + t) * a.yt + (long)h * a.yh;
        const float2 *cs = trig + t * half;
        if (c >= turned) {
            float v[VEC];
            const int e = a.rot + (c - turned) * VEC;
            load_vec<T, VEC>(x + e, v);
            store_vec<T, VEC>(y + e, v);
        } else if (a.pairing == 0) {
            float p[VEC], q[VEC];
            load_vec<T, VEC>(x + c * VEC, p);
            load_vec<T, VEC>(x + half + c * VEC, q);
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
                const float2 w = cs[c * VEC + j];
                const float u = p[j];
                p[j] = u * w.x - q[j] * w.y;
                q[j] = u * w.y + q[j] * w.x;
            }
            store_vec<T, VEC>(y + c * VEC, p);
            store_vec<T, VEC>(y + half + c * VEC, q);
        } else {
            constexpr int W = VEC == 1 ? 2 : VEC;
            float v[W];
            if (VEC == 1) {
                v[0] = (float)x[2 * c];
                v[1] = (float)x[2 * c + 1];
            } else {
                load_vec<T, W>(x + c * W, v);
            }
#pragma unroll
            for (int j = 0; j < W / 2; ++j) {
                const float2 w = cs[c * (W / 2) + j];
                const float u = v[2 * j], z = v[2 * j + 1];
                v[2 * j] = u * w.x - z * w.y;
                v[2 * j + 1] = u * w.y + z * w.x;
            }
            if (VEC == 1) {
                y[2 * c] = (T)v[0];
                y[2 * c + 1] = (T)v[1];
            } else {
                store_vec<T, W>(y + c * W, v);
            }
        }
    }
}

template <typename T>
hipError_t launch_t(RopeArgs &a, bool vec, int cus, hipStream_t st) {
    constexpr int V = sizeof(T) == 4 ? 4 : 8;
    // whole vectors in both halves of the rotated part and in the copied part
    const int half = a.rot / 2;
    vec = vec && (a.D - a.rot) % V == 0 && (a.pairing == 0 ? half % V == 0 : a.rot % V == 0);
    const int v = vec ? V : 1;
    // tokens a block: about four items a thread, but a block for every CU first
    const long items = (long)a.H * (half + (a.D - a.rot)) / v + 1;
    long tb = 4 * kThreads / items;
    tb = tb < a.T / (2 * cus) ? tb : a.T / (2 * cus);
    a.tb = (int)(tb < 1 ? 1 : tb > kMaxTb ? kMaxTb : tb);
    const long piece = kMaxThreads / kThreads * a.tb; // tokens a launch
    if (a.T > piece) {
        for (long done = 0; done < a.T; done += piece) {
            RopeArgs b = a;
            b.x = (const T *)a.x + done * a.xt;
            b.y = (T *)a.y + done * a.yt;
            b.pos = a.pos + done;
            b.T = (int)(a.T - done < piece ? a.T - done : piece);
            const hipError_t e = launch_t<T>(b, vec, cus, st);
            if (e != hipSuccess) return e;
        }
        return hipSuccess;
    }
    const long gx = (a.T + a.tb - 1) / a.tb;
    // few tokens: the heads are split among blocks, which then turn the same angles again
    long gy = gx >= 2 * cus ? 1 : (2 * cus + gx - 1) / gx;
    const long most = (items + kThreads - 1) / kThreads;
    gy = gy < most ? gy : most;
    gy = gy < a.H ? gy : a.H;
    const dim3 grid((unsigned)gx, (unsigned)gy), block(kThreads);
    if (vec)
        hipLaunchKernelGGL((rope_kernel<T, V>), grid, block, 0, st, a);
    else
        hipLaunchKernelGGL((rope_kernel<T, 1>), grid, block, 0, st, a);
    return hipGetLastError();
}

} // namespace

hipError_t launch_rope(RopeArgs &a, int dtype, bool vec, int cus, hipStream_t st) {
    switch (dtype) {
    case WQ_DT_F32: return launch_t<float>(a, vec, cus, st);
    case WQ_DT_BF16: return launch_t<bf16>(a, vec, cus, st);
    default: return launch_t<f16>(a, vec, cus, st);
    }
}

} // namespace wq
