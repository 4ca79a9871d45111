// Quantising a key/value cache as it is written, and reading it back.
//
// D / 8 lanes take RPG rows of one token (keys and values of its heads), 8
// elements a lane and row: a wide load, the row's maximum over the lane group,
// 8 codes back in one store. Where the token lies is found once for its RPG
// rows. Both directions move every byte once and are bound by HBM (few tokens:
// by the chain lengths -> table -> row). Reading 131072 tokens of 8 heads x 128
// from int8 to bf16: 814 MB in 166 us (4.9 TB/s; one row a lane group 290 us);
// a decode step of 64 tokens 4 us each way.
#include "kv_rows.h"

namespace wq {
namespace {

constexpr int kThreads = 256;
// What a lane group works on: a token and its rows first .. first + RPG - 1,
// keys of all heads before values of all heads.
struct Where {
    int tok, first;
    bool any, there; // the token is one of the batch's; it has a place in the cache
    long row, scale; // the place's offsets in the pools for head 0 (bytes, floats)
};

template <int LANES, int RPG>
__device__ __forceinline__ Where token_of(const KvCopyArgs &a) {
    Where w;
    const unsigned parts = (2 * a.c.heads + RPG - 1) / RPG;
    const unsigned r = (blockIdx.y * gridDim.x + blockIdx.x) * (kThreads / LANES) + threadIdx.x / LANES;
    const unsigned tok = r / parts;
    w.any = tok < (unsigned)a.b.T;
    w.tok = w.any ? (int)tok : 0;
    w.first = (int)(r - tok * parts) * RPG;
    return w;
}

// Where the token lies. The lanes of a group read starts and lengths together (one round trip), then the one
// whose sequence holds the token tells the others; the page's entry is the only load that waits for them.
template <int LANES>
__device__ __forceinline__ void locate(const KvCopyArgs &a, Where &w, int lane) {
    int seq = -1, t = -1;
    for (int i = lane; i < a.b.B; i += LANES) {
        const int first = a.b.q_start[i], next = a.b.q_start[i + 1], kv = a.b.kv_len[i];
        if (first <= w.tok && w.tok < next) {
            seq = i;
            t = max(kv, 0) - next + w.tok;
        }
    }
    const int base = (threadIdx.x & 63) - lane;
    const uint64_t hits = __ballot(seq >= 0) >> base & (LANES == 64 ? ~0ull : (1ull << LANES) - 1);
    const int from = base + (hits ? __builtin_ctzll(hits) : 0);
    seq = __shfl(seq, from);
    t = __shfl(t, from);
    w.there = false;
    w.row = w.scale = 0;
    int page, slot;
    if (w.any && hits && find_row(a.c, a.b, seq, t, &page, &slot)) {
        w.there = true;
        w.row = page * a.c.rp + slot * a.c.rs;
        w.scale = page * a.c.sp + slot * a.c.ss;
    }
}

template <typename T, int KIND, int D, bool VEC, int RPG>
__global__ __launch_bounds__(kThreads) void kv_append_kernel(const KvCopyArgs a) {
    constexpr int LANES = D / 8;
    const int lane = threadIdx.x & (LANES - 1), H = a.c.heads;
    Where w = token_of<LANES, RPG>(a);
    float v[RPG][8];
#pragma unroll
    for (int j = 0; j < RPG; ++j) {
        const int s = w.first + j, side = s >= H;
#pragma unroll
        for (int i = 0; i < 8; ++i) v[j][i] = 0.f;
        if (w.any && s < 2 * H)
            load8<T, VEC>((const T *)(side ? a.v : a.k) + (long)w.tok * a.tok + (long)(s - side * H) * a.head + 8 * lane, v[j]);
    }
    locate<LANES>(a, w, lane);
#pragma unroll
    for (int j = 0; j < RPG; ++j) {
        const int s = w.first + j, side = s >= H, head = s - side * H;
        const float top = row_top<LANES>(v[j]);
        if (!w.there || s >= 2 * H) continue;
        uint8_t *row = const_cast<uint8_t *>(side ? a.c.v : a.c.k) + w.row + head * a.c.rh + (long)lane * Codes<KIND>::bytes;
        const float scale = store_codes<KIND>(row, v[j], top);
        if (lane == 0) const_cast<float *>(side ? a.c.vs : a.c.ks)[w.scale + head * a.c.sh] = scale;
    }
}

template <typename T, int KIND, int D, bool VEC, int RPG>
__global__ __launch_bounds__(kThreads) void kv_read_kernel(const KvCopyArgs a) {
    constexpr int LANES = D / 8, W = Codes<KIND>::bytes / 4;
    const int lane = threadIdx.x & (LANES - 1), H = a.c.heads;
    Where w = token_of<LANES, RPG>(a);
    locate<LANES>(a, w, lane);
    if (!w.any) return;
    typedef uint32_t words __attribute__((ext_vector_type(W)));
    words u[RPG];
    float scale[RPG];
#pragma unroll
    for (int j = 0; j < RPG; ++j) {
        const int s = w.first + j, side = s >= H, head = s - side * H;
        scale[j] = 0.f;
        u[j] = (words)(KIND == WQ_KV_I4 ? 0x88888888u : 0u);
        if (w.there && s < 2 * H) {
            u[j] = *reinterpret_cast<const words *>((side ? a.c.v : a.c.k) + w.row + head * a.c.rh + (long)lane * Codes<KIND>::bytes);
            scale[j] = (side ? a.c.vs : a.c.ks)[w.scale + head * a.c.sh];
        }
    }
#pragma unroll
    for (int j = 0; j < RPG; ++j) {
        const int s = w.first + j, side = s >= H, head = s - side * H;
        if (s >= 2 * H) continue;
        float v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if constexpr (KIND == WQ_KV_F16)
                v[i] = (float)__builtin_bit_cast(f16, (uint16_t)(u[j][i / 2] >> (16 * (i & 1))));
            else if constexpr (KIND == WQ_KV_I8)
                v[i] = (float)(int8_t)(u[j][i / 4] >> (8 * (i & 3)));
            else
                v[i] = (float)((int)(u[j][0] >> (4 * i) & 15) - 8);
            v[i] *= scale[j];
        }
        store8<T, VEC>((T *)(side ? a.v : a.k) + (long)w.tok * a.tok + (long)head * a.head + 8 * lane, v);
    }
}

template <typename T, int KIND, int D, bool VEC, int RPG>
hipError_t launch_rpg(const KvCopyArgs &a, bool write, hipStream_t st) {
    const long groups = (long)a.b.T * ((2 * a.c.heads + RPG - 1) / RPG);
    const long blocks = (groups * (D / 8) + kThreads - 1) / kThreads, gy = (blocks + kMaxThreads / kThreads - 1) / (kMaxThreads / kThreads);
    const dim3 grid((unsigned)((blocks + gy - 1) / gy), (unsigned)gy), block(kThreads);
    if (write)
        hipLaunchKernelGGL((kv_append_kernel<T, KIND, D, VEC, RPG>), grid, block, 0, st, a);
    else
        hipLaunchKernelGGL((kv_read_kernel<T, KIND, D, VEC, RPG>), grid, block, 0, st, a);
    return hipGetLastError();
}

template <typename T, int KIND, int D>
hipError_t launch_d(const KvCopyArgs &a, bool write, bool vec, hipStream_t st) {
    if (!vec) return launch_rpg<T, KIND, D, false, 1>(a, write, st);
    // four rows a lane group once that still leaves every CU four blocks
    const long rows = (long)a.b.T * 2 * a.c.heads;
    if (rows * (D / 8) >= 4L * 1024 * kThreads) return launch_rpg<T, KIND, D, true, 4>(a, write, st);
    return launch_rpg<T, KIND, D, true, 1>(a, write, st);
}

template <typename T, int KIND>
hipError_t launch_kind(const KvCopyArgs &a, int dim, bool write, bool vec, hipStream_t st) {
    switch (dim) {
    case 64: return launch_d<T, KIND, 64>(a, write, vec, st);
    case 128: return launch_d<T, KIND, 128>(a, write, vec, st);
    default: return launch_d<T, KIND, 256>(a, write, vec, st);
    }
}

template <typename T>
hipError_t launch_t(const KvCopyArgs &a, int kind, int dim, bool write, bool vec, hipStream_t st) {
    switch (kind) {
    case WQ_KV_F16: return launch_kind<T, WQ_KV_F16>(a, dim, write, vec, st);
    case WQ_KV_I8: return launch_kind<T, WQ_KV_I8>(a, dim, write, vec, st);
    default: return launch_kind<T, WQ_KV_I4>(a, dim, write, vec, st);
    }
}

hipError_t launch_kv(const KvCopyArgs &a, int kind, int dim, int dtype, bool write, bool vec, hipStream_t st) {
    switch (dtype) {
    case WQ_DT_F32: return launch_t<float>(a, kind, dim, write, vec, st);
    case WQ_DT_BF16: return launch_t<bf16>(a, kind, dim, write, vec, st);
    default: return launch_t<f16>(a, kind, dim, write, vec, st);
    }
}

} // namespace

hipError_t launch_kv_append(const KvCopyArgs &a, int kind, int dim, int dtype, bool vec, hipStream_t st) {
    return launch_kv(a, kind, dim, dtype, true, vec, st);
}

hipError_t launch_kv_read(const KvCopyArgs &a, int kind, int dim, int dtype, bool vec, hipStream_t st) {
    return launch_kv(a, kind, dim, dtype, false, vec, st);
}

} // namespace wq
