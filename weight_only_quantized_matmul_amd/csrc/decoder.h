// Internal declarations of the operators between a decoder layer's products:
// argument blocks shared by their C entry points (decoder_api.cpp) and kernel
// files, and the device helpers those share.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

#include "wqmm.h"

constexpr uint32_t kRopeMagic = 0x57515231u; // "WQR1"

struct wq_rope {
    uint32_t magic;
    int rot, pairing, axes;
    double turns[WQ_ROPE_MAX_ROT / 2]; // theta^(-2i/rot) / (2 pi): turns per position
    uint8_t axis[WQ_ROPE_MAX_ROT / 2];
};

namespace wq {

// runtime.cpp: what the entry points share with the matmul calls
int begin_call(int device);                                                    // WQ_OK, WQ_E_NOTINIT, WQ_E_FAULT
int stream_workspace(int device, size_t bytes, hipStream_t st, void **out);    // the stream's workspace
int device_cus(int device);
bool device_is_open(int device);
int device_table(int device, const void *host, size_t bytes, void **out); // a copy in the device's memory
void device_table_free(int device, void *p, size_t bytes);

// A dimension of a launch holds fewer than 2^32 threads; the runtime does not refuse more, it runs what is left of
// their number modulo 2^32. Longer work is launched in pieces or laid over a second dimension, or refused
// (hipErrorNotSupported, WQ_E_UNSUPPORTED to the caller).
constexpr long kMaxThreads = (1L << 32) - 1;

// ---------------------------------------------------------------------------
struct NormArgs {
    const void *x, *res;
    const float *w;
    void *y, *sum;
    float *y_scale;
    long xs, rs, ys, ss;
    float eps;
    int rows, n;
};
hipError_t launch_rmsnorm(const NormArgs &a, int x_dtype, int y_dtype, bool vec, int cus, hipStream_t st);

struct BlockNormArgs {
    const void *x, *gate, *res;
    const float *w_post, *w_pre;
    void *y, *sum;
    long xs, gs, rs, ys, ss;
    float alpha, eps;
    int rows, n;
};
hipError_t launch_block_norm(const BlockNormArgs &a, int x_dtype, int y_dtype, bool vec, int cus, hipStream_t st);

struct RopeArgs {
    const void *x;
    void *y;
    const int *pos;
    long pos_stride, xt, xh, yt, yh;
    int T, H, D, rot, pairing, tb;
    double turns[WQ_ROPE_MAX_ROT / 2];
    uint8_t axis[WQ_ROPE_MAX_ROT / 2];
};
hipError_t launch_rope(RopeArgs &a, int dtype, bool vec, int cus, hipStream_t st);

// ---------------------------------------------------------------------------
// The cache and the batch as kernels see them.
struct KvView {
    const uint8_t *k, *v;
    const float *ks, *vs;
    long rp, rh, rs; // row strides: page, head, slot (bytes)
    long sp, sh, ss; // scale strides (floats)
    int pages, heads, page;
    // position / page = mulhi(position, page_mul) >> page_shift; page_mul 0: a page of one position
    uint32_t page_mul;
    int page_shift;
};

struct BatchView {
    const int *q_start, *kv_len, *table;
    long table_stride;
    int B, T, width;
};

struct KvCopyArgs {
    KvView c;
    BatchView b;
    void *k, *v; // the tokens' side (read by append, written by read)
    long tok, head;
};
hipError_t launch_kv_append(const KvCopyArgs &a, int kind, int dim, int dtype, bool vec, hipStream_t st);
hipError_t launch_kv_read(const KvCopyArgs &a, int kind, int dim, int dtype, bool vec, hipStream_t st);

struct KvRopeArgs {
    KvView c;
    BatchView b;
    const void *q, *k, *v;
    void *q_out;
    const int *pos; // null: the tokens' positions in their sequences
    long pos_stride, qt, qh, ot, oh, tok, head;
    int H, rot, pairing;
    double turns[WQ_ROPE_MAX_ROT / 2];
    uint8_t axis[WQ_ROPE_MAX_ROT / 2];
    int first; // of the launch's tokens
};
hipError_t launch_kv_append_rope(const KvRopeArgs &a, int kind, int dim, int dtype, bool vec, int cus, hipStream_t st);

struct AttnArgs {
    KvView c;
    BatchView b;
    const void *q;
    void *o;
    float *lse;
    long qt, qh, ot, oh;
    float scale;
    int H, causal, window;
};
struct AttnPlan;
struct Partials;
hipError_t launch_attn_few(const AttnArgs &a, const AttnPlan &p, const Partials &pt, int kind, int dim, int dtype, bool vec,
                           bool wide, hipStream_t st);

hipError_t launch_attn_tiled(const AttnArgs &a, const AttnPlan &p, const Partials &pt, int kind, int dim, int dtype, bool vec,
                             bool wide, hipStream_t st);
hipError_t launch_attn_join(const AttnArgs &a, const AttnPlan &p, const Partials &pt, int dim, int dtype, hipStream_t st);

} // namespace wq

// ---------------------------------------------------------------------------
// Device helpers
namespace wq {

typedef __bf16 bf16;
typedef _Float16 f16;

// VEC consecutive elements as floats. VEC > 1: p is aligned to the vector.
template <typename T, int VEC>
__device__ __forceinline__ void load_vec(const T *p, float *v) {
    typedef T vt __attribute__((ext_vector_type(VEC)));
    const vt r = *reinterpret_cast<const vt *>(p);
#pragma unroll
    for (int i = 0; i < VEC; ++i) v[i] = (float)r[i];
}

template <typename T, int VEC>
__device__ __forceinline__ void store_vec(T *p, const float *v) {
    typedef T vt __attribute__((ext_vector_type(VEC)));
    vt r;
#pragma unroll
    for (int i = 0; i < VEC; ++i) r[i] = (T)v[i];
    *reinterpret_cast<vt *>(p) = r;
}

// Position / page, for positions below 2^31.
__device__ __forceinline__ int page_index(const KvView &c, int t) {
    return c.page_mul ? (int)(__umulhi((uint32_t)t, c.page_mul) >> c.page_shift) : t;
}

// Row of position t of sequence b: false if it is not there.
__device__ __forceinline__ bool find_row(const KvView &c, const BatchView &b, int seq, long t, int *page, int *slot) {
    if (t < 0) return false;
    const int i = page_index(c, (int)t);
    if (i >= b.width) return false;
    const int pg = b.table[(long)seq * b.table_stride + i];
    *page = pg;
    *slot = (int)((unsigned)t - (unsigned)i * (unsigned)c.page);
    return pg >= 0 && pg < c.pages;
}

} // namespace wq
