// Internal declarations of the mixture-of-experts operators: the experts' table, argument blocks shared by the C entry
// points (moe_api.cpp) and the kernel files, and the order of positions in a row of codes.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

#include "decoder.h"
#include "moe_plan.h"
#include "wq_internal.h"

namespace wq {

constexpr uint32_t kMoeMagic = 0x57514D31u; // "WQM1"

// What the kernels read of one resident matrix.
struct MoeMatrix {
    const uint8_t *w;
    const float *scales; // O floats, or group-major ng x O
};

struct MoeExpert {
    MoeMatrix gate, up, down;
};

// The shape that the experts' matrices of one kind share.
struct MoeShape {
    int O, I;
    int stride; // bytes a row
    int nfull;  // permuted 1 KiB blocks a row
    int gs, ng;
    int steps;  // 128-byte steps a row
    int kp;     // positions a row with the last step filled up
};

} // namespace wq

struct wq_moe {
    uint32_t magic;
    int device, fmt, E;
    wq::MoeShape in, out; // gate and up; down
    wq::MoeExpert *d_experts;
};

namespace wq {

// ---------------------------------------------------------------------------
struct RouteArgs {
    const void *scores;
    long stride;
    const float *bias;
    int *ids;
    float *weights;
    int T, E, k, groups, top_groups;
    bool sigmoid, normalise;
    float scale;
};
hipError_t launch_route(const RouteArgs &a, int dtype, hipStream_t st);

constexpr int kInlineSlots = 256; // up to as many, the products' blocks find their expert's rows for themselves

// ---------------------------------------------------------------------------
struct MoeArgs {
    const MoeExpert *experts;
    int E, T, k;
    const int *ids;       // [T, k]
    const float *weights; // [T, k]
    const void *x, *add;
    void *y;
    long xs, as, ys;
    MoeShape in, out;
    // x as the products read it: rows of xe_n elements (a multiple of four, zeros behind x's own) of x_size bytes, four-aligned
    const void *xe;
    long xes;
    int xe_n, x_size;
    bool x_bf16;
    int ldh;                 // floats a row of h, a multiple of four
    int operands;              // 1, 2; 4, 8: activations in prepared parts
    MoeForm form_in, form_out; // of gate and up, of down
    // workspace
    MoeWork *plan; // min(E, N), those without rows last; null: the products' blocks plan for themselves
    int *order;    // N slots, with a plan
    void *copy;    // x in rows that can be read four at a time; null: they can
    float *h;      // [N][ldh]
    float *d;      // [N][out.O]
    uint8_t *xp, *hp;      // parts: [T][in.steps] and [N][out.steps] times four planes of a step's positions
    float *xunit, *hunit;  // [T][in.steps], [N][out.steps]
};

hipError_t launch_moe(MoeArgs &a, int fmt, int dtype, hipStream_t st);
hipError_t launch_moe_i8(MoeArgs &a, hipStream_t st);
hipError_t launch_moe_i4(MoeArgs &a, hipStream_t st);
hipError_t launch_moe_i2(MoeArgs &a, hipStream_t st);

} // namespace wq
