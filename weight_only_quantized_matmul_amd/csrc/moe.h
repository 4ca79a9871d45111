// Internal declarations of the mixture-of-experts operators: the experts' table, argument blocks shared by the C entry
// points (moe_api.cpp) and the kernel files, and the order of positions in a row of codes.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

#include "decoder.h"
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
    int planes; // bf16 parts of an element of x: 3 (f32), 2 (f16), 1 (bf16)
    // workspace
    int *plan;        // plan_ints(E, N)
    uint16_t *xp;     // [T][planes][in.kp]
    uint16_t *hp;     // [N][3][out.kp]
    float *d;         // [N][out.O]
};

// The plan: number of chosen experts, then three ints each (expert, first place in the order, rows), then the slots
// t * k + j sorted by expert.
__host__ __device__ inline long plan_ints(int E, long N) { return 4 + 3L * E + N; }

hipError_t launch_moe(const MoeArgs &a, int fmt, int dtype, hipStream_t st);

} // namespace wq
