// C entry points of the mixture-of-experts operators (include/wqmm.h): argument checks and launches.
#include <cmath>
#include <new>

#include "entry.h"
#include "moe.h"

namespace {

bool resident(const wq_tensor *t) { return t != nullptr && t->magic == wq::kTensorMagic; }

wq::MoeShape shape_of(const wq_tensor *t) {
    wq::MoeShape s;
    s.O = t->O;
    s.I = t->I;
    s.stride = (int)t->stride;
    s.nfull = t->nfull;
    s.gs = t->gs;
    s.ng = t->ng;
    s.steps = (int)((t->stride + 127) / 128);
    s.kp = s.steps * 128 * wq::elems_per_byte(t->fmt);
    return s;
}

bool alike(const wq_tensor *a, const wq_tensor *b) {
    return a->device == b->device && a->fmt == b->fmt && a->O == b->O && a->I == b->I && a->gs == b->gs;
}

// A matrix whose bytes 32-bit offsets address and whose positions an int counts.
bool small(const wq_tensor *t) { return (double)t->O * t->stride < 4294967296.0 && t->stride <= (1 << 28); }

wq::MoeMatrix matrix_of(const wq_tensor *t) {
    wq::MoeMatrix m;
    m.w = t->d_w;
    m.scales = t->gs > 0 ? t->d_scales_t : t->d_scales;
    return m;
}

} // namespace

extern "C" {

int wq_moe_route_dev(int device, const void *scores, int dtype, int T, int E, long stride, const float *bias, int gating,
                     int groups, int top_groups, int k, int normalise, float scale, int *ids, float *weights,
                     void *hip_stream) {
    if (!float_type(dtype) || T < 0 || E <= 0 || stride < 0 || k <= 0 || k > E || groups <= 0 || E % groups != 0 ||
        top_groups <= 0 || top_groups > groups || (gating != WQ_GATE_SOFTMAX && gating != WQ_GATE_SIGMOID) || !std::isfinite(scale))
        return WQ_E_INVAL;
    if ((long)(E / groups) * top_groups < k) return WQ_E_INVAL;
    if (E > WQ_MOE_MAX_EXPERTS || k > WQ_MOE_MAX_K || groups > WQ_MOE_MAX_GROUPS) return WQ_E_UNSUPPORTED;
    if (T == 0) return WQ_OK;
    if (scores == nullptr || ids == nullptr || weights == nullptr || !aligned(scores, size_of(dtype)) || !aligned(bias, 4) ||
        !aligned(ids, 4) || !aligned(weights, 4))
        return WQ_E_INVAL;
    const int rc = wq::begin_call(device);
    if (rc != WQ_OK) return rc;
    DeviceScope scope(device);
    wq::RouteArgs a;
    a.scores = scores;
    a.stride = stride;
    a.bias = bias;
    a.ids = ids;
    a.weights = weights;
    a.T = T;
    a.E = E;
    a.k = k;
    a.groups = top_groups == groups ? 1 : groups; // all of them: no choice among groups
    a.top_groups = top_groups == groups ? 1 : top_groups;
    a.sigmoid = gating == WQ_GATE_SIGMOID;
    a.normalise = normalise != 0;
    a.scale = scale;
    return status(wq::launch_route(a, dtype, (hipStream_t)hip_stream));
}

int wq_moe_create(wq_tensor *const *gate, wq_tensor *const *up, wq_tensor *const *down, int E, wq_moe **moe) {
    if (gate == nullptr || up == nullptr || down == nullptr || moe == nullptr || E <= 0) return WQ_E_INVAL;
    if (E > WQ_MOE_MAX_EXPERTS) return WQ_E_UNSUPPORTED;
    for (int e = 0; e < E; ++e) {
        if (!resident(gate[e]) || !resident(up[e]) || !resident(down[e])) return WQ_E_INVAL;
        if (!alike(gate[e], gate[0]) || !alike(up[e], gate[0]) || !alike(down[e], down[0])) return WQ_E_INVAL;
    }
    if (down[0]->device != gate[0]->device || down[0]->fmt != gate[0]->fmt || down[0]->I != gate[0]->O) return WQ_E_INVAL;
    if (gate[0]->fmt == WQ_F32 || !small(gate[0]) || !small(down[0])) return WQ_E_UNSUPPORTED;
    const int device = gate[0]->device;
    if (!wq::device_is_open(device)) return WQ_E_NOTINIT;
    DeviceScope scope(device);
    wq_moe *m = new (std::nothrow) wq_moe;
    wq::MoeExpert *table = new (std::nothrow) wq::MoeExpert[E];
    int rc = m == nullptr || table == nullptr ? WQ_E_OOM : WQ_OK;
    if (rc == WQ_OK) {
        for (int e = 0; e < E; ++e) {
            table[e].gate = matrix_of(gate[e]);
            table[e].up = matrix_of(up[e]);
            table[e].down = matrix_of(down[e]);
        }
        rc = wq::device_table(device, table, (size_t)E * sizeof(wq::MoeExpert), (void **)&m->d_experts);
    }
    delete[] table;
    if (rc != WQ_OK) {
        delete m;
        return rc;
    }
    m->magic = wq::kMoeMagic;
    m->device = device;
    m->fmt = gate[0]->fmt;
    m->E = E;
    m->in = shape_of(gate[0]);
    m->out = shape_of(down[0]);
    *moe = m;
    return WQ_OK;
}

int wq_moe_free(wq_moe *moe) {
    if (moe == nullptr) return WQ_OK;
    if (moe->magic != wq::kMoeMagic) return WQ_E_INVAL;
    DeviceScope scope(moe->device);
    wq::device_table_free(moe->device, moe->d_experts, (size_t)moe->E * sizeof(wq::MoeExpert));
    moe->magic = 0;
    delete moe;
    return WQ_OK;
}

int wq_moe_ffn_dev(const wq_moe *moe, const void *x, int dtype, int T, long x_stride, const int *ids, const float *weights,
                   int k, const void *add, long add_stride, void *y, long y_stride, void *hip_stream) {
    if (moe == nullptr || moe->magic != wq::kMoeMagic || !float_type(dtype) || T < 0 || k <= 0 || x_stride < 0 ||
        y_stride < 0 || (add && add_stride < 0))
        return WQ_E_INVAL;
    if ((long)T * k > WQ_MOE_MAX_ROWS) return WQ_E_UNSUPPORTED;
    if (T == 0) return WQ_OK;
    const int size = size_of(dtype);
    if (x == nullptr || y == nullptr || ids == nullptr || weights == nullptr || !aligned(x, size) || !aligned(y, size) ||
        !aligned(add, size) || !aligned(ids, 4) || !aligned(weights, 4))
        return WQ_E_INVAL;
    int rc = wq::begin_call(moe->device);
    if (rc != WQ_OK) return rc;
    DeviceScope scope(moe->device);
    wq::MoeArgs a;
    a.experts = moe->d_experts;
    a.E = moe->E;
    a.cus = wq::device_cus(moe->device);
    a.T = T;
    a.k = k;
    a.ids = ids;
    a.weights = weights;
    a.x = x;
    a.add = add;
    a.y = y;
    a.xs = x_stride;
    a.as = add_stride;
    a.ys = y_stride;
    a.in = moe->in;
    a.out = moe->out;
    const long N = (long)T * k;
    a.x_size = size;
    a.x_bf16 = dtype == WQ_DT_BF16;
    a.xe_n = (a.in.I + 3) / 4 * 4;
    a.ldh = (a.in.O + 3) / 4 * 4;
    a.active = (int)(a.E * (1.0 - std::pow(1.0 - (k < a.E ? k : a.E) / (double)a.E, T)) + 0.5);
    if (a.active < 1) a.active = 1;
    // Operands for the rows that an expert has on average, with room for those that have more. 17 tokens on 64 experts of 768 x
    // 2048 in int4 (2.4 rows) 44.3 us with two, 48.6 with one, 56.3 with four; 64 tokens on 8 of 2048 x 6144 in int8 (16 rows)
    // 126 us with eight, 159 with four, 232 with two; one token 34.8 us with one, 36.7 with two.
    const double rows = (double)N / a.active;
    // (of the products' blocks, of 256 threads, as many as their smallest tiles of outputs make)
    const double pairs = N <= wq::kInlineSlots || N < a.E ? N : a.E;
    if ((double)T * (a.out.O + 255.0) > wq::kMaxThreads || (double)N * a.out.kp / 16 > wq::kMaxThreads ||
        pairs * (a.in.O + 15.0) * 16 > wq::kMaxThreads || pairs * (a.out.O + 31.0) * 8 > wq::kMaxThreads)
        return WQ_E_UNSUPPORTED;
    a.operands = T <= 4 || rows <= 1.6 ? 1 : T <= 8 || rows <= 4 ? 2 : T <= 16 || rows <= 10 ? 4 : 8;
    const bool parts = a.operands >= 4;
    const bool apart = !parts && (a.in.I % 4 != 0 || x_stride % 4 != 0 || !aligned(x, 4 * size));
    const bool planned = N > wq::kInlineSlots || apart || parts;
    const size_t plan = planned ? (size_t)wq::round_up((N < a.E ? N : a.E) * sizeof(wq::MoeWork), 256) : 0;
    const size_t order = planned ? (size_t)wq::round_up(4 * N, 256) : 0;
    const size_t copy = apart ? (size_t)wq::round_up((long)T * a.xe_n * size, 256) : 0;
    const size_t h = (size_t)wq::round_up(4 * N * a.ldh, 256);
    const int epb = wq::elems_per_byte(moe->fmt);
    const size_t d = (size_t)wq::round_up(4 * N * a.out.O, 256);
    const size_t xp = parts ? (size_t)T * a.in.steps * 512 * epb : 0, hp = parts ? (size_t)N * a.out.steps * 512 * epb : 0;
    const size_t xu = parts ? (size_t)wq::round_up(4L * T * a.in.steps, 256) : 0, hu = parts ? (size_t)4 * N * a.out.steps : 0;
    void *ws = nullptr;
    if ((rc = wq::stream_workspace(moe->device, plan + order + copy + h + d + xp + hp + xu + hu, (hipStream_t)hip_stream, &ws)) != WQ_OK) return rc;
    char *at = (char *)ws;
    a.plan = planned ? (wq::MoeWork *)at : nullptr;
    a.order = (int *)(at += plan);
    a.copy = apart ? at + order : nullptr;
    a.h = (float *)(at += order + copy);
    a.d = (float *)(at += h);
    a.xp = parts ? (uint8_t *)at + d : nullptr;
    a.hp = a.xp + xp;
    a.xunit = (float *)(at + d + xp + hp);
    a.hunit = (float *)(at + d + xp + hp + xu);
    a.xe = apart ? a.copy : x;
    a.xes = apart ? a.xe_n : x_stride;
    return status(wq::launch_moe(a, moe->fmt, dtype, (hipStream_t)hip_stream));
}

} // extern "C"
