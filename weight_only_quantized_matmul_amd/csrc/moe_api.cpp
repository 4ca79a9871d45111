// C entry points of the mixture-of-experts operators (include/wqmm.h): argument checks and launches.
#include <cmath>
#include <cstdio>
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

// Where a call's workspace holds what, in bytes from its start.
struct Layout {
    bool parts, apart, planned;
    size_t order, copy, h, d, xp, hp, xunit, hunit, bytes;
};

// How a call runs: everything of `a` but its buffers, and their places in the workspace. size: bytes of an element of x; x_vec: x
// is aligned to four of them.
int plan_moe(const wq_moe *moe, int size, int T, int k, long x_stride, bool x_vec, int cus, wq::MoeArgs *args, Layout *layout) {
    wq::MoeArgs &a = *args;
    Layout &l = *layout;
    a.experts = moe->d_experts;
    a.E = moe->E;
    a.T = T;
    a.k = k;
    a.in = moe->in;
    a.out = moe->out;
    const long N = (long)T * k;
    a.x_size = size;
    a.xe_n = (a.in.I + 3) / 4 * 4;
    a.ldh = (a.in.O + 3) / 4 * 4;
    // experts that some token chose, on average of an even choice
    int active = (int)(a.E * (1.0 - std::pow(1.0 - (k < a.E ? k : a.E) / (double)a.E, T)) + 0.5);
    if (active < 1) active = 1;
    // Operands for the rows that an expert has on average, with room for those that have more. 17 tokens on 64 experts of 768 x
    // 2048 in int4 (2.4 rows) 42.1 us with two, 45.3 with one, 55.2 with four; 64 tokens on 8 of 2048 x 6144 in int8 (16 rows)
    // 115 us with eight, 154 with four, 213 with two; one token 34.4 us with one, 36.2 with two.
    const double rows = (double)N / active;
    a.operands = T <= 4 || rows <= 1.6 ? 1 : T <= 8 || rows <= 4 ? 2 : T <= 16 || rows <= 10 ? 4 : 8;
    // (of the products' blocks, of 256 threads, as many as their smallest tiles of outputs make)
    const double pairs = N <= wq::kInlineSlots || N < a.E ? N : a.E;
    if ((double)T * (a.out.O + 255.0) > wq::kMaxThreads || (double)N * a.out.kp / 16 > wq::kMaxThreads ||
        pairs * (a.in.O + 15.0) * 16 > wq::kMaxThreads || pairs * (a.out.O + 31.0) * 8 > wq::kMaxThreads)
        return WQ_E_UNSUPPORTED;
    const int epb = wq::elems_per_byte(moe->fmt);
    const auto turned = [&](const wq::MoeShape &s) { return s.gs > 0 && s.gs % (64 * epb) != 0; };
    a.form_in = wq::moe_form(true, a.in.O, a.in.steps, turned(a.in), a.operands, active, cus);
    a.form_out = wq::moe_form(false, a.out.O, a.out.steps, turned(a.out), a.operands, active, cus);
    l.parts = a.operands >= 4;
    l.apart = !l.parts && (a.in.I % 4 != 0 || x_stride % 4 != 0 || !x_vec);
    l.planned = N > wq::kInlineSlots || l.apart || l.parts;
    const auto room = [](double bytes) { return (size_t)wq::round_up((long)bytes, 256); };
    l.order = l.planned ? room((double)(N < a.E ? N : a.E) * sizeof(wq::MoeWork)) : 0;
    l.copy = l.order + (l.planned ? room(4.0 * N) : 0);
    l.h = l.copy + (l.apart ? room((double)T * a.xe_n * size) : 0);
    l.d = l.h + room(4.0 * N * a.ldh);
    l.xp = l.d + room(4.0 * N * a.out.O);
    l.hp = l.xp + (l.parts ? (size_t)T * a.in.steps * 512 * epb : 0);
    l.xunit = l.hp + (l.parts ? (size_t)N * a.out.steps * 512 * epb : 0);
    l.hunit = l.xunit + (l.parts ? room(4.0 * T * a.in.steps) : 0);
    l.bytes = l.hunit + (l.parts ? (size_t)4 * N * a.out.steps : 0);
    return WQ_OK;
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
    Layout l;
    if ((rc = plan_moe(moe, size, T, k, x_stride, aligned(x, 4 * size), wq::device_cus(moe->device), &a, &l)) != WQ_OK) return rc;
    a.ids = ids;
    a.weights = weights;
    a.x = x;
    a.add = add;
    a.y = y;
    a.xs = x_stride;
    a.as = add_stride;
    a.ys = y_stride;
    a.x_bf16 = dtype == WQ_DT_BF16;
    void *ws = nullptr;
    if ((rc = wq::stream_workspace(moe->device, l.bytes, (hipStream_t)hip_stream, &ws)) != WQ_OK) return rc;
    char *at = (char *)ws;
    a.plan = l.planned ? (wq::MoeWork *)at : nullptr;
    a.order = (int *)(at + l.order);
    a.copy = l.apart ? at + l.copy : nullptr;
    a.h = (float *)(at + l.h);
    a.d = (float *)(at + l.d);
    a.xp = l.parts ? (uint8_t *)at + l.xp : nullptr;
    a.hp = l.parts ? (uint8_t *)at + l.hp : nullptr;
    a.xunit = (float *)(at + l.xunit);
    a.hunit = (float *)(at + l.hunit);
    a.xe = l.apart ? a.copy : x;
    a.xes = l.apart ? a.xe_n : x_stride;
    return status(wq::launch_moe(a, moe->fmt, dtype, (hipStream_t)hip_stream));
}

int wq_describe_moe(const wq_moe *moe, int dtype, int T, int k, long x_stride, char *buf, size_t buflen) {
    if (moe == nullptr || moe->magic != wq::kMoeMagic || !float_type(dtype) || T <= 0 || k <= 0 || x_stride < 0 || buf == nullptr || buflen == 0)
        return WQ_E_INVAL;
    if ((long)T * k > WQ_MOE_MAX_ROWS) return WQ_E_UNSUPPORTED;
    wq::MoeArgs a;
    Layout l;
    const int rc = plan_moe(moe, size_of(dtype), T, k, x_stride, true, wq::device_is_open(moe->device) ? wq::device_cus(moe->device) : 256, &a, &l);
    if (rc != WQ_OK) return rc;
    char text[2][96];
    for (int i = 0; i < 2; ++i) {
        const wq::MoeForm &f = i ? a.form_out : a.form_in;
        const int pos = 128 * wq::elems_per_byte(moe->fmt), rows = wq::moe_rows(f.m, f.wk, pos), all = wq::moe_steps((i ? a.out : a.in).steps, f.wk);
        const int one = wq::moe_phase(f.m, f.wk, pos, 1, all), full = wq::moe_phase(f.m, f.wk, pos, rows, all);
        snprintf(text[i], sizeof text[i], "operands=%d waves=%d tiles=%d rows=%d phases=%d-%d", f.m, f.wk, f.tiles, rows, (all + one - 1) / one, (all + full - 1) / full);
    }
    snprintf(buf, buflen, "in %s out %s plan=%d copy=%d workspace=%zu", text[0], text[1], (int)l.planned, (int)l.apart, l.bytes);
    return WQ_OK;
}

} // extern "C"
