// C entry points of the operators between a decoder layer's products
// (include/wqmm.h): argument checks and launches.
#include <climits>
#include <cmath>
#include <cstdio>
#include <new>

#include "attn_common.h"

namespace {

struct DeviceScope { // makes `dev` current, restoring the caller's device after
    int prev = -1;
    bool switched = false;
    explicit DeviceScope(int dev) {
        if (hipGetDevice(&prev) == hipSuccess && prev != dev) switched = hipSetDevice(dev) == hipSuccess;
    }
    ~DeviceScope() {
        if (switched) (void)hipSetDevice(prev);
    }
};

int status(hipError_t e) {
    return e == hipSuccess ? WQ_OK : e == hipErrorOutOfMemory ? WQ_E_OOM : e == hipErrorNotSupported ? WQ_E_UNSUPPORTED : WQ_E_HIP;
}

bool float_type(int t) { return t >= WQ_DT_F32 && t <= WQ_DT_F16; }

int size_of(int t) { return t == WQ_DT_F32 ? 4 : t == WQ_DT_I8 ? 1 : 2; }

bool aligned(const void *p, long a) { return ((uintptr_t)p & (uintptr_t)(a - 1)) == 0; }

// A buffer whose rows start at multiples of `a` bytes (strides in elements of `size` bytes).
bool rows_aligned(const void *p, long s0, long s1, int size, long a) {
    return aligned(p, a) && s0 * size % a == 0 && s1 * size % a == 0;
}

int check_cache(const wq_kv_cache *c) {
    if (c == nullptr || c->k == nullptr || c->v == nullptr || c->k_scale == nullptr || c->v_scale == nullptr)
        return WQ_E_INVAL;
    if (c->kind < WQ_KV_F16 || c->kind > WQ_KV_I4 || c->pages <= 0 || c->heads <= 0 || c->page <= 0 || c->dim <= 0)
        return WQ_E_INVAL;
    if (!aligned(c->k, 16) || !aligned(c->v, 16) || !aligned(c->k_scale, 4) || !aligned(c->v_scale, 4)) return WQ_E_INVAL;
    for (int i = 0; i < 3; ++i)
        if (c->row_stride[i] < 0 || c->row_stride[i] % 16 != 0 || c->scale_stride[i] < 0) return WQ_E_INVAL;
    if ((c->dim != 64 && c->dim != 128 && c->dim != 256) || c->heads > WQ_KV_MAX_HEADS) return WQ_E_UNSUPPORTED;
    return WQ_OK;
}

int check_batch(const wq_kv_batch *b) {
    if (b == nullptr || b->B < 0 || b->T < 0 || b->width < 0 || b->max_q < 0 || b->max_kv < 0 || b->table_stride < 0)
        return WQ_E_INVAL;
    if (b->B == 0 && b->T > 0) return WQ_E_INVAL;
    if (b->T == 0) return WQ_OK;
    if (b->q_start == nullptr || b->kv_len == nullptr || (b->table == nullptr && b->width > 0)) return WQ_E_INVAL;
    if (!aligned(b->q_start, 4) || !aligned(b->kv_len, 4) || !aligned(b->table, 4)) return WQ_E_INVAL;
    return WQ_OK;
}

wq::KvView view(const wq_kv_cache *c) {
    wq::KvView v;
    v.k = (const uint8_t *)c->k;
    v.v = (const uint8_t *)c->v;
    v.ks = c->k_scale;
    v.vs = c->v_scale;
    v.rp = c->row_stride[0];
    v.rh = c->row_stride[1];
    v.rs = c->row_stride[2];
    v.sp = c->scale_stride[0];
    v.sh = c->scale_stride[1];
    v.ss = c->scale_stride[2];
    v.pages = c->pages;
    v.heads = c->heads;
    v.page = c->page;
    // floor(2^(31+L) / page) + 1 with page <= 2^L: exact for positions below 2^31
    int L = 0;
    while ((1L << L) < c->page) ++L;
    v.page_mul = L == 0 ? 0 : (uint32_t)((1ull << (31 + L)) / (unsigned)c->page + 1);
    v.page_shift = L - 1;
    return v;
}

wq::BatchView view(const wq_kv_batch *b) {
    wq::BatchView v;
    v.q_start = b->q_start;
    v.kv_len = b->kv_len;
    v.table = b->table;
    v.table_stride = b->table_stride;
    v.B = b->B;
    v.T = b->T;
    v.width = b->width;
    return v;
}

int kv_copy(const wq_kv_cache *cache, const wq_kv_batch *batch, void *k, void *v, int dtype, long tok, long head,
            bool write, hipStream_t st) {
    int rc = check_cache(cache);
    if (rc == WQ_OK) rc = check_batch(batch);
    if (rc != WQ_OK) return rc;
    if (!float_type(dtype) || tok < 0 || head < 0) return WQ_E_INVAL;
    if (batch->T == 0) return WQ_OK;
    const int size = size_of(dtype);
    if (k == nullptr || v == nullptr || !aligned(k, size) || !aligned(v, size)) return WQ_E_INVAL;
    if ((rc = wq::begin_call(cache->device)) != WQ_OK) return rc;
    if ((long)batch->T * 2 * cache->heads > (long)INT_MAX) return WQ_E_UNSUPPORTED;
    DeviceScope scope(cache->device);
    wq::KvCopyArgs a;
    a.c = view(cache);
    a.b = view(batch);
    a.k = k;
    a.v = v;
    a.tok = tok;
    a.head = head;
    const bool vec = rows_aligned(k, tok, head, size, 16) && aligned(v, 16);
    return status(write ? wq::launch_kv_append(a, cache->kind, cache->dim, dtype, vec, st)
                        : wq::launch_kv_read(a, cache->kind, cache->dim, dtype, vec, st));
}

// How the positions are split: enough waves for every SIMD to have some in
// flight, but no split shorter than pays for its partial result. Lengths that
// are not known are taken from the table's width.
wq::AttnPlan plan_attn(const wq_kv_cache *c, const wq_kv_batch *b, int H, int causal, int window, bool f32, int cus) {
    wq::AttnPlan p;
    const long G = H / c->heads;
    const long q = b->max_q > 0 ? (b->max_q < b->T ? b->max_q : b->T) : ((long)b->T + b->B - 1) / b->B;
    long kv = (long)b->width * c->page;
    if (b->max_kv > 0 && b->max_kv < kv) kv = b->max_kv;
    if (window > 0 && causal && (long)window + q < kv) kv = (long)window + q;
    const int row = c->kind == WQ_KV_F16 ? 2 * c->dim : c->kind == WQ_KV_I8 ? c->dim : c->dim / 2;
    // Up to 64 rows (32 of 256 elements) the few-rows kernel reads the cache once a tile of 32 (16) rows, the second
    // time from L2, and on contexts of a thousand positions beats tiles of which half the rows are empty (60 rows of 128,
    // f32 on int8, 1000 positions: 15 us with one key/value head, tiled 19; 16.5 and 19.7 with eight). On long ones it
    // still does for rows of 64 and for int4 with one head (19531 positions: 14.5 and 20.6, 19.3 and 22.0) but not with
    // eight heads (43 and 31 us).
    p.few = q * G <= (c->dim <= 128 ? 64 : 32);
    p.waves = 4;
    if (p.few) {
        p.rows = q * G > 16 && c->dim <= 128 ? 32 : 16;
        p.step = row <= 64 ? 64 : 32;
    } else {
        // Eight waves share each opened tile where opening is dear (rows of 128 and 256) and their larger tiles still
        // give every CU a block: prefill of 4096 tokens 202 us, with four waves 232. Rows of 64 do better with more,
        // smaller blocks (13 prompts of up to 1695 tokens, window 507: four waves 43 us, eight 91 when they were there).
        const long wave_rows = wq::tiled_rows(c->dim, f32);
        if (c->dim > 64 && (q * G + 8 * wave_rows - 1) / (8 * wave_rows) * b->B * c->heads >= cus) p.waves = 8;
        p.rows = (int)wave_rows * p.waves;
        p.step = c->dim == 256 ? 32 : 64;
    }
    // tiles that are there (the numbers that whole sequences leave unused not counted), and their steps
    const long tiles = (q * G + p.rows - 1) / p.rows * b->B, numbers = wq::tile_count(b->T, G, p.rows, b->B);
    const long steps = (kv + p.step - 1) / p.step + 1;
    const long total = (tiles < numbers ? tiles : numbers) * c->heads * steps;
    if (p.few) {
        long per_wave = total / (cus * 12);
        // many sequences differ in length: shorter splits even that out (64 ragged sequences: 147 us with 512 positions
        // a wave, 173 with 1024); few are split for the chip's sake and pay for each split's start (4 long ones: 146 and 143 us)
        const long most = ((tiles < numbers ? tiles : numbers) * c->heads >= cus ? 512 : 1024) / p.step;
        per_wave = per_wave < 1 ? 1 : per_wave > most ? most : per_wave;
        p.least = (int)(4 * per_wave);
    } else {
        // a block for every CU: no split (its partial results cost more than the tail they save);
        // else enough splits for two blocks a CU
        const long blocks = (tiles < numbers ? tiles : numbers) * c->heads, want = blocks >= cus ? 1 : (2 * cus + blocks - 1) / blocks;
        p.least = (int)((steps + want - 1) / want);
        if (p.least < 4) p.least = 4;
    }
    long n = (steps + p.least - 1) / p.least;
    const long rows = (long)b->T * H;
    const long cap = (256L << 20) / (rows * (c->dim + 2) * 4); // workspace of at most 256 MiB
    n = n > 512 ? 512 : n;
    n = n > cap ? cap : n;
    p.nsplit = (int)(n < 1 ? 1 : n);
    p.ws_bytes = p.nsplit > 1 ? (size_t)rows * p.nsplit * (c->dim + 2) * 4 : 0;
    return p;
}

} // namespace

extern "C" {

int wq_rmsnorm_dev(int device, const void *x, int x_dtype, long x_stride, const void *residual, long res_stride,
                   const float *w, float eps, int rows, int n, void *y, int y_dtype, long y_stride, float *y_scale,
                   void *sum_out, long sum_stride, void *hip_stream) {
    if (!float_type(x_dtype) || (!float_type(y_dtype) && y_dtype != WQ_DT_I8)) return WQ_E_INVAL;
    if (rows < 0 || n <= 0 || x_stride < 0 || y_stride < 0 || !(eps >= 0.f)) return WQ_E_INVAL;
    if ((residual && res_stride < 0) || (sum_out && sum_stride < 0)) return WQ_E_INVAL;
    if (n > WQ_NORM_MAX_N) return WQ_E_UNSUPPORTED;
    if (rows == 0) return WQ_OK;
    if (x == nullptr || w == nullptr || y == nullptr || (y_dtype == WQ_DT_I8) != (y_scale != nullptr)) return WQ_E_INVAL;
    const int sx = size_of(x_dtype), sy = size_of(y_dtype);
    if (!aligned(x, sx) || !aligned(residual, sx) || !aligned(sum_out, sx) || !aligned(y, sy) || !aligned(w, 4) ||
        !aligned(y_scale, 4))
        return WQ_E_INVAL;
    const int rc = wq::begin_call(device);
    if (rc != WQ_OK) return rc;
    DeviceScope scope(device);
    wq::NormArgs a;
    a.x = x;
    a.res = residual;
    a.w = w;
    a.y = y;
    a.sum = sum_out;
    a.y_scale = y_scale;
    a.xs = x_stride;
    a.rs = res_stride;
    a.ys = y_stride;
    a.ss = sum_stride;
    a.eps = eps;
    a.rows = rows;
    a.n = n;
    const int vec = 16 / sx; // elements of a wide load of x
    const long ya = vec * sy < 16 ? vec * sy : 16;
    const bool wide = n % vec == 0 && rows_aligned(x, x_stride, 0, sx, 16) && aligned(w, 16) &&
                      rows_aligned(y, y_stride, 0, sy, ya) && (!residual || rows_aligned(residual, res_stride, 0, sx, 16)) &&
                      (!sum_out || rows_aligned(sum_out, sum_stride, 0, sx, 16));
    return status(wq::launch_rmsnorm(a, x_dtype, y_dtype, wide, wq::device_cus(device), (hipStream_t)hip_stream));
}

int wq_rope_create(int rot, int pairing, double theta, const int *sections, int axes, wq_rope **rope) {
    if (rope == nullptr || sections == nullptr || rot <= 0 || rot % 2 != 0 || (pairing != 0 && pairing != 1) ||
        axes <= 0 || !(theta > 0.0) || !std::isfinite(theta))
        return WQ_E_INVAL;
    if (rot > WQ_ROPE_MAX_ROT || axes > WQ_ROPE_MAX_AXES) return WQ_E_UNSUPPORTED;
    long sum = 0;
    for (int i = 0; i < axes; ++i) {
        if (sections[i] < 0) return WQ_E_INVAL;
        sum += sections[i];
    }
    if (sum != rot / 2) return WQ_E_INVAL;
    wq_rope *r = new (std::nothrow) wq_rope;
    if (r == nullptr) return WQ_E_OOM;
    r->magic = kRopeMagic;
    r->rot = rot;
    r->pairing = pairing;
    r->axes = axes;
    int i = 0;
    for (int ax = 0; ax < axes; ++ax)
        for (int j = 0; j < sections[ax]; ++j, ++i) {
            r->turns[i] = std::pow(theta, -2.0 * i / rot) / (2.0 * M_PI);
            r->axis[i] = (uint8_t)ax;
        }
    *rope = r;
    return WQ_OK;
}

int wq_rope_dev(const wq_rope *rope, int device, const void *x, int dtype, int T, int H, int D, long x_tok,
                long x_head, const int *pos_dev, long pos_stride, void *y, long y_tok, long y_head, void *hip_stream) {
    if (rope == nullptr || rope->magic != kRopeMagic || !float_type(dtype) || T < 0 || H < 0 || D < rope->rot ||
        x_tok < 0 || x_head < 0 || y_tok < 0 || y_head < 0 || pos_stride < 0)
        return WQ_E_INVAL;
    if (D > 65536 || H > WQ_KV_MAX_HEADS) return WQ_E_UNSUPPORTED;
    if (T == 0 || H == 0) return WQ_OK;
    const int size = size_of(dtype);
    if (x == nullptr || y == nullptr || pos_dev == nullptr || !aligned(x, size) || !aligned(y, size) ||
        !aligned(pos_dev, 4))
        return WQ_E_INVAL;
    const int rc = wq::begin_call(device);
    if (rc != WQ_OK) return rc;
    DeviceScope scope(device);
    wq::RopeArgs a;
    a.x = x;
    a.y = y;
    a.pos = pos_dev;
    a.pos_stride = pos_stride;
    a.xt = x_tok;
    a.xh = x_head;
    a.yt = y_tok;
    a.yh = y_head;
    a.T = T;
    a.H = H;
    a.D = D;
    a.rot = rope->rot;
    a.pairing = rope->pairing;
    for (int i = 0; i < rope->rot / 2; ++i) {
        a.turns[i] = rope->turns[i];
        a.axis[i] = rope->axis[i];
    }
    const bool vec = rows_aligned(x, x_tok, x_head, size, 16) && rows_aligned(y, y_tok, y_head, size, 16);
    return status(wq::launch_rope(a, dtype, vec, wq::device_cus(device), (hipStream_t)hip_stream));
}

int wq_rope_free(wq_rope *rope) {
    if (rope == nullptr) return WQ_OK;
    if (rope->magic != kRopeMagic) return WQ_E_INVAL;
    rope->magic = 0;
    delete rope;
    return WQ_OK;
}

int wq_kv_append_dev(const wq_kv_cache *cache, const wq_kv_batch *batch, const void *k_new, const void *v_new,
                     int dtype, long tok, long head, void *hip_stream) {
    return kv_copy(cache, batch, const_cast<void *>(k_new), const_cast<void *>(v_new), dtype, tok, head, true,
                   (hipStream_t)hip_stream);
}

int wq_kv_read_dev(const wq_kv_cache *cache, const wq_kv_batch *batch, void *k_out, void *v_out, int dtype, long tok,
                   long head, void *hip_stream) {
    return kv_copy(cache, batch, k_out, v_out, dtype, tok, head, false, (hipStream_t)hip_stream);
}

int wq_attn_paged_dev(const wq_kv_cache *cache, const wq_kv_batch *batch, const void *q, int dtype, int H, long q_tok,
                      long q_head, float scale, int causal, int window, void *o, long o_tok, long o_head, float *lse,
                      void *hip_stream) {
    int rc = check_cache(cache);
    if (rc == WQ_OK) rc = check_batch(batch);
    if (rc != WQ_OK) return rc;
    if (!float_type(dtype) || H <= 0 || H % cache->heads != 0 || q_tok < 0 || q_head < 0 || o_tok < 0 || o_head < 0 ||
        window < 0 || !std::isfinite(scale))
        return WQ_E_INVAL;
    if (H > WQ_KV_MAX_HEADS || (long)batch->T * (H / cache->heads) > (long)INT_MAX) return WQ_E_UNSUPPORTED;
    if (batch->T == 0) return WQ_OK;
    const int size = size_of(dtype);
    if (q == nullptr || o == nullptr || !aligned(q, size) || !aligned(o, size) || !aligned(lse, 4)) return WQ_E_INVAL;
    if ((rc = wq::begin_call(cache->device)) != WQ_OK) return rc;
    DeviceScope scope(cache->device);
    wq::AttnArgs a;
    a.c = view(cache);
    a.b = view(batch);
    a.q = q;
    a.o = o;
    a.lse = lse;
    a.qt = q_tok;
    a.qh = q_head;
    a.ot = o_tok;
    a.oh = o_head;
    a.scale = scale;
    a.H = H;
    a.causal = causal != 0;
    a.window = window;
    const wq::AttnPlan p = plan_attn(cache, batch, H, a.causal, window, dtype == WQ_DT_F32, wq::device_cus(cache->device));
    wq::Partials pt;
    pt.part = pt.ml = nullptr;
    pt.nsplit = p.nsplit;
    pt.least = p.least;
    if (p.ws_bytes > 0) {
        void *ws = nullptr;
        if ((rc = wq::stream_workspace(cache->device, p.ws_bytes, (hipStream_t)hip_stream, &ws)) != WQ_OK) return rc;
        pt.part = (float *)ws;
        pt.ml = pt.part + (size_t)batch->T * H * p.nsplit * cache->dim;
    }
    const bool vec = rows_aligned(q, q_tok, q_head, size, 16) && rows_aligned(o, o_tok, o_head, size, 16);
    // pools whose rows and scales all lie within 2^32 bytes are addressed by 32-bit offsets
    const auto extent = [&](const long *s) {
        return (double)(cache->pages - 1) * s[0] + (double)(cache->heads - 1) * s[1] + (double)(cache->page - 1) * s[2];
    };
    const bool wide = extent(cache->row_stride) + 2 * cache->dim >= 4294967296.0 ||
                      4 * (extent(cache->scale_stride) + 1) >= 4294967296.0;
    hipError_t e = p.few ? wq::launch_attn_few(a, p, pt, cache->kind, cache->dim, dtype, vec, wide, (hipStream_t)hip_stream)
                         : wq::launch_attn_tiled(a, p, pt, cache->kind, cache->dim, dtype, vec, wide, (hipStream_t)hip_stream);
    if (e == hipSuccess && p.nsplit > 1) e = wq::launch_attn_join(a, p, pt, cache->dim, dtype, (hipStream_t)hip_stream);
    return status(e);
}

int wq_describe_attn(const wq_kv_cache *cache, const wq_kv_batch *batch, int dtype, int H, int causal, int window, char *buf,
                     size_t buflen) {
    int rc = check_cache(cache);
    if (rc == WQ_OK) rc = check_batch(batch);
    if (rc != WQ_OK) return rc;
    if (!float_type(dtype) || H <= 0 || H % cache->heads != 0 || window < 0 || buf == nullptr || buflen == 0) return WQ_E_INVAL;
    if (batch->T == 0) {
        snprintf(buf, buflen, "none");
        return WQ_OK;
    }
    const bool open = cache->device >= 0 && cache->device < WQ_MAX_DEVICES && wq::device_cus(cache->device) > 0;
    const wq::AttnPlan p =
        plan_attn(cache, batch, H, causal != 0, window, dtype == WQ_DT_F32, open ? wq::device_cus(cache->device) : 256);
    const wq::JoinPlan j = wq::plan_join((long)batch->T * H, p.nsplit);
    char kernel[32];
    snprintf(kernel, sizeof kernel, p.few ? "few" : "tiled waves=%d", p.waves);
    snprintf(buf, buflen, "%s rows=%d step=%d splits=%d least=%d join=%dx%d workspace=%zu", kernel, p.rows, p.step, p.nsplit, p.least,
             p.nsplit > 1 ? j.waves : 0, p.nsplit > 1 ? j.at : 0, p.ws_bytes);
    return WQ_OK;
}

} // extern "C"
