/*
 * wqmm.h — C ABI of libwqmm.so, the weight-resident quantized matmul for
 * AMD Instinct MI355X (gfx950).
 *
 * Operation (colibri "第 8 章 · 02 CUDA/Metal/Vulkan 三后端", section 四, the
 * qmatmul.comp header; colibri-analysis "CUDA 后端", section 1, quant_matmul):
 *
 *     y[s,o] = scale[o] * sum_{i<I} dequant(W[o,i]) * x[s,i]
 *
 * W is an [O, I] weight matrix kept resident in device memory in one of four
 * storage formats, with one fp32 scale per output row applied after the sum;
 * x is fp32 [S, I] and y is fp32 [S, O], both row-major with s outer
 * (x[s*I + i], y[s*O + o]).
 *
 * Storage formats (format list: colibri-analysis "CUDA 后端", section 1,
 * row_bytes; codes 0..2 from the Vulkan tensor description in "第 8 章 · 02",
 * section 三; dequant offsets from weight_at in the same section 1):
 *   WQ_F32  4 bytes per element, little-endian IEEE single, used as is;
 *   WQ_I8   1 byte per element, two's complement, used as is;
 *   WQ_I4   2 elements per byte, even element in the low nibble,
 *           value = nibble - 8;
 *   WQ_I2   4 elements per byte, element 4j+k in bits 2k..2k+1 of byte j,
 *           value = code - 2.
 * A packed host row is row_bytes = ceil(I*bits/8) bytes; rows follow each
 * other with no padding; unused high bits of a row's last byte are ignored.
 *
 * Accuracy contract: for every output element,
 *     |y - y_exact| <= 1e-5 * sum_i |scale[o] * q[o,i] * x[s,i]| + 1e-30,
 * and results are deterministic (same inputs, same launch configuration,
 * same bits). Rows whose codes all decode to 0, rows with scale 0 and
 * products that are exact integers sums are reproduced exactly.
 *
 * Errors: every function returns WQ_OK (0) or a negative WQ_E_* code; nothing
 * aborts or exits, and on an error no output is written. A caller that gets
 * an error may fall back to its own CPU path, as the reference engine does
 * when its GPU call fails (colibri-analysis "CUDA 后端", section 3.1).
 *
 * Threads: calls on one device must not overlap from several host threads.
 * Calls on different devices are independent.
 */
#ifndef WQMM_H
#define WQMM_H

#include <stddef.h>

#ifdef __cplusplus
extern "C" {
#endif

#define WQ_MAX_DEVICES 16   /* size of the static device table */
#define WQ_GEMV_MAX_S 8     /* largest S the register GEMV serves (by default f32 only; quantized formats take it at S = 1 and the matrix-core paths above) */

enum wq_fmt { WQ_F32 = 0, WQ_I8 = 1, WQ_I4 = 2, WQ_I2 = 3 };

enum wq_status {
    WQ_OK = 0,
    WQ_E_INVAL = -1,       /* bad argument (NULL pointer, size, format, device list) */
    WQ_E_NODEV = -2,       /* no usable GPU, or the device is not gfx950-capable */
    WQ_E_NOTINIT = -3,     /* device not opened by wq_init */
    WQ_E_OOM = -4,         /* device memory (or WQ_MEM_LIMIT_BYTES budget) exhausted */
    WQ_E_MISMATCH = -5,    /* re-upload with a different device/format/shape */
    WQ_E_HIP = -6,         /* the HIP runtime reported an error */
    WQ_E_FAULT = -7,       /* failure injected with WQ_FAULT (tests of caller fallback) */
    WQ_E_UNSUPPORTED = -8  /* valid request this build cannot serve */
};

typedef struct wq_tensor wq_tensor; /* opaque resident weight tensor */
typedef struct wq_group wq_group;   /* opaque set of tensors run in one launch */

/*
 * Open devices (colibri-analysis "CUDA 后端", section 1, coli_cuda_init: the
 * ordinals are validated and each GPU gets its own context).
 * devices: host array of ndev ordinals; NULL with ndev == 0 opens device 0.
 * Rejects duplicates, negative or out-of-range ordinals and ndev >
 * WQ_MAX_DEVICES (WQ_E_INVAL); no GPU or a non-gfx950 GPU gives WQ_E_NODEV.
 * Calling it again is allowed: already-open devices are kept, and the
 * environment knobs are read again (WQ_FORCE_PATH=gemv|tiled|skinny|auto,
 * WQ_GEMV_MAX_S, WQ_MEM_LIMIT_BYTES, WQ_FAULT=upload|launch,
 * WQ_SKINNY_RING=4|6 (chunks of loads in flight per wave of the few-rows
 * kernel, capped at its spill-free depth; default 2), WQ_WAVES_PER_CU,
 * WQ_TILED_MODE=bf16x3|bf16|fp32, WQ_TILED_SHAPE=BMxBNxBK (a compiled tile shape:
 * 128x96x64, 128x96x128, 64x64x64, 64x64x128, 64x192x64 or 16x128x64 in the
 * bf16x3 mode, the same but 16x128x64 in the bf16 mode, 128x96x32 or 64x64x32
 * in fp32 mode; a 128-deep shape is taken with group scales only when the
 * group size is a multiple of 128, else the automatic choice stands),
 * where WQ_TILED_MODE=bf16 is an opt-in reduced-precision tiled mode for
 * quantized weights (the int4 x 16-bit-activation matrix-unit dispatch in
 * colibri docs "CUDA backend (Linux)", section "The GPU-resident pipeline"):
 * each activation is rounded
 * to the nearest bf16 (ties to even) and multiplied once on the bf16 matrix
 * units. Its results are within the usual bound of the exact product on the
 * rounded activations, hence within 2^-8 * sum_i |scale * q * x| of the exact
 * product on the fp32 ones; the default bf16x3 mode gives up no precision.
 * It applies to calls that take the tiled path only (quantized S > 32 by
 * default),
 * WQ_VERBOSE=1 prints one line per device on stderr).
 */
int wq_init(const int *devices, int ndev);

/*
 * Free and total device memory in bytes (colibri-analysis "CUDA 后端",
 * section 1, coli_cuda_mem_info). free_b/total_b: host pointers, either may be
 * NULL. WQ_E_NOTINIT if the device was not opened.
 */
int wq_mem_info(int device, size_t *free_b, size_t *total_b);

/* Bytes of one packed host row: ceil(I*bits/8); -1 for a bad fmt or I < 0.
 * Host-only, needs no device. */
long wq_row_bytes(int fmt, long I);

/*
 * Upload a weight tensor once and keep it resident (colibri-analysis
 * "CUDA 后端", section 1, coli_cuda_tensor_upload; uploads happen lazily and
 * once, colibri docs "CUDA backend (Linux)", introduction).
 *   t:      in/out handle. *t == NULL: allocate, copy w and scales, set *t.
 *           *t != NULL: nothing is copied; the call only checks that device,
 *           fmt, O and I match the resident tensor (WQ_E_MISMATCH if not).
 *   w:      host pointer to O packed rows of wq_row_bytes(fmt, I) bytes.
 *   scales: host pointer to O floats; may be NULL only for WQ_F32 (scale 1).
 * The copy is synchronous: the caller may free w and scales on return. The
 * library owns the device copy until wq_tensor_free.
 * Errors: WQ_E_INVAL (NULL t or w, bad fmt, O <= 0, I <= 0, missing scales),
 * WQ_E_NOTINIT, WQ_E_OOM, WQ_E_HIP, WQ_E_FAULT (WQ_FAULT=upload).
 */
int wq_tensor_upload(wq_tensor **t, int device, int fmt, int O, int I, const void *w,
                     const float *scales);

/*
 * Upload with group-wise scales: one fp32 scale per (output row o, group of
 * gs consecutive columns) — the group-size field of the Vulkan tensor
 * description (colibri "第 8 章 · 02 CUDA/Metal/Vulkan 三后端", section 三):
 *     y[s,o] = sum_g scales[o*ng + g] * sum_{i in [g*gs, (g+1)*gs)} q[o,i] x[s,i],
 * ng = ceil(I/gs) (the last group may be shorter).
 *   scales: host pointer to O * ng floats, row-major (required).
 *   gs:     group size, a positive multiple of 64 (WQ_E_UNSUPPORTED otherwise;
 *           each 16-byte weight slot and each 64-column tiled step then lies
 *           inside one group). 2 <= S <= 16 runs on the few-rows matrix-core
 *           kernel when gs is a multiple of 128 (int8, int4) or 256 (int2),
 *           else on the tiled path (wq_describe_plan_gs tells which).
 * Formats int8/int4/int2 only (WQ_E_INVAL for WQ_F32 or gs <= 0). Otherwise
 * as wq_tensor_upload; a re-upload also checks gs (WQ_E_MISMATCH). The
 * tensor then works with every matmul call; groups containing such tensors
 * take the grouped few-rows launch (below) when its conditions hold, else
 * one launch per tensor.
 */
int wq_tensor_upload_gs(wq_tensor **t, int device, int fmt, int O, int I, int gs, const void *w,
                        const float *scales);

/*
 * Lazy upload plus a synchronous matmul on host buffers (colibri-analysis
 * "CUDA 后端", section 1, coli_cuda_matmul: upload on first use, copy x in,
 * run, copy y back, all blocking).
 * Same tensor arguments as wq_tensor_upload; x: host [S, I] floats, y: host
 * [S, O] floats (written). S == 0 uploads (if needed) and returns WQ_OK.
 */
int wq_matmul(wq_tensor **t, int device, int fmt, int O, int I, const void *w,
              const float *scales, const float *x, int S, float *y);

/* Synchronous matmul with an already-resident tensor; x, y host pointers.
 * x and y pass through pinned host buffers mapped into the device's address
 * space (library-owned, grown to the largest call, held until the process
 * ends), which kernels on the library stream copy to and from device memory;
 * y is written only when the call succeeds. */
int wq_matmul_t(const wq_tensor *t, const float *x, int S, float *y);

/*
 * Stream-ordered matmul on device buffers, queued on hip_stream (a
 * hipStream_t; NULL = the device's null stream): no copies and no host
 * synchronisation. x_dev: device [S, I] floats, y_dev: device [S, O] floats,
 * both on the tensor's device and 4-byte aligned. The call returns once the
 * work is queued; y_dev is valid after the stream reaches it.
 * Quantized formats at S = 1, f32 at S <= 8: the register GEMV, one kernel
 * launch, no workspace. Quantized 2 <= S <= 32 with I % 4 == 0 and x_dev
 * 16-byte aligned: the few-rows matrix-core kernel, one launch, no
 * workspace (above S = 16 with four waves per block, one block per CU; for
 * S > 20 only where at most one block per CU covers all O rows, else the
 * tiled path). Larger S (or rows the few-rows kernel cannot read in 16-byte
 * runs) with a quantized format (tiled path, bf16x3 mode): two launches that use the
 * stream's workspace (3 * round_up(S, 128) * round_up(fields per row, 128)
 * bf16 values, 16-row padding for S <= 16; when K is split across blocks,
 * a third launch adds ksplit * S * O fp32 partials kept after them;
 * wq_describe_plan prints the size). Each stream has a workspace of its
 * own, so tiled calls on different streams may overlap; it grows on demand,
 * which waits for the device to go idle and allocates. Up to 8 streams per
 * device hold one; the first tiled call on a ninth stream takes over the
 * least recently used stream's workspace (also waiting for the device). The
 * key is the stream handle: a destroyed stream's workspace passes to a new
 * stream that gets the same handle, so let a stream's queued calls finish
 * before destroying it. A call being captured into a HIP graph never waits
 * or allocates: it uses its stream's workspace if that is large enough,
 * else the largest workspace on the device that is, else it returns
 * WQ_E_UNSUPPORTED; so run the largest S once, eagerly, before capturing.
 * A graph keeps the buffer that its calls were captured with: that buffer
 * is never freed and never passes to another stream, whatever calls follow
 * (a stream that needs more gets a new one and leaves the old one, until
 * the process ends, to the graph). The stream whose workspace it was (the one
 * captured, or the one that lent the largest) goes on with the buffer until
 * then, so do not replay the graph while that stream, or another graph with
 * the same buffer, runs calls that use a workspace: results would be wrong.
 */
int wq_matmul_dev(const wq_tensor *t, const float *x_dev, int S, float *y_dev, void *hip_stream);

/*
 * wq_matmul_dev for callers that cannot allocate device memory: code under
 * HIP graph capture, tight serving loops, harnesses that forbid allocation.
 * Same arguments, kernels and results as wq_matmul_dev (bit for bit), but
 * the call never allocates or frees anything: the tiled path's workspace is
 * a fixed device array of WQ_NOALLOC_SCRATCH_BYTES per device, reserved for
 * this call when the library is loaded and held until the process ends (its
 * address is looked up in wq_init). A call whose workspace would exceed it
 * (wq_describe_plan prints the size; e.g. S = 2048 with I = 8192 int8)
 * returns WQ_E_UNSUPPORTED before any launch. Every call on a device shares
 * that device's array, which keeps the last call's contents (each call
 * rewrites every part it reads, so nothing needs clearing): calls that
 * overlap in time on one device -- from two streams, or two host threads --
 * race on it and must not be issued. Calls on different devices do not
 * share it. Errors as wq_matmul_dev, plus WQ_E_UNSUPPORTED.
 */
#define WQ_NOALLOC_SCRATCH_BYTES (32u << 20)
int wq_matmul_dev_noalloc(const wq_tensor *t, const float *x_dev, int S, float *y_dev, void *hip_stream);

/* Size in bytes of the fixed device array wq_matmul_dev_noalloc uses. Host-only. */
size_t wq_noalloc_scratch_bytes(void);

/*
 * Build a group of G resident tensors that run together in one launch (the
 * grouped expert matmul of a mixture-of-experts decode step; grouped expert
 * handling at prefill is described in colibri docs "CUDA backend (Linux)",
 * section "The GPU-resident pipeline"). All tensors must be on the same
 * device and share one format. The work split (balanced by weight bytes) is
 * built once here and kept on the device. The group references the tensors:
 * free the group before any of its tensors.
 */
int wq_grouped_create(wq_tensor *const *ts, int G, wq_group **group);

/*
 * Run every tensor of a plain group (a gated group gives WQ_E_INVAL):
 * y_dev[g] = matmul(ts[g], x_dev[g], S[g]).
 * x_dev, S, y_dev: host arrays of G entries (device pointers inside);
 * S[g] == 0 skips tensor g. When every S[g] <= the grouped GEMV limit
 * (4 for int4 and int2, 8 for int8 and f32) and every row
 * fits one wave of the register GEMV, up to 64 tensors run as ONE launch on
 * hip_stream whatever their shapes (e.g. the gate, up and down projections
 * of 8 experts: 24 tensors with 3 KiB and 1 KiB rows), the work cut into
 * pieces of equal weight bytes when the group is created; more tensors take
 * one launch per 64 (none of this with group-wise scales). Otherwise, when
 * every S[g] <= 32 (16 with group-wise scales), every x_dev[g] is 16-byte
 * aligned, every I % 4 == 0 and every group size is a multiple of 128
 * (int8, int4) or 256 (int2), the
 * tensors run on the few-rows matrix-core kernel, one launch per 32 tensors
 * with S[g] > 0 (blocks of 16 to 64 output rows of one tensor each; the
 * tile is that of the largest S[g]; with any group-scaled tensor the
 * group-scaled kernel, where a row-scaled tensor is one group as long as
 * its row). Otherwise one wq_matmul_dev per
 * tensor, still stream-ordered (the tiled ones share the stream's
 * workspace, in stream order).
 */
int wq_grouped_matmul_dev(wq_group *group, const float *const *x_dev, const int *S,
                          float *const *y_dev, void *hip_stream);

/* Release a group (plain or gated); NULL is a no-op. */
int wq_grouped_free(wq_group *group);

/*
 * Gated feed-forward of a mixture-of-experts layer (the fused gate/up matmul
 * feeding the down projection: the gated up-projection shader
 * qmatmul_gate_up.comp named in colibri "第 8 章 · 02 CUDA/Metal/Vulkan
 * 三后端", learning goals and section recap, whose body and activation the
 * pages do not give; SiLU gating is the reading taken). For expert e:
 *
 *     g = gate_e . x_e,  u = up_e . x_e      (each as wq_matmul_dev computes it)
 *     h_e[s,o] = silu(g[s,o]) * u[s,o],      silu(z) = z / (1 + e^-z)
 *     y_e = down_e . h_e
 *
 * wq_swiglu_create pairs gate[e] with up[e] (host arrays of E tensors, all on
 * one device in one format; gate[e] and up[e] must have the same O, I and
 * group size, else WQ_E_INVAL) into a gated group, freed with
 * wq_grouped_free before its tensors. The group references the tensors.
 *
 * wq_swiglu_matmul_dev: h_dev[e] = h_e, an fp32 [S[e], O_e] device buffer,
 * for x_dev[e] fp32 [S[e], I_e] (host arrays of E device pointers; S[e] == 0
 * skips expert e). Stream-ordered on hip_stream. With every S[e] within the
 * grouped GEMV limit, one scale per row and rows that fit one wave, all experts run
 * in one launch that reads each gate row and up row once and writes h
 * directly (g and u never reach memory); otherwise, on the conditions of
 * the grouped few-rows launch (see wq_grouped_matmul_dev), the gate and up
 * matmuls of up to 16 experts run per launch of the few-rows matrix-core
 * kernel (gate -> h_dev[e], up -> the stream's workspace), then one
 * activation launch per 32 experts; otherwise each expert runs as its own
 * paired launch, or (S above the grouped GEMV limit, or group-wise scales)
 * as gate -> h_dev[e], up -> the stream's workspace, then an activation
 * kernel. The forms through the workspace may grow it (not while the stream
 * is being captured: see wq_matmul_dev; warm up first).
 *
 * Accuracy: g and u meet the matmul contract; h is silu and the product
 * evaluated in fp32 on those values (a few ulps, no further cancellation).
 *
 * wq_swiglu_ffn_dev: the whole layer, both launches stream-ordered on
 * hip_stream: h_dev as above (the caller's intermediate buffers), then
 * y_dev[e] = down_e . h_e through the plain group `down` (wq_grouped_create
 * of the E down tensors, down[e]->I == gate[e]->O, else WQ_E_INVAL);
 * y_dev[e] is fp32 [S[e], O_down_e].
 */
int wq_swiglu_create(wq_tensor *const *gate, wq_tensor *const *up, int E, wq_group **group);
int wq_swiglu_matmul_dev(wq_group *gated, const float *const *x_dev, const int *S,
                         float *const *h_dev, void *hip_stream);
int wq_swiglu_ffn_dev(wq_group *gated, wq_group *down, const float *const *x_dev, const int *S,
                      float *const *h_dev, float *const *y_dev, void *hip_stream);

/* Release a resident tensor (colibri-analysis "CUDA 后端", section 1,
 * coli_cuda_tensor_free). NULL is a no-op. */
int wq_tensor_free(wq_tensor *t);

/* Static description of a status code; never NULL. */
const char *wq_strerror(int code);

/*
 * Introspection for tests and tools: the kernel path wq_matmul_dev would take
 * for (fmt, O, I, S) on this build, written as a NUL-terminated string into
 * buf (e.g. "gemv fmt=2 smax=1 lw=16 kmax=4 k=3 team=1 d=4 rows_per_team=12 grid=256 block=256",
 * "skinny fmt=2 m=2 rpl=2 nb=3 waves=8 ring=2 chunks=48 chunks_per_wave=6 grid=256 block=512 workspace=0",
 * or "tiled fmt=1 mode=bf16x3 bm=128 bn=96 bk=64 tiles_s=4 tiles_o=64 ksplit=1 grid=256 block=512 workspace=...").
 * Host-only: needs no device. Returns WQ_OK or WQ_E_INVAL.
 */
int wq_describe_plan(int fmt, int O, int I, int S, char *buf, size_t buflen);

/* The same for a tensor uploaded with wq_tensor_upload_gs(..., gs, ...)
 * (gs = 0: as wq_describe_plan). WQ_E_INVAL also for gs < 0. */
int wq_describe_plan_gs(int fmt, int O, int I, int S, int gs, char *buf, size_t buflen);

/*
 * Measurement helper (not part of the matmul): the practical HBM read
 * ceiling. Reads `bytes` (a multiple of 16) from the device buffer buf_dev
 * (16-byte aligned) exactly once with the 128-bit non-temporal loads the
 * GEMV streams its weights with: `waves` waves (a positive multiple of 4,
 * blocks of 4 waves) each read one contiguous chunk, keeping
 * loads_in_flight (1, 2, 4, 5, 8, 9, 12, 16, 18, 24 or 36) loads of 1 KiB in
 * flight.
 * out_dev (device, 4-byte aligned) receives 64 * waves words (an
 * exclusive-or of the words read, so the loads cannot be dropped).
 * Stream-ordered on hip_stream, no host synchronisation. It gives the GEMV
 * timings a measured ceiling to be read against (colibri docs "CUDA backend
 * (Linux)" print no kernel-level rates, so the ceiling is measured, not
 * quoted). Errors: WQ_E_INVAL for a bad argument, WQ_E_HIP.
 */
int wq_stream_read_dev(const void *buf_dev, size_t bytes, int waves, int loads_in_flight, unsigned *out_dev,
                       void *hip_stream);

/* ------------------------------------------------------------------------
 * Between a decoder layer's products: the norm before a product, rotary
 * positions of queries and keys, the quantised key/value cache and the
 * attention of new tokens over it. All calls are stream-ordered on hip_stream
 * (a hipStream_t; NULL = the null stream) with device buffers, queue their
 * work without host synchronisation, may be captured into a HIP graph, need
 * wq_init on the device, and give the same bits for the same inputs and the
 * same launch configuration. Strides are in elements unless said otherwise;
 * the last dimension of every buffer is contiguous. Buffers must be aligned
 * to their element type; 16-byte aligned rows take the wide loads and others
 * a slower path with the same results. WQ_FAULT=launch makes each of them
 * return WQ_E_FAULT. Work that no launch holds (attention of more than about
 * 16 million tiles, 2^31 cache rows a call) is refused with WQ_E_UNSUPPORTED.
 */
enum wq_dtype { WQ_DT_F32 = 0, WQ_DT_BF16 = 1, WQ_DT_F16 = 2, WQ_DT_I8 = 3 };

#define WQ_NORM_MAX_N 32768 /* longest row of wq_rmsnorm_dev */
#define WQ_ROPE_MAX_ROT 256 /* most rotated elements of a head */
#define WQ_ROPE_MAX_AXES 8
#define WQ_KV_MAX_HEADS 1024 /* most heads of a cache or of queries */

/*
 * Root-mean-square norm, with the residual's addition:
 *     r = x + residual            (in fp32; residual NULL: r = x)
 *     y = r / sqrt(mean(r^2) + eps) * w
 * x, residual, sum_out: [rows, n] of x_dtype (f32, bf16, f16), row strides
 * x_stride, res_stride, sum_stride; w: n floats; y: [rows, n] of y_dtype, row
 * stride y_stride. sum_out (NULL: not kept) receives r rounded to x_dtype;
 * the norm is taken of the unrounded r. y_dtype WQ_DT_I8 needs y_scale (rows
 * floats): y_scale = max|y| / 127 and the codes are
 * rint(127 * (r*w) / max|r*w|), the quotient in fp64, so y ~ code * y_scale;
 * a row of zeros gets codes 0 and scale 0, a row holding an infinity or a
 * NaN codes 0 and a NaN scale. Finite rows of any size have finite squares
 * here (in float types a row of zeros with eps 0 is 0 / 0, a NaN). sum_out may be x or residual (same stride), and
 * y may be x when the types and strides agree.
 * n <= WQ_NORM_MAX_N (WQ_E_UNSUPPORTED above); rows == 0 is a no-op.
 */
int wq_rmsnorm_dev(int device, const void *x, int x_dtype, long x_stride, const void *residual, long res_stride,
                   const float *w, float eps, int rows, int n, void *y, int y_dtype, long y_stride, float *y_scale,
                   void *sum_out, long sum_stride, void *hip_stream);

/*
 * The norms around a block's output x, with its gate and the residual between them:
 *     z = x / sqrt(mean(x^2) + eps) * w_post      (w_post NULL: z = x)
 *     r = residual + alpha * gate * z             (gate NULL: 1)
 *     y = r / sqrt(mean(r^2) + eps) * w_pre
 * x, gate, residual, sum_out: [rows, n] of x_dtype (f32, bf16, f16) with row
 * strides x_stride, gate_stride (0: one row of gates for all), res_stride,
 * sum_stride; w_post, w_pre: n floats; y: [rows, n] of y_dtype (f32, bf16,
 * f16), row stride y_stride. sum_out (NULL: not kept) receives r rounded to
 * x_dtype; the second norm is taken of the unrounded r. y and w_pre may both be
 * NULL (only sum_out is written). Everything between is fp32; finite rows of
 * any size have finite squares (a row of zeros with eps 0 is 0 / 0, a NaN).
 * sum_out may be x, gate or residual (same stride, and rows that no other row
 * reads), and so may y when the types agree too, but not the one that is
 * sum_out. n <= WQ_NORM_MAX_N (WQ_E_UNSUPPORTED above); rows == 0 is a no-op.
 */
int wq_rmsnorm_block_dev(int device, const void *x, int x_dtype, long x_stride, const float *w_post, const void *gate,
                         long gate_stride, float alpha, const void *residual, long res_stride, const float *w_pre, float eps,
                         int rows, int n, void *y, int y_dtype, long y_stride, void *sum_out, long sum_stride, void *hip_stream);

/*
 * Rotary positions. The first `rot` elements of a head (even, at most
 * WQ_ROPE_MAX_ROT) form rot/2 pairs; pair i is (x[i], x[i + rot/2]) with
 * pairing 0 and (x[2i], x[2i+1]) with pairing 1, and is turned by the angle
 *     pos[axis(i)] * theta^(-2i / rot),
 * where the pairs are dealt to the axes in order: the first sections[0] pairs
 * follow axis 0, the next sections[1] axis 1, and so on (one axis: text;
 * three: time, height and width). Elements past rot are copied. Angles are
 * reduced in fp64, so far positions keep fp32 accuracy.
 *
 * wq_rope_create makes the plan (host memory only; sections: host array of
 * `axes` non-negative counts with sum rot/2; theta > 0); wq_rope_free
 * releases it (NULL is a no-op). wq_rope_dev turns x [T, H, D] (strides
 * x_tok, x_head) into y (y_tok, y_head; may be x itself with x's strides);
 * pos: device int32 [axes, T] with row stride pos_stride.
 */
typedef struct wq_rope wq_rope;
int wq_rope_create(int rot, int pairing, double theta, const int *sections, int axes, wq_rope **rope);
int wq_rope_dev(const wq_rope *rope, int device, const void *x, int dtype, int T, int H, int D, long x_tok,
                long x_head, const int *pos_dev, long pos_stride, void *y, long y_tok, long y_head, void *hip_stream);
int wq_rope_free(wq_rope *rope);

/*
 * A paged, quantised key/value cache: pools the caller owns. A row holds the
 * D = dim codes of one token and head and stands for code * scale:
 *   WQ_KV_F16  2 bytes a code, IEEE half; the scale is a power of two that
 *              puts the row's largest magnitude into [2^14, 2^15];
 *   WQ_KV_I8   1 byte, two's complement, scale = max|x| / 127;
 *   WQ_KV_I4   2 codes a byte, even element in the low half, stored as
 *              code + 8 with codes -7..7, scale = max|x| / 7.
 * Row (page, head, slot) starts at page*row_stride[0] + head*row_stride[1] +
 * slot*row_stride[2] BYTES from k (and from v), its scale at the same sum of
 * scale_stride (in floats) from k_scale (v_scale); k, v and row_stride are
 * multiples of 16 bytes. dim is 64, 128 or 256; `page` slots a page (any
 * number >= 1), `pages` pages, `heads` key/value heads.
 *
 * A batch: the new tokens of B sequences stand one after another, sequence b's
 * at q_start[b] .. q_start[b+1]-1 (device int32 [B+1], ascending from 0 to T);
 * they are the last of its kv_len[b] positions (device int32 [B]), so the i-th
 * new token has position p = kv_len[b] - q_len[b] + i. Position t lies in slot
 * t % page of page table[b*table_stride + t / page] (device int32, `width`
 * entries a sequence; entries past a sequence's end are not read as pages).
 * max_q and max_kv: the longest q_len and kv_len (0: not known); they choose
 * the split of the work only, results are right for any lengths.
 * Positions outside the table, and those whose entry is outside [0, pages),
 * are not there: append skips them, read gives zeros, attention does not see
 * them. Nothing is read or written outside the pools and the T tokens,
 * whatever q_start, kv_len and table hold.
 */
enum wq_kv_kind { WQ_KV_F16 = 0, WQ_KV_I8 = 1, WQ_KV_I4 = 2 };

typedef struct wq_kv_cache {
    int device, kind, pages, heads, page, dim;
    void *k, *v;
    float *k_scale, *v_scale;
    long row_stride[3];
    long scale_stride[3];
} wq_kv_cache;

typedef struct wq_kv_batch {
    int B, T, width, max_q, max_kv;
    long table_stride;
    const int *q_start, *kv_len, *table;
} wq_kv_batch;

/*
 * Quantise the T new tokens' keys and values ([T, heads, dim] of dtype f32,
 * bf16 or f16, strides tok, head for both) into their slots. Codes are
 * rint(x / scale), the quotient in fp64 (ties to even). A row whose largest
 * magnitude is below 2^-100 is stored as zeros with scale 0; a row holding an
 * infinity or a NaN as zero codes with a NaN scale.
 */
int wq_kv_append_dev(const wq_kv_cache *cache, const wq_kv_batch *batch, const void *k_new, const void *v_new,
                     int dtype, long tok, long head, void *hip_stream);

/*
 * Rotary positions and append in one launch: the queries q [T, H, dim] of dtype
 * are turned into q_out (NULL, both: none; q_out may be q with q's strides), the
 * keys k_new are turned, rounded to fp32 and quantised into their slots as by
 * wq_kv_append_dev, the values v_new as they are. Turning follows wq_rope_dev
 * with the plan `rope` (rot <= dim), in fp64 up to that rounding (queries of
 * 16 bits in fp32). pos: device
 * int32 [axes, T], row stride pos_stride; NULL (plans of one axis only): each
 * token's position p in its sequence. Tokens that have no place in the cache
 * are turned all the same; rows past q_start[B] are left as they were.
 */
int wq_kv_append_rope_dev(const wq_kv_cache *cache, const wq_kv_batch *batch, const wq_rope *rope, const void *q, int H,
                          long q_tok, long q_head, void *q_out, long qo_tok, long qo_head, const void *k_new, const void *v_new,
                          int dtype, long tok, long head, const int *pos_dev, long pos_stride, void *hip_stream);

/* The values the batch's T tokens have in the cache, code * scale in fp32
 * rounded to dtype, as k_out, v_out [T, heads, dim] with strides tok, head. */
int wq_kv_read_dev(const wq_kv_cache *cache, const wq_kv_batch *batch, void *k_out, void *v_out, int dtype, long tok,
                   long head, void *hip_stream);

/*
 * Attention of the batch's new tokens over the cache. For token i of sequence
 * b with position p, and query head h reading key/value head h / (H/heads):
 *     s_t = scale * q . k_t,   w = softmax of s over the seen positions t,
 *     o = sum_t w_t v_t,       lse = log sum_t exp(s_t),
 * where t is seen if 0 <= t < kv_len[b], t <= p (causal) and t > p - window
 * (window > 0). A token that sees nothing gets o = 0 and lse = -inf. What
 * unseen positions hold (infinities and NaN among it) never enters a result;
 * a seen value's code that is not finite makes its element of o an infinity
 * or a NaN.
 * q, o: [T, H, dim] of dtype (f32, bf16, f16) with strides; H a multiple of
 * the cache's heads; lse: float [T, H], contiguous, or NULL. The softmax
 * statistics and all sums are fp32; codes enter the matrix units exactly.
 * f32 queries enter as two f16 parts (22 bits and more), 16-bit queries
 * exactly. Probabilities (times their values' scales) of f32 queries enter as
 * three bf16 parts (24 bits) against integer codes, and else as two f16 parts
 * (22 bits, down to 2^-39 of the largest value scale in the row), but for bf16
 * queries of many rows: one f16 part (2^-11), an eighth of what rounding o to
 * bf16 leaves.
 * Where the positions are split among blocks, partial results pass through
 * the stream's workspace as in wq_matmul_dev (it may grow; while the stream
 * is being captured it cannot: warm up first, else WQ_E_UNSUPPORTED; a graph
 * keeps the buffer it was captured with, also after the stream's has grown).
 */
int wq_attn_paged_dev(const wq_kv_cache *cache, const wq_kv_batch *batch, const void *q, int dtype, int H, long q_tok,
                      long q_head, float scale, int causal, int window, void *o, long o_tok, long o_head, float *lse,
                      void *hip_stream);

/*
 * The plan of wq_attn_paged_dev for these sizes as text (host only; buffers
 * are not looked at, 256 CUs where the device is not open), for tests and
 * logs: "few rows=16 step=32 splits=12 least=8 join=4x8 workspace=...", or
 * "tiled waves=8 rows=256 ...": the kernel, rows a tile, positions a step, the
 * most splits of a tile's positions and the fewest steps a split takes, how
 * the join reads them (waves a row x partial rows in flight, 0x0: no splits)
 * and the workspace in bytes.
 */
int wq_describe_attn(const wq_kv_cache *cache, const wq_kv_batch *batch, int dtype, int H, int causal, int window, char *buf,
                     size_t buflen);

/* ------------------------------------------------------------------------
 * A mixture-of-experts layer without the host in between: the choice of each
 * token's experts, and the experts' gated feed-forward over tokens whose
 * experts only the device knows. Stream-ordered and capturable like the calls
 * above.
 */
#define WQ_MOE_MAX_EXPERTS 1024
#define WQ_MOE_MAX_GROUPS 64
#define WQ_MOE_MAX_K 32
#define WQ_MOE_MAX_ROWS 16384 /* most T * k of wq_moe_ffn_dev */

enum wq_gating { WQ_GATE_SOFTMAX = 0, WQ_GATE_SIGMOID = 1 };

/*
 * The k experts of each of T tokens, from the router's scores [T, E] of dtype
 * (f32, bf16, f16; row stride `stride`):
 *     p = softmax over the E scores, or sigmoid of each;   c = p + bias
 * (bias: E floats; NULL: c = p). The experts stand in `groups` groups of
 * E / groups; a group's value is the sum of its two largest c (of its one,
 * where it has one), and only the top_groups groups of largest value are left.
 * ids [T, k] (int32, contiguous) receives the k experts of largest c among
 * them, in descending order; weights [T, k] (floats, contiguous) their p,
 * divided by the sum of the k if `normalise`, times scale. Of equal values the
 * lower index goes first. p, c and sums are fp64. A NaN score counts as -inf,
 * +inf as the largest fp32; where softmax sees -inf only, every p is 0; a sum of
 * 0 leaves weights of 0. A NaN c counts as -inf, and so does a group's value
 * that is none (its two largest c are +inf and -inf).
 * 1 <= k <= E / groups * top_groups. WQ_E_UNSUPPORTED: E > WQ_MOE_MAX_EXPERTS,
 * groups > WQ_MOE_MAX_GROUPS, k > WQ_MOE_MAX_K. T == 0 is a no-op.
 */
int wq_moe_route_dev(int device, const void *scores, int dtype, int T, int E, long stride, const float *bias, int gating,
                     int groups, int top_groups, int k, int normalise, float scale, int *ids, float *weights,
                     void *hip_stream);

/*
 * The layer's E experts: host arrays of resident tensors on one device, all in
 * one quantized format (WQ_F32: WQ_E_UNSUPPORTED), gate[e] and up[e] all of one
 * shape [F, D] and group size, down[e] all of one shape [D_out, F] and group size
 * (else WQ_E_INVAL). A tensor may stand in several places. The layer
 * references the tensors: free it before them. Tensors of 4 GiB and more:
 * WQ_E_UNSUPPORTED.
 */
typedef struct wq_moe wq_moe;
int wq_moe_create(wq_tensor *const *gate, wq_tensor *const *up, wq_tensor *const *down, int E, wq_moe **moe);
int wq_moe_free(wq_moe *moe); /* NULL is a no-op */

/*
 * The layer for a few tokens:
 *     y[t] = add[t] + sum_j weights[t,j] * down_e . h,   e = ids[t,j],
 *     h = silu(gate_e . x[t]) * (up_e . x[t]),           silu(z) = z / (1 + e^-z)
 * x [T, D], add (NULL: zeros) and y [T, D_out] of dtype (f32, bf16, f16) with
 * row strides x_stride, add_stride, y_stride; ids int32 [T, k] and weights float
 * [T, k] contiguous on the device. An id outside [0, E) adds nothing (a place
 * of a batch without a token, an expert that lives elsewhere); an expert that
 * stands twice counts twice. y may be x or add (same stride).
 * The products take codes as they are, and activations (x, and h in fp32) as
 * integers of up to 31 bits: whole multiples of a power of two that those share
 * which meet the same 128 bytes of a resident row (128 elements with int8
 * weights, 256 with int4, 512 with int2, not all side by side), each within
 * 2^-30 of the largest magnitude among them (magnitudes below 2^-96: within
 * 2^-126). Sums over those are exact (with group scales over parts of them),
 * sums over the row fp32 and, with group scales, within 2^-126; the sum over j
 * is fp32 in the order of j, y rounded once. An infinity or NaN in x, or an h
 * that overflows, makes that expert's row for the token NaN. What a token gets
 * does not depend on what the other tokens hold or chose; their number chooses
 * among forms that split the sums differently.
 * It uses the stream's workspace as wq_matmul_dev's tiled path does (it may
 * grow, but not while the stream is being captured).
 * T * k above WQ_MOE_MAX_ROWS, or shapes whose launches could have 2^32 threads
 * (16 * F, 8 * D_out times min(E, T * k)), give WQ_E_UNSUPPORTED. Up to there it
 * takes less time than wq_swiglu_ffn_dev on a group of all experts with rows
 * gathered by expert (which keeps 24 bits of each activation, whatever is
 * multiplied beside it), but for about 1024 rows an expert and more. T == 0 is
 * a no-op.
 */
int wq_moe_ffn_dev(const wq_moe *moe, const void *x, int dtype, int T, long x_stride, const int *ids, const float *weights,
                   int k, const void *add, long add_stride, void *y, long y_stride, void *hip_stream);

/*
 * The plan of wq_moe_ffn_dev for these sizes as text (host only; buffers are
 * not looked at, x counts as aligned, 256 CUs where the device is not open), for
 * tests and logs: "in operands=2 waves=1 tiles=3 rows=8 phases=1-2 out ...
 * plan=0 copy=0 workspace=...". For gate and up (in) and for down (out): operands
 * of four activations, waves along a row of weights, tiles of outputs a block
 * takes one after another, rows of an expert at a time, and the phases in which
 * a block takes the activations of one row and of all of those; plan: a launch
 * sorts the slots by expert; copy: x is copied into aligned rows; and the
 * workspace in bytes.
 */
int wq_describe_moe(const wq_moe *moe, int dtype, int T, int k, long x_stride, char *buf, size_t buflen);

#ifdef __cplusplus
}
#endif

#endif /* WQMM_H */
