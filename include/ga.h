/*
 * ga.h -- fused row-wise gated activations on AMD Instinct MI355X (gfx950).
 *
 * Two operations of a transformer FFN / MoE layer, on rows of an input laid
 * out as [rows, 2d] with the gate in columns [0, d) and up in [d, 2d):
 *
 *   ga_gelu_and_mul_sparse   Gemma3n-style sparse GELU-and-multiply (vLLM PR
 *       48498, "[Performance] Add Triton kernel for Gemma3n sparse GELU",
 *       section Purpose): per row, mean and population std of the gate,
 *       cutoff = mean + z * std, out = gelu_tanh(max(gate - cutoff, 0)) * up,
 *       where gelu_tanh(s) = 0.5 s (1 + tanh(sqrt(2/pi) (s + 0.044715 s^3)))
 *       and z = Phi^-1(target sparsity) (1.6448536 for 95%).
 *   ga_silu_and_mul_bounded  silu(gate) * up over only the live rows of a
 *       capture-sized MoE buffer (Megatron-LM PR 6328, "Size MoE activation
 *       kernel grid to the row count", section What changed and why): the
 *       launch shape depends on the buffer capacity only, and the live count
 *       is read on the device, so one launch can be replayed from a graph
 *       while the count changes.
 *
 * Arithmetic is fp32 inside the kernels; the result is rounded once, to
 * nearest even, to the element type.  Input and output share one element
 * type: fp32, fp16 or bf16.
 *
 * Conventions for every entry point:
 *   - Pointers named in/out/live_rows are DEVICE pointers on the current HIP
 *     device; the caller owns all memory.  Tensors are dense and row-major
 *     (row stride 2d elements for in, d for out).  The library allocates
 *     nothing on the device and keeps no state apart from a per-device cache
 *     of the compute-unit count.
 *   - `stream` is a hipStream_t (NULL = the null stream).  Launches are
 *     asynchronous on that stream and never synchronise, so they may be
 *     recorded into a HIP graph by stream capture.
 *   - All argument checks happen on the host before any HIP call; a rejected
 *     call touches no memory.  ga_last_error() then returns a message.
 *   - Out-of-range device live counts are clamped to [0, rows]; they cannot
 *     be reported (no synchronisation).  A live_rows pointer must be 4-byte
 *     aligned (GA_EINVAL otherwise).
 *   - Any alignment natural to the element type is accepted; when in and out
 *     are 16-byte aligned and a row's bytes are a multiple of 16, 16-byte
 *     vector loads and stores are used.  Otherwise the data still moves as
 *     16-byte vectors of consecutive elements, each one unaligned 16-byte
 *     access (gfx950 runs global memory in unaligned-access mode):
 *     gelu_and_mul_sparse per row (rows up to 8192 vectors; rows of up to 32
 *     vectors packed several to a wavefront, as aligned ones are), the other
 *     ops flat over the output region.
 */
#ifndef GA_H
#define GA_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum { GA_F32 = 0, GA_F16 = 1, GA_BF16 = 2 } ga_dtype;

typedef enum {
    GA_OK = 0,
    GA_EINVAL = 1,       /* malformed argument (null pointer, negative size, ...) */
    GA_EUNSUPPORTED = 2, /* well-formed but outside what the kernels handle;
                            callers fall back to another implementation */
    GA_EHIP = 3          /* the HIP runtime reported an error at launch */
} ga_status;

/* A hipStream_t, passed opaquely so this header needs no HIP include. */
typedef void *ga_stream;

/* Largest d (elements per half row) the kernels take. */
#define GA_MAX_D 65536

/* Launch geometry.  Filled by the planners, or by a caller that wants a
 * specific geometry (a tuning sweep); see ga_gelu_and_mul_sparse_with_plan. */
typedef struct {
    int32_t path;          /* 0: 16-byte vector path, 1: per-element path,
                              2: unaligned path (rows off 16-byte alignment; gelu: per
                                 row, the elementwise ops: flat over the output),
                              3: gelu packed-rows path (short rows of any alignment,
                              several rows per wavefront),
                              4: gelu replicated-statistics path (few rows: `splits`
                                 workgroups per row each reduce the whole gate row and
                                 apply their share; 16-byte rows, no workspace) */
    int32_t waves_per_row; /* gelu: 64-lane wavefronts per workgroup (1,2,4,8,16) */
    int32_t per_lane;      /* gelu vector path: 16-byte gate vectors per lane (1,2,4,8;
                              split rows 1,2,4); gelu element path: gate elements per
                              lane (4,16,64); gelu unaligned path: 16-byte vectors per
                              lane (1..8); gelu packed rows: vectors per lane (1,2,4);
                              silu: items per lane per step (1,2,4) */
    int32_t up_late;       /* gelu vector and unaligned paths: 0 = load the up row together
                              with the gate row (shortest latency), 1 = load it after the
                              statistics, a vector (a chunk) at a time (fewer registers, more
                              rows resident); split rows: 0 only */
    int32_t block;         /* threads per workgroup */
    int32_t splits;        /* gelu vector path: workgroups sharing one row; 1, or 2 .. 16
                              (needs a workspace, see ga_gelu_and_mul_sparse_ws); gelu
                              replicated-statistics path: 2, 4 or 8 */
    int64_t grid;          /* workgroups launched (silu: from the capacity M only) */
    uint32_t spin_limit;   /* split rows: rounds of polls of the row's partials before a
                              workgroup computes the whole row's statistics itself */
    int32_t flags;         /* gelu_and_mul_sparse: 0 or GA_ROUND_INTERMEDIATES (not
                              with split rows); silu: zero */
    int32_t lanes_per_row; /* gelu packed-rows path: lanes sharing one row (4, 8, 16, 32;
                              a 256-lane workgroup holds 256 / lanes_per_row rows);
                              other paths: zero */
    int32_t reserved;      /* zero */
} ga_plan;

/*
 * Round-trip form of gelu_and_mul_sparse (vLLM PR 48498, section
 * Cross-architecture warp and dtype validation and the review thread that
 * follows it: the Triton kernel rounds intermediates to the input dtype so
 * that it reproduces native PyTorch, whose every operation returns a tensor
 * of that dtype).  The pages do not list the rounding points; this library
 * rounds where an eager PyTorch composition of the op stores a tensor: the
 * row mean, the row std, z, z * std, the cutoff mean + z * std, gate -
 * cutoff, the GELU output, and the product.  Statistics are still computed
 * in fp32 from the input values.  For fp32 data the form differs from the
 * default only by the fp32 roundings of those intermediates.  The match with
 * the eager composition covers finite inputs: a NaN in a gate row makes that
 * composition's whole row NaN, while both forms here take max(NaN, 0) as 0.
 */
#define GA_ROUND_INTERMEDIATES 1

/*
 * Sparse GELU-and-multiply.
 *   in        [T, 2d] device array of `dtype`; gate = cols [0,d), up = cols [d,2d).
 *   out       [T, d] device array of `dtype`; must not overlap `in`.
 *   T         rows (tokens), 0 <= T <= INT32_MAX; T == 0 launches nothing.
 *   d         elements per half row, 1 <= d <= GA_MAX_D (larger: GA_EUNSUPPORTED).
 *   dtype     a ga_dtype.
 *   z         cutoff multiplier Phi^-1(target sparsity); must be finite.
 *   live_rows NULL: all T rows.  Else a device int32; rows r with
 *             r >= clamp(*live_rows, 0, T) are left untouched.
 * Returns GA_OK once the launch is enqueued.  A launch is one workgroup per
 * row (rows of up to 32 16-byte vectors: several rows per workgroup); where
 * its work-items would reach 2^32 (T >= 2^26 / waves per row, e.g. T = 2^26
 * rows of d = 512 bf16), the call returns GA_EUNSUPPORTED before any HIP call
 * (split the rows over several calls).
 */
ga_status ga_gelu_and_mul_sparse(const void *in, void *out, int64_t T, int64_t d,
                                 int32_t dtype, float z, const int32_t *live_rows,
                                 ga_stream stream);

/*
 * Bounded SiLU-and-multiply over the live rows of a capture-sized buffer.
 *   in        [M, 2d] device array; gate = cols [0,d), up = cols [d,2d).
 *   out       [M, d] device array; must not overlap `in`.
 *   M         buffer capacity in rows, 0 <= M <= INT32_MAX.
 *   d         1 <= d <= GA_MAX_D.
 *   live_rows required device int32; rows [0, clamp(*live_rows, 0, M)) are
 *             computed, every other row of `out` is left untouched.
 * The grid depends on (M, d, dtype, alignment, device) only, never on the
 * live count, so a captured launch stays valid when the count changes.
 */
ga_status ga_silu_and_mul_bounded(const void *in, void *out, int64_t M, int64_t d,
                                  int32_t dtype, const int32_t *live_rows,
                                  ga_stream stream);

/*
 * Sparse GELU-and-multiply with a workspace, for few rows: when the planner
 * splits each row over several workgroups (T small against the compute-unit
 * count), they exchange per-chunk (mean, M2) partials through `workspace`
 * and combine them (Chan's parallel-variance formula, in a fixed order) so
 * every workgroup of a row uses the same cutoff.  Otherwise this is
 * ga_gelu_and_mul_sparse and the workspace is not touched.
 *   workspace        device memory of at least
 *                    ga_gelu_and_mul_sparse_workspace_bytes(T) bytes, 256-byte
 *                    aligned, zero-filled before its first use; the kernels keep
 *                    it valid for every later call (each call tags its partials
 *                    with the previous call's tag plus 16), so it is zeroed
 *                    once, not per call, and survives graph replay.
 *   Calls that share a workspace must not run concurrently (the same stream
 *   serialises them).  A row's workgroups wait for each other for a bounded
 *   number of polls; past it a workgroup computes the row's statistics on
 *   its own, so a launch always completes with a correct result.
 */
size_t ga_gelu_and_mul_sparse_workspace_bytes(int64_t T);
/* The planner splits rows only in calls of at most this many rows, so a
 * workspace of ga_gelu_and_mul_sparse_workspace_bytes(GA_SPLIT_PLAN_ROWS)
 * bytes (64 KiB) lets every call that the planner would split do so. */
#define GA_SPLIT_PLAN_ROWS 256
ga_status ga_gelu_and_mul_sparse_ws(const void *in, void *out, int64_t T, int64_t d,
                                    int32_t dtype, float z, const int32_t *live_rows,
                                    void *workspace, size_t workspace_bytes, ga_stream stream);

/*
 * ga_gelu_and_mul_sparse_ws without a caller workspace, for callers that
 * cannot allocate device memory (code under HIP graph capture, tight serving
 * loops, harnesses that forbid hipMalloc): the split records live in the
 * library's own static device array (64 KiB per device, held until the
 * process ends).  It allocates nothing and calls no allocating routine.
 *   Same arguments and checks as ga_gelu_and_mul_sparse, and
 *   T <= GA_SPLIT_PLAN_ROWS (larger T: GA_EUNSUPPORTED; such calls never
 *   split rows, and ga_gelu_and_mul_sparse serves them with no memory).
 * The first call on a device also enqueues a zero fill of that device's
 * array on `stream` (recorded into the graph when `stream` is capturing,
 * and then repeated by the next call).  Every call on one device shares its
 * array: calls that overlap in time on one device (other streams, other
 * threads, concurrent graph replays) race and may compute wrong cutoffs;
 * serialise them, e.g. on one stream.
 */
ga_status ga_gelu_and_mul_sparse_noalloc(const void *in, void *out, int64_t T, int64_t d,
                                         int32_t dtype, float z, const int32_t *live_rows,
                                         ga_stream stream);

/*
 * ga_gelu_and_mul_sparse_ws with flags: 0 (the same as _ws) or
 * GA_ROUND_INTERMEDIATES (the round-trip form above; it never splits rows,
 * so the workspace may then be NULL).  Unknown flag bits: GA_EINVAL.
 */
ga_status ga_gelu_and_mul_sparse_ex(const void *in, void *out, int64_t T, int64_t d,
                                    int32_t dtype, float z, const int32_t *live_rows,
                                    int32_t flags, void *workspace, size_t workspace_bytes,
                                    ga_stream stream);

/*
 * GELU-and-multiply without the sparsity step (vLLM PR 48498, section
 * Purpose: the provider is chosen per "approximation mode"):
 * out = gelu(gate) * up, gelu in the tanh form (GA_GELU_TANH, the same
 * constants as above) or the exact form x * Phi(x) (GA_GELU_ERF).
 *   in [T, 2d], out [T, d]; live_rows NULL for all rows, else a device int32
 *   bounding the rows written (as for ga_silu_and_mul_bounded).
 */
typedef enum { GA_GELU_ERF = 0, GA_GELU_TANH = 1 } ga_gelu_approx;
ga_status ga_gelu_and_mul(const void *in, void *out, int64_t T, int64_t d, int32_t dtype,
                          int32_t approximate, const int32_t *live_rows, ga_stream stream);

/*
 * Bounded squared ReLU, not gated (Megatron-LM PR 6328, section Scope and
 * risks, names the squared-ReLU activation kernel as sharing the bounded
 * row pattern): out[r, i] = max(in[r, i], 0)^2 for rows below
 * clamp(*live_rows, 0, M) of in[M, d]; other rows of out[M, d] untouched.
 * live_rows is required; the grid depends on M only.
 */
ga_status ga_squared_relu_bounded(const void *in, void *out, int64_t M, int64_t d, int32_t dtype,
                                  const int32_t *live_rows, ga_stream stream);

/*
 * Sparse GELU-and-multiply fused with the down projection that consumes it
 * (the vLLM page, Test Result, Correctness: the activation's write feeds the
 * layer's downstream projection, and a fused build must keep the two in that
 * order).  For live rows r and output features h:
 *     a[r, k] = gelu_and_mul_sparse(gu)[r, k], rounded once to `dtype`
 *               (the value ga_gelu_and_mul_sparse would store);
 *     y[r, h] = sum over k of a[r, k] * w[h, k], summed in fp32, rounded
 *               once to `dtype`.
 * The plan's form decides how (results within one rounding of the sum of
 * each other; every form is deterministic: fixed summation orders):
 *   GA_DOWN_DECODE  one or two tokens, d up to 16384 (32768 for one token):
 *                   one launch; each workgroup forms its tokens' statistics
 *                   and activation in registers; no workspace.
 *   GA_DOWN_STAGED  two to four tokens, d up to 16384: the activation is
 *                   stored once into the workspace by the library's own
 *                   activation kernel, then a second launch streams the
 *                   weights against it (fp32 dot products).
 *   GA_DOWN_TILED   any T: the activation stored once as in the staged form,
 *                   then a matrix-core product over it; the sum runs over d
 *                   in slices of k_chunk whose fp32 partials are added in
 *                   slice order.  The planner's choice from three tokens.
 *   gu        [T, 2d] device array (gate | up), 16-byte aligned.
 *   w         [H, d] device array, 16-byte aligned: one row of d weights per
 *             output feature (a linear layer's weight layout).
 *   y         [T, H] device array, 16-byte aligned; must not overlap gu or w.
 *   T         0 <= T <= GA_DOWN_MAX_ROWS tokens (more: GA_EUNSUPPORTED; use
 *             ga_gelu_and_mul_sparse and a matrix product).
 *   d         8 <= d <= GA_MAX_D, a multiple of 8 (16-byte rows).
 *   H         16 <= H <= GA_DOWN_MAX_H, a multiple of 16.
 *   dtype     GA_BF16 or GA_F16 (GA_F32: GA_EUNSUPPORTED).
 *   z, live_rows  as for ga_gelu_and_mul_sparse; rows of y at or past the
 *             live count are left untouched.
 *   workspace device memory of ga_gelu_and_mul_sparse_down_workspace_bytes()
 *             bytes, 256-byte aligned, zero-filled before its first use (the
 *             decode form needs none: NULL is accepted).  Each call leaves it
 *             ready for the next (the tiled form's output-tile counters,
 *             kept in a region of their own, are back at zero), so it is
 *             zeroed once and then serves any later calls and shapes that
 *             fit it, and graph replays.  It must not overlap gu, w or y
 *             (GA_EINVAL).  Calls that share a workspace must not overlap in
 *             time (one stream serialises them).
 */
#define GA_DOWN_MAX_ROWS 256
#define GA_DOWN_MAX_H 65536
#define GA_DOWN_DECODE 1
#define GA_DOWN_STAGED 2
#define GA_DOWN_TILED 3
typedef struct {
    int32_t rows_per_block;     /* tokens per workgroup: 16, 32, 64 or 128 in the tiled form; decode
                                   form: 1 or 2; staged form: 2 or 4 (at least T) */
    int32_t features_per_block; /* output features per workgroup: 16 per wavefront feature group in
                                   the tiled form; decode and staged forms: 2, 4 or 8 */
    int32_t waves;              /* wavefronts per workgroup */
    int32_t k_step;             /* tiled form: elements of d per iteration of a workgroup's loop (64,
                                   128 or 256); 0 in the decode and staged forms (each workgroup
                                   covers all of d) */
    int32_t k_chunk;            /* elements of d per workgroup, a multiple of k_step; d in the decode
                                   and staged forms */
    int32_t splits;             /* ceil(d / k_chunk), at most 64: workgroups that share an output tile */
    int32_t form;               /* GA_DOWN_DECODE, GA_DOWN_STAGED or GA_DOWN_TILED */
    int32_t depth;              /* tiled form: steps of loads each wavefront keeps in flight (1-3);
                                   0 in the other forms */
    int64_t grid;               /* workgroups of the product launch */
} ga_down_plan;
ga_status ga_plan_gelu_and_mul_sparse_down(int64_t T, int64_t d, int64_t H, int32_t dtype, ga_down_plan *plan);
/* Workspace for this plan (NULL: the planner's plan for T, d, H). */
size_t ga_gelu_and_mul_sparse_down_workspace_bytes(int64_t T, int64_t d, int64_t H, const ga_down_plan *plan);
ga_status ga_gelu_and_mul_sparse_down(const void *gu, const void *w, void *y, int64_t T, int64_t d, int64_t H,
                                      int32_t dtype, float z, const int32_t *live_rows, void *workspace,
                                      size_t workspace_bytes, ga_stream stream);
ga_status ga_gelu_and_mul_sparse_down_with_plan(const void *gu, const void *w, void *y, int64_t T, int64_t d,
                                                int64_t H, int32_t dtype, float z, const int32_t *live_rows,
                                                const ga_down_plan *plan, void *workspace,
                                                size_t workspace_bytes, ga_stream stream);

/*
 * ---- Training ----
 *
 * The operators below are the training step around the gated activations.
 * They follow the conventions above; any alignment natural to the element
 * type is accepted, with the same kernels for all.  A written array overlaps
 * no other array of the call (GA_EINVAL); an array without an element may be
 * NULL.  live_rows bounds the rows as above (NULL: all); rows at or past it
 * are neither read nor written.  Results do not depend on scheduling: every
 * sum has a fixed order.
 *
 * Activation checkpoint: an array [rows, halves * d] kept in 8 bits for the
 * backward pass.  Each row's halves (gate and up; one half for an ungated
 * array) are cut into blocks of GA_CHECKPOINT_BLOCK = 128 values, the last one
 * shorter.  With m the block's largest magnitude, counted as at least 2^-100:
 *     code  = 127 x / m, the exact quotient rounded to the nearest integer
 *             (ties to even), an int8 in [-127, 127]
 *     scale = m / 127 in fp32
 *     value = code * scale, within m / 254 of x (up to fp32 rounding; a positive
 *             gate - cutoff below m / 254 has code 1: within m / 127)
 * (A 16-bit row's differences from its own mean or cutoff are coded from the
 * fp32 quotient: one within 127 * 2^-21 of a half-integer may go to either side.)
 * A block that holds a NaN, an infinity or a magnitude of 2^126 or more has
 * the scale NaN: all values restored from it are NaN.
 *   codes   int8 [rows, halves, d]
 *   scales  fp32 [rows, halves, ceil(d / 128)]
 *   stats   fp32 [rows, 2], where the codes are relative to their row:
 *           (cutoff, std) for the sparse GELU, whose first half holds
 *           fp32(gate - cutoff); (mean, 1 / std) for layer norm, which holds
 *           fp32(x - mean).
 */
#define GA_CHECKPOINT_BLOCK 128

/* x [rows, d] -> codes, scales (one half).  1 <= d <= GA_MAX_D; rows *
 * ceil(d / 128) < 2^31 (else GA_EUNSUPPORTED). */
ga_status ga_checkpoint_store(const void *in, void *codes, float *scales, int64_t rows, int64_t d, int32_t dtype,
                              const int32_t *live_rows, ga_stream stream);

/* codes, scales -> out [rows, halves * d] of `dtype`: code * scale, plus
 * stats[row][0] in the first half where stats is given, in fp32, rounded once
 * to the type. */
ga_status ga_checkpoint_restore(const void *codes, const float *scales, const float *stats, void *out, int64_t rows,
                                int64_t d, int32_t halves, int32_t dtype, const int32_t *live_rows, ga_stream stream);

/*
 * The activations of the training pair.  f(gate) * up of in [rows, 2d] for
 * SILU, GELU_TANH, GELU_ERF; max(in, 0)^2 of in [rows, d] for SQUARED_RELU;
 * GELU_SPARSE as ga_gelu_and_mul_sparse with cutoff multiplier z (z is not
 * looked at otherwise).
 */
typedef enum {
    GA_ACT_SILU = 0,
    GA_ACT_GELU_TANH = 1,
    GA_ACT_GELU_ERF = 2,
    GA_ACT_SQUARED_RELU = 3,
    GA_ACT_GELU_SPARSE = 4
} ga_activation;

/*
 * The activation's forward pass that keeps its input: one pass over in,
 * writing out [rows, d] (the value of the forward-only entry points, up to
 * fp32 rounding) and codes and scales of in (two halves; one for
 * SQUARED_RELU).  Limits as for ga_checkpoint_store; GELU_SPARSE as for
 * ga_gelu_and_mul_sparse (fewer than 2^32 work-items, 64 to 1024 a row).  GELU_SPARSE: t = fp32(gate - cutoff) is kept in place of the
 * gate, with codes of at least 1 where t > 0, so the backward pass masks
 * exactly the values that the forward pass did; cutoff and std go to stats, which the others do not use (NULL).
 */
ga_status ga_activation_checkpoint(const void *in, void *out, void *codes, float *scales, float *stats, int64_t rows,
                                   int64_t d, int32_t dtype, int32_t activation, float z, const int32_t *live_rows,
                                   ga_stream stream);

/*
 * The gradient dx (in's shape) from dout [rows, d], in fp32, rounded once:
 *     dgate = dout up f'(gate), dup = dout f(gate); squared ReLU 2 max(in, 0) dout
 * GELU_SPARSE, with mean m and std s of the row's gate, t = gate - m - z s,
 * q = dout up gelu'(t) where t > 0 and 0 elsewhere, G the row's sum of q:
 *     dgate = q - (G / d) (1 + z (gate - m) / s), dup = dout gelu(max(t, 0))
 * the gradient through the row's mean and std too; the term with s is 0 where
 * s is 0, as the derivative of a std that is 0 is taken to be.  The row's
 * statistics are summed in fp64 from fp64 differences to one of its values, and
 * gate - cutoff is formed in fp32 from the cutoff as two fp32 numbers (16-bit
 * rows; in fp64 else), which keeps its sign: the side of the cutoff that a value
 * is on does not hang on an fp32 sum.
 * _checkpoint: the same formulas at the values that codes, scales (and stats)
 * stand for; activation and z are those of the forward pass.  What is formed from
 * a block whose scale is NaN is NaN (max(NaN, 0) of a NaN in `in` itself is 0).
 * GELU_SPARSE: a gate block's NaN scale makes the row's G NaN, and with it every
 * dgate of the row; an up block's does where one of its values has t > 0, and
 * nothing is formed from the others.
 */
ga_status ga_activation_backward(const void *dout, const void *in, void *dx, int64_t rows, int64_t d, int32_t dtype,
                                 int32_t activation, float z, const int32_t *live_rows, ga_stream stream);
ga_status ga_activation_backward_checkpoint(const void *dout, const void *codes, const float *scales,
                                            const float *stats, void *dx, int64_t rows, int64_t d, int32_t dtype,
                                            int32_t activation, float z, const int32_t *live_rows, ga_stream stream);

/*
 * Layer norm of in [rows, d]: with the row's mean m and population variance v,
 *     r = 1 / sqrt(v + eps), out = (in - m) r weight + bias
 * stats [rows, 2] = (m, r).  weight and bias (NULL: none) [d] are of
 * weight_dtype, which is dtype or GA_F32.  d <= GA_LAYER_NORM_MAX_D; eps >= 0.
 * A launch has 16 to 1024 work-items a row (16 up to d = 128, 64 up to 1024);
 * where they would reach 2^32 the call returns GA_EUNSUPPORTED.
 * _checkpoint also keeps fp32(in - m) in codes and scales (one half).
 */
#define GA_LAYER_NORM_MAX_D 32768
ga_status ga_layer_norm(const void *in, const void *weight, const void *bias, void *out, float *stats, int64_t rows,
                        int64_t d, int32_t dtype, int32_t weight_dtype, float eps, const int32_t *live_rows,
                        ga_stream stream);
ga_status ga_layer_norm_checkpoint(const void *in, const void *weight, const void *bias, void *out, void *codes,
                                   float *scales, float *stats, int64_t rows, int64_t d, int32_t dtype,
                                   int32_t weight_dtype, float eps, const int32_t *live_rows, ga_stream stream);

/*
 * Layer norm's backward pass from dout [rows, d]: with n = (in - m) r (or r
 * times the value a code stands for) and v = dout weight,
 *     dx = r (v - mean(v) - n mean(v n)) per row
 *     dweight = sum over live rows of dout n, dbias = sum of dout (NULL: not wanted)
 * dx of dtype, dweight and dbias of weight_dtype, sums in fp32.  No live rows:
 * dweight and dbias are zero.  m is the mean that stats hold in fp32; where
 * |m| r > 4, so that its rounding would show, the mean of in - m is taken off n
 * again if it is no more than that rounding (2^-22 |m|).
 *   workspace  ga_layer_norm_backward_workspace_bytes(rows, d) bytes, 16-byte
 *              aligned, any content; calls that share one must not overlap in
 *              time.
 */
size_t ga_layer_norm_backward_workspace_bytes(int64_t rows, int64_t d);
ga_status ga_layer_norm_backward(const void *dout, const void *in, const float *stats, const void *weight, void *dx,
                                 void *dweight, void *dbias, int64_t rows, int64_t d, int32_t dtype,
                                 int32_t weight_dtype, const int32_t *live_rows, void *workspace,
                                 size_t workspace_bytes, ga_stream stream);
ga_status ga_layer_norm_backward_checkpoint(const void *dout, const void *codes, const float *scales,
                                            const float *stats, const void *weight, void *dx, void *dweight,
                                            void *dbias, int64_t rows, int64_t d, int32_t dtype, int32_t weight_dtype,
                                            const int32_t *live_rows, void *workspace, size_t workspace_bytes,
                                            ga_stream stream);

/*
 * The router's balance loss over the n tokens (rows) that count: below the
 * live count and, where mask is given, with a mask byte other than 0.
 *     p = softmax(logits) over the experts, in fp32
 *     counts[e] = number of chosen indices equal to e (int32 [experts])
 *     loss = coefficient * experts / (k n) * sum over e of counts[e] P[e],
 *            P[e] = (sum over tokens of p[t, e]) / n
 * (coefficient when tokens and probabilities are spread evenly; 0 for n = 0).
 *   logits   [rows, experts] of dtype, 1 <= experts <= GA_BALANCE_MAX_EXPERTS
 *   index    [rows, k] int32 or int64 (index_bytes 4 or 8): the experts of each
 *            token; values outside [0, experts) (a dropped choice) are not
 *            counted.  rows * k < 2^31.
 *   offsets  int32 [experts + 1], the running sum of counts: expert e's first
 *            row in a buffer sorted by expert, and in offsets[experts] the
 *            buffer's live rows, which the bounded activations read as
 *            live_rows.
 *   tokens   int32: n.
 * A token whose logits are all -infinity has p = 0.
 * Backward, with counts as constants and dloss a device fp32:
 *     dlogits = dloss coefficient experts / (k n^2) p (counts - sum_j counts[j] p[j])
 * rows of tokens that do not count get 0 (past the live count: untouched).
 * (counts less their mean under p, formed again from the distances to it: a token
 * with a probability next to 1 has small gradients, right to their own roundings)
 *   workspace  as for layer norm, ga_balance_loss_workspace_bytes() bytes.
 */
#define GA_BALANCE_MAX_EXPERTS 1024
size_t ga_balance_loss_workspace_bytes(int64_t rows, int64_t experts);
ga_status ga_balance_loss(const void *logits, const void *index, int32_t index_bytes, const uint8_t *mask, float *loss,
                          int32_t *counts, int32_t *offsets, int32_t *tokens, int64_t rows, int64_t experts, int64_t k,
                          int32_t dtype, float coefficient, const int32_t *live_rows, void *workspace,
                          size_t workspace_bytes, ga_stream stream);
ga_status ga_balance_loss_backward(const void *logits, const uint8_t *mask, const int32_t *counts,
                                   const int32_t *offsets, const int32_t *tokens, const float *dloss, void *dlogits,
                                   int64_t rows, int64_t experts, int64_t k, int32_t dtype, float coefficient,
                                   const int32_t *live_rows, ga_stream stream);

/*
 * ---- The feed-forward layer ----
 *
 * The products around the gated activations, in 16 bits and in microscaled 4
 * bits.  They follow the conventions above.  A written array overlaps no other
 * array of the call (GA_EINVAL).  live_rows bounds the rows (tokens; NULL: all);
 * rows at or past it are neither read nor written.  Every sum has a fixed order.
 * The host knows the capacity `rows` alone and chooses by it: a few live rows of a
 * large buffer take several times as long as a call of as many rows.
 *
 * With the activation's GATED form (SILU, GELU_TANH, GELU_ERF; gate rows of w_in
 * first, then up rows, zd = 2 d) or SQUARED_RELU (not gated, zd = d):
 *     z = x w_in^T                  gate | up
 *     h = act(gate) * up            (SQUARED_RELU: max(z, 0)^2)
 *     y = h w_down^T
 * GELU_SPARSE is refused (GA_EUNSUPPORTED): its cutoff is a statistic of the whole
 * row of z (ga_gelu_and_mul_sparse and ga_gelu_and_mul_sparse_down serve it).
 * Sums are fp32 on the matrix cores.  z is rounded only where it is kept, h once,
 * y once; in fp16 an |h| (a kept |z|) of 65520 or more is an infinity, for
 * SQUARED_RELU from |z| = 256 on.  A NaN in x, a weight or the kept z reaches
 * every output formed from it: max(NaN, 0) is NaN here, in the 4-bit layer and in
 * the backward pass (the activation's own entry points take it as 0).
 *   x       [rows, H], y [rows, H], w_in [zd, H], w_down [H, d] of dtype GA_BF16 or
 *           GA_F16 (GA_F32: GA_EUNSUPPORTED), 16-byte aligned
 *   kept    z in dtype [rows, zd], for the backward pass; NULL: not kept
 *   H, d    8 .. GA_MAX_D, multiples of 8
 *   rows    0 .. 2^31 - 1025; where a launch would have 2^32 work-items or more:
 *           GA_EUNSUPPORTED (rows * max(H, d) of 2^36 or less has fewer)
 *   workspace  ga_feed_forward_workspace_bytes() bytes, 256-byte aligned, any
 *           content; calls that share one must not overlap in time.
 */
size_t ga_feed_forward_workspace_bytes(int64_t rows, int64_t H, int64_t d, int32_t activation);
ga_status ga_feed_forward(const void *x, const void *w_in, const void *w_down, void *y, void *kept, int64_t rows,
                          int64_t H, int64_t d, int32_t dtype, int32_t activation, const int32_t *live_rows,
                          void *workspace, size_t workspace_bytes, ga_stream stream);

/*
 * Its backward pass, from dy [rows, H], x and the kept z:
 *     dh = dy w_down
 *     dz = dh up act'(gate) | dh act(gate)      (SQUARED_RELU: 2 max(z, 0) dh)
 *     dx = dz w_in,  dw_in = dz^T x,  dw_down = dy^T h,  h formed again from z
 * dh stays in fp32; dz and h are rounded to the type once (in fp16 with the same
 * bound), dx, dw_in and dw_down once.  The weights' gradients sum over the live
 * rows (none: zero).
 */
size_t ga_feed_forward_backward_workspace_bytes(int64_t rows, int64_t H, int64_t d, int32_t activation);
ga_status ga_feed_forward_backward(const void *dy, const void *x, const void *kept, const void *w_in, const void *w_down,
                                   void *dx, void *dw_in, void *dw_down, int64_t rows, int64_t H, int64_t d,
                                   int32_t dtype, int32_t activation, const int32_t *live_rows, void *workspace,
                                   size_t workspace_bytes, ga_stream stream);

/*
 * Microscaled 4-bit arrays (OCP MX, MXFP4): a row in blocks of GA_MXFP4_BLOCK = 32
 * values, the last one shorter, each with one power of two.  With m the block's
 * largest magnitude:
 *     scale   byte s, standing for 2^(s - 127): s = max(127 + floor(log2 m) - 2, 0),
 *             0 for m = 0
 *     code    x / 2^(s - 127), exactly, rounded to the nearest of 0, 0.5, 1, 1.5, 2,
 *             3, 4, 6 (ties to the even code), 6 above 6; bit 3 is x's sign
 * A block that holds a NaN or an infinity has s = 255: it stands for NaNs.
 *   codes   uint8 [rows, 16 ceil(d / 32)]: value 2 i of a row in the low and 2 i + 1
 *           in the high half of byte i, past the row's end 0; 16-byte aligned
 *   scales  uint8 [rows, ceil(d / 32)]
 * 1 <= d <= GA_MAX_D; rows * ceil(d / 128) < 2^31 (else GA_EUNSUPPORTED).  The
 * other arrays have any alignment natural to their type.
 */
#define GA_MXFP4_BLOCK 32
ga_status ga_mxfp4_quantize(const void *in, void *codes, uint8_t *scales, int64_t rows, int64_t d, int32_t dtype,
                            const int32_t *live_rows, ga_stream stream);
/* out [rows, d] of `dtype`: the values, rounded once. */
ga_status ga_mxfp4_dequantize(const void *codes, const uint8_t *scales, void *out, int64_t rows, int64_t d,
                              int32_t dtype, const int32_t *live_rows, ga_stream stream);
/* A gated activation (GELU_SPARSE: GA_EUNSUPPORTED) of in [rows, 2d] (SQUARED_RELU
 * [rows, d]), the value that the forward-only entry points store (for SQUARED_RELU
 * max(NaN, 0) = 0 among them), quantised. */
ga_status ga_activation_mxfp4(const void *in, void *codes, uint8_t *scales, int64_t rows, int64_t d, int32_t dtype,
                              int32_t activation, const int32_t *live_rows, ga_stream stream);

/*
 * The product of two such arrays, out[r, i] = sum over k of a[r, k] w[i, k] in fp32,
 * rounded once to dtype (any of the three).  A NaN block makes the outputs of its
 * row NaN.
 *   a codes, scales of [rows, k]; w of [n, k]; out [rows, n], any alignment natural
 *   to its type.  1 <= n < 2^31 - 1024, 1 <= k <= GA_MAX_D.  Where a launch would
 *   have 2^32 work-items or more: GA_EUNSUPPORTED (up to 16 rows: n above 2^27 - 16;
 *   more: not where rows * n is 2^37 or less).
 *   workspace  ga_mxfp4_product_workspace_bytes() bytes (may be 0), as above.
 */
size_t ga_mxfp4_product_workspace_bytes(int64_t rows, int64_t n, int64_t k);
ga_status ga_mxfp4_product(const void *a_codes, const uint8_t *a_scales, const void *w_codes, const uint8_t *w_scales,
                           void *out, int64_t rows, int64_t n, int64_t k, int32_t dtype, const int32_t *live_rows,
                           void *workspace, size_t workspace_bytes, ga_stream stream);

/*
 * The feed-forward layer on 4-bit operands: x is quantised, z = q(x) w_in^T stays
 * in fp32, h = act(gate) up is quantised from fp32, y = q(h) w_down^T.  x and y
 * [rows, H] of dtype GA_BF16 or GA_F16, any alignment natural to the type; w_in
 * [zd, H] and w_down [H, d] as codes and scales.  8 <= H <= GA_MAX_D, a multiple of
 * 8; 32 <= d <= GA_MAX_D, a multiple of 32 (gate and up rows keep blocks of h whole).
 */
size_t ga_feed_forward_mxfp4_workspace_bytes(int64_t rows, int64_t H, int64_t d, int32_t activation);
ga_status ga_feed_forward_mxfp4(const void *x, const void *w_in_codes, const uint8_t *w_in_scales,
                                const void *w_down_codes, const uint8_t *w_down_scales, void *y, int64_t rows, int64_t H,
                                int64_t d, int32_t dtype, int32_t activation, const int32_t *live_rows, void *workspace,
                                size_t workspace_bytes, ga_stream stream);

/*
 * Host-only planners of these products (no HIP call, usable without a GPU): how
 * each would run for these sizes, all rows live.  `product` names one of the
 * layer's; `bits` is 16, or 4 for ga_feed_forward_mxfp4 (the first two).
 */
#define GA_PRODUCT_HIDDEN 0   /* z = x w_in^T, h */
#define GA_PRODUCT_OUT 1      /* y = h w_down^T */
#define GA_PRODUCT_DHIDDEN 2  /* dh = dy w_down, dz, h */
#define GA_PRODUCT_DX 3       /* dx = dz w_in */
#define GA_PRODUCT_DW_IN 4    /* dw_in = dz^T x */
#define GA_PRODUCT_DW_DOWN 5  /* dw_down = dy^T h */
typedef struct {
    int32_t features; /* rows of A of a workgroup's tile (with a gate and an up half: of both); 0: a
                         stream of the weights (up to 16 rows, not in the backward pass) */
    int32_t tokens;   /* rows of B of a tile; 0: a stream */
    int32_t stages;   /* steps of a tile in LDS; 0: a stream */
    int32_t k_step;   /* values of k a step; 0: a stream */
    int32_t splits;   /* slices of k, whose sums a second launch adds; 1: none */
    int32_t joint;    /* 1: the backward pass's last three products in one launch */
    int64_t k_slice;  /* values of k a slice, a multiple of k_step; k where there is one */
    int64_t grid;     /* workgroups of this product (a stream: at most) */
} ga_product_plan;
ga_status ga_plan_feed_forward(int64_t rows, int64_t H, int64_t d, int32_t activation, int32_t bits, int32_t product,
                               ga_product_plan *plan);
ga_status ga_plan_mxfp4_product(int64_t rows, int64_t n, int64_t k, ga_product_plan *plan);

/*
 * Host-only helper: z = Phi^-1(target_sparsity), the cutoff multiplier for
 * a target fraction of zeros (0.95 -> 1.6448536...).  NaN outside (0, 1).
 * Newton's method on the normal CDF, to full double precision.
 */
double ga_z_from_sparsity(double target_sparsity);

/*
 * Host-only planners (no HIP call, usable without a GPU): the geometry the
 * entry points above would launch for these sizes.  `aligned` says whether
 * the 16-byte vector path applies (both base pointers 16-byte aligned and
 * d * element size a multiple of 16); `num_cus` is the device's compute-unit
 * count (256 on MI355X); `with_workspace` allows split rows.
 */
ga_status ga_plan_gelu_and_mul_sparse(int64_t T, int64_t d, int32_t dtype, int32_t aligned,
                                      int32_t num_cus, int32_t with_workspace, ga_plan *plan);
/* The elementwise ops (silu_and_mul_bounded, gelu_and_mul, squared ReLU)
 * share one kernel family and this planner; M is the row capacity. */
ga_status ga_plan_silu_and_mul_bounded(int64_t M, int64_t d, int32_t dtype, int32_t aligned,
                                       int32_t num_cus, ga_plan *plan);

/*
 * The same operations with an explicit geometry (for tuning sweeps and the
 * geometry-independence tests).  The plan must name an instantiated kernel
 * (the values listed in ga_plan) and cover the row: vector path
 * splits * waves_per_row * 64 * per_lane * (16 / element size) >= d, with
 * every split owning at least one vector; element path
 * waves_per_row * 64 * per_lane >= d; unaligned path (any alignment)
 * waves_per_row * 64 * per_lane * e >= d with e = 16 / element size;
 * packed rows (any alignment) lanes_per_row * per_lane * e >= d;
 * else GA_EUNSUPPORTED.
 * `block` and
 * `grid` are derived for gelu; silu takes its grid from the plan.  A split
 * plan needs the workspace described above (else GA_EINVAL) and T <= 65535.
 * `flags` selects the round-trip form for gelu (no split rows with it) and
 * must be zero for silu.  The planners leave it zero.
 */
ga_status ga_gelu_and_mul_sparse_with_plan(const void *in, void *out, int64_t T, int64_t d,
                                           int32_t dtype, float z, const int32_t *live_rows,
                                           const ga_plan *plan, void *workspace,
                                           size_t workspace_bytes, ga_stream stream);
ga_status ga_silu_and_mul_bounded_with_plan(const void *in, void *out, int64_t M, int64_t d,
                                            int32_t dtype, const int32_t *live_rows,
                                            const ga_plan *plan, ga_stream stream);

/*
 * Measurement aid, not part of the activations: a streaming kernel with the
 * same access pattern (read the two halves of rows [0, rows) of in[rows, 2w]
 * 16 bytes at a time, write out[rows, w] = first half XOR second half).  Its
 * bandwidth is the ceiling a row-wise gated activation can reach on the
 * device.  `w_bytes` (bytes per half row) must be a positive multiple of 16
 * and both pointers 16-byte aligned.
 */
ga_status ga_stream_xor_rows(const void *in, void *out, int64_t rows, int64_t w_bytes,
                             ga_stream stream);

/* Static name of a status code. */
const char *ga_status_str(int32_t status);

/* Message describing the last non-OK status returned on this thread. */
const char *ga_last_error(void);

/* Library version: major * 10000 + minor * 100 + patch. */
int32_t ga_version(void);

#ifdef __cplusplus
}
#endif

#endif /* GA_H */
