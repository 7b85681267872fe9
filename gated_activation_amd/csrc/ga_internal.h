// Host-side interface between the C-ABI (api.hip) and the kernel translation
// units.  Each launcher enqueues one kernel on `stream` and returns the HIP
// status of the launch, or hipErrorInvalidValue when no kernel is
// instantiated for the requested geometry.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

namespace ga {

// Enqueues kernel(args...), each argument converted to the kernel's own
// parameter type, and returns this launch's status.
template <typename... P>
hipError_t launch_kernel(void (*kernel)(P...), dim3 grid, dim3 block, hipStream_t stream,
                         typename std::common_type<P>::type... args) {
    void *pointers[] = {(void *)&args...};
    return hipLaunchKernel((const void *)kernel, grid, block, pointers, 0, stream);
}

// Geometries with a compiled kernel.
bool gelu_vec_available(int dtype, int waves, int vec_per_lane, int up_late);
bool gelu_elem_available(int dtype, int waves, int elem_per_lane);
// Elementwise activation ops sharing one kernel family.
enum : int { OP_SILU_MUL = 0, OP_GELU_TANH_MUL = 1, OP_GELU_ERF_MUL = 2, OP_SQUARED_RELU = 3, OP_COUNT = 4 };
bool act_available(int op, int path, int dtype, int per_lane);

constexpr int SILU_BLOCK = 256;

// Split-row gelu workspace: one record per row, the same layout for every T
// and split count: SPLIT_MAX 16-byte slots of two 64-bit words,
// {uint32 tag, fp32 mean} and {uint32 tag, fp32 M2}.
constexpr int SPLIT_MAX = 16;
constexpr int SPLIT_SLOT_BYTES = 16;  // slot stride: the two words, packed (one slot per cache line measured slower)
constexpr size_t SPLIT_RECORD_BYTES = (size_t)SPLIT_MAX * SPLIT_SLOT_BYTES;
inline size_t split_workspace_bytes(int64_t T) { return (size_t)T * SPLIT_RECORD_BYTES; }
bool gelu_split_available(int dtype, int waves, int vec_per_lane, int splits);
hipError_t launch_gelu_split(int dtype, int waves, int vec_per_lane, int splits, const void *in, void *out,
                             int32_t T, int32_t d, int32_t nvec, float z, const int32_t *live, void *workspace,
                             uint32_t spin_limit, hipStream_t stream);

// Replicated-statistics path for few rows: REP (2, 4, 8) workgroups per row,
// each reducing the whole gate row itself and applying its REP-th share;
// grid = gelu_rep_grid(T, REP) (rows rounded up to groups of 8).
bool gelu_rep_available(int dtype, int waves, int vec_per_lane, int rep);
int64_t gelu_rep_grid(int64_t T, int rep);
hipError_t launch_gelu_rep(int dtype, int waves, int vec_per_lane, int rep, const void *in, void *out, int32_t T,
                           int32_t d, int32_t nvec, float z, const int32_t *live, hipStream_t stream);

// The activation fused with the down projection y = a . w^T (w: [H, d]).
// At most DOWN_MAX_SPLITS slices of d per row in the tiled form.
constexpr int DOWN_MAX_SPLITS = 64;

// Decode form of the fused op, for T <= tmax tokens (1 or 2): one launch, no
// workspace; workgroups of f output features (2, 4 or 8) over all of d,
// grid ceil(H / f).  Available where a kernel of that geometry reaches d.
bool gelu_down_decode_available(int dtype, int tmax, int f, int waves, int64_t d);
hipError_t launch_gelu_down_decode(int dtype, int tmax, int f, int waves, const void *gu, const void *w, void *y,
                                   int32_t T, int32_t d, int32_t H, float z, const int32_t *live,
                                   hipStream_t stream);

// Workspace of the staged and tiled forms: [0, 256) unused, the tiled
// product's output-tile counters at a fixed place (DOWN_MAX_TILES words,
// zero between calls: each tile's last workgroup resets its own), the stored
// activation ([T, d]) from DOWN_ACT_OFFSET, then the tiled product's fp32
// partial tiles.
constexpr int64_t DOWN_TILE_CNT_OFFSET = 256;
constexpr int64_t DOWN_MAX_TILES = 16384;
constexpr int64_t DOWN_ACT_OFFSET = DOWN_TILE_CNT_OFFSET + DOWN_MAX_TILES * 4;
__host__ __device__ inline int64_t down_tiled_part_offset(int64_t T, int64_t d) {
    return DOWN_ACT_OFFSET + (T * d * 2 + 255) / 256 * 256;
}

// Tiled form's product launch, for any T: y = a . w^T with a the stored
// activation at workspace + DOWN_ACT_OFFSET; workgroups of tm tokens x bh
// features x kc elements of d (grid ceil(T / tm) * ceil(H / bh) * ceil(d / kc));
// several slices of d add their partials through the workspace
// (gelu_down_tiled_workspace_bytes), at most DOWN_MAX_TILES output tiles.
bool gelu_down_tiled_available(int dtype, int tm, int bh, int waves, int kstep, int depth);
size_t gelu_down_tiled_workspace_bytes(int64_t T, int64_t d, int64_t H, int tm, int bh, int64_t kc);
hipError_t launch_gelu_down_tiled(int dtype, int tm, int bh, int waves, int kstep, int depth, int32_t kc, const void *a,
                                  const void *w, void *y, int32_t T, int32_t d, int32_t H, const int32_t *live,
                                  void *workspace, hipStream_t stream);

// Staged form's product launch, for T <= tmax tokens (2 or 4): y = a . w^T
// with a the stored activation ([T, d], rows past the live count not read);
// workgroups of f output features over all of d, grid ceil(H / f).
bool gelu_down_staged_available(int dtype, int tmax, int f, int waves, int64_t d);
hipError_t launch_gelu_down_staged(int dtype, int tmax, int f, int waves, const void *a, const void *w, void *y,
                                   int32_t T, int32_t d, int32_t H, const int32_t *live, hipStream_t stream);

// Packed-rows path for short rows: ROWS_BLOCK threads per workgroup,
// lanes_per_row in {4, 8, 16, 32} lanes per row, vec_per_lane in {1, 2, 4};
// grid = ceil(T / (ROWS_BLOCK / lanes_per_row)).  nvec: the row's 16-byte
// vectors (a partial last one included); unaligned: rows or bases off 16-byte
// alignment (unaligned 16-byte vectors).
constexpr int ROWS_BLOCK = 256;
bool gelu_rows_available(int dtype, int lanes_per_row, int vec_per_lane);
hipError_t launch_gelu_rows(int dtype, int lanes_per_row, int vec_per_lane, bool round_trip, bool unaligned,
                            int64_t grid, const void *in, void *out, int32_t T, int32_t d, int32_t nvec, float z,
                            const int32_t *live, hipStream_t stream);

// Unaligned path for rows that are not 16-byte aligned: waves 1, 2, 4, 8, 16;
// vectors per lane 1 .. 8 (vector j = elements [j * 16 / es, (j + 1) * 16 / es),
// one unaligned 16-byte access); up_late 0 (up loaded with the gate) or 1
// (one vector at a time after the statistics).
bool gelu_unaligned_available(int dtype, int waves, int vec_per_lane, int up_late);
hipError_t launch_gelu_unaligned(int dtype, int waves, int vec_per_lane, int up_late, bool round_trip,
                                 int64_t grid, const void *in, void *out, int32_t T, int32_t d, float z,
                                 const int32_t *live, hipStream_t stream);

// round_trip selects the form that rounds each intermediate (mean, std, z,
// z * std, cutoff, gate - cutoff, GELU output) to the element type.
hipError_t launch_gelu_vec(int dtype, int waves, int vec_per_lane, int up_late, bool round_trip, int64_t grid,
                           const void *in, void *out, int32_t T, int32_t d, int32_t nvec,
                           float z, const int32_t *live, hipStream_t stream);

hipError_t launch_gelu_elem(int dtype, int waves, int elem_per_lane, bool round_trip, int64_t grid,
                            const void *in, void *out, int32_t T, int32_t d,
                            float z, const int32_t *live, hipStream_t stream);

// path 0: 16-byte items (nitems_row = d / elements per 16 bytes),
// path 1: single elements (nitems_row = d), path 2: unaligned 16-byte vectors
// numbered flat over the live output region (nitems_row = d).  live may be
// null (all M rows).
hipError_t launch_act(int op, int path, int dtype, int per_lane, int64_t grid, const void *in, void *out,
                      int32_t M, uint32_t nitems_row, const int32_t *live, hipStream_t stream);

hipError_t launch_xor_rows(int64_t grid, const void *in, void *out, int32_t rows,
                           uint32_t nvec_row, hipStream_t stream);

// ---------------------------------------------------------------------------
// Training kernels.  Codes are int8 [rows, halves * d], scales fp32
// [rows, halves * ceil(d / 128)], stats fp32 [rows, 2]; any alignment natural
// to the type.
// ---------------------------------------------------------------------------
// Elementwise: rows * halves * ceil(d / 128) < 2^31.  op: OP_* above, or -1 for
// the plain store of an [rows, d] array (out unused).
hipError_t launch_checkpoint_store(int dtype, int op, const void *in, void *out, void *codes, float *scales,
                                   int32_t rows, uint32_t d, const int32_t *live, hipStream_t stream);
hipError_t launch_checkpoint_restore(int dtype, const void *codes, const float *scales, const float *stats, void *out,
                                     int32_t rows, uint32_t d, int32_t halves, const int32_t *live,
                                     hipStream_t stream);
// From in (x) where it is not null, else from codes and scales.
hipError_t launch_act_backward(int dtype, int op, const void *dout, const void *in, const void *codes,
                               const float *scales, void *dx, int32_t rows, uint32_t d, const int32_t *live,
                               hipStream_t stream);

// Sparse GELU, d <= 65536: one team of sparse_train_waves(d) wavefronts a row.
int sparse_train_waves(int64_t d);
hipError_t launch_sparse_store(int dtype, const void *in, void *out, void *codes, float *scales, float *stats,
                               int32_t rows, int32_t d, float z, const int32_t *live, hipStream_t stream);
hipError_t launch_sparse_backward(int dtype, const void *dout, const void *in, const void *codes, const float *scales,
                                  const float *stats, void *dx, int32_t rows, int32_t d, float z, const int32_t *live,
                                  hipStream_t stream);

// Layer norm, d <= LN_MAX_D.  wide: weight, bias and their gradients are fp32,
// else of `dtype`.  With codes, the forward also keeps fp32(x - mean) there.
constexpr int64_t LN_MAX_D = 32768;
// The forward's launch has layer_norm_lanes(d) work-items a row.
int layer_norm_lanes(int64_t d);
hipError_t launch_layer_norm(int dtype, bool wide, const void *in, const void *weight, const void *bias, void *out,
                             void *codes, float *scales, float *stats, int32_t rows, int32_t d, float eps,
                             const int32_t *live, hipStream_t stream);
// Groups of rows in the backward's launch, each of which leaves one partial row
// of the weight's and the bias' gradient in the workspace ([groups, 2, d] fp32;
// none with one group), after three sums of each row for each 8192 columns where
// a row is wider.  kept: from codes and scales, else from in.
int layer_norm_groups(int64_t rows, int64_t d, bool f32, int cus);
size_t layer_norm_workspace_bytes(int64_t rows, int64_t d, int groups);
hipError_t launch_layer_norm_backward(int dtype, bool wide, const void *dout, const void *in, const void *codes,
                                      const float *scales, const float *stats, const void *weight, void *dx,
                                      void *dweight, void *dbias, bool kept, int32_t rows, int32_t d,
                                      const int32_t *live, int groups, int cus, float *workspace, hipStream_t stream);

// Balance loss, E <= BALANCE_MAX_E experts.  wide_index: int64 indices.
constexpr int64_t BALANCE_MAX_E = 1024;
int balance_groups(int64_t rows, int64_t experts, int cus);
inline size_t balance_workspace_bytes(int groups, int64_t experts) {
    return groups <= 1 ? 0 : (size_t)groups * (2 * (size_t)experts + 1) * 4;
}
hipError_t launch_balance(int dtype, const void *logits, const void *index, bool wide_index, const uint8_t *mask,
                          float *loss, int32_t *counts, int32_t *offsets, int32_t *tokens, int32_t rows, int32_t experts,
                          int32_t k, float coefficient, const int32_t *live, int groups, void *workspace,
                          hipStream_t stream);
hipError_t launch_balance_backward(int dtype, const void *logits, const uint8_t *mask, const int32_t *counts,
                                   const int32_t *offsets, const int32_t *tokens, const float *dloss, void *dlogits,
                                   int32_t rows, int32_t experts, int32_t k, float coefficient, const int32_t *live,
                                   int cus, hipStream_t stream);

// ---------------------------------------------------------------------------
// The feed-forward layer's products, 16-bit and microscaled 4-bit operands
// (ga_tile.h, ga_mx.h).
// ---------------------------------------------------------------------------
// How one product of F features, T tokens and K values runs: up to
// PRODUCT_FEW_TOKENS tokens, both operands with k contiguous, as a stream of the
// weights (ga_stream.h); else in tiles (ga_tile.h) of 256 features (half as many
// where a gate and an up half share a tile) x 256 tokens, 128 x 192, 128 x 128
// with two or four stages (DEEP), or 128 x 64 or 64 x 64, these with k in `splits` slices of
// k_split values whose partial sums a second launch adds (splits * T * F fp32, twice
// that with two halves).
enum : int { PRODUCT_BIG, PRODUCT_WIDE, PRODUCT_MID, PRODUCT_DEEP, PRODUCT_SLIM, PRODUCT_THIN, PRODUCT_FEW };
constexpr int64_t PRODUCT_FEW_TOKENS = 16, PRODUCT_FEW_WIDE = 4096;  // from so many features on 16 a workgroup
struct ProductPlan {
    int tile, threads, splits;  // threads: of a workgroup
    int32_t k_split;
    int64_t workgroups;
    size_t partial_bytes;
};
// strided: how many operands have k strided (one: A); step: values of k a step (64
// of 16 bits, 256 of 4)
ProductPlan plan_product(int64_t F, int64_t T, int64_t K, bool halves, int strided, int step);

// The backward pass's dx, dw_in and dw_down: in one launch where together, x in 64 x
// 64 tiles, in and down in 128 x 128; cut_w: these two with k in slices (with the
// partial sums of all three one after another).
struct ThreePlan {
    bool together, cut_w;
    ProductPlan x, in, down;
};
ThreePlan plan_three(int64_t rows, int64_t H, int64_t d, int64_t zd);

// Bytes of workspace, and where its parts begin.
struct FeedForwardSpace {
    size_t hidden, gradient, partial, total;
};
FeedForwardSpace feed_forward_space(int64_t rows, int64_t H, int64_t d, int halves);
FeedForwardSpace feed_forward_backward_space(int64_t rows, int64_t H, int64_t d, int halves);

// op: OP_* above; kept may be null.  _f16, _bf16: of one type.
hipError_t launch_feed_forward_f16(int op, const void *x, const void *w_in, const void *w_down, void *y, void *kept,
                                   int32_t rows, int32_t H, int32_t d, const int32_t *live, uint8_t *workspace,
                                   hipStream_t stream);
hipError_t launch_feed_forward_bf16(int op, const void *x, const void *w_in, const void *w_down, void *y, void *kept,
                                    int32_t rows, int32_t H, int32_t d, const int32_t *live, uint8_t *workspace,
                                    hipStream_t stream);
hipError_t launch_feed_forward_backward_f16(int op, const void *dy, const void *x, const void *kept, const void *w_in,
                                            const void *w_down, void *dx, void *dw_in, void *dw_down, int32_t rows,
                                            int32_t H, int32_t d, const int32_t *live, uint8_t *workspace,
                                            hipStream_t stream);
hipError_t launch_feed_forward_backward_bf16(int op, const void *dy, const void *x, const void *kept, const void *w_in,
                                             const void *w_down, void *dx, void *dw_in, void *dw_down, int32_t rows,
                                             int32_t H, int32_t d, const int32_t *live, uint8_t *workspace,
                                             hipStream_t stream);
hipError_t launch_feed_forward(int dtype, int op, const void *x, const void *w_in, const void *w_down, void *y, void *kept,
                               int32_t rows, int32_t H, int32_t d, const int32_t *live, uint8_t *workspace,
                               hipStream_t stream);
hipError_t launch_feed_forward_backward(int dtype, int op, const void *dy, const void *x, const void *kept,
                                        const void *w_in, const void *w_down, void *dx, void *dw_in, void *dw_down,
                                        int32_t rows, int32_t H, int32_t d, const int32_t *live, uint8_t *workspace,
                                        hipStream_t stream);

// op: OP_*, or -1 for x itself.
hipError_t launch_mxfp4_quantize(int dtype, int op, const void *in, void *codes, uint8_t *scales, int32_t rows,
                                 uint32_t d, const int32_t *live, hipStream_t stream);
hipError_t launch_mxfp4_dequantize(int dtype, const void *codes, const uint8_t *scales, void *out, int32_t rows,
                                   uint32_t d, const int32_t *live, hipStream_t stream);
// out [rows, n] of `dtype` from a [rows, k] and w [n, k].
size_t mxfp4_product_space(int64_t rows, int64_t n, int64_t k);
hipError_t launch_mxfp4_product(int dtype, const void *a, const uint8_t *a_scales, const void *w, const uint8_t *w_scales,
                                void *out, int32_t rows, int32_t n, int32_t k, const int32_t *live, uint8_t *workspace,
                                hipStream_t stream);
struct FeedForward4Space {
    size_t x_codes, x_scales, h_codes, h_scales, partial, total;
};
FeedForward4Space feed_forward_mxfp4_space(int64_t rows, int64_t H, int64_t d, int halves);
hipError_t launch_feed_forward_mxfp4(int dtype, int op, const void *x, const void *w_in, const uint8_t *w_in_scales,
                                     const void *w_down, const uint8_t *w_down_scales, void *y, int32_t rows, int32_t H,
                                     int32_t d, const int32_t *live, uint8_t *workspace, hipStream_t stream);

}  // namespace ga
