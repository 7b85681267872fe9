// The feed-forward layer's entry points of the C-ABI: argument checks and
// dispatch.  As in api.hip, every check runs on the host before any HIP call.
#include <stddef.h>

#include "../../include/ga.h"
#include "ga_host.h"
#include "ga_internal.h"

namespace {

using ga::check_regions;
using ga::check_sizes;
using ga::elem_size;
using ga::fail;
using ga::op_of;
using ga::Region;

int halves_of(int32_t activation) { return activation == GA_ACT_SQUARED_RELU ? 1 : 2; }

ga_status check_activation(const char *op, int32_t activation) {
    if (activation < GA_ACT_SILU || activation > GA_ACT_GELU_SPARSE)
        return fail(GA_EINVAL, "%s: unknown activation %d", op, (int)activation);
    if (activation == GA_ACT_GELU_SPARSE)
        return fail(GA_EUNSUPPORTED, "%s: the sparse GELU's cutoff is a statistic of the whole row", op);
    return GA_OK;
}

// rows, H and d of the layer.
ga_status check_layer(const char *op, int64_t rows, int64_t H, int64_t d, int64_t d_step, int32_t dtype,
                      int32_t activation) {
    ga_status st = check_sizes(op, rows, d, GA_MAX_D, dtype);
    if (st != GA_OK || (st = check_sizes(op, rows, H, GA_MAX_D, dtype)) != GA_OK ||
        (st = check_activation(op, activation)) != GA_OK)
        return st;
    if (dtype == GA_F32) return fail(GA_EUNSUPPORTED, "%s: bf16 or fp16 only", op);
    if (H % 8 != 0 || d % d_step != 0)
        return fail(GA_EUNSUPPORTED, "%s: H = %lld is not a multiple of 8 or d = %lld of %lld", op, (long long)H, (long long)d,
                    (long long)d_step);
    return GA_OK;
}

ga_status check_workspace(const char *op, const void *workspace, size_t bytes, size_t need) {
    if (bytes < need || (need > 0 && workspace == nullptr))
        return fail(GA_EINVAL, "%s: workspace of %zu bytes, %zu needed", op, workspace == nullptr ? 0 : bytes, need);
    return GA_OK;
}

// One product's launch has fewer than 2^32 work-items; rows and features are counted
// a few tiles past their end in 32 bits.
ga_status check_product(const char *op, int64_t F, int64_t T, int64_t K, bool halves, int strided, int step) {
    if (T > INT32_MAX - 1024) return fail(GA_EUNSUPPORTED, "%s: %lld rows (at most 2^31 - 1025)", op, (long long)T);
    const ga::ProductPlan p = ga::plan_product(F, T, K, halves, strided, step);
    if (p.workgroups * p.threads > (int64_t)UINT32_MAX)
        return fail(GA_EUNSUPPORTED, "%s: a product of %lld features and %lld rows needs %lld workgroups of %d work-items (2^32 or more)",
                    op, (long long)F, (long long)T, (long long)p.workgroups, p.threads);
    return GA_OK;
}

static_assert(sizeof(ga_product_plan) == 40 && offsetof(ga_product_plan, grid) == 32, "ga_product_plan layout");

void describe(const ga::ProductPlan &p, int64_t K, int step, bool joint, ga_product_plan *out) {
    static const int32_t shapes[][3] = {{256, 256, 2}, {128, 192, 2}, {128, 128, 2}, {128, 128, 4},
                                        {128, 64, 4},  {64, 64, 4},   {0, 0, 0}};
    static_assert(ga::PRODUCT_BIG == 0 && ga::PRODUCT_WIDE == 1 && ga::PRODUCT_MID == 2 && ga::PRODUCT_DEEP == 3 &&
                      ga::PRODUCT_SLIM == 4 && ga::PRODUCT_THIN == 5 && ga::PRODUCT_FEW == 6,
                  "shapes");
    const int32_t *s = shapes[p.tile];
    *out = ga_product_plan{s[0], s[1], s[2], s[0] == 0 ? 0 : step, p.splits, joint, p.splits == 1 ? K : p.k_split, p.workgroups};
}

bool layer_sizes(int64_t rows, int64_t H, int64_t d, int32_t activation) {
    return rows >= 1 && rows <= INT32_MAX && H >= 1 && H <= GA_MAX_D && d >= 1 && d <= GA_MAX_D && op_of(activation) >= 0;
}

size_t mx_codes(int64_t rows, int64_t d) { return (size_t)rows * (size_t)((d + GA_MXFP4_BLOCK - 1) / GA_MXFP4_BLOCK) * 16; }
size_t mx_scales(int64_t rows, int64_t d) { return mx_codes(rows, d) / 16; }

ga_status quantize(const char *op, const void *in, void *codes, uint8_t *scales, int64_t rows, int64_t d, int64_t halves,
                   int32_t dtype, int kernel_op, const int32_t *live_rows, ga_stream stream) {
    const size_t es = elem_size(dtype);
    const Region regions[] = {{"in", in, (size_t)rows * halves * d * es, es, false, false},
                              {"live_rows", live_rows, 4, 4, false, true},
                              {"codes", codes, mx_codes(rows, d), 16, true, false},
                              {"scales", scales, mx_scales(rows, d), 1, true, false}};
    ga_status st = check_regions(op, regions);
    if (st != GA_OK || (st = ga::check_blocks(op, rows * ga::blocks_of(d))) != GA_OK) return st;
    if (rows == 0) return GA_OK;
    return ga::launched(op, ga::launch_mxfp4_quantize(dtype, kernel_op, in, codes, scales, (int32_t)rows, (uint32_t)d,
                                                      live_rows, (hipStream_t)stream));
}

}  // namespace

extern "C" {

// ---------------------------------------------------------------------------
// 16 bits
// ---------------------------------------------------------------------------
size_t ga_feed_forward_workspace_bytes(int64_t rows, int64_t H, int64_t d, int32_t activation) {
    return layer_sizes(rows, H, d, activation) ? ga::feed_forward_space(rows, H, d, halves_of(activation)).total : 0;
}

ga_status ga_feed_forward(const void *x, const void *w_in, const void *w_down, void *y, void *kept, int64_t rows,
                          int64_t H, int64_t d, int32_t dtype, int32_t activation, const int32_t *live_rows,
                          void *workspace, size_t workspace_bytes, ga_stream stream) {
    const char *op = "ga_feed_forward";
    ga_status st = check_layer(op, rows, H, d, 8, dtype, activation);
    if (st != GA_OK) return st;
    const int64_t zd = halves_of(activation) * d;
    const Region regions[] = {{"x", x, (size_t)rows * H * 2, 16, false, false},
                              {"w_in", w_in, (size_t)zd * H * 2, 16, false, false},
                              {"w_down", w_down, (size_t)H * d * 2, 16, false, false},
                              {"live_rows", live_rows, 4, 4, false, true},
                              {"y", y, (size_t)rows * H * 2, 16, true, false},
                              {"kept", kept, kept == nullptr ? 0 : (size_t)rows * zd * 2, 16, true, true},
                              {"workspace", workspace, workspace_bytes, 256, true, true}};
    if ((st = check_regions(op, regions)) != GA_OK ||
        (st = check_workspace(op, workspace, workspace_bytes, ga_feed_forward_workspace_bytes(rows, H, d, activation))) != GA_OK ||
        (st = check_product(op, d, rows, H, zd != d, 0, 64)) != GA_OK || (st = check_product(op, H, rows, d, false, 0, 64)) != GA_OK)
        return st;
    if (rows == 0) return GA_OK;
    return ga::launched(op, ga::launch_feed_forward(dtype, op_of(activation), x, w_in, w_down, y, kept, (int32_t)rows,
                                                    (int32_t)H, (int32_t)d, live_rows, (uint8_t *)workspace,
                                                    (hipStream_t)stream));
}

size_t ga_feed_forward_backward_workspace_bytes(int64_t rows, int64_t H, int64_t d, int32_t activation) {
    return layer_sizes(rows, H, d, activation) ? ga::feed_forward_backward_space(rows, H, d, halves_of(activation)).total : 0;
}

ga_status ga_feed_forward_backward(const void *dy, const void *x, const void *kept, const void *w_in, const void *w_down,
                                   void *dx, void *dw_in, void *dw_down, int64_t rows, int64_t H, int64_t d,
                                   int32_t dtype, int32_t activation, const int32_t *live_rows, void *workspace,
                                   size_t workspace_bytes, ga_stream stream) {
    const char *op = "ga_feed_forward_backward";
    ga_status st = check_layer(op, rows, H, d, 8, dtype, activation);
    if (st != GA_OK) return st;
    const int64_t zd = halves_of(activation) * d;
    const Region regions[] = {{"dy", dy, (size_t)rows * H * 2, 16, false, false},
                              {"x", x, (size_t)rows * H * 2, 16, false, false},
                              {"kept", kept, (size_t)rows * zd * 2, 16, false, false},
                              {"w_in", w_in, (size_t)zd * H * 2, 16, false, false},
                              {"w_down", w_down, (size_t)H * d * 2, 16, false, false},
                              {"live_rows", live_rows, 4, 4, false, true},
                              {"dx", dx, (size_t)rows * H * 2, 16, true, false},
                              {"dw_in", dw_in, (size_t)zd * H * 2, 16, true, false},
                              {"dw_down", dw_down, (size_t)H * d * 2, 16, true, false},
                              {"workspace", workspace, workspace_bytes, 256, true, true}};
    if ((st = check_regions(op, regions)) != GA_OK ||
        (st = check_workspace(op, workspace, workspace_bytes,
                              ga_feed_forward_backward_workspace_bytes(rows, H, d, activation))) != GA_OK ||
        (st = check_product(op, d, rows, H, false, 1, 64)) != GA_OK || (st = check_product(op, H, rows, zd, false, 1, 64)) != GA_OK)
        return st;
    return ga::launched(op, ga::launch_feed_forward_backward(dtype, op_of(activation), dy, x, kept, w_in, w_down, dx, dw_in,
                                                             dw_down, (int32_t)rows, (int32_t)H, (int32_t)d, live_rows,
                                                             (uint8_t *)workspace, (hipStream_t)stream));
}

// ---------------------------------------------------------------------------
// Microscaled 4 bits
// ---------------------------------------------------------------------------
ga_status ga_mxfp4_quantize(const void *in, void *codes, uint8_t *scales, int64_t rows, int64_t d, int32_t dtype,
                            const int32_t *live_rows, ga_stream stream) {
    const char *op = "ga_mxfp4_quantize";
    const ga_status st = check_sizes(op, rows, d, GA_MAX_D, dtype);
    return st != GA_OK ? st : quantize(op, in, codes, scales, rows, d, 1, dtype, -1, live_rows, stream);
}

ga_status ga_activation_mxfp4(const void *in, void *codes, uint8_t *scales, int64_t rows, int64_t d, int32_t dtype,
                              int32_t activation, const int32_t *live_rows, ga_stream stream) {
    const char *op = "ga_activation_mxfp4";
    ga_status st = check_sizes(op, rows, d, GA_MAX_D, dtype);
    if (st != GA_OK || (st = check_activation(op, activation)) != GA_OK) return st;
    return quantize(op, in, codes, scales, rows, d, halves_of(activation), dtype, op_of(activation), live_rows, stream);
}

ga_status ga_mxfp4_dequantize(const void *codes, const uint8_t *scales, void *out, int64_t rows, int64_t d,
                              int32_t dtype, const int32_t *live_rows, ga_stream stream) {
    const char *op = "ga_mxfp4_dequantize";
    ga_status st = check_sizes(op, rows, d, GA_MAX_D, dtype);
    if (st != GA_OK) return st;
    const size_t es = elem_size(dtype);
    const Region regions[] = {{"codes", codes, mx_codes(rows, d), 16, false, false},
                              {"scales", scales, mx_scales(rows, d), 1, false, false},
                              {"live_rows", live_rows, 4, 4, false, true},
                              {"out", out, (size_t)rows * d * es, es, true, false}};
    if ((st = check_regions(op, regions)) != GA_OK || (st = ga::check_blocks(op, rows * ga::blocks_of(d))) != GA_OK) return st;
    if (rows == 0) return GA_OK;
    return ga::launched(op, ga::launch_mxfp4_dequantize(dtype, codes, scales, out, (int32_t)rows, (uint32_t)d, live_rows,
                                                        (hipStream_t)stream));
}

size_t ga_mxfp4_product_workspace_bytes(int64_t rows, int64_t n, int64_t k) {
    if (rows < 1 || rows > INT32_MAX || n < 1 || n > INT32_MAX || k < 1 || k > GA_MAX_D) return 0;
    return ga::mxfp4_product_space(rows, n, k);
}

ga_status ga_mxfp4_product(const void *a_codes, const uint8_t *a_scales, const void *w_codes, const uint8_t *w_scales,
                           void *out, int64_t rows, int64_t n, int64_t k, int32_t dtype, const int32_t *live_rows,
                           void *workspace, size_t workspace_bytes, ga_stream stream) {
    const char *op = "ga_mxfp4_product";
    ga_status st = check_sizes(op, rows, k, GA_MAX_D, dtype);
    if (st != GA_OK) return st;
    if (n < 1) return fail(GA_EINVAL, "%s: n = %lld must be >= 1", op, (long long)n);
    if (n > INT32_MAX - 1024) return fail(GA_EUNSUPPORTED, "%s: n = %lld above 2^31 - 1025", op, (long long)n);
    const size_t es = elem_size(dtype);
    const Region regions[] = {{"a_codes", a_codes, mx_codes(rows, k), 16, false, false},
                              {"a_scales", a_scales, mx_scales(rows, k), 1, false, false},
                              {"w_codes", w_codes, mx_codes(n, k), 16, false, false},
                              {"w_scales", w_scales, mx_scales(n, k), 1, false, false},
                              {"live_rows", live_rows, 4, 4, false, true},
                              {"out", out, (size_t)rows * n * es, es, true, false},
                              {"workspace", workspace, workspace_bytes, 256, true, true}};
    if ((st = check_regions(op, regions)) != GA_OK ||
        (st = check_workspace(op, workspace, workspace_bytes, ga_mxfp4_product_workspace_bytes(rows, n, k))) != GA_OK ||
        (st = check_product(op, n, rows, k, false, 0, 256)) != GA_OK)
        return st;
    if (rows == 0) return GA_OK;
    return ga::launched(op, ga::launch_mxfp4_product(dtype, a_codes, a_scales, w_codes, w_scales, out, (int32_t)rows,
                                                     (int32_t)n, (int32_t)k, live_rows, (uint8_t *)workspace,
                                                     (hipStream_t)stream));
}

size_t ga_feed_forward_mxfp4_workspace_bytes(int64_t rows, int64_t H, int64_t d, int32_t activation) {
    return layer_sizes(rows, H, d, activation) ? ga::feed_forward_mxfp4_space(rows, H, d, halves_of(activation)).total : 0;
}

ga_status ga_feed_forward_mxfp4(const void *x, const void *w_in_codes, const uint8_t *w_in_scales,
                                const void *w_down_codes, const uint8_t *w_down_scales, void *y, int64_t rows, int64_t H,
                                int64_t d, int32_t dtype, int32_t activation, const int32_t *live_rows, void *workspace,
                                size_t workspace_bytes, ga_stream stream) {
    const char *op = "ga_feed_forward_mxfp4";
    ga_status st = check_layer(op, rows, H, d, GA_MXFP4_BLOCK, dtype, activation);
    if (st != GA_OK) return st;
    const int64_t zd = halves_of(activation) * d;
    const Region regions[] = {{"x", x, (size_t)rows * H * 2, 2, false, false},
                              {"w_in_codes", w_in_codes, mx_codes(zd, H), 16, false, false},
                              {"w_in_scales", w_in_scales, mx_scales(zd, H), 1, false, false},
                              {"w_down_codes", w_down_codes, mx_codes(H, d), 16, false, false},
                              {"w_down_scales", w_down_scales, mx_scales(H, d), 1, false, false},
                              {"live_rows", live_rows, 4, 4, false, true},
                              {"y", y, (size_t)rows * H * 2, 2, true, false},
                              {"workspace", workspace, workspace_bytes, 256, true, true}};
    if ((st = check_regions(op, regions)) != GA_OK ||
        (st = check_workspace(op, workspace, workspace_bytes,
                              ga_feed_forward_mxfp4_workspace_bytes(rows, H, d, activation))) != GA_OK ||
        (st = ga::check_blocks(op, rows * ga::blocks_of(H))) != GA_OK ||
        (st = check_product(op, d, rows, H, zd != d, 0, 256)) != GA_OK ||
        (st = check_product(op, H, rows, d, false, 0, 256)) != GA_OK)
        return st;
    if (rows == 0) return GA_OK;
    return ga::launched(op, ga::launch_feed_forward_mxfp4(dtype, op_of(activation), x, w_in_codes, w_in_scales, w_down_codes,
                                                          w_down_scales, y, (int32_t)rows, (int32_t)H, (int32_t)d, live_rows,
                                                          (uint8_t *)workspace, (hipStream_t)stream));
}

// ---------------------------------------------------------------------------
// Planners
// ---------------------------------------------------------------------------
ga_status ga_plan_feed_forward(int64_t rows, int64_t H, int64_t d, int32_t activation, int32_t bits, int32_t product,
                               ga_product_plan *plan) {
    const char *op = "ga_plan_feed_forward";
    if (plan == nullptr) return fail(GA_EINVAL, "%s: null plan", op);
    if (bits != 4 && bits != 16) return fail(GA_EINVAL, "%s: %d bits", op, (int)bits);
    if (product < GA_PRODUCT_HIDDEN || product > (bits == 4 ? GA_PRODUCT_OUT : GA_PRODUCT_DW_DOWN))
        return fail(GA_EINVAL, "%s: no product %d in %d bits", op, (int)product, (int)bits);
    const ga_status st = check_layer(op, rows, H, d, bits == 4 ? GA_MXFP4_BLOCK : 8, GA_BF16, activation);
    if (st != GA_OK) return st;
    if (rows < 1) return fail(GA_EINVAL, "%s: no rows", op);
    const bool pair = halves_of(activation) == 2;
    const int64_t zd = halves_of(activation) * d;
    const struct {
        int64_t F, T, K;
        bool halves;
        int strided;
    } of[] = {{d, rows, H, pair, 0}, {H, rows, d, false, 0}, {d, rows, H, false, 1},
              {H, rows, zd, false, 1}, {H, zd, rows, false, 2}, {d, H, rows, false, 2}};
    const auto &p = of[product];
    const int step = bits == 4 ? 256 : 64;
    if (product >= GA_PRODUCT_DX) {
        const ga::ThreePlan three = ga::plan_three(rows, H, d, zd);
        if (three.together) {
            describe(product == GA_PRODUCT_DX ? three.x : product == GA_PRODUCT_DW_IN ? three.in : three.down, p.K, step, true, plan);
            return GA_OK;
        }
    }
    describe(ga::plan_product(p.F, p.T, p.K, p.halves, p.strided, step), p.K, step, false, plan);
    return GA_OK;
}

ga_status ga_plan_mxfp4_product(int64_t rows, int64_t n, int64_t k, ga_product_plan *plan) {
    const char *op = "ga_plan_mxfp4_product";
    if (plan == nullptr) return fail(GA_EINVAL, "%s: null plan", op);
    const ga_status st = check_sizes(op, rows, k, GA_MAX_D, GA_BF16);
    if (st != GA_OK) return st;
    if (rows < 1 || n < 1 || n > INT32_MAX) return fail(GA_EINVAL, "%s: %lld x %lld outputs", op, (long long)rows, (long long)n);
    describe(ga::plan_product(n, rows, k, false, 0, 256), k, 256, false, plan);
    return GA_OK;
}

}  // extern "C"
