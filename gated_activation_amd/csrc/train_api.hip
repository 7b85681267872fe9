// The training entry points of the C-ABI: argument checks and dispatch.  As in
// api.hip, every check runs on the host before any HIP call.
#include <cmath>

#include "../../include/ga.h"
#include "ga_host.h"
#include "ga_internal.h"

static_assert(GA_LAYER_NORM_MAX_D == ga::LN_MAX_D && GA_BALANCE_MAX_EXPERTS == ga::BALANCE_MAX_E, "limits");

namespace {

using ga::elem_size;
using ga::fail;
using ga::overlaps;

// One array of a call, for the checks that all share.
struct Region {
    const char *name;
    const void *at;
    size_t bytes;
    size_t align;
    bool written;
    bool optional;
};

// Null, misaligned and overlapping arrays.  Arrays without a byte may be null;
// one that is written overlaps no other.
template <int N>
ga_status check_regions(const char *op, const Region (&r)[N]) {
    for (int i = 0; i < N; ++i) {
        if (r[i].at == nullptr) {
            if (r[i].optional || r[i].bytes == 0) continue;
            return fail(GA_EINVAL, "%s: null %s", op, r[i].name);
        }
        if ((uintptr_t)r[i].at % r[i].align != 0)
            return fail(GA_EINVAL, "%s: %s is not aligned to %zu bytes", op, r[i].name, r[i].align);
        for (int j = 0; j < i; ++j) {
            if (r[j].at == nullptr || !(r[i].written || r[j].written) || r[i].bytes == 0 || r[j].bytes == 0) continue;
            if (overlaps(r[i].at, r[i].bytes, r[j].at, r[j].bytes))
                return fail(GA_EINVAL, "%s: %s and %s overlap", op, r[j].name, r[i].name);
        }
    }
    return GA_OK;
}

ga_status check_sizes(const char *op, int64_t rows, int64_t d, int64_t most_d, int32_t dtype) {
    if (rows < 0 || rows > INT32_MAX)
        return fail(GA_EINVAL, "%s: row count %lld out of [0, 2^31)", op, (long long)rows);
    if (d < 1) return fail(GA_EINVAL, "%s: d = %lld must be >= 1", op, (long long)d);
    if (elem_size(dtype) == 0) return fail(GA_EINVAL, "%s: unknown dtype %d", op, (int)dtype);
    if (d > most_d) return fail(GA_EUNSUPPORTED, "%s: d = %lld above %lld", op, (long long)d, (long long)most_d);
    return GA_OK;
}

int64_t blocks_of(int64_t d) { return (d + GA_CHECKPOINT_BLOCK - 1) / GA_CHECKPOINT_BLOCK; }

// Elementwise kernels number the blocks of 128 values in 31 bits; the launches
// of kernels that give a row `lanes` work-items have fewer than 2^32.
ga_status check_blocks(const char *op, int64_t blocks) {
    if (blocks > INT32_MAX)
        return fail(GA_EUNSUPPORTED, "%s: %lld blocks of 128 values in one call (2^31 or more)", op, (long long)blocks);
    return GA_OK;
}

ga_status check_items(const char *op, int64_t rows, int64_t lanes) {
    if (rows * lanes + 1024 > (int64_t)UINT32_MAX)
        return fail(GA_EUNSUPPORTED, "%s: %lld rows of %lld lanes in one launch (2^32 work-items or more)", op,
                    (long long)rows, (long long)lanes);
    return GA_OK;
}

int op_of(int32_t activation) {
    switch (activation) {
    case GA_ACT_SILU: return ga::OP_SILU_MUL;
    case GA_ACT_GELU_TANH: return ga::OP_GELU_TANH_MUL;
    case GA_ACT_GELU_ERF: return ga::OP_GELU_ERF_MUL;
    case GA_ACT_SQUARED_RELU: return ga::OP_SQUARED_RELU;
    default: return -1;
    }
}

ga_status check_activation(const char *op, int32_t activation, float z) {
    if (activation < GA_ACT_SILU || activation > GA_ACT_GELU_SPARSE)
        return fail(GA_EINVAL, "%s: unknown activation %d", op, (int)activation);
    if (activation == GA_ACT_GELU_SPARSE && !std::isfinite(z)) return fail(GA_EINVAL, "%s: z is not finite", op);
    return GA_OK;
}

int64_t halves_of(int32_t activation) { return activation == GA_ACT_SQUARED_RELU ? 1 : 2; }

ga_status check_rows_fit(const char *op, int32_t activation, int64_t rows, int64_t d) {
    if (activation == GA_ACT_GELU_SPARSE) return check_items(op, rows, 64 * ga::sparse_train_waves(d));
    return check_blocks(op, rows * blocks_of(d));
}

ga_status check_weight_type(const char *op, int32_t dtype, int32_t weight_dtype) {
    if (weight_dtype != dtype && weight_dtype != GA_F32)
        return fail(GA_EINVAL, "%s: weight dtype %d is neither fp32 nor the rows' %d", op, (int)weight_dtype, (int)dtype);
    return GA_OK;
}

constexpr int kMostCus = 256;  // what workspaces are sized for

ga_status usable_cus(int *cus) {
    const ga_status st = ga::current_cus(cus);
    if (st == GA_OK && *cus > kMostCus) *cus = kMostCus;
    return st;
}

ga_status layer_norm(const char *op, const void *in, const void *weight, const void *bias, void *out, void *codes,
                     float *scales, float *stats, bool keep, int64_t rows, int64_t d, int32_t dtype,
                     int32_t weight_dtype, float eps, const int32_t *live_rows, ga_stream stream) {
    ga_status st = check_sizes(op, rows, d, ga::LN_MAX_D, dtype);
    if (st != GA_OK || (st = check_weight_type(op, dtype, weight_dtype)) != GA_OK) return st;
    if (!(eps >= 0.0f) || !std::isfinite(eps)) return fail(GA_EINVAL, "%s: eps is not a finite number >= 0", op);
    const size_t es = elem_size(dtype), ws = elem_size(weight_dtype), n = (size_t)rows * d;
    const Region regions[] = {{"in", in, n * es, es, false, false},
                              {"weight", weight, (size_t)d * ws, ws, false, false},
                              {"bias", bias, (size_t)d * ws, ws, false, true},
                              {"live_rows", live_rows, 4, 4, false, true},
                              {"out", out, n * es, es, true, false},
                              {"stats", stats, (size_t)rows * 8, 4, true, false},
                              {"codes", codes, keep ? n : 0, 1, true, !keep},
                              {"scales", scales, keep ? (size_t)rows * blocks_of(d) * 4 : 0, 4, true, !keep}};
    if ((st = check_regions(op, regions)) != GA_OK || (st = check_items(op, rows, ga::layer_norm_lanes(d))) != GA_OK)
        return st;
    if (rows == 0) return GA_OK;
    return ga::launched(op, ga::launch_layer_norm(dtype, weight_dtype == GA_F32, in, weight, bias, out,
                                                  keep ? codes : nullptr, scales, stats, (int32_t)rows, (int32_t)d, eps,
                                                  live_rows, (hipStream_t)stream));
}

ga_status layer_norm_backward(const char *op, const void *dout, const void *in, const void *codes, const float *scales,
                              const float *stats, bool kept, const void *weight, void *dx, void *dweight, void *dbias,
                              int64_t rows, int64_t d, int32_t dtype, int32_t weight_dtype, const int32_t *live_rows,
                              void *workspace, size_t workspace_bytes, ga_stream stream) {
    ga_status st = check_sizes(op, rows, d, ga::LN_MAX_D, dtype);
    if (st != GA_OK || (st = check_weight_type(op, dtype, weight_dtype)) != GA_OK) return st;
    const size_t es = elem_size(dtype), ws = elem_size(weight_dtype), n = (size_t)rows * d;
    const Region regions[] = {{"dout", dout, n * es, es, false, false},
                              {"in", in, kept ? 0 : n * es, es, false, kept},
                              {"codes", codes, kept ? n : 0, 1, false, !kept},
                              {"scales", scales, kept ? (size_t)rows * blocks_of(d) * 4 : 0, 4, false, !kept},
                              {"stats", stats, (size_t)rows * 8, 4, false, false},
                              {"weight", weight, (size_t)d * ws, ws, false, false},
                              {"live_rows", live_rows, 4, 4, false, true},
                              {"dx", dx, n * es, es, true, false},
                              {"dweight", dweight, (size_t)d * ws, ws, true, false},
                              {"dbias", dbias, (size_t)d * ws, ws, true, true},
                              {"workspace", workspace, workspace_bytes, 16, true, true}};
    if ((st = check_regions(op, regions)) != GA_OK) return st;
    const size_t need = ga_layer_norm_backward_workspace_bytes(rows, d);
    if (workspace_bytes < need || (need > 0 && workspace == nullptr))
        return fail(GA_EINVAL, "%s: workspace of %zu bytes, %zu needed", op, workspace == nullptr ? 0 : workspace_bytes,
                    need);
    int cus = 0;
    if ((st = usable_cus(&cus)) != GA_OK) return st;
    return ga::launched(op, ga::launch_layer_norm_backward(
                                dtype, weight_dtype == GA_F32, dout, kept ? nullptr : in, kept ? codes : nullptr, scales,
                                stats, weight, dx, dweight, dbias, kept, (int32_t)rows, (int32_t)d, live_rows,
                                ga::layer_norm_groups(rows, d, dtype == GA_F32, cus), cus, (float *)workspace, (hipStream_t)stream));
}

ga_status check_balance(const char *op, int64_t rows, int64_t experts, int64_t k, int32_t dtype, float coefficient) {
    if (rows < 0 || rows > INT32_MAX)
        return fail(GA_EINVAL, "%s: row count %lld out of [0, 2^31)", op, (long long)rows);
    if (experts < 1 || k < 1) return fail(GA_EINVAL, "%s: experts and k must be >= 1", op);
    if (elem_size(dtype) == 0) return fail(GA_EINVAL, "%s: unknown dtype %d", op, (int)dtype);
    if (!std::isfinite(coefficient)) return fail(GA_EINVAL, "%s: coefficient is not finite", op);
    if (experts > ga::BALANCE_MAX_E)
        return fail(GA_EUNSUPPORTED, "%s: %lld experts, at most %lld", op, (long long)experts,
                    (long long)ga::BALANCE_MAX_E);
    if (k > INT32_MAX || rows * k > INT32_MAX)
        return fail(GA_EUNSUPPORTED, "%s: rows * k is 2^31 or more (counts are int32)", op);
    return GA_OK;
}

}  // namespace

extern "C" {

// ---------------------------------------------------------------------------
// Activation checkpoints
// ---------------------------------------------------------------------------
ga_status ga_checkpoint_store(const void *in, void *codes, float *scales, int64_t rows, int64_t d, int32_t dtype,
                              const int32_t *live_rows, ga_stream stream) {
    const char *op = "ga_checkpoint_store";
    ga_status st = check_sizes(op, rows, d, GA_MAX_D, dtype);
    if (st != GA_OK) return st;
    const size_t es = elem_size(dtype), n = (size_t)rows * d;
    const Region regions[] = {{"in", in, n * es, es, false, false},
                              {"live_rows", live_rows, 4, 4, false, true},
                              {"codes", codes, n, 1, true, false},
                              {"scales", scales, (size_t)rows * blocks_of(d) * 4, 4, true, false}};
    if ((st = check_regions(op, regions)) != GA_OK || (st = check_blocks(op, rows * blocks_of(d))) != GA_OK) return st;
    if (rows == 0) return GA_OK;
    return ga::launched(op, ga::launch_checkpoint_store(dtype, -1, in, nullptr, codes, scales, (int32_t)rows,
                                                        (uint32_t)d, live_rows, (hipStream_t)stream));
}

ga_status ga_checkpoint_restore(const void *codes, const float *scales, const float *stats, void *out, int64_t rows,
                                int64_t d, int32_t halves, int32_t dtype, const int32_t *live_rows, ga_stream stream) {
    const char *op = "ga_checkpoint_restore";
    ga_status st = check_sizes(op, rows, d, GA_MAX_D, dtype);
    if (st != GA_OK) return st;
    if (halves != 1 && halves != 2) return fail(GA_EINVAL, "%s: halves = %d is neither 1 nor 2", op, (int)halves);
    const size_t es = elem_size(dtype), n = (size_t)rows * halves * d;
    const Region regions[] = {{"codes", codes, n, 1, false, false},
                              {"scales", scales, (size_t)rows * halves * blocks_of(d) * 4, 4, false, false},
                              {"stats", stats, (size_t)rows * 8, 4, false, true},
                              {"live_rows", live_rows, 4, 4, false, true},
                              {"out", out, n * es, es, true, false}};
    if ((st = check_regions(op, regions)) != GA_OK ||
        (st = check_blocks(op, rows * halves * blocks_of(d))) != GA_OK)
        return st;
    if (rows == 0) return GA_OK;
    return ga::launched(op, ga::launch_checkpoint_restore(dtype, codes, scales, stats, out, (int32_t)rows, (uint32_t)d,
                                                          halves, live_rows, (hipStream_t)stream));
}

ga_status ga_activation_checkpoint(const void *in, void *out, void *codes, float *scales, float *stats, int64_t rows,
                                   int64_t d, int32_t dtype, int32_t activation, float z, const int32_t *live_rows,
                                   ga_stream stream) {
    const char *op = "ga_activation_checkpoint";
    ga_status st = check_sizes(op, rows, d, GA_MAX_D, dtype);
    if (st != GA_OK || (st = check_activation(op, activation, z)) != GA_OK) return st;
    const bool sparse = activation == GA_ACT_GELU_SPARSE;
    const size_t es = elem_size(dtype), n = (size_t)rows * d, h = (size_t)halves_of(activation);
    const Region regions[] = {{"in", in, h * n * es, es, false, false},
                              {"live_rows", live_rows, 4, 4, false, true},
                              {"out", out, n * es, es, true, false},
                              {"codes", codes, h * n, 1, true, false},
                              {"scales", scales, (size_t)rows * h * blocks_of(d) * 4, 4, true, false},
                              {"stats", stats, sparse ? (size_t)rows * 8 : 0, 4, true, !sparse}};
    if ((st = check_regions(op, regions)) != GA_OK || (st = check_rows_fit(op, activation, rows, d)) != GA_OK) return st;
    if (rows == 0) return GA_OK;
    const hipStream_t s = (hipStream_t)stream;
    return ga::launched(op, sparse ? ga::launch_sparse_store(dtype, in, out, codes, scales, stats, (int32_t)rows,
                                                             (int32_t)d, z, live_rows, s)
                                   : ga::launch_checkpoint_store(dtype, op_of(activation), in, out, codes, scales,
                                                                 (int32_t)rows, (uint32_t)d, live_rows, s));
}

ga_status ga_activation_backward(const void *dout, const void *in, void *dx, int64_t rows, int64_t d, int32_t dtype,
                                 int32_t activation, float z, const int32_t *live_rows, ga_stream stream) {
    const char *op = "ga_activation_backward";
    ga_status st = check_sizes(op, rows, d, GA_MAX_D, dtype);
    if (st != GA_OK || (st = check_activation(op, activation, z)) != GA_OK) return st;
    const size_t es = elem_size(dtype), n = (size_t)rows * d, h = (size_t)halves_of(activation);
    const Region regions[] = {{"dout", dout, n * es, es, false, false},
                              {"in", in, h * n * es, es, false, false},
                              {"live_rows", live_rows, 4, 4, false, true},
                              {"dx", dx, h * n * es, es, true, false}};
    if ((st = check_regions(op, regions)) != GA_OK || (st = check_rows_fit(op, activation, rows, d)) != GA_OK) return st;
    if (rows == 0) return GA_OK;
    const hipStream_t s = (hipStream_t)stream;
    return ga::launched(op, activation == GA_ACT_GELU_SPARSE
                                ? ga::launch_sparse_backward(dtype, dout, in, nullptr, nullptr, nullptr, dx,
                                                             (int32_t)rows, (int32_t)d, z, live_rows, s)
                                : ga::launch_act_backward(dtype, op_of(activation), dout, in, nullptr, nullptr, dx,
                                                          (int32_t)rows, (uint32_t)d, live_rows, s));
}

ga_status ga_activation_backward_checkpoint(const void *dout, const void *codes, const float *scales,
                                            const float *stats, void *dx, int64_t rows, int64_t d, int32_t dtype,
                                            int32_t activation, float z, const int32_t *live_rows, ga_stream stream) {
    const char *op = "ga_activation_backward_checkpoint";
    ga_status st = check_sizes(op, rows, d, GA_MAX_D, dtype);
    if (st != GA_OK || (st = check_activation(op, activation, z)) != GA_OK) return st;
    const bool sparse = activation == GA_ACT_GELU_SPARSE;
    const size_t es = elem_size(dtype), n = (size_t)rows * d, h = (size_t)halves_of(activation);
    const Region regions[] = {{"dout", dout, n * es, es, false, false},
                              {"codes", codes, h * n, 1, false, false},
                              {"scales", scales, (size_t)rows * h * blocks_of(d) * 4, 4, false, false},
                              {"stats", stats, sparse ? (size_t)rows * 8 : 0, 4, false, !sparse},
                              {"live_rows", live_rows, 4, 4, false, true},
                              {"dx", dx, h * n * es, es, true, false}};
    if ((st = check_regions(op, regions)) != GA_OK || (st = check_rows_fit(op, activation, rows, d)) != GA_OK) return st;
    if (rows == 0) return GA_OK;
    const hipStream_t s = (hipStream_t)stream;
    return ga::launched(op, sparse ? ga::launch_sparse_backward(dtype, dout, nullptr, codes, scales, stats, dx,
                                                                (int32_t)rows, (int32_t)d, z, live_rows, s)
                                   : ga::launch_act_backward(dtype, op_of(activation), dout, nullptr, codes, scales, dx,
                                                             (int32_t)rows, (uint32_t)d, live_rows, s));
}

// ---------------------------------------------------------------------------
// Layer norm
// ---------------------------------------------------------------------------
ga_status ga_layer_norm(const void *in, const void *weight, const void *bias, void *out, float *stats, int64_t rows,
                        int64_t d, int32_t dtype, int32_t weight_dtype, float eps, const int32_t *live_rows,
                        ga_stream stream) {
    return layer_norm("ga_layer_norm", in, weight, bias, out, nullptr, nullptr, stats, false, rows, d, dtype,
                      weight_dtype, eps, live_rows, stream);
}

ga_status ga_layer_norm_checkpoint(const void *in, const void *weight, const void *bias, void *out, void *codes,
                                   float *scales, float *stats, int64_t rows, int64_t d, int32_t dtype,
                                   int32_t weight_dtype, float eps, const int32_t *live_rows, ga_stream stream) {
    return layer_norm("ga_layer_norm_checkpoint", in, weight, bias, out, codes, scales, stats, true, rows, d, dtype,
                      weight_dtype, eps, live_rows, stream);
}

size_t ga_layer_norm_backward_workspace_bytes(int64_t rows, int64_t d) {
    if (rows < 1 || rows > INT32_MAX || d < 1 || d > ga::LN_MAX_D) return 0;
    // of any row type: 16-bit rows have more teams to a workgroup, so fp32 rows the more groups
    return ga::layer_norm_workspace_bytes(rows, d, ga::layer_norm_groups(rows, d, true, kMostCus));
}

ga_status ga_layer_norm_backward(const void *dout, const void *in, const float *stats, const void *weight, void *dx,
                                 void *dweight, void *dbias, int64_t rows, int64_t d, int32_t dtype,
                                 int32_t weight_dtype, const int32_t *live_rows, void *workspace,
                                 size_t workspace_bytes, ga_stream stream) {
    return layer_norm_backward("ga_layer_norm_backward", dout, in, nullptr, nullptr, stats, false, weight, dx, dweight,
                               dbias, rows, d, dtype, weight_dtype, live_rows, workspace, workspace_bytes, stream);
}

ga_status ga_layer_norm_backward_checkpoint(const void *dout, const void *codes, const float *scales,
                                            const float *stats, const void *weight, void *dx, void *dweight,
                                            void *dbias, int64_t rows, int64_t d, int32_t dtype, int32_t weight_dtype,
                                            const int32_t *live_rows, void *workspace, size_t workspace_bytes,
                                            ga_stream stream) {
    return layer_norm_backward("ga_layer_norm_backward_checkpoint", dout, nullptr, codes, scales, stats, true, weight,
                               dx, dweight, dbias, rows, d, dtype, weight_dtype, live_rows, workspace, workspace_bytes,
                               stream);
}

// ---------------------------------------------------------------------------
// Balance loss
// ---------------------------------------------------------------------------
size_t ga_balance_loss_workspace_bytes(int64_t rows, int64_t experts) {
    if (rows < 1 || rows > INT32_MAX || experts < 1 || experts > ga::BALANCE_MAX_E) return 0;
    return ga::balance_workspace_bytes(ga::balance_groups(rows, experts, kMostCus), experts);
}

ga_status ga_balance_loss(const void *logits, const void *index, int32_t index_bytes, const uint8_t *mask, float *loss,
                          int32_t *counts, int32_t *offsets, int32_t *tokens, int64_t rows, int64_t experts, int64_t k,
                          int32_t dtype, float coefficient, const int32_t *live_rows, void *workspace,
                          size_t workspace_bytes, ga_stream stream) {
    const char *op = "ga_balance_loss";
    ga_status st = check_balance(op, rows, experts, k, dtype, coefficient);
    if (st != GA_OK) return st;
    if (index_bytes != 4 && index_bytes != 8)
        return fail(GA_EINVAL, "%s: indices of %d bytes (4 or 8)", op, (int)index_bytes);
    const size_t es = elem_size(dtype);
    const Region regions[] = {{"logits", logits, (size_t)rows * experts * es, es, false, false},
                              {"index", index, (size_t)rows * k * index_bytes, (size_t)index_bytes, false, false},
                              {"mask", mask, (size_t)rows, 1, false, true},
                              {"live_rows", live_rows, 4, 4, false, true},
                              {"loss", loss, 4, 4, true, false},
                              {"counts", counts, (size_t)experts * 4, 4, true, false},
                              {"offsets", offsets, (size_t)(experts + 1) * 4, 4, true, false},
                              {"tokens", tokens, 4, 4, true, false},
                              {"workspace", workspace, workspace_bytes, 16, true, true}};
    if ((st = check_regions(op, regions)) != GA_OK) return st;
    const size_t need = ga_balance_loss_workspace_bytes(rows, experts);
    if (workspace_bytes < need || (need > 0 && workspace == nullptr))
        return fail(GA_EINVAL, "%s: workspace of %zu bytes, %zu needed", op, workspace == nullptr ? 0 : workspace_bytes,
                    need);
    int cus = 0;
    if ((st = usable_cus(&cus)) != GA_OK) return st;
    return ga::launched(op, ga::launch_balance(dtype, logits, index, index_bytes == 8, mask, loss, counts, offsets,
                                               tokens, (int32_t)rows, (int32_t)experts, (int32_t)k, coefficient,
                                               live_rows, ga::balance_groups(rows, experts, cus), workspace,
                                               (hipStream_t)stream));
}

ga_status ga_balance_loss_backward(const void *logits, const uint8_t *mask, const int32_t *counts,
                                   const int32_t *offsets, const int32_t *tokens, const float *dloss, void *dlogits,
                                   int64_t rows, int64_t experts, int64_t k, int32_t dtype, float coefficient,
                                   const int32_t *live_rows, ga_stream stream) {
    const char *op = "ga_balance_loss_backward";
    ga_status st = check_balance(op, rows, experts, k, dtype, coefficient);
    if (st != GA_OK) return st;
    const size_t es = elem_size(dtype);
    const Region regions[] = {{"logits", logits, (size_t)rows * experts * es, es, false, false},
                              {"mask", mask, (size_t)rows, 1, false, true},
                              {"counts", counts, (size_t)experts * 4, 4, false, false},
                              {"offsets", offsets, (size_t)(experts + 1) * 4, 4, false, false},
                              {"tokens", tokens, 4, 4, false, false},
                              {"dloss", dloss, 4, 4, false, false},
                              {"live_rows", live_rows, 4, 4, false, true},
                              {"dlogits", dlogits, (size_t)rows * experts * es, es, true, false}};
    if ((st = check_regions(op, regions)) != GA_OK) return st;
    if (rows == 0) return GA_OK;
    int cus = 0;
    if ((st = usable_cus(&cus)) != GA_OK) return st;
    return ga::launched(op, ga::launch_balance_backward(dtype, logits, mask, counts, offsets, tokens, dloss, dlogits,
                                                        (int32_t)rows, (int32_t)experts, (int32_t)k, coefficient,
                                                        live_rows, cus, (hipStream_t)stream));
}

}  // extern "C"
