"""Fused row-wise gated activations for AMD MI355X (gfx950).

A thin Python binding over libga.so (include/ga.h): it checks tensor shapes,
dtypes and contiguity, and passes device pointers, sizes and the current HIP
stream through the C-ABI.  Every step of the computation runs in the HIP
kernels; PyTorch only supplies device memory and the stream.  If the library
is not built, importing this package raises: there is no fallback.

    gelu_and_mul_sparse(x, z)           x: [T, 2d] -> [T, d] (round_intermediates=True:
                                        the round-trip form)
    gelu_and_mul_sparse_noalloc(x, z)   the same for T <= 256 rows, no workspace
                                        (the library's own static array)
    gelu_and_mul_sparse_down(x, w)      x: [T, 2d], w: [H, d] -> [T, H]: the activation
                                        fused with the down projection (bf16 / fp16)
    silu_and_mul_bounded(x, live_rows)  x: [M, 2d] -> [M, d] (live rows only)
    gelu_and_mul(x, approximate)        x: [T, 2d] -> [T, d] (tanh or erf GELU)
    squared_relu_bounded(x, live_rows)  x: [M, d]  -> [M, d] (live rows only)
    z_from_sparsity(p)                  Phi^-1(p), host-side

Training (no autograd graph: each backward is its own call):

    activation_checkpoint(x, activation)        -> out, Checkpoint (x kept in 8 bits)
    activation_backward(dout, kept, activation) kept: the Checkpoint or x -> dx
    checkpoint_store(x), checkpoint_restore(checkpoint, dtype)
    layer_norm(x, weight, bias)                 -> y, stats
    layer_norm_checkpoint(x, weight, bias)      -> y, Checkpoint (x - mean in 8 bits)
    layer_norm_backward(dy, kept, weight, stats) -> dx, dweight, dbias
    balance_loss(logits, experts)               -> Balance (loss, counts, offsets, tokens)
    balance_loss_backward(logits, balance, dloss) -> dlogits

The feed-forward layer, its products and the activation (bf16 / fp16):

    feed_forward(x, w_in, w_down, activation)         -> y = (act(gate) * up) w_down^T
    feed_forward_train(x, w_in, w_down, activation)   -> y, kept (gate | up)
    feed_forward_backward(dy, x, kept, w_in, w_down, activation) -> dx, dw_in, dw_down

and in microscaled 4 bits (Mxfp4: codes, scales, d):

    mxfp4_quantize(x), mxfp4_dequantize(q, dtype)
    activation_mxfp4(x, activation)                   -> Mxfp4 of the activation's result
    mxfp4_product(a, w, dtype)                        -> a w^T
    feed_forward_mxfp4(x, w_in, w_down, activation)   -> y

How these products run (host only): plan_feed_forward(rows, H, d, activation, product),
plan_mxfp4_product(rows, n, d) -> ProductPlan
"""
from ._lib import (  # noqa: F401
    GA_BF16, GA_F16, GA_F32, GA_OK, GA_EINVAL, GA_EUNSUPPORTED, GA_EHIP, GA_MAX_D, GA_ROUND_INTERMEDIATES,
    GaError, Plan, Z_SPARSITY_095, lib, library_path,
    gelu_and_mul_sparse, gelu_and_mul_sparse_noalloc, silu_and_mul_bounded, stream_xor_rows,
    gelu_and_mul, squared_relu_bounded, z_from_sparsity,
    plan_gelu_and_mul_sparse, plan_silu_and_mul_bounded, workspace_for,
    reserve_workspace, held_workspaces, GA_SPLIT_PLAN_ROWS, WORKSPACE_BYTES,
    DownPlan, GA_DOWN_MAX_ROWS, GA_DOWN_DECODE, GA_DOWN_STAGED, GA_DOWN_TILED,
    gelu_and_mul_sparse_down, plan_gelu_and_mul_sparse_down,
    gelu_and_mul_sparse_down_workspace_bytes, reserve_down_workspace,
)
from ._train import (  # noqa: F401
    GA_ACT_SILU, GA_ACT_GELU_TANH, GA_ACT_GELU_ERF, GA_ACT_SQUARED_RELU, GA_ACT_GELU_SPARSE, ACTIVATIONS,
    GA_CHECKPOINT_BLOCK, GA_LAYER_NORM_MAX_D, GA_BALANCE_MAX_EXPERTS, Checkpoint, Balance,
    checkpoint_store, checkpoint_restore, activation_checkpoint, activation_backward,
    layer_norm, layer_norm_checkpoint, layer_norm_backward, layer_norm_backward_workspace_bytes,
    balance_loss, balance_loss_backward, balance_loss_workspace_bytes,
)
from ._feed_forward import (  # noqa: F401
    GA_MXFP4_BLOCK, Mxfp4, feed_forward, feed_forward_train, feed_forward_backward, feed_forward_workspace_bytes,
    feed_forward_backward_workspace_bytes, mxfp4_quantize, mxfp4_dequantize, activation_mxfp4, mxfp4_product,
    mxfp4_product_workspace_bytes, feed_forward_mxfp4, feed_forward_mxfp4_workspace_bytes,
    ProductPlan, plan_feed_forward, plan_mxfp4_product, GA_PRODUCT_HIDDEN, GA_PRODUCT_OUT, GA_PRODUCT_DHIDDEN,
    GA_PRODUCT_DX, GA_PRODUCT_DW_IN, GA_PRODUCT_DW_DOWN,
)
