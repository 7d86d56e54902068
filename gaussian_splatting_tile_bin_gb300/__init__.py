"""GB300-native tile-binned 2-D Gaussian splat rasterizer.

The compute path is libgsr.so (hand-written sm_103a CUDA kernels behind the C
ABI in include/gsr.h); this package is its thin Python binding:

    ctx = Context(0)
    bins = bin_splats(ctx, splats, depths, width, height)
    out_rgbw, final_T, last = rasterize_forward(ctx, splats, bins)
    grad = rasterize_backward(ctx, splats, bins, dl_dout, final_T, last)

and on either side the projection of 3-D Gaussians and its backward:

    splats, depths = project_forward(ctx, gaussians, camera)
    dl_dgaussians = project_backward(ctx, gaussians, camera, grad)

and the operators of a decoder that predicts those Gaussians from images, each
with its backward:

    y, mean, rstd = group_norm_forward(ctx, features, groups, weight, bias, activation="silu")
    k = rotary_forward(ctx, k, positions, rotary_frequencies(sections), sections)
    out, lse = cross_attention_forward(ctx, q, k, v, kv_lengths=lengths, key_mask=mask)
    y, total, mean, rstd = layer_norm_forward(ctx, x, weight, bias, residual=residual)
    out, final, states = gated_recurrence_forward(ctx, x, forget, gate, initial=state, reverse=True)
"""
from ._abi import (LIB_PATH, Bins, Context, GsrError, bin_splats, cross_attention_backward,
                   cross_attention_forward, gated_recurrence_backward, gated_recurrence_forward, group_norm_backward,
                   group_norm_forward, layer_norm_backward, layer_norm_forward, peak_kernel, project_backward,
                   project_forward, rasterize_backward, rasterize_forward, rotary_backward, rotary_forward,
                   rotary_frequencies)

__all__ = ["LIB_PATH", "Bins", "Context", "GsrError", "bin_splats", "rasterize_forward",
           "rasterize_backward", "project_forward", "project_backward", "peak_kernel",
           "group_norm_forward", "group_norm_backward", "rotary_forward", "rotary_backward",
           "rotary_frequencies", "cross_attention_forward", "cross_attention_backward",
           "layer_norm_forward", "layer_norm_backward", "gated_recurrence_forward", "gated_recurrence_backward"]
