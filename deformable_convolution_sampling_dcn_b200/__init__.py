"""B200 (sm_100a) modulated deformable sampling-aggregation core.

Thin Python front end of libdcn_b200.so (C ABI in include/dcn_b200.h):

    dcn_core_forward / dcn_core_backward     DCNv2/v3/v4 sampling core
    dcn_core_forward_proj                    the core fused with its 1x1 projection (DCNv4 module)
    dcn_deform_conv_forward                  modulated deformable convolution, weight per point (DCNv2)
    deform_agg_forward / deform_agg_backward Sparse4D multi-camera aggregation
    deform_roi_pool_forward                  deformable RoI pooling
    dcn_proj_adapters_forward                1x1 projection with low-rank adapters of many requests
    dcn_add_rms_norm_forward / _backward     residual addition + root-mean-square norm, 8-bit output
    dcn_grad_norm / dcn_clip_grads           global gradient norm over many tensors (GradList), clipping
    DCNCoreFunction, DeformAggFunction,
    AddRmsNormFunction                       autograd wrappers over the above
    shard_range                              batch split for one-process-per-GPU runs

PyTorch only allocates device memory and supplies the current stream; every
arithmetic step runs in the library's CUDA kernels.
"""
from __future__ import annotations

from typing import Tuple

import torch

from ._binding import (ABI_VERSION, EXPORTS, AddRmsNorm, DadaptParams, DaggParams, DclipParams, DcnError, DcnParams,
                       DnormParams, DroiParams, GradList, core_params, dcn_add_rms_norm_backward, dcn_add_rms_norm_forward,
                       dcn_clip_grads, dcn_core_backward, dcn_core_forward, dcn_core_forward_proj, dcn_core_output_hw,
                       dcn_deform_conv_forward, dcn_grad_norm, dcn_proj_adapters_forward,
                       deform_agg_backward,
                       deform_agg_forward, deform_roi_pool_forward, lib)

__all__ = ["dcn_core_forward", "dcn_core_forward_proj", "dcn_deform_conv_forward", "dcn_core_backward", "dcn_core_output_hw", "deform_agg_forward",
           "deform_agg_backward", "deform_roi_pool_forward", "DroiParams", "DCNCoreFunction", "DeformAggFunction", "shard_range", "lib", "DcnError",
           "DcnParams", "DaggParams", "core_params", "EXPORTS", "ABI_VERSION", "dcn_add_rms_norm_forward",
           "dcn_add_rms_norm_backward", "AddRmsNorm", "AddRmsNormFunction", "dcn_grad_norm", "dcn_clip_grads",
           "GradList", "DnormParams", "DclipParams", "dcn_proj_adapters_forward", "DadaptParams"]


class DCNCoreFunction(torch.autograd.Function):
    """autograd over dcn_core_forward/backward (x, offset, mask all differentiable)."""

    @staticmethod
    def forward(ctx, x, offset, mask, group: int, kernel=(3, 3), stride=(1, 1), pad=(1, 1), dil=(1, 1),
                offset_scale: float = 1.0, softmax: bool = False):
        ctx.cfg = dict(group=group, kernel=kernel, stride=stride, pad=pad, dil=dil, offset_scale=offset_scale,
                       softmax=softmax)
        ctx.save_for_backward(x, offset, mask)
        return dcn_core_forward(x, offset, mask, **ctx.cfg)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, grad_out):
        x, offset, mask = ctx.saved_tensors
        gx, goff, gm = dcn_core_backward(x, offset, mask, grad_out.contiguous(), **ctx.cfg)
        return gx, goff, gm, None, None, None, None, None, None, None


class DeformAggFunction(torch.autograd.Function):
    """autograd over deform_agg_forward/backward (feat, locations, weights differentiable)."""

    @staticmethod
    def forward(ctx, feat, spatial_shape, scale_start_index, sampling_location, weights):
        ctx.save_for_backward(feat, spatial_shape, scale_start_index, sampling_location, weights)
        return deform_agg_forward(feat, spatial_shape, scale_start_index, sampling_location, weights)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, grad_out):
        feat, ss, st, loc, w = ctx.saved_tensors
        gf, gl, gw = deform_agg_backward(feat, ss, st, loc, w, grad_out.contiguous())
        return gf, None, None, gl, gw


class AddRmsNormFunction(torch.autograd.Function):
    """autograd over dcn_add_rms_norm_forward/backward: (out, h) of x, residual and weight, all
    differentiable; residual and weight may be None, h is x + residual (x itself without one).

    Inside a CUDA graph capture, let no uncaptured autograd graph of the same leaves live: PyTorch would run their
    gradients' accumulation on the stream of that graph and end the capture with an error."""

    @staticmethod
    def forward(ctx, x, residual, weight, eps: float = 1e-6):
        o = dcn_add_rms_norm_forward(x, residual, weight, eps=eps, save_rstd=True)
        h = x if residual is None else o.residual_out
        ctx.save_for_backward(h, o.rstd, weight)
        ctx.eps, ctx.has_residual = eps, residual is not None
        ctx.set_materialize_grads(False)
        return o.out, (h.view_as(h) if residual is None else h)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, grad_out, grad_h):
        h, rstd, weight = ctx.saved_tensors
        if grad_out is None:
            gw = torch.zeros_like(weight) if ctx.needs_input_grad[2] else None
            return grad_h, (grad_h if ctx.has_residual else None), gw, None
        gx, gw = dcn_add_rms_norm_backward(grad_out.contiguous(), h, rstd, weight, eps=ctx.eps,
                                           grad_residual_out=None if grad_h is None else grad_h.contiguous(),
                                           need_grad_weight=ctx.needs_input_grad[2])
        return gx, (gx if ctx.has_residual else None), gw, None


def shard_range(total: int, world: int, rank: int) -> Tuple[int, int]:
    """Contiguous [lo, hi) share of `total` independent batch images for
    `rank` of `world` processes.  Images are independent in the forward and
    the backward (grad_x of image b only receives from image b), so a batch
    split needs no exchange between ranks."""
    if world < 1 or not 0 <= rank < world:
        raise ValueError("bad rank/world")
    base, extra = divmod(int(total), int(world))
    lo = rank * base + min(rank, extra)
    return lo, lo + base + (1 if rank < extra else 0)
