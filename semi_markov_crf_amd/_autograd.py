"""What the differentiable calls share.  Their gradients run in the library's kernels, which
autograd cannot look into."""

from __future__ import annotations

import torch


class _FirstOrder(torch.autograd.Function):
    @staticmethod
    def forward(ctx, name, compute, *tensors):
        ctx.name = name
        return compute()

    @staticmethod
    def backward(ctx, *grads):
        raise RuntimeError(f"{ctx.name} has no second derivatives: its gradient cannot be differentiated")


def first_order(name, compute, *tensors):
    """compute(), the gradients of `name` as functions of `tensors`.  Under create_graph=True they
    belong to the graph, so that a derivative taken through them raises instead of missing them."""
    if not torch.is_grad_enabled():
        return compute()
    return _FirstOrder.apply(name, compute, *tensors)
