"""What the package's autograd functions share."""
from __future__ import annotations

import functools

import torch


class _NoSecond(torch.autograd.Function):
    """n gradients as they are, tied to what they were computed from; their own backward raises."""

    @staticmethod
    def forward(ctx, name, n, *tensors):
        ctx.name = name
        return tuple(t.view_as(t) for t in tensors[:n])

    @staticmethod
    def backward(ctx, *_):
        raise RuntimeError("%s has no second derivatives: its gradients cannot be differentiated" % ctx.name)


def first_order(backward):
    """For a Function's backward whose kernels build no graph (the decorator goes under staticmethod).

    Under create_graph=True its gradients depend on the saved tensors and on
    the incoming gradients, so that differentiating them raises instead of
    leaving terms out.  An incoming gradient that is handed on keeps its graph.
    The forward has to save every input that the gradients depend on.
    """
    @functools.wraps(backward)
    def run(ctx, *dys):
        with torch.no_grad():
            grads = backward(ctx, *dys)
        if not torch.is_grad_enabled():
            return grads
        own = [i for i, t in enumerate(grads) if t is not None and not any(t is d for d in dys)]
        roots = [t for t in (*ctx.saved_tensors, *dys) if t is not None and t.requires_grad]
        if not own or not roots:
            return grads
        name = backward.__qualname__.split(".")[0]
        tied = _NoSecond.apply(name, len(own), *(grads[i] for i in own), *roots)
        grads = list(grads)
        for i, t in zip(own, tied):
            grads[i] = t
        return tuple(grads)
    return run
