"""Newton-Schulz orthogonalisation of stacks of blocks as a differentiable torch function, and the
views that cut a fused parameter into its blocks."""
from __future__ import annotations

import functools

import torch
from torch.autograd import forward_ad

from . import binding as mb

KJ_COEFFS = (3.4445, -4.7750, 2.0315)


def row_blocks(p, rows: int):
    """A [n * rows, cols] matrix as the stack of its n row blocks (heads of a fused projection)."""
    if p.dim() != 2 or rows <= 0 or p.shape[0] % rows:
        raise ValueError(f"cannot cut shape {tuple(p.shape)} into blocks of {rows} rows")
    return p.unflatten(0, (p.shape[0] // rows, rows))


def col_blocks(p, cols: int):
    """A [rows, n * cols] matrix as the stack of its n column blocks (a fused input projection)."""
    if p.dim() != 2 or cols <= 0 or p.shape[1] % cols:
        raise ValueError(f"cannot cut shape {tuple(p.shape)} into blocks of {cols} columns")
    return p.unflatten(1, (p.shape[1] // cols, cols)).transpose(0, 1)


def _unit_last(t):
    """t itself where the library can read it in place (unit stride in the last dimension, row pitch of
    at least a row), else a dense copy."""
    ok = (t.shape[-1] == 1 or t.stride(-1) == 1) and (t.shape[-2] == 1 or t.stride(-2) >= t.shape[-1])
    return t if ok else t.contiguous()


@functools.lru_cache(maxsize=64)
def _schedule(coeffs: tuple, steps: int, eps: float):
    per_step = coeffs if isinstance(coeffs[0], tuple) else (coeffs,) * steps
    if len(per_step) != steps:
        raise ValueError(f"{len(per_step)} coefficient triples for {steps} steps")
    return mb.Schedule(per_step, eps=eps)


class _Orthogonalize(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, schedule, dtype):
        y = torch.empty(x.shape, dtype=dtype, device=x.device)
        saved = mb.orthogonalize_alloc([mb.Stack(_unit_last(x.detach()), y)], schedule, keep=True)
        ctx.schedule, ctx.dtype = schedule, x.dtype
        ctx.save_for_backward(saved)
        return y

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dy):
        (saved,) = ctx.saved_tensors
        if dy.dtype not in (torch.bfloat16, torch.float16, torch.float32):
            dy = dy.float()
        dx = torch.empty(dy.shape, dtype=ctx.dtype, device=dy.device)
        mb.orthogonalize_backward_alloc([mb.Stack(_unit_last(dy), dx)], ctx.schedule, saved)
        return dx, None, None


def orthogonalize(x, steps: int = 5, coeffs=KJ_COEFFS, eps: float = 1e-7, dtype=None):
    """Every [rows, cols] block of x ([rows, cols] or [count, rows, cols]; bf16, fp16 or fp32) after
    `steps` Newton-Schulz iterations with `coeffs` ((a, b, c), or a sequence of `steps` of them), in
    `dtype` (x's own if None).  Differentiable with respect to x, once and in reverse mode (an input
    with a forward-mode tangent is refused); without a gradient to come (no grad mode, an input that
    needs none) no iterates are kept.  Forward and backward can be captured in a CUDA graph; as for any
    backward pass, no graph of the same leaves made outside the capture may still be alive then.

    With the optimizer's coefficients the singular values of the result lie near 1 (0.7 to 1.2); a
    parametrisation that needs orthonormal blocks takes converging ones, such as (1.875, -1.25, 0.375).
    The iterates run on the tensor cores in fp16 with scales of their own (see ns_orthogonalize_stacks
    in the C header for the accuracy).  Long runs of the optimizer's iterations (more than 13, unless two
    or three converging ones follow) leave nothing of a gradient and are refused where one is to come."""
    coeffs = tuple(tuple(map(float, c)) if isinstance(c, (tuple, list)) else float(c) for c in coeffs)
    if forward_ad.unpack_dual(x).tangent is not None:
        raise NotImplementedError("orthogonalize has no forward-mode derivative")
    schedule, dtype = _schedule(coeffs, steps, eps), dtype if dtype is not None else x.dtype
    if torch.is_grad_enabled() and x.requires_grad:
        return _Orthogonalize.apply(x, schedule, dtype)
    y = torch.empty(x.shape, dtype=dtype, device=x.device)
    mb.orthogonalize_alloc([mb.Stack(_unit_last(x.detach()), y)], schedule)
    return y
