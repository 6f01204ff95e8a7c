"""The gradient of stacked-block orthogonalisation where its range runs out first.  References in 64 bits."""
import pytest
import torch

import stack_reference as ref
from matrix_orthogonalising_optimizer_02_b200 import binding as mb

pytestmark = pytest.mark.gpu

BF, FP = torch.bfloat16, torch.float32


def blocks(seed, count, rows, cols, dtype=FP, std=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn((count, rows, cols), generator=g, device="cuda") * std).to(dtype)


def gradient(x, dy, sch):
    """(output, gradient of the input, device status) through the C ABI's calls."""
    y, dx = torch.empty_like(x), torch.empty_like(x)
    stacks, grads = [mb.Stack(x, y)], [mb.Stack(dy, dx)]
    saved = mb.workspace(mb.ns_stacks_saved_size(stacks, sch))
    ws = mb.workspace(mb.ns_stacks_workspace_size(stacks, sch, True))
    mb.ns_orthogonalize_stacks(stacks, sch, ws, saved=saved)
    back = mb.workspace(mb.ns_stacks_backward_workspace_size(grads, sch))
    mb.ns_orthogonalize_stacks_backward(grads, sch, saved, back)
    return y, dx, mb.device_status(back)


@pytest.mark.parametrize("shape", [(2, 160, 300), (2, 300, 160), (2, 40, 300)], ids=str)
@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("size", [1e-30, 1e-36, 1e-39])
def test_gradients_that_have_nearly_died_out(shape, dtype, size):
    """Blocks of norm about `size` * 200, every third element exactly zero, the first block zero all over.  Values
    below 2^-126 lie at steps of 2^-149 (fp32) or 2^-133 (bf16): they are the call's input as they are, and an element
    of the result is rounded by half such a step, whose norm joins the tolerance."""
    x = blocks(1, *shape, dtype, std=1e-2)
    dy = blocks(2, *shape, FP) * size
    dy.view(-1)[::3] = 0
    dy[0] = 0
    dy = dy.to(dtype)
    coeffs = [ref.STABLE] * 5
    _, dx, status = gradient(x, dy, mb.Schedule(coeffs))
    assert status == mb.MUON_OK
    assert bool((dx[0] == 0).all())
    want = ref.ns_grad(x[1], dy[1], coeffs)
    step = 2.0 ** (-150 if dtype == FP else -134) * (shape[1] * shape[2]) ** 0.5
    assert float((dx[1].double() - want).norm()) <= ref.tol_stable(dtype) * float(want.norm()) + step
