"""The gradient of stacked-block orthogonalisation where its range runs out first: gradients that have nearly died out,
and schedules of many iterations.  References in 64 bits."""
import pytest
import torch

import stack_reference as ref
from matrix_orthogonalising_optimizer_02_b200 import binding as mb
from matrix_orthogonalising_optimizer_02_b200 import stacks as ms

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


def hybrid(n, last=2):
    return [ref.KJ] * n + [ref.STABLE] * last


# The optimizer's polynomial maps [0.68, 1.2] into itself; its |p'| is 1.55 there in the mean square: each iteration
# beyond the five of 2 tol_kj multiplies what earlier ones have rounded by 1.7 at most on average.  A converging
# iteration behind them has 0.23 there, and multiplies by 0.25.
def tol_long(n, last, dtype):
    return 2 * ref.tol_kj(dtype) * max(1.0, 1.7 ** (n - 5) * 0.25 ** last)


@pytest.mark.parametrize("shape", [(2, 160, 256), (1, 300, 200), (3, 96, 200), (2, 512, 768), (2, 64, 2100), (3, 200, 24)], ids=str)
@pytest.mark.parametrize("coeffs,tol", [
    ([ref.STABLE] * 10, ref.tol_stable(FP)), ([ref.STABLE] * 16, ref.tol_stable(FP)), ([ref.STABLE] * 32, ref.tol_stable(FP)),
    ([(2.0, -1.5, 0.5)] * 32, ref.tol_stable(FP)), (hybrid(8), tol_long(8, 2, FP)), (hybrid(12), tol_long(12, 2, FP)),
    ([ref.KJ] * 8, tol_long(8, 0, FP)), ([ref.KJ] * 10, tol_long(10, 0, FP))],
    ids=["stable10", "stable16", "stable32", "other32", "hybrid8", "hybrid12", "kj8", "kj10"])
def test_gradient_through_many_iterations(shape, coeffs, tol):
    """The derivative's bound grows by the largest |p'| every iteration, the gradient itself does not: what the planes
    hold has to follow the gradient.  Both directions are compared."""
    x, dy = blocks(3, *shape, std=0.5), blocks(4, *shape, std=1e-2)
    y, dx, status = gradient(x, dy, mb.Schedule(coeffs))
    assert status == mb.MUON_OK
    for b in range(shape[0]):
        assert ref.rel(y[b], ref.ns(x[b], coeffs)) <= tol, b
        assert ref.rel(dx[b], ref.ns_grad(x[b], dy[b], coeffs)) <= tol, b


@pytest.mark.parametrize("shape", [(4, 160, 256), (4, 96, 200)], ids=str)
def test_blocks_of_one_long_call_are_scaled_apart(shape):
    """Gradients of 1e-20 and 1e12, one along the smallest direction (which grows by a factor a every iteration), a zero
    one and one that is not finite, side by side."""
    coeffs = [ref.STABLE] * 24
    x, dy = blocks(5, *shape, std=0.5), blocks(6, *shape, std=1.0)
    u, s, v = torch.linalg.svd(x[1].double(), full_matrices=False)
    s = torch.logspace(0, -6, s.numel(), device="cuda", dtype=torch.float64)
    x[1] = ((u * s) @ v).float()
    dy[1] = torch.outer(u[:, -1], v[-1]).float()
    dy[0] *= 1e-20
    dy[2] *= 1e12
    dy[3, 1, 1] = float("inf")
    _, dx, status = gradient(x, dy, mb.Schedule(coeffs))
    assert status == mb.MUON_ERR_NONFINITE
    assert bool(torch.isnan(dx[3]).any())
    for b in (0, 2):
        assert ref.rel(dx[b], ref.ns_grad(x[b], dy[b], coeffs)) <= ref.tol_stable(FP), b
    assert bool(torch.isfinite(dx[1]).all())
    dy[0] = 0
    _, dx, _ = gradient(x, dy, mb.Schedule(coeffs))
    assert bool((dx[0] == 0).all())
    assert ref.rel(dx[2], ref.ns_grad(x[2], dy[2], coeffs)) <= ref.tol_stable(FP)


def test_a_schedule_without_a_gradient_is_refused_where_one_is_to_come():
    x = blocks(7, 2, 160, 200, std=0.5)
    with torch.no_grad():
        assert bool(torch.isfinite(ms.orthogonalize(x, steps=16)).all())
    with pytest.raises(mb.MuonError):
        ms.orthogonalize(x.requires_grad_(True), steps=16)
    (dx,) = torch.autograd.grad(ms.orthogonalize(x, steps=12), x, x.detach())
    assert bool(torch.isfinite(dx).all())


def test_gradients_of_many_classes_and_iterations():
    """More operations than one launch of a chain takes, and more classes; the scales carry over from launch to launch."""
    coeffs = [ref.STABLE] * 32
    shapes = [(1 + i % 2, 136 + 8 * i, 300 - 4 * i) for i in range(14)] + [(2, 20 + i, 50) for i in range(3)]
    xs, dys = [blocks(20 + i, *s, std=0.5) for i, s in enumerate(shapes)], [blocks(60 + i, *s) for i, s in enumerate(shapes)]
    ys, dxs = [torch.empty_like(x) for x in xs], [torch.empty_like(x) for x in xs]
    sch = mb.Schedule(coeffs)
    stacks, grads = [mb.Stack(*p) for p in zip(xs, ys)], [mb.Stack(*p) for p in zip(dys, dxs)]
    saved = mb.workspace(mb.ns_stacks_saved_size(stacks, sch))
    mb.ns_orthogonalize_stacks(stacks, sch, mb.workspace(mb.ns_stacks_workspace_size(stacks, sch, True)), saved=saved)
    back = mb.workspace(mb.ns_stacks_backward_workspace_size(grads, sch))
    mb.ns_orthogonalize_stacks_backward(grads, sch, saved, back)
    assert mb.device_status(back) == mb.MUON_OK
    for i, (x, y, dy, dx) in enumerate(zip(xs, ys, dys, dxs)):
        assert ref.rel(y[-1], ref.ns(x[-1], coeffs)) <= ref.tol_stable(FP), i
        assert ref.rel(dx[-1], ref.ns_grad(x[-1], dy[-1], coeffs)) <= ref.tol_stable(FP), i
