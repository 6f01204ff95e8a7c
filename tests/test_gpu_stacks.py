"""Stacked-block orthogonalisation, its gradient and the Muon step on stacks against 64 bits."""
import pytest
import torch

import stack_reference as ref
from matrix_orthogonalising_optimizer_02_b200 import binding as mb
from matrix_orthogonalising_optimizer_02_b200 import stacks as ms
from matrix_orthogonalising_optimizer_02_b200.optim import AdamW, StackedMuon, clip_scale

pytestmark = pytest.mark.gpu

BF, HF, FP = torch.bfloat16, torch.float16, torch.float32
T = 5


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def padded(count, rows, cols, pad, dtype, fill=7.0):
    """A [count, rows, cols] view whose rows lie `pad` elements further apart, and its buffer."""
    buf = torch.full((count, rows, cols + pad), fill, dtype=dtype, device="cuda")
    return buf[:, :, :cols], buf


def blocks(seed, count, rows, cols, dtype, std=1e-3):
    return (torch.randn((count, rows, cols), generator=gen(seed), device="cuda") * std).to(dtype)


def run(stacks, sch, saved=None, stream=None):
    ws = mb.workspace(mb.ns_stacks_workspace_size(stacks, sch, saved is not None))
    mb.ns_orthogonalize_stacks(stacks, sch, ws, saved=saved, stream=stream)
    return ws


SHAPES = [(1, 1, 1), (3, 1, 7), (2, 9, 1), (5, 13, 29), (4, 64, 768), (3, 100, 52), (2, 300, 520), (1, 257, 1000),
          (1, 1000, 257), (7, 128, 136), (2, 129, 640), (1, 64, 16384), (33, 8, 8), (1, 768, 768), (1, 530, 530)]


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("x_dtype,y_dtype,pad", [(BF, BF, 0), (FP, HF, 3), (HF, FP, 8)])
@pytest.mark.parametrize("coeffs,tol", [(ref.KJ, ref.tol_kj), (ref.STABLE, ref.tol_stable)], ids=["kj", "stable"])
def test_forward(shape, x_dtype, y_dtype, pad, coeffs, tol):
    x, _ = padded(*shape, pad, x_dtype)
    x.copy_(blocks(1, *shape, x_dtype))
    y, buf = padded(*shape, pad, y_dtype)
    ws = run([mb.Stack(x, y)], mb.Schedule.fixed(T, coeffs))
    assert mb.device_status(ws) == mb.MUON_OK
    for b in range(shape[0]):
        want = ref.ns(x[b], [coeffs] * T)
        most = ref.tol_vector([coeffs] * T, y_dtype) if min(shape[1:]) == 1 else tol(y_dtype)
        assert ref.rel(y[b], want) <= most, b
    if pad:
        assert bool((buf[:, :, shape[2]:] == 7.0).all())


def _gradient_like(seed, count, rows, cols, noise=0.0):
    """A falling spectrum (i^-0.7), or rank 16 with noise."""
    k = min(rows, cols)
    g = gen(seed)
    fall = torch.arange(1, k + 1, device="cuda", dtype=FP) ** -0.7
    if noise:
        fall = (torch.arange(k, device="cuda") < 16).float()
    u = torch.matmul(torch.randn((count, rows, k), generator=g, device="cuda") * fall,
                     torch.randn((count, k, cols), generator=g, device="cuda"))
    return u + noise * torch.randn(u.shape, generator=g, device="cuda")


@pytest.mark.parametrize("shape", [(3, 64, 768), (2, 512, 512), (1, 700, 300)], ids=str)
@pytest.mark.parametrize("noise", [0.0, 0.03])
def test_forward_keeps_small_singular_directions(shape, noise):
    """The term a X carries 22 bits, so blocks with tiny singular values hold the same tolerance;
    bf16 iterates are 2e-2 and 1e-1 off here."""
    x = _gradient_like(2, *shape, noise=noise)
    y = torch.empty_like(x)
    run([mb.Stack(x, y)], mb.Schedule.fixed(T, ref.KJ))
    for b in range(shape[0]):
        assert ref.rel(y[b], ref.ns(x[b], [ref.KJ] * T)) <= ref.tol_kj(FP), b


@pytest.mark.parametrize("rows,cols", [(40, 96), (300, 200)])
def test_a_block_does_not_touch_its_neighbours(rows, cols):
    x = blocks(3, 5, rows, cols, FP)
    x[1] = 0
    x[2, 0, 0] = float("nan")
    x[3, rows - 1, cols - 1] = float("inf")
    y = torch.empty_like(x)
    ws = run([mb.Stack(x, y)], mb.Schedule.fixed(T))
    assert mb.device_status(ws) == mb.MUON_ERR_NONFINITE
    assert mb.device_status(ws) == mb.MUON_OK     # read and cleared
    assert bool((y[1] == 0).all())
    assert bool(torch.isnan(y[2]).all()) and bool(torch.isnan(y[3]).all())
    for b in (0, 4):
        assert ref.rel(y[b], ref.ns(x[b], [ref.KJ] * T)) <= ref.tol_kj(FP)
    ws2 = run([mb.Stack(x[:1], y[:1])], mb.Schedule.fixed(T))
    assert mb.device_status(ws2) == mb.MUON_OK


@pytest.mark.parametrize("size", [1e-20, 1e-3, 1e18])
def test_any_magnitude(size):
    """Sums of squares are formed in fp64; with an eps far below the norm the result does not
    depend on the magnitude."""
    x = blocks(4, 2, 96, 200, FP, std=1.0) * size
    y = torch.empty_like(x)
    run([mb.Stack(x, y)], mb.Schedule.fixed(T, eps=1e-25))
    for b in range(2):
        assert ref.rel(y[b], ref.ns(x[b], [ref.KJ] * T, 1e-25)) <= ref.tol_kj(FP)


def test_one_huge_element():
    x = torch.zeros((1, 700, 900), device="cuda")
    x[0, 5, 6] = 3e4
    y = torch.empty_like(x)
    run([mb.Stack(x, y)], mb.Schedule.fixed(T))
    assert ref.rel(y[0], ref.ns(x[0], [ref.KJ] * T)) <= ref.tol_kj(FP)


def test_hybrid_schedule():
    sch = mb.Schedule.hybrid()
    x = _gradient_like(5, 2, 200, 333)
    y = torch.empty_like(x)
    run([mb.Stack(x, y)], sch)
    for b in range(2):   # ends with converging iterations: as for those
        assert ref.rel(y[b], ref.ns(x[b], sch.coeffs)) <= ref.tol_kj(FP)


def test_views_and_in_place():
    """Column blocks, interleaved rows, a repeated input, and an output that is the input."""
    coeffs = [ref.KJ] * T
    w = blocks(6, 1, 48, 3 * 40, BF)[0]
    cols, rows = ms.col_blocks(w, 40), w.view(16, 3, 120).transpose(0, 1)
    for v in (cols, rows):
        y = torch.empty(v.shape, dtype=FP, device="cuda")
        run([mb.Stack(v, y)], mb.Schedule.fixed(T))
        for b in range(3):
            assert ref.rel(y[b], ref.ns(v[b], coeffs)) <= ref.tol_kj(FP)
    one = blocks(7, 1, 33, 65, BF)
    y = torch.empty((4, 33, 65), dtype=BF, device="cuda")
    run([mb.Stack(one.expand(4, 33, 65), y)], mb.Schedule.fixed(T))
    assert all(torch.equal(y[b], y[0]) for b in range(4))
    for rc in ((3, 72, 128), (2, 31, 77)):
        x = blocks(8, *rc, BF)
        y = torch.empty_like(x)
        run([mb.Stack(x, y)], mb.Schedule.fixed(T))
        run([mb.Stack(x, x)], mb.Schedule.fixed(T))
        assert torch.equal(x, y)


def test_many_stacks_in_one_call():
    """More shapes than one launch holds, several stacks of one shape, mixed types; each equals a call
    of its own."""
    shapes = [(1 + i % 3, 8 + 5 * i, 16 + 3 * i) for i in range(20)] + [(2, 24, 40)] * 150
    st = [mb.Stack(blocks(20 + i, *s, (BF, HF, FP)[i % 3]), torch.empty(s, dtype=(HF, FP, BF)[i % 3], device="cuda"))
          for i, s in enumerate(shapes)]
    ws = run(st, mb.Schedule.fixed(T))
    assert mb.device_status(ws) == mb.MUON_OK
    for i, s in enumerate(st):
        y = torch.empty_like(s.Y)
        run([mb.Stack(s.X, y)], mb.Schedule.fixed(T))
        assert ref.rel(s.Y, y) <= 2 * ref.half_step(y.dtype), i   # a 16-bit result may be rounded twice
        assert ref.rel(s.Y[0], ref.ns(s.X[0], [ref.KJ] * T)) <= ref.tol_kj(y.dtype), i


@pytest.mark.parametrize("shape", [(2, 1, 1), (3, 1, 9), (2, 11, 5), (4, 64, 200), (2, 96, 641), (1, 300, 130),
                                   (2, 256, 256), (1, 520, 1032)], ids=str)
@pytest.mark.parametrize("dtype", [BF, FP])
def test_gradient(shape, dtype):
    """Against the formulas in 64 bits (which a CPU test holds against differences)."""
    x = blocks(9, *shape, dtype, std=0.5)
    dy = blocks(10, *shape, dtype, std=1e-2)
    coeffs = [ref.STABLE] * T
    leaf = x.clone().requires_grad_(True)
    y = ms.orthogonalize(leaf, steps=T, coeffs=ref.STABLE)
    (dx,) = torch.autograd.grad(y, leaf, dy)
    assert dx.dtype == dtype and y.dtype == dtype
    for b in range(shape[0]):
        want = ref.ns_grad(x[b], dy[b], coeffs)
        assert ref.rel(y[b], ref.ns(x[b], coeffs)) <= ref.tol_stable(dtype)
        if min(shape[1:]) == 1:
            # a vector's direction alone survives: with sigma = 1 the radial part cancels, so the error
            # counts against the parts that cancel, |dy| (max |p'|)^T / N <= 1.9^5 |dy| / N
            n = float(x[b].double().norm())
            bound = 1.9 ** 5 * float(dy[b].double().norm()) / n * ref.tol_stable(dtype)
            assert float((dx[b].double() - want).norm()) <= bound
        else:
            assert ref.rel(dx[b], want) <= ref.tol_stable(dtype)


def test_gradient_with_the_optimizers_schedule_and_magnitudes():
    """The derivative of the optimizer's polynomial neither grows nor shrinks evenly; the backward
    reads A, B and X in fp16, so twice the forward's tolerance stands.  Gradients of 1e-12 and 1e6."""
    for size in (1e-12, 1.0, 1e6):
        x, dy = blocks(11, 2, 120, 264, FP), blocks(12, 2, 120, 264, FP, std=1.0) * size
        leaf = x.clone().requires_grad_(True)
        (dx,) = torch.autograd.grad(ms.orthogonalize(leaf), leaf, dy)
        for b in range(2):
            assert ref.rel(dx[b], ref.ns_grad(x[b], dy[b], [ref.KJ] * T)) <= 2 * ref.tol_kj(FP)


def test_gradient_aligned_with_the_smallest_direction():
    """The largest growth: a rank-one gradient along a tiny singular direction stays in range."""
    u, s, v = torch.linalg.svd(torch.randn((64, 96), generator=gen(13), device="cuda", dtype=torch.float64))
    s = torch.logspace(0, -3, 64, device="cuda", dtype=torch.float64)
    x = (u * s) @ v[:64]
    dy = torch.outer(u[:, -1], v[63])
    leaf = x.float()[None].requires_grad_(True)
    (dx,) = torch.autograd.grad(ms.orthogonalize(leaf), leaf, dy.float()[None])
    assert ref.rel(dx[0], ref.ns_grad(x.float(), dy.float(), [ref.KJ] * T)) <= 2 * ref.tol_kj(FP)


def test_gradient_special_blocks():
    x = blocks(14, 4, 24, 40, FP)
    x[1] = 0
    dy = blocks(15, 4, 24, 40, FP)
    dy[2] = 0
    dy[3, 0, 0] = float("nan")
    leaf = x.clone().requires_grad_(True)
    (dx,) = torch.autograd.grad(ms.orthogonalize(leaf, coeffs=ref.STABLE, eps=1e-3), leaf, dy)
    want = [ref.ns_grad(x[b], dy[b], [ref.STABLE] * T, 1e-3) for b in range(4)]
    assert ref.rel(dx[0], want[0]) <= ref.tol_stable(FP)
    assert ref.rel(dx[1], want[1]) <= ref.tol_stable(FP)
    assert bool((dx[2] == 0).all()) and bool(torch.isnan(dx[3]).all())


def test_gradient_of_broadcast_and_strided():
    """One block shared by several uses, a strided input, and an output gradient without strides."""
    x = blocks(16, 1, 40, 56, FP, std=0.1)[0]
    leaf = x.clone().requires_grad_(True)
    y = ms.orthogonalize(leaf.expand(3, 40, 56), coeffs=ref.STABLE)
    dy = blocks(17, 3, 40, 56, FP)
    y.backward(dy)
    want = sum(ref.ns_grad(x, dy[b], [ref.STABLE] * T) for b in range(3))
    assert ref.rel(leaf.grad, want) <= 3 * ref.tol_stable(FP)
    fused = blocks(18, 1, 40, 112, BF, std=0.1)[0].clone().requires_grad_(True)
    ms.orthogonalize(ms.col_blocks(fused, 56), coeffs=ref.STABLE).sum().backward()
    for b in range(2):
        part = fused.detach()[:, 56 * b:56 * (b + 1)]
        want = ref.ns_grad(part, torch.ones_like(part), [ref.STABLE] * T)
        assert ref.rel(fused.grad[:, 56 * b:56 * (b + 1)], want) <= ref.tol_stable(BF)


def muon_stack(seed, count, rows, cols, pad, w_dtype=BF, g_dtype=BF):
    w, wb = padded(count, rows, cols, pad, w_dtype)
    g, _ = padded(count, rows, cols, pad + 1 if pad else 0, g_dtype)
    m, mbuf = padded(count, rows, cols, pad, FP)
    w.copy_(blocks(seed, count, rows, cols, w_dtype, 0.02))
    g.copy_(blocks(seed + 1, count, rows, cols, g_dtype, 1e-3))
    m.copy_(blocks(seed + 2, count, rows, cols, FP, 1e-2))
    return mb.MuonStack(w, g, m), (wb, mbuf)


@pytest.mark.parametrize("w_dtype,g_dtype,pad,nesterov,mode", [
    (BF, BF, 0, True, "moonlight"), (FP, HF, 5, False, "kellerjordan"), (HF, FP, 8, True, "mup"),
    (BF, FP, 1, False, "naive")])
def test_muon_step(w_dtype, g_dtype, pad, nesterov, mode):
    lr, beta, wd, gs = 0.02, 0.95, 0.1, 0.37
    shapes = [(3, 64, 200), (2, 257, 130), (1, 31, 31), (2, 64, 200)]
    st, bufs = zip(*(muon_stack(30 + 3 * i, *s, pad, w_dtype, g_dtype) for i, s in enumerate(shapes)))
    st[0].G[1] = 0
    st[0].M[1] = 0
    old = [(s.W.clone(), s.M.clone()) for s in st]
    hp = mb.hyper(lr, beta, wd, nesterov, mode)
    ws = mb.workspace(mb.muon_stacks_workspace_size(st, hp))
    mb.muon_step_stacks(st, hp, ws, grad_scale=torch.tensor([gs], device="cuda"))
    assert mb.device_status(ws) == mb.MUON_OK
    f = lambda x: float(torch.tensor(x, dtype=FP))  # noqa: E731  the call takes fp32 factors
    for s, (w0, m0), (wb, mbuf) in zip(st, old, bufs):
        for b in range(s.W.shape[0]):
            w, m, o = ref.muon(w0[b], s.G[b], m0[b], f(lr), f(beta), f(wd), nesterov, mode, [ref.KJ] * T, gs=f(gs))
            # M: the product with the scale and the fused multiply-add round once each
            assert bool(((s.M[b].double() - m).abs() <= 2.0 ** -23 * (m0[b].abs() + s.G[b].float().abs())).all())
            # W: the chain's error in O times the step, and the rounding of W (two in fp32 before it)
            step = lr * ref.scale(*w.shape, mode)
            bound = step * ref.tol_kj(FP) * o.norm() + (ref.half_step(w_dtype) + 2.0 ** -23) * w.norm() + 1e-12
            assert float((s.W[b].double() - w).norm()) <= float(bound)
        if pad:
            assert bool((wb[:, :, s.W.shape[2]:] == 7.0).all()) and bool((mbuf[:, :, s.W.shape[2]:] == 7.0).all())
    idle = (1 - f(lr) * f(wd)) * old[0][0][1].double()
    err = (st[0].W[1].double() - idle).abs()
    assert bool((err <= (ref.half_step(w_dtype) * 1.01 + 2.0 ** -23) * idle.abs() + 2.0 ** -25).all())


def test_bad_gradient_scale_reaches_every_block():
    st, _ = muon_stack(40, 2, 16, 24, 0)
    hp = mb.hyper(0.02)
    ws = mb.workspace(mb.muon_stacks_workspace_size([st], hp))
    mb.muon_step_stacks([st], hp, ws, grad_scale=torch.tensor([float("nan")], device="cuda"))
    assert mb.device_status(ws) == mb.MUON_ERR_NONFINITE
    assert bool(torch.isnan(st.W.float()).all())


def test_graphs_that_share_a_workspace_and_streams():
    """A call is captured without a call before it; two graphs that share a workspace replay in turn
    and equal eager calls bitwise; two streams run calls side by side in workspaces of their own."""
    sch = mb.Schedule.fixed(T)
    xs = [blocks(50 + i, 3, 40, 100 + 8 * i, BF) for i in range(2)]
    ys = [torch.zeros_like(x) for x in xs]
    ws = mb.workspace(max(mb.ns_stacks_workspace_size([mb.Stack(x, y)], sch) for x, y in zip(xs, ys)))
    graphs = []
    for x, y in zip(xs, ys):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            mb.ns_orthogonalize_stacks([mb.Stack(x, y)], sch, ws)
        graphs.append(g)
    want = [torch.empty_like(y) for y in ys]
    for seed in (60, 61):
        for i, x in enumerate(xs):
            x.copy_(blocks(seed + 10 * i, *x.shape, BF))
            run([mb.Stack(x, want[i])], sch)
        for g in graphs + graphs[::-1]:
            g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(ys, want))
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for y in ys:
        y.zero_()
    torch.cuda.synchronize()
    keep = [run([mb.Stack(x, y)], sch, stream=s) for x, y, s in zip(xs, ys, streams)]
    torch.cuda.synchronize()
    assert len(keep) == 2 and all(torch.equal(a, b) for a, b in zip(ys, want))


def test_repeatable():
    x = blocks(70, 4, 130, 300, FP)
    out = []
    for _ in range(3):
        leaf = x.clone().requires_grad_(True)
        y = ms.orthogonalize(leaf)
        (dx,) = torch.autograd.grad(y, leaf, x)
        out.append((y.detach(), dx))
    assert all(torch.equal(a, b) for o in out[1:] for a, b in zip(out[0], o))


@pytest.mark.parametrize("sizes", [[1], [7, 8, 9], [4096, 4097, 100003], [0, 5, 0], [3] * 700])
@pytest.mark.parametrize("g_dtype,w_dtype,off", [(BF, BF, 0), (HF, FP, 1), (FP, HF, 3)])
def test_norm_and_adamw(sizes, g_dtype, w_dtype, off):
    def flat(seed, n, dtype, std):   # tensors that begin `off` elements into a buffer
        return (torch.randn(n + off, generator=gen(seed), device="cuda") * std).to(dtype)[off:]
    ts = [mb.AdamWTensor(flat(4 * i, n, w_dtype, 0.1), flat(4 * i + 1, n, g_dtype, 1.0),
                         flat(4 * i + 2, n, FP, 0.1), flat(4 * i + 3, n, FP, 0.1).square_()) for i, n in enumerate(sizes)]
    grads = [t.G for t in ts]
    out = torch.empty(2, device="cuda")
    ws = mb.workspace(mb.grad_norm_workspace_size(grads))
    mb.grad_norm_batched(grads, 0.5, out, ws)
    assert mb.device_status(ws) == mb.MUON_OK
    norm = torch.cat([g.double() for g in grads]).norm()
    # fp64 sums: only the roundings of the two results to fp32
    assert abs(float(out[0]) - float(norm)) <= 2.0 ** -23 * float(norm)
    assert abs(float(out[1]) - min(1.0, 0.5 / (float(norm) + 1e-6))) <= 2.0 ** -23
    h = dict(lr=1e-2, beta1=0.9, beta2=0.95, eps=1e-8, weight_decay=0.1)
    old = [(t.W.clone(), t.m.clone(), t.v.clone()) for t in ts]
    mb.adamw_step_batched(ts, mb.adamw_hyper(**h), 7, grad_scale=out[1:])
    for t, (w0, m0, v0) in zip(ts, old):
        w, m, v = ref.adamw(w0, t.G, m0, v0, 7, 1e-2, 0.9, 0.95, 1e-8, 0.1, gs=float(out[1]))
        g = t.G.double().abs() * float(out[1])
        # m, v: factors and products in fp32, at most 4 and 6 roundings of 2^-24 of the larger term
        assert bool(((t.m.double() - m).abs() <= 4 * 2.0 ** -24 * (m0.double().abs() + g)).all())
        assert bool(((t.v.double() - v).abs() <= 6 * 2.0 ** -24 * (v0.double() + g * g)).all())
        # W: m's error (cancellation included), v's, a square root, a division and the factors: 16
        # roundings of 2^-24 of u's size taken without cancellation, and W's own rounding (fp16 has
        # values below 2^-14 at a fixed step)
        size = ((m0.double().abs() + g) / (1 - 0.9 ** 7)) / (torch.sqrt(v / (1 - 0.95 ** 7)) + 1e-8)
        bound = 16 * 2.0 ** -24 * (1e-2 * size + w0.double().abs()) + ref.half_step(w_dtype) * w.abs() * 1.01 + 2.0 ** -25
        assert bool(((t.W.double() - w).abs() <= bound).all())


def test_norm_special_values():
    big = [torch.full((5000,), 1e30, device="cuda"), torch.full((3,), 1e-30, device="cuda")]
    out = torch.empty(2, device="cuda")
    ws = mb.workspace(mb.grad_norm_workspace_size(big))
    mb.grad_norm_batched(big, 1.0, out, ws)
    assert abs(float(out[0]) / (1e30 * 5000 ** 0.5) - 1) <= 1e-6
    mb.grad_norm_batched(big[1:], 1.0, out, ws)
    assert float(out[1]) == 1.0 and float(out[0]) > 0
    big[0][17] = float("nan")
    mb.grad_norm_batched(big, 1.0, out, ws)
    assert bool(torch.isnan(out).all()) and mb.device_status(ws) == mb.MUON_ERR_NONFINITE
    big[0][17] = float("inf")
    mb.grad_norm_batched(big, 1.0, out, ws)
    assert float(out[0]) == float("inf") and float(out[1]) == 0.0
    empty = [torch.empty(0, device="cuda")]
    mb.grad_norm_batched(empty, 1.0, out, mb.workspace(mb.grad_norm_workspace_size(empty)))
    assert float(out[0]) == 0.0 and float(out[1]) == 1.0


def test_adamw_captured_steps_advance():
    """A captured step reads its number on the device: replays equal eager steps."""
    def make():
        return [mb.AdamWTensor(blocks(80, 1, 1, 1000, BF)[0, 0].clone(), blocks(81, 1, 1, 1000, BF)[0, 0],
                               torch.zeros(1000, device="cuda"), torch.zeros(1000, device="cuda"))]
    a, b = make(), make()
    hp = mb.adamw_hyper(lr=1e-2)
    step = torch.zeros(1, dtype=torch.int64, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step += 1
        mb.adamw_step_batched(a, hp, step)
    for t in range(1, 5):
        g.replay()
        mb.adamw_step_batched(b, hp, t)
    torch.cuda.synchronize()
    assert int(step) == 4
    # the corrections come from pow() on either side: each within an ulp or two of fp32
    assert torch.equal(a[0].m, b[0].m) and torch.equal(a[0].v, b[0].v)
    assert ref.rel(a[0].W, b[0].W) <= ref.half_step(BF)


class _Tiny(torch.nn.Module):
    """Embedding, a fused QKV whose heads are blocks, a stack of experts, a bias, a head with orthonormal
    rows by parametrisation."""

    def __init__(self):
        super().__init__()
        g = torch.Generator().manual_seed(0)
        r = lambda *s: torch.nn.Parameter(torch.randn(s, generator=g) * 0.1)  # noqa: E731
        self.emb, self.qkv, self.experts, self.bias, self.head = r(50, 24), r(3 * 24, 24), r(2, 40, 24), r(40), r(13, 40)

    def forward(self, tokens, orth):
        x = self.emb[tokens]
        q, k, v = (x @ self.qkv.T).chunk(3, dim=-1)
        x = torch.softmax(q @ k.transpose(-1, -2), dim=-1) @ v
        x = torch.stack([x @ e.T for e in self.experts]).sum(0) + self.bias
        return (torch.tanh(x) @ orth(self.head).T).square().mean()


def test_a_training_step_of_all_of_them():
    """Forward and backward through the orthogonalised head, the norm over all gradients, Muon on the
    blocks and AdamW on the rest, against the same in 64 bits."""
    model, twin = _Tiny().cuda(), _Tiny().double().cuda()
    tokens = torch.randint(0, 50, (2, 9), generator=torch.Generator().manual_seed(1)).cuda()
    muon = StackedMuon([{"params": [model.qkv], "row_block": 8}, {"params": [model.experts]}], lr=0.02, weight_decay=0.1)
    adam = AdamW([model.emb, model.bias, model.head], lr=1e-2, betas=(0.9, 0.95))
    state = {n: [torch.zeros_like(p), torch.zeros_like(p)] for n, p in twin.named_parameters()}

    def orth64(p):
        u = p / (torch.linalg.vector_norm(p) + 1e-7)
        for _ in range(T):
            a, b, c = ref.STABLE
            m = u @ u.T
            u = a * u + (b * m + c * m @ m) @ u
        return u
    for t in (1, 2):
        with torch.no_grad():   # steps do not compound: each starts from the first side's weights
            for p, q in zip(model.parameters(), twin.parameters()):
                q.copy_(p)
        for m in (model, twin):
            m.zero_grad()
        model(tokens, lambda p: ms.orthogonalize(p, coeffs=ref.STABLE)).backward()
        twin(tokens, orth64).backward()
        for (n, p), q in zip(model.named_parameters(), twin.parameters()):
            # the loss is smooth and its other parts run in fp32: the head's error, 2 tol_stable, reaches
            # every gradient once
            assert ref.rel(p.grad, q.grad) <= 2 * ref.tol_stable(FP) + 1e-5, n
        out = clip_scale(model.parameters(), 0.01)
        norm = torch.cat([p.grad.double().flatten() for p in model.parameters()]).norm()
        assert abs(float(out[0]) / float(norm) - 1) <= 2.0 ** -22
        gs = min(1.0, 0.01 / (float(norm) + 1e-6))
        old = {n: p.detach().clone() for n, p in model.named_parameters()}
        muon.step(grad_scale=out[1:])
        adam.step(grad_scale=out[1:])
        for n, p in model.named_parameters():
            s = state[n]
            if n in ("qkv", "experts"):
                cut = (lambda x: x.unflatten(0, (9, 8))) if n == "qkv" else (lambda x: x)
                for b in range(cut(p).shape[0]):
                    w, m, o = ref.muon(cut(old[n])[b], cut(p.grad)[b], cut(s[0])[b], 0.02, 0.95, 0.1, True, "moonlight",
                                       [ref.KJ] * T, gs=gs)
                    step = 0.02 * ref.scale(*w.shape, "moonlight")
                    err = float((cut(p.detach())[b].double() - w).norm())
                    assert err <= 2 * step * ref.tol_kj(FP) * float(o.norm()) + 1e-6 * float(w.norm()), (n, b)
                    cut(s[0])[b] = m
            else:
                w, m, v = ref.adamw(old[n], p.grad, s[0], s[1], t, 1e-2, 0.9, 0.95, 1e-8, 0.01, gs=gs)
                assert ref.rel(p, w) <= 1e-5, n
                s[0], s[1] = m, v


# ---------------------------------------------------------------- how calls are made
_FRESH = """
import torch
from matrix_orthogonalising_optimizer_02_b200 import binding as mb, stacks as ms
x = torch.randn({shape}, device="cuda")
dy = torch.randn_like(x)
leaf = x.clone().requires_grad_(True)
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    y = ms.orthogonalize(leaf)
    (dx,) = torch.autograd.grad(y, leaf, dy)
for seed in range(3):
    with torch.no_grad():
        leaf.copy_(torch.randn_like(x))
    g.replay()
    torch.cuda.synchronize()
    got = y.detach().clone(), dx.clone()
    twin = leaf.detach().clone().requires_grad_(True)
    z = ms.orthogonalize(twin)
    (dz,) = torch.autograd.grad(z, twin, dy)
    assert torch.equal(got[0], z.detach()) and torch.equal(got[1], dz)
print("equal")
"""


@pytest.mark.parametrize("shape", [(2, 300, 200), (3, 64, 400), (2, 200, 64)], ids=str)
def test_first_call_of_a_process_is_a_captured_forward_and_backward(shape):
    import pathlib
    import subprocess
    import sys
    out = subprocess.run([sys.executable, "-c", _FRESH.format(shape=shape)], capture_output=True, text=True, timeout=300,
                         cwd=pathlib.Path(__file__).resolve().parents[1])
    assert out.returncode == 0 and "equal" in out.stdout, out.stderr[-2000:]


def test_streams_run_chains_side_by_side():
    """Two streams, several calls each, workspaces of their own; each equals the call alone."""
    sch = mb.Schedule.fixed(T)
    xs = [blocks(90 + i, 4, 320, 400 + 64 * i, BF) for i in range(2)]
    want = [torch.empty_like(x) for x in xs]
    for x, y in zip(xs, want):
        run([mb.Stack(x, y)], sch)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in xs]
    ys = [[torch.empty_like(x) for _ in range(6)] for x in xs]
    torch.cuda.synchronize()
    keep = [run([mb.Stack(xs[i], ys[i][k])], sch, stream=streams[i]) for k in range(6) for i in range(2)]
    torch.cuda.synchronize()
    assert all(mb.device_status(ws) == mb.MUON_OK for ws in keep)
    assert all(torch.equal(y, w) for per, w in zip(ys, want) for y in per)


def test_backward_twice_and_many_graphs_alive():
    x = blocks(100, 3, 150, 222, FP).requires_grad_(True)
    dy = [blocks(101 + i, 3, 150, 222, FP, std=1.0) for i in range(2)]
    ys = [ms.orthogonalize(x) for _ in range(2)]
    first = [torch.autograd.grad(y, x, d, retain_graph=True)[0] for y, d in zip(ys, dy)]
    again = [torch.autograd.grad(y, x, d)[0] for y, d in zip(ys, dy)]
    assert all(torch.equal(a, b) for a, b in zip(first, again))
    assert ref.rel(first[1][2], ref.ns_grad(x[2].detach(), dy[1][2], [ref.KJ] * T)) <= 2 * ref.tol_kj(FP)


def test_no_iterates_are_kept_without_a_gradient(monkeypatch):
    kept, call = [], mb.orthogonalize_alloc
    monkeypatch.setattr(mb, "orthogonalize_alloc", lambda s, sch, keep=False: kept.append(keep) or call(s, sch, keep))
    x = blocks(110, 2, 40, 60, FP).requires_grad_(True)
    y = ms.orthogonalize(x)
    with torch.no_grad():
        z = ms.orthogonalize(x)
    w = ms.orthogonalize(x.detach())
    assert kept == [True, False, False] and y.requires_grad and not z.requires_grad and not w.requires_grad
    for v in (y, z, w):
        assert ref.rel(v[1], ref.ns(x[1].detach(), [ref.KJ] * T)) <= ref.tol_kj(FP)


def test_many_classes_and_iterations():
    """More classes than one launch of a chain takes, and more operations."""
    shapes = [(1, 136 + 8 * i, 300 - 4 * i) for i in range(14)] + [(2, 20 + i, 50) for i in range(3)]
    coeffs = [ref.STABLE] * 32
    xs = [blocks(120 + i, *s, FP) for i, s in enumerate(shapes)]
    ys = [torch.empty_like(x) for x in xs]
    run([mb.Stack(x, y) for x, y in zip(xs, ys)], mb.Schedule(coeffs))
    for x, y in zip(xs, ys):   # converging iterations: the last ones contract what went before
        assert ref.rel(y[-1], ref.ns(x[-1], coeffs)) <= ref.tol_stable(FP)


def test_many_stacks_of_longer_sides():
    """More stacks than one launch of a pass takes, through every pass."""
    n = 135
    x = blocks(140, n, 136, 144, FP)
    xs = [x[i:i + 1] for i in range(n)]
    dy = blocks(141, n, 136, 144, FP, std=1.0)
    ys, dx = [torch.empty_like(v) for v in xs], [torch.empty_like(v) for v in xs]
    sch = mb.Schedule.fixed(T)
    stacks = [mb.Stack(a, b) for a, b in zip(xs, ys)]
    saved = mb.workspace(mb.ns_stacks_saved_size(stacks, sch))
    run(stacks, sch, saved=saved)
    grads = [mb.Stack(dy[i:i + 1], dx[i]) for i in range(n)]
    ws = mb.workspace(mb.ns_stacks_backward_workspace_size(grads, sch))
    mb.ns_orthogonalize_stacks_backward(grads, sch, saved, ws)
    w = [torch.zeros_like(v) for v in xs]
    hp = mb.hyper(1.0, 0.0, 0.0, False, "naive", sch)
    muon = [mb.MuonStack(a, b, torch.zeros_like(b)) for a, b in zip(w, xs)]
    mb.muon_step_stacks(muon, hp, mb.workspace(mb.muon_stacks_workspace_size(muon, hp)))
    for i in (0, 63, 127, 128, 134):
        want = ref.ns(x[i], [ref.KJ] * T)
        assert ref.rel(ys[i][0], want) <= ref.tol_kj(FP), i
        assert ref.rel(-w[i][0], want) <= ref.tol_kj(FP), i
        assert ref.rel(dx[i][0], ref.ns_grad(x[i], dy[i], [ref.KJ] * T)) <= 2 * ref.tol_kj(FP), i


@pytest.mark.parametrize("rows,cols", [(40, 96), (150, 200)])
def test_offsets_beyond_32_bits(rows, cols):
    """Blocks, and rows, that lie further apart than 2^32 bytes or 2^31 elements reach."""
    far = 2 ** 32 + 24
    buf = torch.empty(far + rows * cols, dtype=BF, device="cuda")
    x = buf.as_strided((2, rows, cols), (far, cols, 1))
    x.copy_(blocks(150, 2, rows, cols, BF))
    y = torch.empty((2, rows, cols), device="cuda")
    run([mb.Stack(x, y)], mb.Schedule.fixed(T))
    want = [ref.ns(b, [ref.KJ] * T) for b in x]
    assert all(ref.rel(a, b) <= ref.tol_kj(FP) for a, b in zip(y, want))
    run([mb.Stack(x, x)], mb.Schedule.fixed(T))
    assert all(ref.rel(a, b) <= ref.tol_kj(BF) for a, b in zip(x, want))
    pitch = 2 ** 32 // (rows - 1) & ~7       # the last row begins beyond 2^31 elements
    z = buf.as_strided((rows, cols), (pitch, 1))
    z.copy_(blocks(151, 1, rows, cols, BF)[0])
    y = torch.empty((rows, cols), device="cuda")
    run([mb.Stack(z, y)], mb.Schedule.fixed(T))
    assert ref.rel(y, ref.ns(z, [ref.KJ] * T)) <= ref.tol_kj(FP)


def test_more_blocks_than_a_group_takes():
    """The call goes through its blocks in groups of some 5 GiB of workspace."""
    n = 9000
    x = blocks(160, n, 200, 264, BF)
    y = torch.empty_like(x)
    ws = run([mb.Stack(x, y)], mb.Schedule.fixed(T))
    assert ws.numel() < 6 * 2 ** 30 and mb.device_status(ws) == mb.MUON_OK
    for b in list(range(0, n, 1500)) + [n - 1]:
        assert ref.rel(y[b], ref.ns(x[b], [ref.KJ] * T)) <= ref.tol_kj(BF), b
    # every block was done: none is left as it was allocated, and all have a full block's norm
    norms = torch.linalg.vector_norm(y.float(), dim=(1, 2))
    assert float(norms.min()) > 0.6 * 200 ** 0.5 and float(norms.max()) < 1.3 * 200 ** 0.5


def test_a_tensor_beyond_31_bits_of_elements():
    n = 2 ** 31 + 9
    w, g = torch.zeros(n, dtype=BF, device="cuda"), torch.zeros(n, dtype=BF, device="cuda")
    m, v = torch.zeros(n, device="cuda"), torch.zeros(n, device="cuda")
    g[-5:] = 3.0
    g[:4] = 4.0
    out = torch.empty(2, device="cuda")
    mb.grad_norm_batched([g], 1.0, out, mb.workspace(mb.grad_norm_workspace_size([g])))
    assert abs(float(out[0]) - 109 ** 0.5) <= 2.0 ** -22 * 109 ** 0.5
    mb.adamw_step_batched([mb.AdamWTensor(w, g, m, v)], mb.adamw_hyper(lr=0.5, weight_decay=0.0), 1)
    # the first step moves every element with a gradient by lr
    assert bool((w[:4] == -0.5).all()) and bool((w[-5:] == -0.5).all()) and float(w.float().sum()) == -4.5


def test_optimizers_carry_their_state_in_fp32():
    """State dicts, and copies, of bf16 parameters' optimizers go on as the original does."""
    import copy
    p = [torch.nn.Parameter(blocks(170, 2, 24, 40, BF, std=0.1)), torch.nn.Parameter(blocks(171, 1, 5, 7, BF, std=0.1)[0])]
    q = [torch.nn.Parameter(x.detach().clone()) for x in p]

    def make(x):
        return StackedMuon(x[:1], lr=0.02), AdamW(x[1:], lr=1e-2)

    def step(x, opts, seed):
        for i, t in enumerate(x):
            t.grad = blocks(seed + i, *t.shape, BF) if t.dim() == 3 else blocks(seed + i, 1, *t.shape, BF)[0]
        for o in opts:
            o.step()
    a, b = make(p), make(q)
    step(p, a, 180)
    for x, y in zip(p, q):
        y.data.copy_(x.data)
    for o, n in zip(a, b):
        n.load_state_dict(copy.deepcopy(o.state_dict()))
        assert all(v.dtype == FP for s in n.state.values() for v in s.values() if torch.is_tensor(v))
    step(p, a, 190)
    step(q, b, 190)
    assert all(torch.equal(x, y) for x, y in zip(p, q))
    twin = copy.deepcopy(a[0])
    for t in twin.param_groups[0]["params"]:
        t.grad = blocks(200, 2, 24, 40, BF)
    twin.step()


@pytest.mark.parametrize("shape", [(5, 128, 256), (3, 128, 1024), (2, 120, 2048), (2, 128, 2049), (40, 96, 641), (16, 64, 768),
                                   (9, 7, 500), (200, 24, 40), (1, 128, 128), (6, 2048, 64), (2, 2049, 100), (20, 641, 96),
                                   (4, 300, 7), (3, 777, 128)], ids=str)
@pytest.mark.parametrize("dtype,pad", [(HF, 0), (FP, 3), (BF, 8)])
@pytest.mark.parametrize("coeffs,tol", [(ref.KJ, lambda t: 2 * ref.tol_kj(t)), (ref.STABLE, ref.tol_stable)],
                         ids=["kj", "stable"])
def test_gradient_of_short_sides(shape, dtype, pad, coeffs, tol):
    """Blocks whose short side is at most 128, of every cluster size, on either side of the longest slab; arrays
    with and without whole 16-byte rows.  Tolerances as above."""
    count = shape[0]
    x, dy = blocks(210, *shape, dtype, std=0.5), blocks(211, *shape, FP, std=1e-2)
    dy = dy.to(dtype)
    leaf, buf = padded(*shape, pad, dtype)
    leaf.copy_(x)
    dyv, _ = padded(*shape, pad, dtype)
    dyv.copy_(dy)
    dx, out = padded(*shape, pad, dtype)
    sch = mb.Schedule.fixed(T, coeffs)
    y = torch.empty_like(x)
    stacks, grads = [mb.Stack(leaf, y)], [mb.Stack(dyv, dx)]
    saved = mb.workspace(mb.ns_stacks_saved_size(stacks, sch))
    run(stacks, sch, saved=saved)
    ws = mb.workspace(mb.ns_stacks_backward_workspace_size(grads, sch))
    mb.ns_orthogonalize_stacks_backward(grads, sch, saved, ws)
    assert mb.device_status(ws) == mb.MUON_OK
    for b in sorted({0, 1 % count, count // 2, count - 1}):
        assert ref.rel(dx[b], ref.ns_grad(x[b], dy[b], [coeffs] * T)) <= tol(dtype), b
    if pad:
        assert bool((out[:, :, shape[2]:] == 7.0).all())


def test_gradient_of_short_sides_at_any_magnitude():
    """Gradients from 1e-30 to 1e30, a zero gradient, and one that is not finite, side by side."""
    x = blocks(212, 5, 40, 300, FP, std=0.5)
    dy = blocks(213, 5, 40, 300, FP, std=1.0)
    dy[0] *= 1e-30
    dy[1] *= 1e30
    dy[2] = 0
    dy[3, 39, 299] = float("inf")
    sch = mb.Schedule.fixed(T)
    dx = torch.empty_like(x)
    stacks, grads = [mb.Stack(x, torch.empty_like(x))], [mb.Stack(dy, dx)]
    saved = mb.workspace(mb.ns_stacks_saved_size(stacks, sch))
    run(stacks, sch, saved=saved)
    ws = mb.workspace(mb.ns_stacks_backward_workspace_size(grads, sch))
    mb.ns_orthogonalize_stacks_backward(grads, sch, saved, ws)
    assert mb.device_status(ws) == mb.MUON_ERR_NONFINITE
    assert bool((dx[2] == 0).all()) and bool(torch.isnan(dx[3]).any())
    for b in (0, 1, 4):
        assert ref.rel(dx[b], ref.ns_grad(x[b], dy[b], [ref.KJ] * T)) <= 2 * ref.tol_kj(FP), b


@pytest.mark.parametrize("dtype", [BF, HF, FP])
def test_norm_of_long_tensors(dtype):
    """Whole chunks: runs of zeros, values whose squares leave fp32's range, an infinity."""
    n = 5 * 4096 + 17
    g = blocks(220, 1, 1, n, dtype, std=1.0)[0, 0]
    g[4096:9000] = 0
    out, ws = torch.empty(2, device="cuda"), mb.workspace(mb.grad_norm_workspace_size([g]))
    sizes = [1.0, 1e-30, 1e25] if dtype != HF else [1.0, 2.0 ** -20]     # fp16: down to its subnormals
    for size in sizes:
        h = (g.double() * size).to(dtype)
        mb.grad_norm_batched([h], 1.0, out, ws)
        norm = float(h.double().norm())
        assert abs(float(out[0]) - norm) <= 2.0 ** -23 * norm, size   # 2^-24 of the sums, 2^-24 of the result
    h[4] = float("inf")
    mb.grad_norm_batched([h], 1.0, out, ws)
    assert float(out[0]) == float("inf") and mb.device_status(ws) == mb.MUON_ERR_NONFINITE


@pytest.mark.parametrize("shape", [(151, 64, 320), (151, 320, 64), (149, 33, 65), (149, 65, 33), (79, 64, 1024), (75, 1000, 61),
                                   (201, 1, 5), (160, 64, 64)], ids=str)
@pytest.mark.parametrize("x_dtype,y_dtype,pad", [(BF, BF, 0), (FP, HF, 8), (HF, FP, 3)])
def test_more_short_blocks_than_run_at_once(shape, x_dtype, y_dtype, pad):
    """Two to a cluster, an odd number of them, neighbours of every kind: with a zero block, one that is not finite
    and sizes far apart.  What the padding holds stays."""
    n = shape[0]
    x, _ = padded(*shape, pad, x_dtype)
    x.copy_(blocks(230, *shape, x_dtype))
    x[2] = 0
    x[5, -1, -1] = float("nan")
    x[6] *= 64
    x[9, 0, 0] = float("inf")
    y, buf = padded(*shape, pad, y_dtype)
    ws = run([mb.Stack(x, y)], mb.Schedule.fixed(T, ref.STABLE))
    assert mb.device_status(ws) == mb.MUON_ERR_NONFINITE
    assert bool(torch.isnan(y[5]).all()) and bool(torch.isnan(y[9]).all()) and bool((y[2] == 0).all())
    ok = [b for b in list(range(12)) + [n // 2, n - 2, n - 1] if b not in (2, 5, 9)]
    for b in ok:
        want = ref.ns(x[b], [ref.STABLE] * T)
        most = ref.tol_vector([ref.STABLE] * T, y_dtype) if min(shape[1:]) == 1 else ref.tol_stable(y_dtype)
        assert ref.rel(y[b], want) <= most, b
    assert int(torch.isnan(y.float()).flatten(1).any(dim=1).sum()) == 2
    if pad:
        assert bool((buf[:, :, shape[2]:] == 7.0).all())


@pytest.mark.parametrize("shape,counts", [((64, 1024), (50, 33)), ((60, 333), (101, 1, 90)), ((300, 24), (160,))], ids=str)
def test_steps_and_gradients_of_more_short_blocks_than_run_at_once(shape, counts):
    """Several stacks of one shape, whose last blocks stay alone."""
    sch = mb.Schedule.fixed(T)
    w = [blocks(240 + i, c, *shape, BF, std=0.1) for i, c in enumerate(counts)]
    g = [blocks(250 + i, c, *shape, BF) for i, c in enumerate(counts)]
    m = [blocks(260 + i, c, *shape, FP) for i, c in enumerate(counts)]
    old = [(a.clone(), b.clone()) for a, b in zip(w, m)]
    hp = mb.hyper(0.02, 0.95, 0.1, True, "moonlight", sch)
    st = [mb.MuonStack(a, b, c) for a, b, c in zip(w, g, m)]
    ws = mb.workspace(mb.muon_stacks_workspace_size(st, hp))
    mb.muon_step_stacks(st, hp, ws)
    assert mb.device_status(ws) == mb.MUON_OK
    step = 0.02 * ref.scale(*shape, "moonlight")
    for i, c in enumerate(counts):
        for b in sorted({0, c // 2, c - 1}):
            ww, mm, o = ref.muon(old[i][0][b], g[i][b], old[i][1][b], 0.02, 0.95, 0.1, True, "moonlight", [ref.KJ] * T)
            assert ref.rel(m[i][b], mm) <= 2 * 2.0 ** -23
            bound = step * ref.tol_kj(FP) * o.norm() + (ref.half_step(BF) + 2.0 ** -23) * ww.norm() + 1e-12
            assert float((w[i][b].double() - ww).norm()) <= float(bound), (i, b)
    # iterates kept two to a cluster, read one to a cluster
    ys, dx = [torch.empty_like(a) for a in m], [torch.empty_like(a) for a in m]
    dy = [blocks(270 + i, c, *shape, FP, std=1.0) for i, c in enumerate(counts)]
    stacks, grads = [mb.Stack(a, b) for a, b in zip(m, ys)], [mb.Stack(a, b) for a, b in zip(dy, dx)]
    saved = mb.workspace(mb.ns_stacks_saved_size(stacks, sch))
    run(stacks, sch, saved=saved)
    ws = mb.workspace(mb.ns_stacks_backward_workspace_size(grads, sch))
    mb.ns_orthogonalize_stacks_backward(grads, sch, saved, ws)
    for i, c in enumerate(counts):
        for b in sorted({0, c // 2, c - 1}):
            assert ref.rel(ys[i][b], ref.ns(m[i][b], [ref.KJ] * T)) <= ref.tol_kj(FP), (i, b)
            assert ref.rel(dx[i][b], ref.ns_grad(m[i][b], dy[i][b], [ref.KJ] * T)) <= 2 * ref.tol_kj(FP), (i, b)


@pytest.mark.parametrize("n,rows,cols", [(161, 64, 100), (41, 60, 1500), (77, 640, 33), (3, 90, 400)])
def test_gradient_of_short_blocks_beside_bad_ones(n, rows, cols):
    """An input, or a gradient, that is not finite makes its own block's gradient NaN and no other's."""
    x = blocks(280, n, rows, cols, FP, std=0.5)
    dy = blocks(281, n, rows, cols, FP, std=1.0)
    x[0, 3, 3] = float("nan")
    dy[n - 2, 1, 1] = float("inf")
    if n > 8:
        dy[4] = 0
        x[7] = 0
    sch = mb.Schedule.fixed(T, ref.STABLE)
    dx = torch.empty_like(x)
    stacks, grads = [mb.Stack(x, torch.empty_like(x))], [mb.Stack(dy, dx)]
    saved = mb.workspace(mb.ns_stacks_saved_size(stacks, sch))
    run(stacks, sch, saved=saved)
    ws = mb.workspace(mb.ns_stacks_backward_workspace_size(grads, sch))
    mb.ns_orthogonalize_stacks_backward(grads, sch, saved, ws)
    assert mb.device_status(ws) == mb.MUON_ERR_NONFINITE
    assert bool(torch.isnan(dx[0]).all()) and bool(torch.isnan(dx[n - 2]).all())
    assert int(torch.isnan(dx).flatten(1).any(dim=1).sum()) == 2
    for b in [b for b in list(range(12)) + [n - 3, n - 1] if b < n and b not in (0, n - 2)]:
        want = ref.ns_grad(x[b], dy[b], [ref.STABLE] * T)
        if n > 8 and b == 4:
            assert bool((dx[b] == 0).all())
        else:
            assert ref.rel(dx[b], want) <= ref.tol_stable(FP), b


@pytest.mark.parametrize("rows,cols,pad", [(64, 200, 0), (64, 201, 0), (200, 64, 3), (257, 130, 0)])
def test_a_decay_to_zero_keeps_what_is_not_finite(rows, cols, pad):
    """lr * weight decay = 1 takes every weight to zero before the step, and a NaN or an infinity to NaN, on every path."""
    st, _ = muon_stack(300, 2, rows, cols, pad)
    st.W[1, 3, 5], st.W[1, 6, 7] = float("nan"), float("inf")
    m0 = st.M.clone()
    hp = mb.hyper(1.0, 0.95, 1.0, True, "naive")
    mb.muon_step_stacks([st], hp, mb.workspace(mb.muon_stacks_workspace_size([st], hp)))
    assert bool(torch.isnan(st.W[1, 3, 5])) and bool(torch.isnan(st.W[1, 6, 7]))
    assert int(torch.isnan(st.W.float()).sum()) == 2
    f = lambda x: float(torch.tensor(x, dtype=FP))  # noqa: E731
    want = ref.muon(torch.zeros_like(st.W[0]), st.G[0], m0[0], 1.0, f(0.95), 1.0, True, "naive", [ref.KJ] * T)[0]
    assert ref.rel(st.W[0], want) <= ref.tol_kj(BF)


def test_a_captured_step_outlives_its_workspaces_growth():
    """A parameter meets its first gradient after the capture, and the workspace grows: the graph goes on writing to its own,
    and to nothing that was allocated since."""
    a, b = blocks(310, 2, 160, 200, FP, std=0.1), blocks(311, 3, 300, 400, FP, std=0.1)
    p, q = torch.nn.Parameter(a.clone()), torch.nn.Parameter(b.clone())
    twin = torch.nn.Parameter(a.clone())
    opt, other = StackedMuon([p, q], lr=0.02), StackedMuon([twin], lr=0.02)
    p.grad = blocks(312, 2, 160, 200, FP)
    twin.grad = p.grad.clone()
    opt.step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        opt.step()
    size = opt._ws.get(1, p.device).numel()
    q.grad = blocks(313, 3, 300, 400, FP)
    opt.step()
    assert opt._ws.get(1, p.device).numel() > size
    junk = [torch.full((size,), 7, dtype=torch.uint8, device="cuda") for _ in range(8)]
    for seed in (314, 315):
        p.grad.copy_(blocks(seed, 2, 160, 200, FP))
        graph.replay()
    torch.cuda.synchronize()
    assert all(bool((j == 7).all()) for j in junk)
    for g in (312, 312, 314, 315):          # eager, eager beside q, replay, replay
        twin.grad.copy_(blocks(g, 2, 160, 200, FP))
        other.step()
    assert torch.equal(p, twin)
