"""CPU checks of the stacked-block operators, the gradient norm and AdamW: the reverse formulas against
differences, workspace queries, and the refusal of every argument the calls do not take (these calls
return before any CUDA call)."""
import ctypes

import pytest
import torch

import stack_reference as ref
from matrix_orthogonalising_optimizer_02_b200 import binding as mb
from matrix_orthogonalising_optimizer_02_b200 import stacks as ms
from matrix_orthogonalising_optimizer_02_b200.optim import AdamW, StackedMuon, clip_scale

P = 1 << 20
WS = ctypes.c_void_p(1 << 24)


@pytest.mark.parametrize("shape", [(1, 1), (1, 6), (5, 8), (9, 4)])
@pytest.mark.parametrize("coeffs", [ref.KJ, ref.STABLE])
def test_reverse_formulas_against_differences(shape, coeffs):
    """Central differences in 64 bits with step h are off by h^2 f'''/6 plus eps f / h: with
    h = 1e-5 and |f'''| up to 1e4 that is 2e-7 at most; 1e-5 leaves room."""
    gen = torch.Generator().manual_seed(3)
    u = torch.randn(shape, generator=gen, dtype=torch.float64)
    dy = torch.randn(shape, generator=gen, dtype=torch.float64)
    grad = ref.ns_grad(u, dy, [coeffs] * 3, eps=0.1)
    h = 1e-5
    for i in range(shape[0]):
        for j in range(shape[1]):
            e = torch.zeros(shape, dtype=torch.float64)
            e[i, j] = h
            d = ((ref.ns(u + e, [coeffs] * 3, 0.1) - ref.ns(u - e, [coeffs] * 3, 0.1)) * dy).sum() / (2 * h)
            assert abs(float(d - grad[i, j])) <= 1e-5


def _ns(count=2, rows=16, cols=24, **kw):
    d = dict(X=P, Y=P + (1 << 19), x_stride=rows * cols, y_stride=rows * cols, x_ld=cols, y_ld=cols, count=count,
             rows=rows, cols=cols, x_dtype=mb.MUON_BF16, y_dtype=mb.MUON_BF16)
    d.update(kw)
    arr = (mb.NsStackDesc * 1)()
    arr[0] = mb.NsStackDesc(**d)
    return arr


def _orth(arr, n=1, sch=None, saved=None, saved_bytes=0, ws=WS, ws_bytes=1 << 30):
    sch = sch or mb.Schedule.fixed(5)
    return mb.load().ns_orthogonalize_stacks(arr, n, ctypes.byref(sch.c), saved, saved_bytes, ws, ws_bytes, None)


INVALID, SHAPE, ALIGN, SMALL = (mb.MUON_ERR_INVALID_ARG, mb.MUON_ERR_UNSUPPORTED_SHAPE, mb.MUON_ERR_ALIGNMENT,
                                mb.MUON_ERR_WORKSPACE_TOO_SMALL)


@pytest.mark.parametrize("change,status", [
    (dict(X=None), INVALID), (dict(Y=None), INVALID), (dict(count=0), INVALID), (dict(rows=0), INVALID),
    (dict(cols=-1), INVALID), (dict(x_dtype=3), INVALID), (dict(y_dtype=-1), INVALID), (dict(x_ld=23), INVALID),
    (dict(y_stride=-1), INVALID), (dict(y_stride=0), INVALID), (dict(y_stride=100), INVALID),
    (dict(rows=32769, x_stride=1 << 30, y_stride=1 << 30), SHAPE), (dict(X=P + 1), ALIGN),
    (dict(Y=P + 2, y_dtype=mb.MUON_F32), ALIGN), (dict(count=(1 << 20) + 1), SHAPE),
])
def test_refused_stacks(change, status):
    arr = _ns(**change)
    s = mb.Schedule.fixed(5)
    assert _orth(arr) == status
    assert mb.load().ns_stacks_workspace_size(arr, 1, ctypes.byref(s.c), 0) == 0
    assert mb.load().ns_stacks_saved_size(arr, 1, ctypes.byref(s.c)) == 0
    assert mb.load().ns_stacks_backward_workspace_size(arr, 1, ctypes.byref(s.c)) == 0
    assert mb.load().ns_orthogonalize_stacks_backward(arr, 1, ctypes.byref(s.c), WS, 1 << 30, WS, 1 << 30,
                                                      None) == status


@pytest.mark.parametrize("sch", [
    mb.Schedule([]), mb.Schedule.fixed(5, n_split_iters=1), mb.Schedule.fixed(5, fp32_mode=True),
    mb.Schedule.fixed(5, eps=0.0), mb.Schedule([(float("nan"), 0, 0)]), mb.Schedule([(100.0, 0.0, 0.0)]),
    mb.Schedule([(3.0, 1.0, 1.0)] * 4), mb.Schedule.fixed(33)], ids=str)
def test_refused_schedules(sch):
    assert _orth(_ns(), sch=sch) == INVALID
    assert mb.load().ns_stacks_workspace_size(_ns(), 1, ctypes.byref(sch.c), 0) == 0


def test_refused_workspaces_and_counts():
    lib, s = mb.load(), mb.Schedule.fixed(5)
    need = lib.ns_stacks_workspace_size(_ns(), 1, ctypes.byref(s.c), 0)
    assert need > 0
    assert _orth(_ns(), ws_bytes=need - 1) == SMALL
    assert _orth(_ns(), ws=None) == INVALID
    assert _orth(_ns(), ws=ctypes.c_void_p((1 << 24) + 16)) == ALIGN
    assert _orth(_ns(), n=0) == INVALID
    assert _orth(None) == INVALID
    kept = lib.ns_stacks_saved_size(_ns(), 1, ctypes.byref(s.c))
    assert _orth(_ns(), saved=ctypes.c_void_p(1 << 26), saved_bytes=kept - 1) == SMALL
    assert _orth(_ns(), saved=ctypes.c_void_p((1 << 26) + 8), saved_bytes=kept) == ALIGN
    back = lib.ns_stacks_backward_workspace_size(_ns(), 1, ctypes.byref(s.c))

    def b(saved, sb, ws, wb):
        return lib.ns_orthogonalize_stacks_backward(_ns(), 1, ctypes.byref(s.c), saved, sb, ws, wb, None)
    assert b(None, kept, WS, back) == INVALID
    assert b(WS, kept - 1, WS, back) == SMALL
    assert b(WS, kept, WS, back - 1) == SMALL
    assert b(WS, kept, None, back) == INVALID


def test_side_by_side_blocks_are_taken():
    """Column blocks of a fused matrix, and interleaved rows: written blocks that do not overlap."""
    s, lib = mb.Schedule.fixed(5), mb.load()
    cols = _ns(count=3, rows=16, cols=8, x_stride=8, y_stride=8, x_ld=24, y_ld=24)
    rows = _ns(count=4, rows=16, cols=24, x_stride=24, y_stride=24, x_ld=96, y_ld=96)
    over = _ns(count=4, rows=16, cols=8, x_stride=8, y_stride=8, x_ld=24, y_ld=24)
    assert lib.ns_stacks_workspace_size(cols, 1, ctypes.byref(s.c), 0) > 0
    assert lib.ns_stacks_workspace_size(rows, 1, ctypes.byref(s.c), 0) > 0
    assert lib.ns_stacks_workspace_size(over, 1, ctypes.byref(s.c), 0) == 0


def _muon(**kw):
    d = dict(W=P, G=P, M=P, w_stride=384, g_stride=384, m_stride=384, w_ld=24, g_ld=24, m_ld=24, count=2, rows=16,
             cols=24, w_dtype=mb.MUON_BF16, g_dtype=mb.MUON_F16)
    d.update(kw)
    arr = (mb.MuonStackDesc * 1)()
    arr[0] = mb.MuonStackDesc(**d)
    return arr


@pytest.mark.parametrize("change,status", [
    (dict(W=None), INVALID), (dict(G=None), INVALID), (dict(M=None), INVALID), (dict(g_dtype=9), INVALID),
    (dict(m_stride=0), INVALID), (dict(w_ld=8), INVALID), (dict(M=P + 2), ALIGN), (dict(cols=40000, w_ld=40000,
     g_ld=40000, m_ld=40000, w_stride=1 << 24, m_stride=1 << 24), SHAPE)])
def test_refused_muon_stacks(change, status):
    hp = mb.hyper(0.02)
    lib = mb.load()
    assert lib.muon_step_stacks(_muon(**change), 1, ctypes.byref(hp[0]), None, WS, 1 << 30, None) == status
    assert lib.muon_stacks_workspace_size(_muon(**change), 1, ctypes.byref(hp[0])) == 0


def test_refused_muon_hyper():
    lib = mb.load()
    for hp in (mb.hyper(float("nan")), mb.hyper(0.1, beta=float("inf")), mb.hyper(0.1, schedule=mb.Schedule([]))):
        assert lib.muon_step_stacks(_muon(), 1, ctypes.byref(hp[0]), None, WS, 1 << 30, None) == INVALID
    hp = mb.hyper(0.1)
    assert lib.muon_step_stacks(_muon(), 1, ctypes.byref(hp[0]), ctypes.c_void_p(P + 2), WS, 1 << 30, None) == ALIGN
    assert lib.muon_step_stacks(_muon(), 1, ctypes.byref(hp[0]), None, WS, 255, None) == SMALL
    assert lib.muon_step_stacks(_muon(), 1, None, None, WS, 1 << 30, None) == INVALID


def _adam(**kw):
    d = dict(W=P, G=P, m=P, v=P, n=100, w_dtype=mb.MUON_BF16, g_dtype=mb.MUON_BF16)
    d.update(kw)
    arr = (mb.AdamWTensorDesc * 1)()
    arr[0] = mb.AdamWTensorDesc(**d)
    return arr


@pytest.mark.parametrize("change,status", [
    (dict(W=None), INVALID), (dict(G=None), INVALID), (dict(m=None), INVALID), (dict(v=None), INVALID),
    (dict(n=-1), INVALID), (dict(w_dtype=3), INVALID), (dict(G=P + 1), ALIGN), (dict(v=P + 2), ALIGN)])
def test_refused_adamw_tensors(change, status):
    hp = mb.adamw_hyper()
    hp.step = 1
    assert mb.load().adamw_step_batched(_adam(**change), 1, ctypes.byref(hp), None, None) == status


def test_refused_adamw_hyper_and_norm():
    lib = mb.load()
    for change in (dict(lr=float("nan")), dict(beta1=1.0), dict(beta2=-0.1), dict(eps=-1.0), dict(eps=float("inf"))):
        hp = mb.adamw_hyper(**change)
        hp.step = 1
        assert lib.adamw_step_batched(_adam(), 1, ctypes.byref(hp), None, None) == INVALID
    hp = mb.adamw_hyper()
    assert lib.adamw_step_batched(_adam(), 1, ctypes.byref(hp), None, None) == INVALID          # step 0
    hp.step = 1
    assert lib.adamw_step_batched(_adam(), 0, ctypes.byref(hp), None, None) == INVALID
    assert lib.adamw_step_batched(_adam(), 1, None, None, None) == INVALID
    assert lib.adamw_step_batched(_adam(), 1, ctypes.byref(hp), ctypes.c_void_p(P + 1), None) == ALIGN
    one = ctypes.c_float(1.0)
    need = lib.grad_norm_workspace_size(_adam(), 1)
    assert need > 0 and lib.grad_norm_workspace_size(_adam(n=-1), 1) == 0
    assert lib.grad_norm_batched(_adam(), 1, one, None, WS, need, None) == INVALID
    assert lib.grad_norm_batched(_adam(), 1, ctypes.c_float(0.0), WS, WS, need, None) == INVALID
    assert lib.grad_norm_batched(_adam(), 1, ctypes.c_float(float("nan")), WS, WS, need, None) == INVALID
    assert lib.grad_norm_batched(_adam(), 1, one, WS, WS, need - 1, None) == SMALL
    assert lib.grad_norm_batched(_adam(), 1, one, ctypes.c_void_p(P + 2), WS, need, None) == ALIGN


def test_workspaces_grow_with_the_blocks_up_to_a_group():
    s, lib = mb.Schedule.fixed(5), mb.load()

    def size(count, rows=4096, cols=4096):
        return lib.ns_stacks_workspace_size(_ns(count=count, rows=rows, cols=cols, x_ld=cols, y_ld=cols,
                                                x_stride=rows * cols, y_stride=rows * cols), 1, ctypes.byref(s.c), 0)
    assert size(1) < size(2) < size(20)
    assert size(100) == size(200) <= (5 << 30) + (1 << 20)


def test_views_of_fused_parameters():
    w = torch.arange(24).reshape(6, 4)
    r = ms.row_blocks(w, 2)
    assert r.shape == (3, 2, 4) and torch.equal(r[1], w[2:4]) and r.data_ptr() == w.data_ptr()
    c = ms.col_blocks(w, 2)
    assert c.shape == (2, 6, 2) and torch.equal(c[1], w[:, 2:]) and c.data_ptr() == w.data_ptr()
    for bad in (4, 0):
        with pytest.raises(ValueError):
            ms.row_blocks(w, bad)
    with pytest.raises(ValueError):
        ms.col_blocks(w, 3)


def test_front_ends_refuse():
    par = torch.nn.Parameter
    with pytest.raises(ValueError):
        StackedMuon([par(torch.zeros(8))])
    with pytest.raises(ValueError):
        StackedMuon([par(torch.zeros(8, 8))], scale_mode="bogus")
    with pytest.raises(ValueError):
        StackedMuon([par(torch.zeros(8, 8))], row_block=3)
    with pytest.raises(ValueError):
        StackedMuon([par(torch.zeros(8, 8))], row_block=4, col_block=4)
    with pytest.raises(ValueError):
        StackedMuon([par(torch.zeros(8, 8, dtype=torch.float64))])
    with pytest.raises(ValueError):
        AdamW([par(torch.zeros(8, dtype=torch.float64))])
    with pytest.raises(ValueError):
        clip_scale([par(torch.zeros(8))], 1.0)
    with pytest.raises(ValueError):
        ms.orthogonalize(torch.zeros(4, 4), steps=3, coeffs=[ref.KJ] * 2)
    with pytest.raises(ValueError):   # host tensors
        ms.orthogonalize(torch.zeros(4, 4))


def test_blocks_on_chip_need_no_planes():
    """Where the iterations and the reverse pass run on chip, the workspaces hold no planes; the kept iterates do."""
    s, lib = mb.Schedule.fixed(5), mb.load()
    d = _ns(count=96, rows=64, cols=2048, x_ld=2048, y_ld=2048, x_stride=64 * 2048, y_stride=64 * 2048)
    assert lib.ns_stacks_workspace_size(d, 1, ctypes.byref(s.c), 0) < 4096
    assert lib.ns_stacks_workspace_size(d, 1, ctypes.byref(s.c), 1) < 4096
    assert lib.ns_stacks_backward_workspace_size(d, 1, ctypes.byref(s.c)) < 4096
    assert lib.ns_stacks_saved_size(d, 1, ctypes.byref(s.c)) >= 5 * 2 * 96 * 64 * 2048


@pytest.mark.parametrize("coeffs,taken", [
    ([ref.KJ] * 5, True), ([ref.KJ] * 12, True), ([ref.KJ] * 8 + [ref.STABLE] * 2, True), ([ref.KJ] * 16 + [ref.STABLE] * 2, True),
    ([ref.STABLE] * 32, True), ([(2.0, -1.5, 0.5)] * 32, True), ([(1.5, -0.5, 0.0)] * 32, True),
    ([ref.KJ] * 16, False), ([ref.KJ] * 32, False), ([ref.KJ] * 30 + [ref.STABLE], False)],
    ids=["kj5", "kj12", "hybrid", "hybrid16", "stable32", "other32", "quadratic32", "kj16", "kj32", "kj30 stable1"])
def test_schedules_through_which_no_gradient_survives(coeffs, taken):
    """Roundings that grow from iteration to iteration leave no correct digit in a gradient: such a schedule is refused
    where one is to come (a forward call without one takes it)."""
    lib, s = mb.load(), mb.Schedule(coeffs)
    d = _ns()
    sch = ctypes.byref(s.c)
    assert lib.ns_stacks_workspace_size(d, 1, sch, 0) > 0
    for size in (lib.ns_stacks_workspace_size(d, 1, sch, 1), lib.ns_stacks_saved_size(d, 1, sch),
                 lib.ns_stacks_backward_workspace_size(d, 1, sch)):
        assert (size > 0) == taken
    if not taken:
        assert _orth(d, sch=s, saved=WS, saved_bytes=1 << 30) == INVALID
        assert lib.ns_orthogonalize_stacks_backward(d, 1, sch, WS, 1 << 30, WS, 1 << 30, None) == INVALID


@pytest.mark.skipif(torch.cuda.is_available(), reason="the calls have to fail: without a device they do before any launch")
def test_a_failing_call_names_an_error_that_was_pending():
    """An error of earlier work does not become the call's own, and does not vanish either."""
    lib, hp = mb.load(), mb.adamw_hyper()
    hp.step = 1
    cudart = ctypes.CDLL("libcudart.so.12")
    calls = [lambda: _orth(_ns(rows=300, cols=400, x_ld=400, y_ld=400, x_stride=1 << 18, y_stride=1 << 18)),
             lambda: lib.adamw_step_batched(_adam(), 1, ctypes.byref(hp), None, None),
             lambda: lib.grad_norm_batched(_adam(), 1, ctypes.c_float(1.0), WS, WS, 1 << 30, None)]
    for call in calls:
        assert cudart.cudaSetDevice(99) != 0               # an unrelated call fails
        assert call() == mb.MUON_ERR_CUDA
        assert b"was pending on entry" in lib.muon_last_error()
