"""CPU checks of the torch front-ends of the stacked-block operators and AdamW; the library's calls are replaced by
recorders."""
import pytest
import torch
import torch.autograd.forward_ad as forward_ad

from matrix_orthogonalising_optimizer_02_b200 import binding as mb
from matrix_orthogonalising_optimizer_02_b200 import stacks as ms


@pytest.mark.parametrize("requires_grad", [False, True])
@pytest.mark.parametrize("grad_mode", [False, True])
def test_orthogonalize_refuses_forward_mode(monkeypatch, requires_grad, grad_mode):
    """A tangent would be dropped silently: the operator has a reverse derivative alone."""
    calls = []

    def record(stacks, schedule, keep=False):
        calls.append(keep)
        stacks[0].Y.zero_()
        return torch.zeros(1) if keep else None
    monkeypatch.setattr(mb, "orthogonalize_alloc", record)
    x = torch.randn(4, 6, requires_grad=requires_grad)
    with torch.set_grad_enabled(grad_mode), forward_ad.dual_level():
        with pytest.raises(NotImplementedError):
            ms.orthogonalize(forward_ad.make_dual(x, torch.ones(4, 6)))
        assert not calls
        y = ms.orthogonalize(x)      # beside a dual level, without a tangent
    assert calls == [requires_grad and grad_mode] and y.shape == x.shape
    with pytest.raises(NotImplementedError):
        torch.func.jvp(ms.orthogonalize, (x.detach(),), (torch.ones(4, 6),))


def test_adamw_refuses_a_capture(monkeypatch):
    """The number of the step is a host integer: a replay would go on with the captured one's corrections."""
    from matrix_orthogonalising_optimizer_02_b200.optim import AdamW
    steps = []
    monkeypatch.setattr(mb, "adamw_step_batched", lambda tensors, hp, step, grad_scale=None: steps.append(step))
    p = torch.nn.Parameter(torch.ones(8))
    p.grad = torch.ones(8)
    opt = AdamW([p])
    opt.step()
    monkeypatch.setattr(torch.cuda, "is_available", lambda: True)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: True)
    with pytest.raises(RuntimeError, match="captured"):
        opt.step()
    assert steps == [1] and opt.state[p]["step"] == 1
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    opt.step()
    assert steps == [1, 2]


class _Buffer:
    """Stands for a workspace tensor."""

    def __init__(self, nbytes):
        self.nbytes, self.streams = nbytes, []

    def numel(self):
        return self.nbytes

    def record_stream(self, stream):
        self.streams.append(stream)


@pytest.fixture
def fake_cuda(monkeypatch):
    state = {"capturing": False, "stream": "one"}
    monkeypatch.setattr(mb, "workspace", lambda nbytes, device=None: _Buffer(nbytes))
    monkeypatch.setattr(torch.cuda, "is_available", lambda: True)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: state["capturing"])
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: state["stream"])
    return state


def test_a_workspace_that_a_capture_has_used_stays(fake_cuda):
    """A graph goes on writing to the workspace it was captured with: growing must not give it back."""
    import gc
    import weakref

    from matrix_orthogonalising_optimizer_02_b200.optim import _Workspaces
    pool = _Workspaces()
    plain = weakref.ref(pool.get(100, "cuda:0"))
    pool.get(200, "cuda:0")
    gc.collect()
    assert plain() is None                          # never captured: given back
    fake_cuda["capturing"] = True
    held = [weakref.ref(pool.get(150, "cuda:0"))]
    assert held[0]().numel() == 200
    held.append(weakref.ref(pool.get(300, "cuda:0")))   # grown inside a capture
    fake_cuda["capturing"] = False
    last = pool.get(400, "cuda:0")
    gc.collect()
    assert all(w() is not None for w in held) and last.numel() == 400
    assert pool.get(10, "cuda:1").numel() == 10


def test_a_workspace_used_on_another_stream_waits_for_it(fake_cuda):
    """The allocator must not hand a dropped workspace to its own stream while another one still uses it."""
    from matrix_orthogonalising_optimizer_02_b200.optim import _Workspaces
    pool = _Workspaces()
    ws = pool.get(100, "cuda:0")
    assert pool.get(100, "cuda:0") is ws and ws.streams == []
    fake_cuda["stream"] = "two"
    assert pool.get(50, "cuda:0") is ws and ws.streams == ["two"]
    assert pool.get(200, "cuda:0").streams == []


def test_state_dicts_leave_the_workspaces(fake_cuda):
    """A graph that was captured before a state was loaded still has its workspace."""
    import copy

    from matrix_orthogonalising_optimizer_02_b200.optim import StackedMuon
    opt = StackedMuon([torch.nn.Parameter(torch.zeros(4, 6))])
    ws = opt._ws.get(100, "cuda:0")
    opt.load_state_dict(copy.deepcopy(opt.state_dict()))
    assert opt._ws.get(100, "cuda:0") is ws
    assert copy.deepcopy(opt)._ws.get(100, "cuda:0") is not ws    # a copy has its own


def test_adamw_goes_on_from_torchs_state(monkeypatch):
    """torch.optim.AdamW keeps the number of the step in a tensor, one per parameter."""
    from matrix_orthogonalising_optimizer_02_b200.optim import AdamW
    shapes = [(3, 5), (7,)]
    theirs = [torch.nn.Parameter(torch.ones(s, dtype=torch.bfloat16)) for s in shapes]
    ours = [torch.nn.Parameter(torch.ones(s, dtype=torch.bfloat16)) for s in shapes]
    a, b = torch.optim.AdamW(theirs, lr=0.5, weight_decay=0.25), AdamW(ours)
    for _ in range(2):
        for p in theirs:
            p.grad = torch.ones_like(p)
        a.step()
    b.load_state_dict(a.state_dict())
    assert b.param_groups[0]["lr"] == 0.5 and b.param_groups[0]["weight_decay"] == 0.25
    for p, q in zip(theirs, ours):
        s = b.state[q]
        assert type(s["step"]) is int and s["step"] == 2
        assert s["exp_avg"].dtype == s["exp_avg_sq"].dtype == torch.float32
        assert torch.equal(s["exp_avg"], a.state[p]["exp_avg"].float())
    calls = []
    monkeypatch.setattr(mb, "adamw_step_batched", lambda t, hp, step, grad_scale=None: calls.append((len(t), step)))
    for q in ours:
        q.grad = torch.ones_like(q)
    b.step()
    assert calls == [(2, 3)]                       # one call for both parameters
    b.load_state_dict(b.state_dict())              # and its own
    assert b.state[ours[0]]["step"] == 3


@pytest.mark.parametrize("change", [dict(amsgrad=True), dict(maximize=True), dict(decoupled_weight_decay=False)], ids=str)
def test_adamw_refuses_a_state_of_another_rule(change):
    from matrix_orthogonalising_optimizer_02_b200.optim import AdamW
    p = torch.nn.Parameter(torch.ones(4))
    state = torch.optim.AdamW([p]).state_dict()
    state["param_groups"][0].update(change)
    opt = AdamW([p], lr=0.125)
    with pytest.raises(ValueError):
        opt.load_state_dict(state)
    assert opt.param_groups[0]["lr"] == 0.125      # left as it was


def test_a_refused_adamw_step_does_not_count(monkeypatch):
    from matrix_orthogonalising_optimizer_02_b200.optim import AdamW

    def refuse(*args, **kw):
        raise ValueError("refused")
    p = torch.nn.Parameter(torch.ones(4))
    p.grad = torch.ones(4)
    opt = AdamW([p])
    monkeypatch.setattr(mb, "adamw_step_batched", refuse)
    with pytest.raises(ValueError):
        opt.step()
    steps = []
    monkeypatch.setattr(mb, "adamw_step_batched", lambda t, hp, step, grad_scale=None: steps.append(step))
    opt.step()
    assert steps == [1]


def test_a_parameter_without_elements_takes_no_step(monkeypatch):
    """A rank without experts, say: beside others, and alone."""
    from matrix_orthogonalising_optimizer_02_b200.optim import StackedMuon
    calls = []
    monkeypatch.setattr(mb, "muon_stacks_workspace_size", lambda stacks, hp: 256)
    monkeypatch.setattr(mb, "muon_step_stacks", lambda stacks, hp, ws, grad_scale=None: calls.append([s.W for s in stacks]))
    monkeypatch.setattr(mb, "workspace", lambda nbytes, device=None: _Buffer(nbytes))
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: "one")
    full, none = torch.nn.Parameter(torch.ones(2, 4, 6)), torch.nn.Parameter(torch.ones(0, 4, 6))
    flat = torch.nn.Parameter(torch.ones(0, 6))
    for p in (full, none, flat):
        p.grad = torch.ones_like(p)
    opt = StackedMuon([{"params": [full, none]}, {"params": [flat], "row_block": 4}])
    opt.step()
    assert len(calls) == 1 and [w.shape for w in calls[0]] == [full.shape]
    opt.load_state_dict(opt.state_dict())


def test_a_first_step_refuses_a_capture(fake_cuda, monkeypatch):
    """The momentum would be made inside the graph, and every replay would begin by setting it to zero."""
    from matrix_orthogonalising_optimizer_02_b200.optim import StackedMuon
    calls = []
    monkeypatch.setattr(mb, "muon_stacks_workspace_size", lambda stacks, hp: 256)
    monkeypatch.setattr(mb, "muon_step_stacks", lambda stacks, hp, ws, grad_scale=None: calls.append(len(stacks)))
    a, b = torch.nn.Parameter(torch.ones(4, 6)), torch.nn.Parameter(torch.ones(6, 4))
    opt = StackedMuon([a, b])
    a.grad = torch.ones_like(a)
    fake_cuda["capturing"] = True
    with pytest.raises(RuntimeError, match="captured"):
        opt.step()
    assert not calls and not opt.state[a]
    fake_cuda["capturing"] = False
    opt.step()
    fake_cuda["capturing"] = True
    opt.step()
    b.grad = torch.ones_like(b)            # its first
    with pytest.raises(RuntimeError, match="captured"):
        opt.step()
    assert calls == [1, 1]


def test_host_tensors_are_refused_as_such():
    from matrix_orthogonalising_optimizer_02_b200.optim import AdamW, Muon, MuonCayley, StackedMuon
    for cls in (AdamW, Muon, MuonCayley, StackedMuon):
        p = torch.nn.Parameter(torch.ones(16, 8))
        p.grad = torch.ones_like(p)
        with pytest.raises(ValueError):
            cls([p]).step()
