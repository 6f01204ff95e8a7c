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
