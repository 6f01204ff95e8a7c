"""torch.optim front-ends over the C ABI (argument marshalling only).

``Muon`` mirrors the constructor of the ``Muon`` class on the "Muon优化器" page
(linsight.cn/f25d614e.html, "Muon 算法伪代码与 PyTorch 实现"): lr, momentum,
weight_decay, nesterov, ns_steps, scale_mode.  ``MuonCayley`` mirrors the optimizer of
the Stiefel-manifold page (mlqm.cn/news/1339166, §4.3) for its Cayley branch.  Both hand
every matrix of a parameter group to one library call per step; grouping parameters
into Muon matrices and AdamW tensors stays with the caller, as the pages advise, so
these classes accept 2-D parameters only.  ``StackedMuon`` takes the fused and stacked forms of
such matrices (heads of a QKV weight, experts, any sizes), ``AdamW`` the rest, and
``clip_scale`` the gradient norm over all of them.
"""
from __future__ import annotations

import torch

from . import binding as mb
from . import stacks as ms

KJ_COEFFS = (3.4445, -4.7750, 2.0315)


def _check_matrix(p):
    if p.dim() != 2:
        raise ValueError(f"Muon handles 2-D weight matrices only, got shape {tuple(p.shape)}; "
                         "give embeddings, heads, biases and norms to AdamW")
    if p.dtype not in (torch.bfloat16, torch.float32):
        raise ValueError(f"unsupported parameter dtype {p.dtype}")


def _capturing() -> bool:
    return torch.cuda.is_available() and torch.cuda.is_current_stream_capturing()


class _Workspaces:
    """One workspace per device, grown to the largest request: the library's calls are
    ordered on the current stream, so successive calls can share it.  A buffer that a CUDA
    graph was captured with is never given back: its replays go on writing there.  One that
    another stream than its own has used is given back when that stream is done with it."""

    def __init__(self):
        self.bufs = {}
        self.captured = []

    def get(self, nbytes, device):
        ws, own = self.bufs.get(device, (None, None))
        # a host tensor's workspace goes to the call that refuses it
        stream = torch.cuda.current_stream(device) if torch.device(device).type == "cuda" else None
        if ws is None or ws.numel() < nbytes:
            ws, own = mb.workspace(nbytes, device=device), stream
            self.bufs[device] = ws, own
        if _capturing():
            if not any(ws is c for c in self.captured):
                self.captured.append(ws)
        elif stream != own:
            ws.record_stream(stream)
        return ws


class Muon(torch.optim.Optimizer):
    """Momentum orthogonalised by Newton-Schulz, one grouped CUDA step per param group."""

    def __init__(self, params, lr=1e-3, momentum=0.95, weight_decay=0.01, nesterov=True, ns_steps=5,
                 scale_mode="moonlight", coeffs=None, n_split_iters=0, fp32_mode=False, eps=1e-7):
        if scale_mode not in mb.SCALE_MODES:
            raise ValueError(f"scale_mode must be one of {sorted(mb.SCALE_MODES)}")
        defaults = dict(lr=lr, momentum=momentum, weight_decay=weight_decay, nesterov=nesterov, ns_steps=ns_steps,
                        scale_mode=scale_mode, coeffs=coeffs, n_split_iters=n_split_iters, fp32_mode=fp32_mode,
                        eps=eps)
        super().__init__(params, defaults)
        for g in self.param_groups:
            for p in g["params"]:
                _check_matrix(p)
        self._ws = _Workspaces()

    @torch.no_grad()
    def step(self, closure=None):
        loss = None
        if closure is not None:
            with torch.enable_grad():
                loss = closure()
        for group in self.param_groups:
            mats = []
            for p in group["params"]:
                if p.grad is None:
                    continue
                state = self.state[p]
                if "momentum_buffer" not in state:
                    state["momentum_buffer"] = torch.zeros(p.shape, dtype=torch.float32, device=p.device)
                mats.append(mb.Matrix(p.data, p.grad.contiguous(), state["momentum_buffer"]))
            if not mats:
                continue
            coeffs = group["coeffs"] or [KJ_COEFFS] * group["ns_steps"]
            sch = mb.Schedule(coeffs, n_split_iters=group["n_split_iters"], fp32_mode=group["fp32_mode"],
                              eps=group["eps"])
            hp = mb.hyper(group["lr"], group["momentum"], group["weight_decay"], group["nesterov"],
                          group["scale_mode"], sch)
            ws = self._ws.get(mb.muon_step_workspace_size(mats, hp), mats[0].W.device)
            mb.muon_step_batched(mats, hp, ws)
        return loss


class MuonCayley(torch.optim.Optimizer):
    """Stiefel-manifold Muon: EMA momentum, column centering, tangent projection and the
    Cayley retraction in Woodbury form.  Parameters are fp32 and orthonormal along their
    shorter side: a tall n x k parameter has orthonormal columns, a wide one orthonormal
    rows and is updated as its transpose inside the library (page §4.4)."""

    def __init__(self, params, lr=3e-3, momentum=0.9, center=True):
        super().__init__(params, dict(lr=lr, momentum=momentum, center=center))
        for g in self.param_groups:
            for p in g["params"]:
                _check_matrix(p)
                if p.dtype != torch.float32:
                    raise ValueError("MuonCayley needs fp32 parameters")
        self._ws = _Workspaces()

    @torch.no_grad()
    def step(self, closure=None):
        loss = None
        if closure is not None:
            with torch.enable_grad():
                loss = closure()
        for group in self.param_groups:
            for p in group["params"]:
                if p.grad is None:
                    continue
                state = self.state[p]
                if "momentum_buffer" not in state:
                    state["momentum_buffer"] = torch.zeros_like(p)
                n, k = p.shape
                ws = self._ws.get(mb.muon_cayley_workspace_size(1, n, k), p.device)
                mb.muon_cayley_step(p.data, p.grad.contiguous(), state["momentum_buffer"], group["lr"],
                                    group["momentum"], ws, center=group["center"])
        return loss


def clip_scale(params, max_norm: float, workspaces=None):
    """A device tensor [norm, scale] of the parameters' gradients: their norm together and
    min(1, max_norm / (norm + 1e-6)).  scale = out[1:] goes to the step() of StackedMuon and AdamW as
    `grad_scale`, which leaves the gradients as they are and needs no synchronisation."""
    grads = [p.grad.contiguous() for p in params if p.grad is not None]
    if not grads:
        raise ValueError("no parameter has a gradient")
    out = torch.empty(2, dtype=torch.float32, device=grads[0].device)
    ws = (workspaces or _Workspaces()).get(mb.grad_norm_workspace_size(grads), grads[0].device)
    mb.grad_norm_batched(grads, max_norm, out, ws)
    return out


class _Fp32State(torch.optim.Optimizer):
    """Keeps its state in fp32 through load_state_dict, which casts it to the parameter's type otherwise."""

    def load_state_dict(self, state_dict):
        super().load_state_dict(state_dict)
        saved = [i for g in state_dict["param_groups"] for i in g["params"]]
        params = [p for g in self.param_groups for p in g["params"]]
        for i, p in zip(saved, params):
            for k, v in state_dict["state"].get(i, {}).items():
                if k == "step":        # a host integer here; torch.optim.AdamW has it in a tensor
                    self.state[p][k] = int(v)
                elif torch.is_tensor(v):
                    self.state[p][k] = v.to(device=p.device, dtype=torch.float32, copy=True)


class StackedMuon(_Fp32State):
    """The Muon step on blocks of parameters: a 3-D parameter [count, rows, cols] is a stack of blocks
    (experts); a 2-D one is a block, or, with the group option ``row_block`` or ``col_block``, a stack
    of blocks of that many rows or columns (heads of a fused QKV weight, the halves of a fused gate/up
    weight).  Any sizes; bf16, fp16 or fp32 parameters.  One grouped call per param group.  step() can be
    captured in a CUDA graph once every parameter with a gradient has taken a step."""

    def __init__(self, params, lr=1e-3, momentum=0.95, weight_decay=0.01, nesterov=True, ns_steps=5,
                 scale_mode="moonlight", coeffs=None, eps=1e-7, row_block=None, col_block=None):
        if scale_mode not in mb.SCALE_MODES:
            raise ValueError(f"scale_mode must be one of {sorted(mb.SCALE_MODES)}")
        super().__init__(params, dict(lr=lr, momentum=momentum, weight_decay=weight_decay, nesterov=nesterov,
                                      ns_steps=ns_steps, scale_mode=scale_mode, coeffs=coeffs, eps=eps,
                                      row_block=row_block, col_block=col_block))
        for g in self.param_groups:
            for p in g["params"]:
                if p.dtype not in (torch.bfloat16, torch.float16, torch.float32):
                    raise ValueError(f"unsupported parameter dtype {p.dtype}")
                self._blocks(p, g)
        self._ws = _Workspaces()

    def __setstate__(self, state):     # copies and pickles carry the state alone; load_state_dict comes here too
        super().__setstate__(state)
        self.__dict__.setdefault("_ws", _Workspaces())

    @staticmethod
    def _blocks(t, group):
        if group["row_block"] is not None and group["col_block"] is not None:
            raise ValueError("give row_block or col_block, not both")
        if t.dim() == 2 and group["row_block"] is not None:
            return ms.row_blocks(t, group["row_block"])
        if t.dim() == 2 and group["col_block"] is not None:
            return ms.col_blocks(t, group["col_block"])
        if t.dim() not in (2, 3):
            raise ValueError(f"StackedMuon handles matrices and stacks of them, got shape {tuple(t.shape)}; "
                             "give embeddings, heads, biases and norms to AdamW")
        return t

    @torch.no_grad()
    def step(self, closure=None, grad_scale=None):
        loss = None
        if closure is not None:
            with torch.enable_grad():
                loss = closure()
        for group in self.param_groups:
            stacks = []
            for p in group["params"]:
                if p.grad is None or p.numel() == 0:     # a rank without experts, say
                    continue
                state = self.state[p]
                if "momentum_buffer" not in state:
                    if _capturing():
                        raise RuntimeError("a parameter's first step cannot be captured: every replay would begin with "
                                           "its momentum at zero")
                    state["momentum_buffer"] = torch.zeros(p.shape, dtype=torch.float32, device=p.device)
                stacks.append(mb.MuonStack(*(self._blocks(t, group) for t in
                                             (p.data, p.grad.contiguous(), state["momentum_buffer"]))))
            if not stacks:
                continue
            coeffs = group["coeffs"] or [KJ_COEFFS] * group["ns_steps"]
            hp = mb.hyper(group["lr"], group["momentum"], group["weight_decay"], group["nesterov"],
                          group["scale_mode"], mb.Schedule(coeffs, eps=group["eps"]))
            ws = self._ws.get(mb.muon_stacks_workspace_size(stacks, hp), stacks[0].W.device)
            mb.muon_step_stacks(stacks, hp, ws, grad_scale=grad_scale)
        return loss


class AdamW(_Fp32State):
    """AdamW for what Muon does not take, one grouped call per param group.  Parameters of any shape,
    dense, bf16, fp16 or fp32; moments in fp32.  The number of the step is a host integer, so step() refuses
    to be captured in a CUDA graph (binding.adamw_step_batched takes a device step count for that)."""

    def __init__(self, params, lr=1e-3, betas=(0.9, 0.999), eps=1e-8, weight_decay=0.01):
        super().__init__(params, dict(lr=lr, betas=betas, eps=eps, weight_decay=weight_decay))
        for g in self.param_groups:
            for p in g["params"]:
                if p.dtype not in (torch.bfloat16, torch.float16, torch.float32):
                    raise ValueError(f"unsupported parameter dtype {p.dtype}")

    def load_state_dict(self, state_dict):
        """Takes a state of torch.optim.AdamW too, where its rule is this one."""
        for g in state_dict["param_groups"]:
            if g.get("amsgrad") or g.get("maximize") or (g.get("weight_decay") and not g.get("decoupled_weight_decay", True)):
                raise ValueError("the state is of another rule than AdamW's (amsgrad, maximize or weight decay in the gradient)")
        super().load_state_dict(state_dict)

    @torch.no_grad()
    def step(self, closure=None, grad_scale=None):
        if _capturing():
            raise RuntimeError("AdamW.step() cannot be captured: every replay would use the captured step's number")
        loss = None
        if closure is not None:
            with torch.enable_grad():
                loss = closure()
        for group in self.param_groups:
            by_step = {}
            for p in group["params"]:
                if p.grad is None:
                    continue
                state = self.state[p]
                if "step" not in state:
                    state["step"] = 0
                    state["exp_avg"] = torch.zeros(p.shape, dtype=torch.float32, device=p.device)
                    state["exp_avg_sq"] = torch.zeros(p.shape, dtype=torch.float32, device=p.device)
                states, tensors = by_step.setdefault(state["step"] + 1, ([], []))
                states.append(state)
                tensors.append(mb.AdamWTensor(p.data, p.grad.contiguous(), state["exp_avg"], state["exp_avg_sq"]))
            hp = mb.adamw_hyper(group["lr"], *group["betas"], group["eps"], group["weight_decay"])
            for step, (states, tensors) in by_step.items():
                mb.adamw_step_batched(tensors, hp, step, grad_scale=grad_scale)
                for state in states:       # a refused call has not counted
                    state["step"] = step
        return loss
