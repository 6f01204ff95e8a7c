"""The workloads that time the stacked-block operators and AdamW: their inputs, their plain form and their exact values.

Four operators, as a training program uses them:
  orth   Newton-Schulz orthogonalisation of stacks of equal blocks (heads, experts), any sizes, strided views
  grad   the same through autograd: the orthogonalised blocks and the gradient of their input
  muon   the whole Muon step on such stacks, the gradient scaled by a clip factor that is on the device
  adamw  the global gradient norm with its clip factor, and AdamW on what Muon does not take
and `train`: one optimizer step of a small model, norm, Muon and AdamW together.

`own` chooses between the plain form and this package's operators.
"""
import math

import torch

own = False

KJ = (3.4445, -4.7750, 2.0315)          # an optimizer's updates
STABLE = (1.875, -1.25, 0.375)          # an orthogonal parametrisation: converges to the polar factor
STEPS = 5
EPS = 1e-7
LR, BETA, DECAY = 0.02, 0.95, 0.1
ADAM = dict(lr=3e-4, beta1=0.9, beta2=0.95, eps=1e-8, weight_decay=0.1)
MAX_NORM = 1.0
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def listed():
    return [
        # one layer's query heads of a 768-wide model: the smallest call, a few launches' latency
        {"name": "orth-heads", "op": "orth", "count": 12, "rows": 64, "cols": 768, "x": "bf16", "y": "bf16", "pad": 0},
        # stacked experts with odd sides in a padded buffer, fp32 gradients accumulated over micro-batches
        {"name": "orth-experts-odd", "op": "orth", "count": 24, "rows": 509, "cols": 1021, "x": "fp32", "y": "bf16",
         "pad": 3},
        # a whole MLP matrix of a 7B model, tall
        {"name": "orth-mlp", "op": "orth", "count": 1, "rows": 11008, "cols": 4096, "x": "bf16", "y": "bf16", "pad": 0},
        # orthogonally parametrised heads, ragged width
        {"name": "grad-heads", "op": "grad", "count": 16, "rows": 96, "cols": 641, "x": "fp16", "pad": 0},
        # two orthogonally parametrised square projections
        {"name": "grad-square", "op": "grad", "count": 2, "rows": 2048, "cols": 2048, "x": "bf16", "pad": 0},
        # four layers' rectangular projections of the same parametrisation, tall
        {"name": "grad-tall", "op": "grad", "count": 4, "rows": 1408, "cols": 520, "x": "bf16", "pad": 0},
        # fused QKV of a 7B layer, one block per head
        {"name": "muon-qkv-heads", "op": "muon", "count": 96, "rows": 128, "cols": 4096, "pad": 0, "idle": 0},
        # stacked experts' down projections; two experts saw no token
        {"name": "muon-experts", "op": "muon", "count": 16, "rows": 2048, "cols": 1408, "pad": 0, "idle": 2},
        # the gate and up halves of a small fused matrix, side by side in its rows
        {"name": "muon-fused-small", "op": "muon", "count": 2, "rows": 320, "cols": 257, "pad": 257, "idle": 0},
        # norms and biases of a small model: many short tensors
        {"name": "adamw-small", "op": "adamw", "tensors": 50, "width": 768, "vocab": 0, "g": "fp32"},
        # a 7B model's embedding, head and norms
        {"name": "adamw-embedding", "op": "adamw", "tensors": 65, "width": 4096, "vocab": 32000, "g": "bf16"},
        # one optimizer step of a small model: clip, Muon on its blocks, AdamW on the rest
        {"name": "train-step", "op": "train", "layers": 4, "width": 1024, "head": 64, "ff": 2752, "vocab": 32003},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    op = rng.choice(["orth", "orth", "grad", "muon", "muon", "adamw", "train"])
    if op == "adamw":
        return {"op": op, "tensors": _log(rng, 1, 400), "width": _log(rng, 1, 8192),
                "vocab": rng.choice([0, _log(rng, 100, 20000)]), "g": rng.choice(["bf16", "fp16", "fp32"])}
    if op == "train":
        head = rng.choice([32, 64, 80, 128])
        return {"op": op, "layers": _log(rng, 1, 6), "width": head * rng.randint(2, 8), "head": head,
                "ff": _log(rng, 200, 2000), "vocab": _log(rng, 500, 30000)}
    while True:
        rows, cols, count = _log(rng, 16, 4096), _log(rng, 16, 4096), _log(rng, 1, 64)
        small, large = min(rows, cols), max(rows, cols)
        if count * small * small * large <= (3e10 if op == "grad" else 1e11) and count * small * large <= 4e7:
            break
    c = {"op": op, "count": count, "rows": rows, "cols": cols, "pad": rng.choice([0, 0, rng.randint(1, 64)])}
    if op == "muon":
        c["idle"] = rng.choice([0, 0, min(1, count - 1)])
    else:
        c["x"] = rng.choice(["bf16", "fp16"]) if op == "grad" else rng.choice(["bf16", "fp16", "fp32"])
    if op == "orth":
        c["y"] = "bf16"
    return c


# ------------------------------------------------------------------------------------------ inputs
def _view(count, rows, cols, pad, dtype):
    """[count, rows, cols] inside a buffer whose rows are `pad` elements longer."""
    return torch.zeros((count, rows, cols + pad), dtype=dtype, device="cuda")[:, :, :cols]


def _gradient(gen, count, rows, cols, std=1e-3):
    """Blocks with the falling spectrum of a layer's gradient (sigma_i ~ i^-0.7), of element size about std."""
    k = min(rows, cols)
    fall = torch.arange(1, k + 1, device="cuda", dtype=torch.float32) ** -0.7
    fall = fall / fall.norm()
    left = torch.randn((count, rows, k), generator=gen, device="cuda")
    right = torch.randn((count, k, cols), generator=gen, device="cuda")
    return torch.matmul(left * fall, right) * std


def _near_orthogonal(gen, count, rows, cols):
    """Blocks of a trained orthogonal parametrisation: a random matrix two Newton-Schulz steps towards its polar factor."""
    x = torch.randn((count, rows, cols), generator=gen, device="cuda")
    x = x / (math.sqrt(rows) + math.sqrt(cols))
    for _ in range(2):
        x = 1.5 * x - 0.5 * torch.matmul(x, torch.matmul(x.transpose(1, 2), x)) if cols <= rows else \
            1.5 * x - 0.5 * torch.matmul(torch.matmul(x, x.transpose(1, 2)), x)
    return x


def _muon_state(gen, count, rows, cols, pad, idle):
    st = {"W": _view(count, rows, cols, pad, torch.bfloat16), "G": _view(count, rows, cols, pad, torch.bfloat16),
          "M": _view(count, rows, cols, pad, torch.float32)}
    st["W"].copy_(torch.randn((count, rows, cols), generator=gen, device="cuda") * 0.02)
    st["G"].copy_(_gradient(gen, count, rows, cols))
    st["M"].copy_(_gradient(gen, count, rows, cols, std=1e-2))
    if idle:
        st["G"][:idle] = 0
        st["M"][:idle] = 0
    return st


def _adam_state(gen, shape, g):
    st = {"W": (torch.randn(shape, generator=gen, device="cuda") * 0.02).to(torch.bfloat16),
          "G": (torch.randn(shape, generator=gen, device="cuda") * 1e-3).to(g),
          "m": torch.randn(shape, generator=gen, device="cuda") * 1e-4,
          "v": torch.randn(shape, generator=gen, device="cuda").square() * 1e-6}
    return st


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    c, op, st = case, case["op"], {"case": case, "step": 100}
    if op in ("orth", "grad"):
        x = _view(c["count"], c["rows"], c["cols"], c["pad"], TYPES[c["x"]])
        make = _gradient if op == "orth" else _near_orthogonal
        x.copy_(make(gen, c["count"], c["rows"], c["cols"]))
        st["X"] = x
        if op == "grad":
            st["dY"] = (torch.randn(x.shape, generator=gen, device="cuda") * 1e-2).to(x.dtype)
    elif op == "muon":
        st["stacks"] = [_muon_state(gen, c["count"], c["rows"], c["cols"], c["pad"], c["idle"])]
        st["scale"] = torch.full((1,), 0.37, device="cuda")
    elif op == "adamw":
        shapes = [(c["width"] + i % 3,) for i in range(c["tensors"])] + [(c["vocab"], c["width"])] * (2 if c["vocab"] else 0)
        st["tensors"] = [_adam_state(gen, s, TYPES[c["g"]]) for s in shapes]
    else:
        d, h, f, n = c["width"], c["head"], c["ff"], c["layers"]
        st["stacks"] = []
        for _ in range(n):
            st["stacks"].append(_muon_state(gen, 3 * d // h, h, d, 0, 0))   # fused QKV, a block per head
            st["stacks"].append(_muon_state(gen, 1, d, d, 0, 0))            # attention output
            st["stacks"].append(_muon_state(gen, 2, f, d, 0, 0))            # fused gate and up
            st["stacks"].append(_muon_state(gen, 1, d, f, 0, 0))            # down
        shapes = [(c["vocab"], d)] + [(d,)] * (2 * n + 1)
        st["tensors"] = [_adam_state(gen, s, torch.bfloat16) for s in shapes]
    return st


# ------------------------------------------------------------------------------------------ the plain form
def _plain_ns(u, coeffs=KJ):
    x = u.float()
    x = x / (x.square().sum(dim=(1, 2), keepdim=True, dtype=torch.float64).sqrt().float() + EPS)
    a, b, c = coeffs
    tall = x.shape[1] > x.shape[2]
    for _ in range(STEPS):
        if tall:
            g = torch.matmul(x.transpose(1, 2), x)
            x = a * x + torch.matmul(x, b * g + c * torch.matmul(g, g))
        else:
            g = torch.matmul(x, x.transpose(1, 2))
            x = a * x + torch.matmul(b * g + c * torch.matmul(g, g), x)
    return x


def _plain_muon(st, scale):
    w, m = st["W"], st["M"]
    g = st["G"].float() * scale
    m.copy_(BETA * m + g)
    o = _plain_ns(BETA * m + g)
    step = LR * 0.2 * math.sqrt(max(w.shape[1:]))
    w.copy_(((1 - LR * DECAY) * w.float() - step * o).to(w.dtype))


def _plain_norm(grads):
    total = torch.zeros((), dtype=torch.float64, device="cuda")
    for g in grads:
        total = total + g.float().square().sum(dtype=torch.float64)
    norm = total.sqrt().float()
    return norm, torch.clamp(MAX_NORM / (norm + 1e-6), max=1.0)


def _plain_adamw(st, scale, t):
    w, m, v, h = st["W"], st["m"], st["v"], ADAM
    g = st["G"].float() * scale
    m.copy_(h["beta1"] * m + (1 - h["beta1"]) * g)
    v.copy_(h["beta2"] * v + (1 - h["beta2"]) * g * g)
    u = (m / (1 - h["beta1"] ** t)) / ((v / (1 - h["beta2"] ** t)).sqrt() + h["eps"])
    w.copy_(((1 - h["lr"] * h["weight_decay"]) * w.float() - h["lr"] * u).to(w.dtype))


def _run_plain(st):
    c, op = st["case"], st["case"]["op"]
    if op == "orth":
        return _plain_ns(st["X"]).to(TYPES[c["y"]])
    if op == "grad":
        x = st["X"].detach().float().requires_grad_(True)
        y = _plain_ns(x, STABLE)
        (dx,) = torch.autograd.grad(y, x, st["dY"].float())
        return y.detach().to(st["X"].dtype), dx.to(st["X"].dtype)
    out = {}
    if op == "muon":
        scale = st["scale"]
    else:
        every = [s["G"] for s in st.get("stacks", [])] + [t["G"] for t in st["tensors"]]
        out["norm"], scale = _plain_norm(every)
    for s in st.get("stacks", []):
        _plain_muon(s, scale)
    for t in st.get("tensors", []):
        _plain_adamw(t, scale, st["step"])
    return _updated(st, out)


# ------------------------------------------------------------------------------------------ this package's operators
def _run_own(st):
    from matrix_orthogonalising_optimizer_02_b200 import binding as mb
    from matrix_orthogonalising_optimizer_02_b200 import stacks as ms
    c, op = st["case"], st["case"]["op"]
    if op == "orth":
        return ms.orthogonalize(st["X"], steps=STEPS, coeffs=KJ, eps=EPS, dtype=TYPES[c["y"]])
    if op == "grad":
        x = st["X"].detach().requires_grad_(True)
        y = ms.orthogonalize(x, steps=STEPS, coeffs=STABLE, eps=EPS)
        (dx,) = torch.autograd.grad(y, x, st["dY"])
        return y.detach(), dx
    out = {}
    if op == "muon":
        scale = st["scale"]
    else:
        every = [s["G"] for s in st.get("stacks", [])] + [t["G"] for t in st["tensors"]]
        if "norm_ws" not in st:
            st["norm_ws"] = mb.workspace(mb.grad_norm_workspace_size(every))
            st["norm"] = torch.empty(2, device="cuda")
        mb.grad_norm_batched(every, MAX_NORM, st["norm"], st["norm_ws"])
        out["norm"], scale = st["norm"][0], st["norm"][1:]
    if st.get("stacks"):
        stacks = [mb.MuonStack(s["W"], s["G"], s["M"]) for s in st["stacks"]]
        hp = mb.hyper(LR, BETA, DECAY, nesterov=True, schedule=mb.Schedule.fixed(STEPS, KJ, eps=EPS))
        if "muon_ws" not in st:
            st["muon_ws"] = mb.workspace(mb.muon_stacks_workspace_size(stacks, hp))
        mb.muon_step_stacks(stacks, hp, st["muon_ws"], grad_scale=scale)
    if st.get("tensors"):
        tensors = [mb.AdamWTensor(t["W"], t["G"], t["m"], t["v"]) for t in st["tensors"]]
        mb.adamw_step_batched(tensors, mb.adamw_hyper(**ADAM), step=st["step"], grad_scale=scale)
    return _updated(st, out)


# The updated buffers; of many alike, the first and the last ones.
def _updated(st, out):
    stacks, tensors = st.get("stacks", []), st.get("tensors", [])
    for i, s in enumerate(stacks[:4] + stacks[4:][-4:]):
        out["stack%d" % i] = {"W": s["W"], "M": s["M"]}
    long = [t for t in tensors if t["W"].dim() == 2]
    short = [t for t in tensors if t["W"].dim() == 1]
    for i, t in enumerate(long):
        out["long%d" % i] = {"W": t["W"], "m": t["m"], "v": t["v"]}
    for i, t in enumerate(short[:4] + short[4:][-4:]):
        out["short%d" % i] = {"W": t["W"], "m": t["m"], "v": t["v"]}
    return out


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ------------------------------------------------------------------------------------------ floors
def _ns_work(count, rows, cols):
    r, s = min(rows, cols), max(rows, cols)
    direct = STEPS * (3.0 * r * r * s + float(r) ** 3)      # symmetric products counted once
    through_gram = 3.0 * r * r * s + 4.0 * STEPS * float(r) ** 3
    return count * min(direct, through_gram)


def _sizes(case):
    c, op = case, case["op"]
    if op in ("orth", "grad", "muon"):
        return [(c["count"], c["rows"], c["cols"])], 0
    if op == "adamw":
        return [], sum(c["width"] + i % 3 for i in range(c["tensors"])) + 2 * c["vocab"] * c["width"]
    d, h, f, n = c["width"], c["head"], c["ff"], c["layers"]
    return [(3 * d // h, h, d), (1, d, d), (2, f, d), (1, d, f)] * n, c["vocab"] * d + (2 * n + 1) * d


def work(case):
    blocks, rest = _sizes(case)
    op, size = case["op"], {"bf16": 2, "fp16": 2, "fp32": 4}
    n = float(sum(k * r * s for k, r, s in blocks))
    flops = sum(_ns_work(*b) for b in blocks)
    if op == "orth":
        return {"bytes": n * (size[case["x"]] + size[case["y"]]), "flops": flops}
    if op == "grad":
        k, r, s = blocks[0]
        small, large = min(r, s), max(r, s)
        flops += k * STEPS * (6.0 * small * small * large + 2.0 * float(small) ** 3)
        return {"bytes": n * 4 * size[case["x"]], "flops": flops}
    g = size[case["g"]] if op == "adamw" else 2
    norm = 0 if op == "muon" else 1                          # the norm reads every gradient once more
    return {"bytes": n * (4 + 8 + 2 * (1 + norm)) + rest * (4 + 16 + g * (1 + norm)), "flops": flops + 20.0 * rest}


# ------------------------------------------------------------------------------------------ exact values, in 64 bits
def _exact_iterates(u, coeffs):
    """All iterates, blocks turned wide."""
    x = u.double()
    n = torch.linalg.vector_norm(x, dim=(1, 2), keepdim=True)
    xs = [x / (n + EPS)]
    a, b, c = coeffs
    for _ in range(STEPS):
        x = xs[-1]
        g = x @ x.mT
        q = b * g + c * (g @ g)
        q.diagonal(dim1=1, dim2=2).add_(a)
        xs.append(q @ x)
    return xs, n


def _wide(x):
    return x.mT if x.shape[1] > x.shape[2] else x


def _exact_ns(u):
    x = _exact_iterates(_wide(u), KJ)[0][-1]
    return x.mT if u.shape[1] > u.shape[2] else x


def _exact_grad(u, dy):
    """The reverse pass written out: with S = sym(D X^T) and P = bS + c(SA + AS), dX = aD + BD + 2PX."""
    xs, n = _exact_iterates(_wide(u), STABLE)
    d = _wide(dy).double()
    a, b, c = STABLE
    for x in reversed(xs[:-1]):
        g = x @ x.mT
        s = d @ x.mT
        s = 0.5 * (s + s.mT)
        p = b * s + c * (s @ g + g @ s)
        d = a * d + b * (g @ d) + c * (g @ (g @ d)) + 2.0 * (p @ x)
    w = _wide(u).double()
    along = (d * w).sum(dim=(1, 2), keepdim=True) / (n * (n + EPS) ** 2)
    dx = d / (n + EPS) - along * w
    y = xs[-1]
    return (y.mT, dx.mT) if u.shape[1] > u.shape[2] else (y, dx)


def _exact_step(st, out, scale):
    """The step on copies: the updated buffers in 64 bits, laid out as run() returns them."""
    new = {"stacks": [], "tensors": []}
    for s in st.get("stacks", []):
        g = s["G"].double() * scale
        m = BETA * s["M"].double() + g
        u = BETA * m + g
        o = torch.zeros_like(u)
        live = u.abs().amax(dim=(1, 2)) > 0
        o[live] = _exact_ns(u[live])
        w = (1 - LR * DECAY) * s["W"].double() - LR * 0.2 * math.sqrt(max(u.shape[1:])) * o
        new["stacks"].append({"W": w, "M": m})
    h, t = ADAM, st["step"]
    for x in st.get("tensors", []):
        g = x["G"].double() * scale
        m = h["beta1"] * x["m"].double() + (1 - h["beta1"]) * g
        v = h["beta2"] * x["v"].double() + (1 - h["beta2"]) * g ** 2
        w = x["W"].double() * (1 - h["lr"] * h["weight_decay"])
        w -= h["lr"] / (1 - h["beta1"] ** t) * m / (torch.sqrt(v) / math.sqrt(1 - h["beta2"] ** t) + h["eps"])
        new["tensors"].append({"W": w, "m": m, "v": v})
    return _updated(new, out)


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "orth":
        return _exact_ns(st["X"])
    if op == "grad":
        return _exact_grad(st["X"], st["dY"])
    out, scale = {}, None
    if op == "muon":
        scale = st["scale"].double()
    else:
        squares = [torch.linalg.vector_norm(s["G"].double()) ** 2 for s in st.get("stacks", []) + st["tensors"]]
        out["norm"] = torch.stack(squares).sum().sqrt()
        scale = min(1.0, MAX_NORM / (float(out["norm"]) + 1e-6))
    return _exact_step(st, out, scale)
