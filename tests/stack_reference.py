"""Plain 64-bit forms of the stacked-block operators, the gradient norm and AdamW, for the tests."""
import math

import torch

KJ = (3.4445, -4.7750, 2.0315)
STABLE = (1.875, -1.25, 0.375)

# Half a step of fp16, the type the iterates are held in, relative to a value.
U16 = torch.finfo(torch.float16).eps / 2


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


# Tolerances (relative, 2-norm of a block), from the roundings of the method.  An iteration rounds
# A, B and the multiplied plane of X once each; a rounding of a plane is at most U16 per element,
# and over a block its 2-norm is about U16 / sqrt(3) of the plane's.  Independent errors of five
# iterations add up to sqrt(15) U16 / sqrt(3) = 2.3 U16 where later iterations keep errors as they
# are; the optimizer's polynomial amplifies them on the way (|p'| up to 3.5 on small singular values, each
# of which it moves up through a few iterations): a factor of 4 covers that for blocks without tiny
# singular values.  A converging polynomial contracts (p'(1) = 0): 2.3 U16 stands with a margin of 2.
def tol_kj(dtype):
    return 4 * 2.3 * U16 + half_step(dtype)


def tol_stable(dtype):
    return 2 * 2.3 * U16 + half_step(dtype)


# A vector has one singular value, so nothing averages.  Its path is known (sigma_0 = 1), and so is the worst
# case: with lambda = sigma^2 and q = b lambda + c lambda^2, a relative rounding u of A moves
# p(sigma) = sigma (a + q) by u sigma lambda |b + 2 c lambda|, those of B and of the multiplied plane of X
# by u sigma |q| each, and an earlier error goes on by |p'(sigma)|.  For the optimizer's schedule the
# sum after five iterations is 41 u; for the converging one 2.2 u.
def tol_vector(coeffs, dtype):
    s, e = 1.0, 0.0
    for a, b, c in coeffs:
        lam = s * s
        q = b * lam + c * lam * lam
        e = abs(a + 3 * b * lam + 5 * c * lam * lam) * e + U16 * s * (lam * abs(b + 2 * c * lam) + 2 * abs(q))
        s = s * (a + q)
    return e / abs(s) + half_step(dtype)


def ns(u, coeffs, eps=1e-7):
    """X_T of one block in 64 bits; coeffs: a list of (a, b, c)."""
    x = u.double()
    x = x / (torch.linalg.vector_norm(x) + eps)
    for a, b, c in coeffs:
        if x.shape[0] > x.shape[1]:
            g = x.T @ x
            x = a * x + x @ (b * g + c * (g @ g))
        else:
            g = x @ x.T
            x = a * x + (b * g + c * (g @ g)) @ x
    return x


def ns_grad(u, dy, coeffs, eps=1e-7):
    """Gradient of <dy, ns(u)>, from the reverse formulas."""
    if u.shape[0] > u.shape[1]:
        return ns_grad(u.T, dy.T, coeffs, eps).T
    x = u.double()
    n = torch.linalg.vector_norm(x)
    xs = [x / (n + eps)]
    for a, b, c in coeffs:
        g = xs[-1] @ xs[-1].T
        xs.append(a * xs[-1] + (b * g + c * (g @ g)) @ xs[-1])
    d = dy.double()
    for (a, b, c), x in zip(reversed(coeffs), reversed(xs[:-1])):
        g = x @ x.T
        s = 0.5 * (d @ x.T + x @ d.T)
        p = b * s + c * (s @ g + g @ s)
        d = a * d + (b * g + c * (g @ g)) @ d + 2 * p @ x
    out = d / (n + eps)
    if n > 0:
        out = out - u.double() * (d * u.double()).sum() / (n * (n + eps) ** 2)
    return out


def scale(rows, cols, mode):
    return {"moonlight": 0.2 * math.sqrt(max(rows, cols)), "kellerjordan": math.sqrt(max(1.0, rows / cols)),
            "mup": math.sqrt(rows / cols), "naive": 1.0}[mode]


def muon(w, g, m, lr, beta, wd, nesterov, mode, coeffs, gs=1.0, eps=1e-7):
    """(W, M, O) after one step of one block."""
    g = g.double() * gs
    m = beta * m.double() + g
    u = beta * m + g if nesterov else m
    o = ns(u, coeffs, eps)
    return (1 - lr * wd) * w.double() - lr * scale(*w.shape, mode) * o, m, o


def adamw(w, g, m, v, t, lr, b1, b2, eps, wd, gs=1.0):
    g = g.double() * gs
    m = b1 * m.double() + (1 - b1) * g
    v = b2 * v.double() + (1 - b2) * g * g
    u = (m / (1 - b1 ** t)) / (torch.sqrt(v / (1 - b2 ** t)) + eps)
    return (1 - lr * wd) * w.double() - lr * u, m, v


def rel(got, want):
    got, want = got.detach().double(), want.detach().double()
    d, n = torch.linalg.vector_norm(got - want), torch.linalg.vector_norm(want)
    return float(d / n) if n > 0 else float(d)
