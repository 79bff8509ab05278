"""Plain 64-bit forms of the token embedding, the gated recurrence and the
vocabulary loss, for the tests: loops in the order of the definitions, on the
CPU, with what bounds the rounding of a result in fewer bits.

Bounds. A sum of n products taken in 32 bits in any order is off by at most
about n 2^-24 times the sum of the products' absolute values (each partial sum
and each product is rounded by half a step, 2^-24 relative); a result in its
storage type is off by half a step more, eps / 2 of that type. So every bound
below is  count * 2^-24 * (the same expression in absolute values) + eps / 2 *
|result|, with a count that is derived where it is used."""
from __future__ import annotations

import math

import torch

F32_STEP = 2.0 ** -24


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def within(got, ref, size, count, what):
    """|got - ref| <= count 2^-24 size + half a step of |ref|, value by value;
    values below the type's normal range may be off by its smallest one."""
    assert tuple(got.shape) == tuple(ref.shape), (what, got.shape, ref.shape)
    tiny = torch.finfo(got.dtype).tiny
    u = half_step(got.dtype)
    got, ref = got.detach().double().cpu(), ref.detach().double().cpu()
    size = torch.as_tensor(size, dtype=torch.float64).cpu()
    assert torch.isfinite(got).all(), f"{what}: non-finite"
    if not ref.numel():
        return
    slack = count * F32_STEP * size
    bound = slack + u * (ref.abs() + slack) + tiny
    worst = float(((got - ref).abs() / bound).max())
    assert worst <= 1.0, f"{what}: {worst:.3f} times the bound"


def lengths(lens, B, L):
    return [L] * B if lens is None else [min(max(int(n), 0), L) for n in lens]


# ---- embedding ----------------------------------------------------------------
def embedding(ids, weight, scale=1.0, lens=None):
    B, L = ids.shape
    V, D = weight.shape
    out = torch.zeros(B, L, D, dtype=torch.float64)
    for b, n in enumerate(lengths(lens, B, L)):
        for t in range(n):
            if 0 <= int(ids[b, t]) < V:
                out[b, t] = weight[int(ids[b, t])].double() * scale
    return out


def embedding_grad(ids, gy, V, scale=1.0, lens=None):
    """(gradient, the same in absolute values, tokens of each row)."""
    B, L, D = gy.shape
    dw, size, count = (torch.zeros(V, D, dtype=torch.float64) for _ in range(3))
    for b, n in enumerate(lengths(lens, B, L)):
        for t in range(n):
            v = int(ids[b, t])
            if 0 <= v < V:
                dw[v] += scale * gy[b, t].double()
                size[v] += abs(scale) * gy[b, t].double().abs()
                count[v] += 1
    return dw, size, count


# ---- gated recurrence ---------------------------------------------------------
def gated(x, r, i, A, state=None, lens=None, absolute=False):
    """(out, state_out), float64; absolute: of |x| and |state|."""
    x, r, i, A = (t.double() for t in (x, r, i, A))
    B, L, C = x.shape
    if absolute:
        x = x.abs()
    outs, ends = [], []
    for b, n in enumerate(lengths(lens, B, L)):
        h = state[b].double() if state is not None else x.new_zeros(C)
        if absolute:
            h = h.abs()
        rows = []
        for t in range(n):
            log_a = A * torch.sigmoid(r[b, t])
            h = torch.exp(log_a) * h + torch.sqrt(-torch.expm1(2 * log_a)) * torch.sigmoid(i[b, t]) * x[b, t]
            rows.append(h)
        rows += [x.new_zeros(C)] * (L - n)
        outs.append(torch.stack(rows) if rows else x.new_zeros(0, C))
        ends.append(h)
    return torch.stack(outs), torch.stack(ends)


def gated_grads(x, r, i, A, gy, state=None, lens=None, grad_state=None, absolute=False):
    """Gradients by the formula, and with ``absolute`` the same expression with
    every term taken in absolute value."""
    x, r, i, A, gy = (t.double() for t in (x, r, i, A, gy))
    B, L, C = x.shape
    mag = (lambda t: t.abs()) if absolute else (lambda t: t)
    x, gy = mag(torch.nan_to_num(x)), mag(gy)
    d = {k: torch.zeros(B, L, C, dtype=torch.float64) for k in ("x", "r", "i")}
    d["A"] = torch.zeros(C, dtype=torch.float64)
    dstate = torch.zeros(B, C, dtype=torch.float64)
    for b, n in enumerate(lengths(lens, B, L)):
        h = [mag(state[b].double()) if state is not None else x.new_zeros(C)]
        s, w = torch.sigmoid(r[b]), torch.sigmoid(i[b])
        a, left = torch.exp(A * s), -torch.expm1(2 * A * s)
        beta = left.sqrt()
        for t in range(n):
            h.append(a[t] * h[-1] + beta[t] * w[t] * x[b, t])
        carry = mag(grad_state[b].double()) if grad_state is not None else x.new_zeros(C)
        for t in range(n - 1, -1, -1):
            g = gy[b, t] + carry
            slope = torch.where(left[t] > 0, a[t] ** 2 / beta[t], torch.zeros_like(beta[t]))
            u = w[t] * x[b, t]
            k = g * (a[t] * h[t] + slope * u) if absolute else g * (a[t] * h[t] - slope * u)
            d["r"][b, t] = k * mag(A) * s[t] * (1 - s[t])
            d["A"] += k * s[t]
            d["x"][b, t] = g * beta[t] * w[t]
            d["i"][b, t] = g * beta[t] * x[b, t] * w[t] * (1 - w[t])
            carry = a[t] * g
        dstate[b] = carry
    if state is not None:
        d["state"] = dstate
    return d


# ---- vocabulary loss ----------------------------------------------------------
def vocab_loss(x, weight, targets, lens=None):
    """(loss, lse), float64 [B, L]."""
    B, L, D = x.shape
    V = weight.shape[0]
    x, weight = x.double(), weight.double()
    loss, lse = torch.zeros(2, B, L, dtype=torch.float64)
    for b, n in enumerate(lengths(lens, B, L)):
        for t in range(n):
            z = weight @ x[b, t]
            m = z.max()
            lse[b, t] = m + math.log(float(torch.exp(z - m).sum()))
            if 0 <= int(targets[b, t]) < V:
                loss[b, t] = lse[b, t] - z[int(targets[b, t])]
    return loss, lse


def vocab_loss_grads(x, weight, targets, grad, lens=None):
    """{"x", "weight"} and the same sums in absolute values."""
    B, L, D = x.shape
    V = weight.shape[0]
    x, weight = x.double(), weight.double()
    dx, sx = torch.zeros(2, B, L, D, dtype=torch.float64)
    dw, sw = torch.zeros(2, V, D, dtype=torch.float64)
    for b, n in enumerate(lengths(lens, B, L)):
        for t in range(n):
            if not 0 <= int(targets[b, t]) < V:
                continue
            p = torch.softmax(weight @ x[b, t], 0)
            p[int(targets[b, t])] -= 1
            G = float(grad[b, t]) * p
            dx[b, t] = G @ weight
            sx[b, t] = G.abs() @ weight.abs()
            dw += G[:, None] * x[b, t]
            sw += G.abs()[:, None] * x[b, t].abs()
    return {"x": dx, "weight": dw}, {"x": sx, "weight": sw}
