"""Plain 64-bit forms of the token-sequence operators, for the tests: loops
over tokens and heads in the order of the definitions, on the CPU."""
from __future__ import annotations

import math

import torch


def conv(x, w, bias=None, state=None, lens=None, silu=True):
    """(out, state_out), float64; x [B, L, C], w [C, K]."""
    x, w = x.double(), w.double()
    B, L, C = x.shape
    K = w.shape[1]
    outs, ends = [], []
    for b in range(B):
        n = L if lens is None else min(max(int(lens[b]), 0), L)
        head = state[b].double() if state is not None else x.new_zeros(K - 1, C)
        xx = torch.cat([head, x[b, :n]], 0)
        rows = []
        for t in range(n):
            pre = (w.T * xx[t:t + K]).sum(0)
            if bias is not None:
                pre = pre + bias.double()
            rows.append(pre * torch.sigmoid(pre) if silu else pre)
        rows += [x.new_zeros(C)] * (L - n)
        outs.append(torch.stack(rows) if rows else x.new_zeros(0, C))
        ends.append(xx[n:n + K - 1])
    return torch.stack(outs), torch.stack(ends)


def scan(x, dt, A, Bm, Cm, D=None, z=None, dt_bias=None, state=None, lens=None, softplus=True):
    """(out, state_out), float64; Bm, Cm [B, L, G, N]."""
    x, dt, A, Bm, Cm = (t.double() for t in (x, dt, A, Bm, Cm))
    B, L, C = x.shape
    G, N = Bm.shape[2], A.shape[1]
    outs, ends = [], []
    for b in range(B):
        n = L if lens is None else min(max(int(lens[b]), 0), L)
        h = state[b].double() if state is not None else x.new_zeros(C, N)
        rows = []
        for t in range(n):
            d = dt[b, t] if dt_bias is None else dt[b, t] + dt_bias.double()
            if softplus:
                d = torch.logaddexp(d, torch.zeros_like(d))
            Bt = Bm[b, t].repeat_interleave(C // G, 0)
            Ct = Cm[b, t].repeat_interleave(C // G, 0)
            h = torch.exp(d[:, None] * A) * h + (d * x[b, t])[:, None] * Bt
            y = (Ct * h).sum(1)
            if D is not None:
                y = y + D.double() * x[b, t]
            if z is not None:
                zz = z[b, t].double()
                y = y * zz * torch.sigmoid(zz)
            rows.append(y)
        rows += [x.new_zeros(C)] * (L - n)
        outs.append(torch.stack(rows) if rows else x.new_zeros(0, C))
        ends.append(h)
    return torch.stack(outs), torch.stack(ends)


def attention(q, k, v, mask=None, scale=None):
    """(out, lse), float64; q [B, Lq, Hq, E], k, v [B, Lk, Hkv, E]."""
    q, k, v = q.double(), k.double(), v.double()
    B, Lq, Hq, E = q.shape
    Hkv = k.shape[2]
    scale = E ** -0.5 if scale is None else scale
    outs, lses = [], []
    for b in range(B):
        keys = torch.arange(k.shape[1])
        if mask is not None:
            keys = keys[mask[b].cpu()]
        per, per_l = [], []
        for h in range(Hq):
            j = h // (Hq // Hkv)
            if len(keys) == 0:
                per.append(torch.zeros(Lq, E, dtype=torch.float64))
                per_l.append(torch.full((Lq,), -math.inf, dtype=torch.float64))
                continue
            s = scale * (q[b, :, h] @ k[b, keys, j].T)
            per_l.append(torch.logsumexp(s, 1))
            per.append(torch.exp(s - per_l[-1][:, None]) @ v[b, keys, j])
        outs.append(torch.stack(per, 1))
        lses.append(torch.stack(per_l, 0))
    return torch.stack(outs), torch.stack(lses)


def gradients(fn, inputs: dict, wrt, grad_out, grad_state=None):
    """dL/dname for name in wrt, L = <fn(**inputs)[0], grad_out> (+ <second
    result, grad_state>), by automatic differentiation in 64 bits."""
    leaf = {n: (t.double().detach().requires_grad_(True) if n in wrt else t) for n, t in inputs.items()}
    out, state = fn(**leaf)
    loss = (out * grad_out.double()).sum()
    if grad_state is not None:
        loss = loss + (state * grad_state.double()).sum()
    if not loss.requires_grad:      # nothing to compute: no tokens, no keys
        return {n: torch.zeros_like(leaf[n]) for n in wrt}
    got = torch.autograd.grad(loss, [leaf[n] for n in wrt], allow_unused=True)
    return {n: torch.zeros_like(leaf[n]) if g is None else g for n, g in zip(wrt, got)}


def difference(fn, inputs: dict, name, direction, grad_out, eps=1e-4):
    """d/de L(inputs[name] + e direction) at 0 by a central difference in 64
    bits (error O(eps^2))."""
    def loss(e):
        moved = dict(inputs)
        moved[name] = inputs[name].double() + e * direction.double()
        return float((fn(**moved)[0] * grad_out.double()).sum())
    return (loss(eps) - loss(-eps)) / (2 * eps)
