"""Cases of the token-sequence operators: the causal convolution and the
selective scan of a state space block (whole prompts, training, single
tokens), and cross attention of image or text tokens to an encoder's states.

``run`` computes one pass: with ``own`` true by the framework's entry points,
otherwise in a plain form of elementary torch operations in 32 bits."""
from __future__ import annotations

import math

import torch

own = False

DEV = "cuda:0"
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
BYTES = {"f32": 4, "bf16": 2}


# --------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------
def listed():
    return [
        # one new token for each of 32 sequences in a serving loop
        dict(name="conv_step", op="conv", train=False, dtype="bf16", B=32, L=1, C=2304, K=4,
             ragged=False, state=True),
        # a batch of prompts of different lengths, padded to the longest
        dict(name="conv_prompts", op="conv", train=False, dtype="bf16", B=8, L=4096, C=2304, K=4,
             ragged=True, state=True),
        # a training step with odd sizes in full precision
        dict(name="conv_train_odd", op="conv", train=True, dtype="f32", B=3, L=1021, C=1153, K=3,
             ragged=False, state=False),
        # one new token for each of 64 sequences
        dict(name="scan_step", op="scan", train=False, dtype="bf16", B=64, L=1, C=2304, N=16, G=1,
             ragged=False, state=True, gate=True),
        # one long prompt alone: few channels against the card, a long axis
        dict(name="scan_long_prompt", op="scan", train=False, dtype="bf16", B=1, L=8192, C=2304,
             N=16, G=1, ragged=False, state=False, gate=True),
        # a batch of prompts of different lengths
        dict(name="scan_prompts", op="scan", train=False, dtype="bf16", B=16, L=2048, C=2304, N=16,
             G=1, ragged=True, state=True, gate=True),
        # a training step of ordinary size
        dict(name="scan_train", op="scan", train=True, dtype="bf16", B=8, L=2048, C=2304, N=16,
             G=1, ragged=False, state=False, gate=True),
        # odd sizes, grouped B and C, full precision
        dict(name="scan_train_odd", op="scan", train=True, dtype="f32", B=2, L=333, C=202, N=9,
             G=2, ragged=True, state=True, gate=False),
        # a decoder's one token over a long document's states, shared heads
        dict(name="attn_one_token", op="attn", train=False, dtype="bf16", B=8, Lq=1, Lk=8192,
             Hq=32, Hkv=8, E=128, mask=True),
        # the pixels of a 2048 x 1024 latent of 320 channels reading a prompt
        dict(name="attn_latent", op="attn", train=False, dtype="bf16", B=1, Lq=2048 * 1024, Lk=77,
             Hq=5, Hkv=5, E=64, mask=True),
        # a training step on long states with shared heads
        dict(name="attn_train", op="attn", train=True, dtype="bf16", B=2, Lq=4096, Lk=2048, Hq=16,
             Hkv=4, E=128, mask=True),
        # odd lengths and head size, full precision
        dict(name="attn_train_odd", op="attn", train=True, dtype="f32", B=2, Lq=333, Lk=129, Hq=6,
             Hkv=3, E=40, mask=True),
    ]


def _log(rng, lo, hi):
    """A whole number between lo and hi, its logarithm uniform."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    """One more case of the ranges above."""
    op = rng.choice(["conv", "scan", "attn"])
    train = rng.random() < 0.5
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op == "conv":
        B, C, K = _log(rng, 1, 32), _log(rng, 64, 4608), rng.choice([2, 3, 4])
        top = min(8192, (8 * 4096 * 2304) // (B * C * (4 if train else 1)))
        L = 1 if not train and rng.random() < 0.3 else _log(rng, 2, max(2, top))
        return dict(op=op, train=train, dtype=dtype, B=B, L=L, C=C, K=K,
                    ragged=rng.random() < 0.5, state=rng.random() < 0.5 or L == 1)
    if op == "scan":
        B, G = _log(rng, 1, 64), rng.choice([1, 1, 2])
        C, N = G * _log(rng, 32, 2304), rng.choice([4, 8, 9, 16, 16, 24])
        top = min(8192, (16 * 2048 * 2304 * 16) // (B * C * N * (4 if train else 1)))
        top = min(top, 2048) if train else top
        L = 1 if not train and rng.random() < 0.3 else _log(rng, 2, max(2, top))
        return dict(op=op, train=train, dtype=dtype, B=B, L=L, C=C, N=N, G=G,
                    ragged=rng.random() < 0.5, state=rng.random() < 0.5 or L == 1,
                    gate=rng.random() < 0.7)
    E, Hkv, share = rng.choice([32, 40, 64, 72, 96, 128]), _log(rng, 1, 16), rng.choice([1, 1, 2, 4])
    B, Hq = _log(rng, 1, 16), Hkv * share
    Lk = _log(rng, 1, 8192)
    # f32 costs about 16 times bf16's matrix time, a training step about 3.5 times a forward pass
    most = (4096 * 2048 * 2 * 16 * 128) // (16 if dtype == "f32" else 1) // (1 if train else 1)
    top = max(1, min(65536, most // (B * Hq * E * Lk), (1 << 30) // (B * Hq * Lk)))
    Lq = 1 if not train and rng.random() < 0.3 else _log(rng, 1, top)
    return dict(op=op, train=train, dtype=dtype, B=B, Lq=Lq, Lk=Lk, Hq=Hq, Hkv=Hkv, E=E,
                mask=rng.random() < 0.6)


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------
def _lens(c, gen):
    """Sequence lengths: the longest fills the batch, one may be empty."""
    if not c["ragged"]:
        return None
    n = torch.randint(0 if c["B"] > 2 else 1, c["L"] + 1, (c["B"],), generator=gen, device=DEV)
    n[0] = c["L"]
    if c["B"] > 3:
        n[2] = 0
    return n.to(torch.int32)


def prepare(c, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    t = TYPES[c["dtype"]]

    def normal(*shape, std=1.0, kind=t):
        x = torch.empty(shape, dtype=kind, device=DEV)
        return x.normal_(0.0, std, generator=gen)

    s = {"case": c}
    if c["op"] == "conv":
        B, L, C, K = c["B"], c["L"], c["C"], c["K"]
        s["x"] = normal(B, L, C)
        s["w"], s["bias"] = normal(C, K, std=K ** -0.5), normal(C, std=0.1)
        s["state"] = normal(B, K - 1, C) if c["state"] else None
        s["lens"] = _lens(c, gen)
        s["state_out"] = torch.empty((B, K - 1, C), dtype=t, device=DEV)
        if c["train"]:
            s["gy"] = normal(B, L, C)
    elif c["op"] == "scan":
        B, L, C, N, G = c["B"], c["L"], c["C"], c["N"], c["G"]
        s["x"], s["dt"] = normal(B, L, C), normal(B, L, C, std=0.5)
        s["z"] = normal(B, L, C) if c["gate"] else None
        # B and C as a projection leaves them: slices of one row
        bc = normal(B, L, 2 * G * N)
        s["Bm"] = bc[..., :G * N].unflatten(-1, (G, N))
        s["Cm"] = bc[..., G * N:].unflatten(-1, (G, N))
        n = torch.arange(1, N + 1, device=DEV, dtype=torch.float32)
        s["A"] = -n * torch.exp(normal(C, N, std=0.1, kind=torch.float32))
        s["D"] = normal(C, kind=torch.float32)
        # step sizes between 0.001 and 0.1 after the softplus
        u = torch.rand(C, generator=gen, device=DEV) * (math.log(0.1) - math.log(0.001))
        u = torch.exp(u + math.log(0.001))
        s["dt_bias"] = u + torch.log(-torch.expm1(-u))
        s["state"] = normal(B, C, N, std=0.3, kind=torch.float32) if c["state"] else None
        s["lens"] = _lens(c, gen)
        s["state_out"] = torch.empty((B, C, N), dtype=torch.float32, device=DEV)
        if c["train"]:
            s["gy"] = normal(B, L, C)
    else:
        B, Lq, Lk, Hq, Hkv, E = (c[k] for k in ("B", "Lq", "Lk", "Hq", "Hkv", "E"))
        s["q"] = normal(B, Lq, Hq, E)
        s["k"], s["v"] = normal(B, Lk, Hkv, E), normal(B, Lk, Hkv, E)
        s["mask"] = None
        if c["mask"]:
            # right padding, one prompt empty in larger batches, a few single tokens dropped
            n = torch.randint((Lk + 1) // 2, Lk + 1, (B,), generator=gen, device=DEV)
            if B > 2:
                n[1] = 0
            m = torch.arange(Lk, device=DEV)[None] < n[:, None]
            s["mask"] = m & (torch.rand((B, Lk), generator=gen, device=DEV) > 0.02)
        if c["train"]:
            s["gy"] = normal(B, Lq, Hq, E)
    return s


# --------------------------------------------------------------------------
# plain forms, 32 bits
# --------------------------------------------------------------------------
def _silu(x):
    return x / (1 + torch.exp(-x))


def _silu_slope(x):
    sg = 1 / (1 + torch.exp(-x))
    return sg * (1 + x * (1 - sg))


def _live(s, B, L):
    """[B, L, 1]: 1 where a token is no padding."""
    if s["lens"] is None:
        return None
    return (torch.arange(L, device=DEV)[None] < s["lens"][:, None])[..., None]


def _keep(x, live):
    return x if live is None else torch.where(live, x, torch.zeros_like(x))


def _conv_plain(s):
    c = s["case"]
    B, L, C, K = c["B"], c["L"], c["C"], c["K"]
    t = TYPES[c["dtype"]]
    live = _live(s, B, L)
    x = _keep(s["x"].float(), live)
    before = s["state"].float() if s["state"] is not None else x.new_zeros(B, K - 1, C)
    w = s["w"].float()
    xx = torch.cat([before, x], 1)
    pre = s["bias"].float() + sum(w[:, j] * xx[:, j:j + L] for j in range(K))
    out = _keep(_silu(pre), live).to(t)
    n = s["lens"].long() if s["lens"] is not None else torch.full((B,), L, device=DEV)
    at = n[:, None] + torch.arange(K - 1, device=DEV)[None]
    r = {"out": out, "state": torch.gather(xx, 1, at[..., None].expand(-1, -1, C)).to(t)}
    if c["train"]:
        dpre = _keep(s["gy"].float() * _silu_slope(pre), live)
        dxx = torch.zeros_like(xx)
        for j in range(K):
            dxx[:, j:j + L] += w[:, j] * dpre
        r["dw"] = torch.stack([(dpre * xx[:, j:j + L]).sum((0, 1)) for j in range(K)], 1).to(t)
        r["dbias"] = dpre.sum((0, 1)).to(t)
        r["dx"] = _keep(dxx[:, K - 1:], live).to(t)
        if s["state"] is not None:
            r["dstate"] = dxx[:, :K - 1].to(t)
    return r


def _heads(x, C):
    """[B, L, G, N] in 32 bits, and the channel's group index."""
    G = x.shape[2]
    return x.float(), torch.arange(C, device=DEV) // (C // G)


def _scan_plain(s):
    c = s["case"]
    B, L, C, N = c["B"], c["L"], c["C"], c["N"]
    t = TYPES[c["dtype"]]
    live = _live(s, B, L)
    x, raw = _keep(s["x"].float(), live), s["dt"].float() + s["dt_bias"]
    dl = torch.clamp(raw, min=0) + torch.log1p(torch.exp(-torch.abs(raw)))
    dl = _keep(dl, live)                       # a step of zero leaves the state as it is
    A, (Bm, grp), Cm = s["A"], _heads(s["Bm"], C), s["Cm"].float()
    if live is not None:
        Bm, Cm = _keep(Bm, live[..., None]), _keep(Cm, live[..., None])
    h = s["state"].clone() if s["state"] is not None else x.new_zeros(B, C, N)
    dlx = dl * x
    y = torch.empty_like(x)
    kept = x.new_empty(L + 1, B, C, N) if c["train"] else None
    if c["train"]:
        kept[0] = h
    for i in range(L):
        h = torch.exp(dl[:, i, :, None] * A) * h + dlx[:, i, :, None] * Bm[:, i, grp]
        y[:, i] = (h * Cm[:, i, grp]).sum(-1)
        if c["train"]:
            kept[i + 1] = h
    y = y + s["D"] * x
    z = s["z"].float() if s["z"] is not None else None
    out = y if z is None else y * _silu(z)
    r = {"out": _keep(out, live).to(t), "state": h}
    if not c["train"]:
        return r
    gy = _keep(s["gy"].float(), live)
    if z is not None:
        r["dz"] = _keep(gy * y * _silu_slope(z), live).to(t)
        gy = gy * _silu(z)
    G = Bm.shape[2]
    g = torch.zeros_like(h)
    dA, dB, dC = torch.zeros_like(A), torch.empty_like(Bm), torch.empty_like(Cm)
    du, ddl = torch.empty_like(x), torch.empty_like(x)
    for i in range(L - 1, -1, -1):
        g = g + gy[:, i, :, None] * Cm[:, i, grp]
        a = torch.exp(dl[:, i, :, None] * A)
        back = g * a
        moved = back * kept[i]
        du[:, i] = (g * Bm[:, i, grp]).sum(-1)
        ddl[:, i] = (moved * A).sum(-1)
        dA += (moved * dl[:, i, :, None]).sum(0)
        dC[:, i] = (gy[:, i, :, None] * kept[i + 1]).reshape(B, G, C // G, N).sum(2)
        dB[:, i] = (dlx[:, i, :, None] * g).reshape(B, G, C // G, N).sum(2)
        g = back
    ddt = _keep((ddl + x * du) / (1 + torch.exp(-raw)), live)
    r |= {"dx": _keep(s["D"] * gy + dl * du, live).to(t), "ddt": ddt.to(t), "dA": dA,
          "dB": _keep(dB, None if live is None else live[..., None]).to(t),
          "dC": _keep(dC, None if live is None else live[..., None]).to(t),
          "dD": (gy * x).sum((0, 1)), "ddt_bias": ddt.sum((0, 1))}
    if s["state"] is not None:
        r["dstate"] = g
    return r


def _attn_plain(s):
    c = s["case"]
    B, Lq, Lk, Hq, Hkv, E = (c[k] for k in ("B", "Lq", "Lk", "Hq", "Hkv", "E"))
    t, g, scale = TYPES[c["dtype"]], c["Hq"] // c["Hkv"], c["E"] ** -0.5

    def rows(x):   # [B, Lq, Hq, E] -> [B, Hkv, g * Lq, E]: the heads that share keys, one after another
        return x.float().reshape(B, Lq, Hkv, g, E).permute(0, 2, 3, 1, 4).reshape(B, Hkv, g * Lq, E)

    def unrows(x):
        return x.reshape(B, Hkv, g, Lq, E).permute(0, 3, 1, 2, 4).reshape(B, Lq, Hq, E)

    q = rows(s["q"])
    k, v = (s[n].float().permute(0, 2, 1, 3).contiguous() for n in ("k", "v"))
    p = torch.matmul(q * scale, k.transpose(2, 3).contiguous())
    if s["mask"] is not None:
        p.masked_fill_(~s["mask"][:, None, None, :], -math.inf)
        m = p.amax(-1, keepdim=True)
        m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    else:
        m = p.amax(-1, keepdim=True)
    p.sub_(m).exp_()
    l = p.sum(-1, keepdim=True)
    p.div_(torch.where(l == 0, torch.ones_like(l), l))
    o = torch.matmul(p, v)
    r = {"out": unrows(o).to(t)}
    if c["train"]:
        do = rows(s["gy"])
        dv = torch.matmul(p.transpose(2, 3).contiguous(), do)
        ds = torch.matmul(do, v.transpose(2, 3).contiguous())
        ds.sub_((do * o).sum(-1, keepdim=True)).mul_(p)
        r["dq"] = unrows(torch.matmul(ds, k) * scale).to(t)
        r["dk"] = (torch.matmul(ds.transpose(2, 3).contiguous(), q) * scale).transpose(1, 2).to(t)
        r["dv"] = dv.transpose(1, 2).to(t)
    return r


# --------------------------------------------------------------------------
# one pass
# --------------------------------------------------------------------------
def run(s):
    c = s["case"]
    if not own:
        return {"conv": _conv_plain, "scan": _scan_plain, "attn": _attn_plain}[c["op"]](s)
    import linear_spatial_propagation_line_amd as g

    if c["op"] == "conv":
        out = g.causal_conv(s["x"], s["w"], s["bias"], state=s["state"], lens=s["lens"],
                            state_out=s["state_out"])
        r = {"out": out, "state": s["state_out"]}
        if c["train"]:
            d = g.causal_conv_backward(s["x"], s["w"], s["bias"], s["gy"], state=s["state"],
                                       lens=s["lens"])
            r |= {"dx": d["x"], "dw": d["weight"], "dbias": d["bias"]}
            if s["state"] is not None:
                r["dstate"] = d["state"]
        return r
    if c["op"] == "scan":
        args = (s["x"], s["dt"], s["A"], s["Bm"], s["Cm"])
        par = dict(D=s["D"], z=s["z"], dt_bias=s["dt_bias"], state=s["state"], lens=s["lens"])
        saved = g.selective_scan_saved(*args) if c["train"] else None
        out = g.selective_scan(*args, **par, state_out=s["state_out"], saved=saved)
        r = {"out": out, "state": s["state_out"]}
        if c["train"]:
            d = g.selective_scan_backward(*args, s["gy"], **par, saved=saved)
            r |= {"dx": d["x"], "ddt": d["dt"], "dA": d["A"], "dB": d["B"], "dC": d["C"],
                  "dD": d["D"], "ddt_bias": d["dt_bias"]}
            if s["z"] is not None:
                r["dz"] = d["z"]
            if s["state"] is not None:
                r["dstate"] = d["state"]
        return r
    if not c["train"]:
        return {"out": g.cross_attention(s["q"], s["k"], s["v"], mask=s["mask"])}
    lse = torch.empty((c["B"], c["Hq"], c["Lq"]), dtype=torch.float32, device=DEV)
    out = g.cross_attention(s["q"], s["k"], s["v"], mask=s["mask"], lse=lse)
    d = g.cross_attention_backward(s["q"], s["k"], s["v"], out, lse, s["gy"], mask=s["mask"])
    return {"out": out, "dq": d["q"], "dk": d["k"], "dv": d["v"]}


# --------------------------------------------------------------------------
# the definitions in 64 bits; gradients by automatic differentiation
# --------------------------------------------------------------------------
def exact(c, seed):
    s = prepare(c, seed)
    grad = c["train"]

    def wide(name):
        v = s.get(name)
        if v is None:
            return None
        return v.double().detach().requires_grad_(grad)

    if c["op"] == "conv":
        B, L, C, K = c["B"], c["L"], c["C"], c["K"]
        x, w, bias, st = wide("x"), wide("w"), wide("bias"), wide("state")
        outs, ends = [], []
        for b in range(B):
            n = L if s["lens"] is None else int(s["lens"][b])
            head = st[b] if st is not None else x.new_zeros(K - 1, C)
            row = torch.cat([head, x[b, :n]], 0)
            taps = row.unfold(0, K, 1) if n else row.new_zeros(0, C, K)   # [n, C, K]
            pre = (taps * w).sum(-1) + bias
            outs.append(torch.cat([torch.nn.functional.silu(pre), x.new_zeros(L - n, C)], 0))
            ends.append(row[n:])
        out = torch.stack(outs)
        r = {"out": out.detach(), "state": torch.stack(ends).detach()}
        if grad:
            ins = {"dx": x, "dw": w, "dbias": bias} | ({} if st is None else {"dstate": st})
            got = torch.autograd.grad(out, list(ins.values()), s["gy"].double())
            r |= dict(zip(ins, got))
        return r
    if c["op"] == "scan":
        B, L, C, N, G = c["B"], c["L"], c["C"], c["N"], c["G"]
        # the states of all steps are kept for the gradient: at most about 60 GB
        if grad and B * L * C * N * 8 * 8 > 60e9:
            return None
        x, dt, z, A, D, bias, st, Bm, Cm = (wide(k) for k in (
            "x", "dt", "z", "A", "D", "dt_bias", "state", "Bm", "Cm"))
        n = torch.full((B,), L, device=DEV) if s["lens"] is None else s["lens"]
        dl = torch.logaddexp(dt + bias, torch.zeros_like(dt))
        h = st if st is not None else x.new_zeros(B, C, N)
        ys = []
        for i in range(L):
            per = [m[:, i].repeat_interleave(C // G, 1) for m in (Bm, Cm)]
            new = h * torch.exp(dl[:, i, :, None] * A) + (dl[:, i] * x[:, i])[..., None] * per[0]
            on = (i < n)[:, None]
            h = torch.where(on[..., None], new, h)
            y = torch.einsum("bcn,bcn->bc", h, per[1]) + D * x[:, i]
            if z is not None:
                y = y * torch.nn.functional.silu(z[:, i])
            ys.append(torch.where(on, y, torch.zeros_like(y)))
        out = torch.stack(ys, 1)
        r = {"out": out.detach(), "state": h.detach()}
        if grad:
            ins = {"dx": x, "ddt": dt, "dA": A, "dB": Bm, "dC": Cm, "dD": D, "ddt_bias": bias}
            if z is not None:
                ins["dz"] = z
            if st is not None:
                ins["dstate"] = st
            r |= dict(zip(ins, torch.autograd.grad(out, list(ins.values()), s["gy"].double())))
        return r
    B, Lq, Hq, Hkv, E = (c[k] for k in ("B", "Lq", "Hq", "Hkv", "E"))
    q, k, v = wide("q"), wide("k"), wide("v")
    outs, got = [], {"dq": [], "dk": [], "dv": []}
    for b in range(B):
        keys = torch.arange(c["Lk"], device=DEV)
        if s["mask"] is not None:
            keys = keys[s["mask"][b]]
        heads, dq, dk, dv = [], [], torch.zeros_like(k[b]), torch.zeros_like(v[b])
        for h in range(Hq):
            j = h // (Hq // Hkv)
            qq, kk, vv = (u.detach().requires_grad_(grad) for u in (q[b, :, h], k[b, :, j], v[b, :, j]))
            if len(keys):
                o = torch.softmax(qq @ kk[keys].T / math.sqrt(E), -1) @ vv[keys]
            else:
                o = qq * 0
            heads.append(o.detach())
            if grad:
                d = torch.autograd.grad(o, (qq, kk, vv), s["gy"][b, :, h].double(), allow_unused=True)
                dq.append(d[0])
                dk[:, j] += 0 if d[1] is None else d[1]
                dv[:, j] += 0 if d[2] is None else d[2]
        outs.append(torch.stack(heads, 1))
        if grad:
            got["dq"].append(torch.stack(dq, 1))
            got["dk"].append(dk.detach())
            got["dv"].append(dv.detach())
    r = {"out": torch.stack(outs)}
    if grad:
        r |= {n: torch.stack(x) for n, x in got.items()}
    return r


# --------------------------------------------------------------------------
# what a pass cannot do without
# --------------------------------------------------------------------------
def work(c):
    e = BYTES[c["dtype"]]
    if c["op"] == "conv":
        B, L, C, K = c["B"], c["L"], c["C"], c["K"]
        rows, tail = B * L * C, B * (K - 1) * C
        b = e * (2 * rows + C * (K + 1) + tail * (2 if c["state"] else 1))
        f = rows * (2 * K + 5)
        if c["train"]:       # grad_out in; the gradients of x, the weights and the state out
            b += e * (2 * rows + C * (K + 1) + (tail if c["state"] else 0))
            f += rows * (6 * K + 8)
        return {"bytes": b, "flops": f}
    if c["op"] == "scan":
        B, L, C, N, G = c["B"], c["L"], c["C"], c["N"], c["G"]
        rows, bc, st = B * L * C, 2 * B * L * G * N, 4 * B * C * N
        nz = 1 if c["gate"] else 0
        b = e * (rows * (3 + nz) + bc) + 4 * C * (N + 2) + st * (2 if c["state"] else 1)
        f = rows * (N * 7 + 12)
        if c["train"]:
            b += e * (rows * (3 + nz) + bc) + 4 * C * (N + 2) + (st if c["state"] else 0)
            f += rows * (N * 16 + 20)
        return {"bytes": b, "flops": f}
    B, Lq, Lk, Hq, Hkv, E = (c[k] for k in ("B", "Lq", "Lk", "Hq", "Hkv", "E"))
    qb, kb = e * B * Lq * Hq * E, e * B * Lk * Hkv * E
    b = 2 * qb + 2 * kb + (B * Lk if c["mask"] else 0)
    f = 4 * B * Hq * Lq * Lk * E
    if c["train"]:
        b += 2 * qb + 2 * kb
        f += 10 * B * Hq * Lq * Lk * E
    return {"bytes": b, "flops": f}
