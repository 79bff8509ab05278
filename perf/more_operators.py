"""Cases of the prompt side's operators from token ids to the training loss: the
embedding lookup with its gradient by sorted tokens, the gated linear recurrence
(whole prompts, training, single tokens), and the softmax cross entropy over a
vocabulary, taken from hidden states and the vocabulary's weights.

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
        # the next token of each of 32 sequences in a serving loop
        dict(name="embed_step", op="embed", train=False, dtype="bf16", B=32, L=1, V=65536, D=2304,
             ragged=False, scaled=True),
        # a training step: 32768 tokens into a large table's gradient
        dict(name="embed_train", op="embed", train=True, dtype="bf16", B=8, L=4096, V=65536, D=2304,
             ragged=True, scaled=True),
        # odd sizes, a small table with many tokens for each row, full precision
        dict(name="embed_train_odd", op="embed", train=True, dtype="f32", B=3, L=1021, V=703, D=1153,
             ragged=True, scaled=False),
        # one new token for each of 64 sequences
        dict(name="gated_step", op="gated", train=False, dtype="bf16", B=64, L=1, C=2304,
             ragged=False, state=True),
        # a batch of prompts of different lengths, padded to the longest
        dict(name="gated_prompts", op="gated", train=False, dtype="bf16", B=8, L=4096, C=2304,
             ragged=True, state=True),
        # one long document alone: few channels against the card, a long axis
        dict(name="gated_long", op="gated", train=False, dtype="bf16", B=1, L=32768, C=2304,
             ragged=False, state=False),
        # a training step of ordinary size
        dict(name="gated_train", op="gated", train=True, dtype="bf16", B=8, L=2048, C=2304,
             ragged=False, state=False),
        # odd sizes, full precision, from a state on
        dict(name="gated_train_odd", op="gated", train=True, dtype="f32", B=3, L=1021, C=1153,
             ragged=True, state=True),
        # the log-probabilities of one token for each of 32 sequences
        dict(name="loss_step", op="loss", train=False, dtype="bf16", B=32, L=1, V=65536, D=2304,
             ragged=False),
        # prompts of different lengths scored
        dict(name="loss_score", op="loss", train=False, dtype="bf16", B=8, L=512, V=65536, D=2304,
             ragged=True),
        # a training step, a vocabulary that is no multiple of any tile
        dict(name="loss_train", op="loss", train=True, dtype="bf16", B=4, L=2048, V=50001, D=2304,
             ragged=False),
        # odd sizes, rows of no whole pieces, full precision
        dict(name="loss_train_odd", op="loss", train=True, dtype="f32", B=3, L=111, V=5003, D=333,
             ragged=True),
    ]


def _log(rng, lo, hi):
    """A whole number between lo and hi, its logarithm uniform."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _width(rng, lo, hi):
    """A row's width: mostly whole pieces of eight values, one in four any."""
    n = _log(rng, lo, hi)
    return n if rng.random() < 0.25 else max(lo, n - n % 8)


def draw(rng):
    """One more case of the ranges above."""
    op = rng.choice(["embed", "gated", "loss"])
    train = rng.random() < 0.6
    dtype = rng.choice(["bf16", "bf16", "f32"])
    wide = 2 if dtype == "f32" else 1
    if op == "embed":
        D = _width(rng, 64, 4608)
        V = _log(rng, 64, min(131072, 65536 * 2304 // (D * wide)))
        B = _log(rng, 1, 32)
        top = min(8192, 32768 * 2304 // (B * D * wide))
        L = 1 if not train and rng.random() < 0.3 else _log(rng, 1, max(2, top))
        return dict(op=op, train=train, dtype=dtype, B=B, L=L, V=V, D=D, ragged=rng.random() < 0.5,
                    scaled=rng.random() < 0.5)
    if op == "gated":
        B, C = _log(rng, 1, 64), _width(rng, 64, 4608)
        top = min(32768, (8 * 4096 * 2304) // (B * C * wide * (2 if train else 1)))
        L = 1 if not train and rng.random() < 0.3 else _log(rng, 2, max(2, top))
        return dict(op=op, train=train, dtype=dtype, B=B, L=L, C=C, ragged=rng.random() < 0.5,
                    state=rng.random() < 0.5 or L == 1)
    D, B = _width(rng, 64, 4608), _log(rng, 1, 32)
    V = _log(rng, 256, 131072)
    # f32 costs about 8 times bf16's matrix time, a training step 4 times a forward pass
    most = 8192 * 50001 * 2304 // (8 if dtype == "f32" else 1)
    top = max(1, min(8192, most // (V * D * B), (1 << 29) // (V * B)))
    L = 1 if not train and rng.random() < 0.3 else _log(rng, 1, top)
    return dict(op=op, train=train, dtype=dtype, B=B, L=L, V=V, D=D, ragged=rng.random() < 0.5)


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


def _ids(c, gen):
    """Token ids as text has them: rank k about as often as 1 / k, so that the
    commonest is one in some fifteen and most rows of a large table have none."""
    u = torch.rand((c["B"], c["L"]), generator=gen, device=DEV, dtype=torch.float64)
    ids = torch.exp(u * math.log(c["V"] + 1)).long() - 1
    return ids.clamp_(0, c["V"] - 1)


def prepare(c, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    t = TYPES[c["dtype"]]

    def normal(*shape, std=1.0, kind=t):
        x = torch.empty(shape, dtype=kind, device=DEV)
        return x.normal_(0.0, std, generator=gen)

    s = {"case": c}
    if c["op"] == "embed":
        s["ids"] = _ids(c, gen)
        s["weight"] = normal(c["V"], c["D"], std=c["D"] ** -0.5)
        s["scale"] = c["D"] ** 0.5 if c["scaled"] else 1.0
        s["lens"] = _lens(c, gen)
        if c["train"]:
            s["gy"] = normal(c["B"], c["L"], c["D"])
    elif c["op"] == "gated":
        B, L, C = c["B"], c["L"], c["C"]
        # the two gates as one projection leaves them: slices of its rows
        gates = normal(B, L, 2 * C)
        s["x"], s["r"], s["i"] = normal(B, L, C), gates[..., :C], gates[..., C:]
        # a token's decay between 0.9 and 0.999 at an eighth of the rate
        u = torch.rand(C, generator=gen, device=DEV)
        s["A"] = 8.0 * torch.log(0.9 + 0.099 * u)
        s["state"] = normal(B, C, kind=torch.float32) if c["state"] else None
        s["lens"] = _lens(c, gen)
        s["state_out"] = torch.empty((B, C), dtype=torch.float32, device=DEV)
        if c["train"]:
            s["gy"] = normal(B, L, C)
    else:
        B, L, V, D = c["B"], c["L"], c["V"], c["D"]
        s["x"], s["weight"] = normal(B, L, D), normal(V, D, std=2.0 * D ** -0.5)
        s["targets"] = _ids(c, gen)
        # a few tokens take no part
        drop = torch.rand((B, L), generator=gen, device=DEV) < 0.02
        s["targets"] = torch.where(drop, torch.full_like(s["targets"], -100), s["targets"])
        s["lens"] = _lens(c, gen)
        if c["train"]:
            # the weight of each token in the loss
            s["gl"] = torch.rand((B, L), generator=gen, device=DEV) + 0.5
    return s


# --------------------------------------------------------------------------
# plain forms, 32 bits
# --------------------------------------------------------------------------
def _live(s):
    """[B, L]: true where a token is no padding; None without lengths."""
    if s["lens"] is None:
        return None
    return torch.arange(s["case"]["L"], device=DEV)[None] < s["lens"][:, None]


def _keep(x, live):
    return x if live is None else torch.where(live[..., None], x, torch.zeros_like(x))


def _embed_plain(s):
    c, t = s["case"], TYPES[s["case"]["dtype"]]
    live = _live(s)
    r = {"out": _keep((s["weight"][s["ids"]].float() * s["scale"]), live).to(t)}
    if c["train"]:
        gy = _keep(s["gy"].float(), live) * s["scale"]
        dw = torch.zeros((c["V"], c["D"]), dtype=torch.float32, device=DEV)
        r["dweight"] = dw.index_add_(0, s["ids"].flatten(), gy.flatten(0, 1)).to(t)
    return r


def _sigmoid(x):
    return 1 / (1 + torch.exp(-x))


def _recur(a, b):
    """h[t] = a[t] h[t - 1] + b[t] over the second axis, in steps that double."""
    d, L = 1, a.shape[1]
    while d < L:
        b = torch.cat([b[:, :d], torch.addcmul(b[:, d:], a[:, d:], b[:, :-d])], 1)
        if 2 * d < L:
            a = torch.cat([a[:, :d], a[:, d:] * a[:, :-d]], 1)
        d *= 2
    return b


def _gated_plain(s):
    c, t = s["case"], TYPES[s["case"]["dtype"]]
    live = _live(s)
    A, x = s["A"], s["x"].float()
    sr, si = _sigmoid(s["r"].float()), _sigmoid(s["i"].float())
    log_a = _keep(A * sr, live)                     # padding leaves the state as it is
    a, left = torch.exp(log_a), -torch.expm1(2 * log_a)
    beta = torch.sqrt(left)
    u = _keep(si * x, live)
    b = beta * u
    if s["state"] is not None:
        b[:, 0] += a[:, 0] * s["state"]
    h = _recur(a, b)
    r = {"out": _keep(h, live).to(t), "state": h[:, -1].contiguous()}
    if not c["train"]:
        return r
    gy = _keep(s["gy"].float(), live)
    # the same recurrence from the end, with the decay of the token after
    after = torch.cat([a[:, 1:], torch.zeros_like(a[:, :1])], 1)
    g = _recur(after.flip(1), gy.flip(1)).flip(1)
    first = s["state"][:, None] if s["state"] is not None else torch.zeros_like(h[:, :1])
    before = torch.cat([first, h[:, :-1]], 1)
    slope = torch.where(left > 0, a * a / torch.where(left > 0, beta, torch.ones_like(beta)),
                        torch.zeros_like(a))
    k = _keep(g * (a * before - slope * u), live)
    du = _keep(g * beta, live)
    r |= {"dx": (du * si).to(t), "dr": (k * A * sr * (1 - sr)).to(t),
          "di": (du * x * si * (1 - si)).to(t), "dA": (k * sr).sum((0, 1))}
    if s["state"] is not None:
        r["dstate"] = a[:, 0] * g[:, 0]
    return r


def _loss_plain(s):
    c, t = s["case"], TYPES[s["case"]["dtype"]]
    live, V = _live(s), c["V"]
    on = (s["targets"] >= 0) & (s["targets"] < V)
    if live is not None:
        on &= live
    on = on.flatten()
    target = torch.where(on, s["targets"].flatten(), torch.zeros_like(s["targets"]).flatten())
    x, w = s["x"].flatten(0, 1).float(), s["weight"].float()
    if live is not None:
        x = torch.where(live.flatten()[:, None], x, torch.zeros_like(x))
    p = torch.matmul(x, w.t())
    at = p.gather(1, target[:, None])[:, 0]
    m = p.amax(1)
    p.sub_(m[:, None]).exp_()
    total = p.sum(1)
    lse = m + torch.log(total)
    zero = torch.zeros_like(lse)
    shape = (c["B"], c["L"])
    r = {"loss": torch.where(on, lse - at, zero).view(shape),
         "lse": (lse if live is None else torch.where(live.flatten(), lse, zero)).view(shape)}
    if c["train"]:
        g = torch.where(on, s["gl"].flatten(), zero)
        p.mul_((g / total)[:, None])
        rows = torch.arange(p.shape[0], device=DEV)
        p[rows, target] -= g
        r["dx"] = torch.matmul(p, w).view(s["x"].shape).to(t)
        r["dweight"] = torch.matmul(p.t(), x).to(t)
    return r


# --------------------------------------------------------------------------
# one pass
# --------------------------------------------------------------------------
def run(s):
    c = s["case"]
    if not own:
        return {"embed": _embed_plain, "gated": _gated_plain, "loss": _loss_plain}[c["op"]](s)
    import linear_spatial_propagation_line_amd as g

    if c["op"] == "embed":
        r = {"out": g.token_embedding(s["ids"], s["weight"], scale=s["scale"], lens=s["lens"])}
        if c["train"]:
            d = g.token_embedding_backward(s["ids"], s["gy"], c["V"], scale=s["scale"], lens=s["lens"])
            r["dweight"] = d["weight"]
        return r
    if c["op"] == "gated":
        args = (s["x"], s["r"], s["i"], s["A"])
        par = dict(state=s["state"], lens=s["lens"])
        saved = g.gated_recurrence_saved(s["x"]) if c["train"] else None
        out = g.gated_recurrence(*args, **par, state_out=s["state_out"], saved=saved)
        r = {"out": out, "state": s["state_out"]}
        if c["train"]:
            d = g.gated_recurrence_backward(*args, s["gy"], **par, saved=saved)
            r |= {"dx": d["x"], "dr": d["r"], "di": d["i"], "dA": d["A"]}
            if s["state"] is not None:
                r["dstate"] = d["state"]
        return r
    lse = torch.empty((c["B"], c["L"]), dtype=torch.float32, device=DEV)
    r = {"loss": g.vocab_loss(s["x"], s["weight"], s["targets"], lens=s["lens"], lse=lse), "lse": lse}
    if c["train"]:
        d = g.vocab_loss_backward(s["x"], s["weight"], s["targets"], lse, s["gl"], lens=s["lens"])
        r |= {"dx": d["x"], "dweight": d["weight"]}
    return r


# --------------------------------------------------------------------------
# the definitions in 64 bits; gradients by automatic differentiation
# --------------------------------------------------------------------------
def exact(c, seed):
    s = prepare(c, seed)
    n = [c["L"]] * c["B"] if s["lens"] is None else s["lens"].tolist()
    if c["op"] == "embed":
        w = s["weight"].double().requires_grad_(c["train"])
        rows = []
        for b in range(c["B"]):
            got = torch.nn.functional.embedding(s["ids"][b, :n[b]], w) * s["scale"]
            rows.append(torch.nn.functional.pad(got, (0, 0, 0, c["L"] - n[b])))
        out = torch.stack(rows)
        r = {"out": out.detach()}
        if c["train"]:
            r["dweight"] = torch.autograd.grad(out, w, s["gy"].double())[0]
        return r
    if c["op"] == "gated":
        leaf = {k: s[k].double().detach().requires_grad_(c["train"])
                for k in ("x", "r", "i", "A", "state") if s[k] is not None}
        x, rr, ii, A = (leaf[k] for k in ("x", "r", "i", "A"))
        log_a = A * torch.sigmoid(rr)
        drive = torch.sqrt(-torch.expm1(2 * log_a)) * torch.sigmoid(ii) * x
        a = torch.exp(log_a)
        h = leaf["state"] if "state" in leaf else x.new_zeros(c["B"], c["C"])
        top = torch.tensor(n, device=DEV)
        a, drive, ys = a.unbind(1), drive.unbind(1), []
        for i in range(c["L"]):
            new = torch.addcmul(drive[i], a[i], h)
            if s["lens"] is None:
                h = new
                ys.append(new)
            else:
                on = (i < top)[:, None]
                h = torch.where(on, new, h)
                ys.append(torch.where(on, new, torch.zeros_like(new)))
        out = torch.stack(ys, 1)
        r = {"out": out.detach(), "state": h.detach()}
        if c["train"]:
            got = torch.autograd.grad(out, list(leaf.values()), s["gy"].double())
            r |= {"d" + k: v for k, v in zip(leaf, got)}
        return r
    x = s["x"].double().requires_grad_(c["train"])
    w = s["weight"].double().requires_grad_(c["train"])
    losses, lses = [], []
    for b in range(c["B"]):
        z = x[b, :n[b]] @ w.T
        lse = torch.logsumexp(z, 1)
        t = s["targets"][b, :n[b]]
        on = (t >= 0) & (t < c["V"])
        one = torch.where(on, lse - z.gather(1, t.clamp(0, c["V"] - 1)[:, None])[:, 0], torch.zeros_like(lse))
        pad = (0, c["L"] - n[b])
        losses.append(torch.nn.functional.pad(one, pad))
        lses.append(torch.nn.functional.pad(lse.detach(), pad))
    loss = torch.stack(losses)
    r = {"loss": loss.detach(), "lse": torch.stack(lses)}
    if c["train"]:
        r["dx"], r["dweight"] = torch.autograd.grad(loss, (x, w), s["gl"].double())
    return r


# --------------------------------------------------------------------------
# what a pass cannot do without
# --------------------------------------------------------------------------
def work(c):
    e = BYTES[c["dtype"]]
    if c["op"] == "embed":
        T, V, D = c["B"] * c["L"], c["V"], c["D"]
        b = 8 * T + e * D * (min(T, V) + T)
        f = T * D
        if c["train"]:
            b += e * D * (T + V)
            f += T * D
        return {"bytes": b, "flops": f}
    if c["op"] == "gated":
        rows, st = c["B"] * c["L"] * c["C"], 4 * c["B"] * c["C"]
        b = e * rows * 4 + 4 * c["C"] + st * (2 if c["state"] else 1)
        f = rows * 20
        if c["train"]:
            b += e * rows * 4 + 4 * c["C"] + (st if c["state"] else 0)
            f += rows * 30
        return {"bytes": b, "flops": f}
    T, V, D = c["B"] * c["L"], c["V"], c["D"]
    b = e * D * (T + V) + 16 * T
    f = 2 * T * V * D
    if c["train"]:
        b += e * D * (T + V) + 4 * T
        f += 4 * T * V * D
    return {"bytes": b, "flops": f}
