"""The vocabulary loss and its gradients on the GPU against their plain 64-bit
forms, at the sizes, targets and lengths where they can go wrong.

Bounds. A logit is a sum of D products in 32 bits: off by at most
E = (D + 2) 2^-24 max_v sum |x| |w_v|. lse is a maximum and a sum of V
exponentials whose arguments are rounded at most 4 times and which are added
in parts, at most 200 sums deep: off by E + 2^-24 (200 + 8 max|z| + 2 |lse|); the
loss by E more. An entry of G = g (p - onehot) is then off by the factor
r = 2 E + 2^-24 (200 + 8 max|z| + 2 |lse|) of p, and by half a step of its type as
an operand (none at the target); the gradients are sums of V or T such
products, each sum rounded."""
from __future__ import annotations

import pytest
import torch

import linear_spatial_propagation_line_amd as g
import plain_prompt as plain

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
F32, BF16 = torch.float32, torch.bfloat16
NAN = float("nan")
S = plain.F32_STEP


def rows_of(t, extra=5, offset=3):
    wide = torch.full(t.shape[:-1] + (t.shape[-1] + extra,), NAN, dtype=t.dtype, device=t.device)
    wide[..., offset:offset + t.shape[-1]] = t
    return wide[..., offset:offset + t.shape[-1]]


CASES = [
    # B, L, V, D, dtype, targets, lens
    (1, 1, 1, 1, F32, torch.int64, None),
    (1, 1, 2, 8, BF16, torch.int32, None),
    (2, 1, 300, 64, BF16, torch.int64, None),
    (3, 5, 129, 33, F32, torch.int64, (5, 0, 2)),          # odd rows, an empty entry
    (2, 33, 257, 72, BF16, torch.int64, (33, 7)),          # one past a tile of the vocabulary
    (2, 40, 255, 40, F32, torch.int32, None),
    (4, 70, 500, 136, BF16, torch.int64, (70, 0, 1, 37)),  # more tokens than one small tile
    (1, 257, 1000, 264, BF16, torch.int64, None),          # one past a tile of tokens, of the width
    (1, 300, 90, 257, F32, torch.int64, (260,)),
    (2, 64, 700, 7, BF16, torch.int64, None),              # rows of no whole pieces
    (3, 0, 20, 12, F32, torch.int64, None),                # no tokens
    (0, 4, 20, 16, BF16, torch.int64, None),
    (2, 9, 40, 520, BF16, torch.int32, (-3, 99)),          # lengths are clamped
]


def case(B, L, V, D, dtype, tt, lens, seed=0, drop=True):
    gen = torch.Generator().manual_seed(500 + seed)
    x = torch.randn(B, L, D, generator=gen).to(dtype)
    w = (torch.randn(V, D, generator=gen) * 2 * D ** -0.5).to(dtype)
    t = torch.randint(0, V, (B, L), generator=gen)
    if drop and t.numel() > 8:
        t.view(-1)[1::7], t.view(-1)[5::11], t.view(-1)[3::13] = -1, V, -100
        if tt is torch.int64:
            t.view(-1)[6::17] = (1 << 32) + 1
    gl = torch.randn(B, L, generator=gen)
    for b, n in enumerate(plain.lengths(lens, B, L)):
        x[b, n:], gl[b, n:] = NAN, NAN
    return x, w, t.to(tt), gl, None if lens is None else torch.tensor(lens, dtype=torch.int32)


def errors(x, w, lens):
    """([B, L] bounds of lse, of a probability's factor)."""
    xd, wd = torch.nan_to_num(x.double()), w.double()
    z = xd @ wd.T
    E = (x.shape[2] + 2) * S * (xd.abs() @ wd.abs().T).amax(-1)
    rest = S * (200 + 8 * z.abs().amax(-1) + 2 * torch.logsumexp(z, -1).abs())
    return E + rest, 2 * E + rest


def check_bound(got, ref, bound, what):
    assert tuple(got.shape) == tuple(ref.shape), what
    got = got.detach().double().cpu()
    assert torch.isfinite(got).all(), f"{what}: non-finite"
    if ref.numel():
        worst = float(((got - ref).abs() / (bound + 1e-38)).max())
        assert worst <= 1.0, f"{what}: {worst:.3f} times the bound"


def check(c, x, w, t, gl, lens, view=False):
    B, L, V, D = c[:4]
    d = [v.to(DEV) for v in (x, w, t, gl)]
    dl = None if lens is None else lens.to(DEV)
    if view:
        d[0] = rows_of(d[0])
        wide = torch.full((B, L + 3), 1, dtype=t.dtype, device=DEV)
        wide[:, 2:2 + L] = d[2]
        d[2] = wide[:, 2:2 + L]
    lse = torch.full((B, L), NAN, device=DEV)
    loss = g.vocab_loss(d[0], d[1], d[2], lens=dl, lse=lse)
    ref, ref_lse = plain.vocab_loss(x, w, t, lens)
    if B * L:
        e_lse, factor = errors(x, w, lens)
    else:
        e_lse = factor = torch.zeros(B, L, dtype=torch.float64)
    check_bound(lse, ref_lse, e_lse + S * ref_lse.abs(), "lse")
    check_bound(loss, ref, 2 * e_lse + S * ref.abs(), "loss")
    got = g.vocab_loss_backward(d[0], d[1], d[2], lse, d[3], lens=dl)
    assert set(got) == {"x", "weight"}
    dref, size = plain.vocab_loss_grads(x, w, t, torch.nan_to_num(gl), lens)
    u, f = plain.half_step(x.dtype), float(factor.max()) if factor.numel() else 0.0
    part = (0.0 if x.dtype == F32 else u) + f
    for k, n in (("x", V), ("weight", B * L)):
        slack = (part + (n + 8) * S) * size[k]
        if k == "x":        # p - 1 at the target, off by r p beside a small p - 1
            slack = slack + f * gl.nan_to_num().abs().double()[..., None] * w.double().abs().amax(0)
        else:
            slack = slack + f * (gl.nan_to_num().abs().double()[..., None] * x.nan_to_num().double().abs()).sum((0, 1))
        check_bound(got[k], dref[k], slack + u * (dref[k].abs() + slack), "d" + k)


@pytest.mark.parametrize("c", CASES)
@pytest.mark.parametrize("view", [False, True])
def test_vocab_loss(c, view):
    check(c, *case(*c), view=view)


def test_without_lse():
    x, w, t, _, _ = case(2, 33, 257, 72, BF16, torch.int64, None)
    lse = torch.empty(2, 33, device=DEV)
    a = g.vocab_loss(x.to(DEV), w.to(DEV), t.to(DEV), lse=lse)
    assert torch.equal(a, g.vocab_loss(x.to(DEV), w.to(DEV), t.to(DEV)))


def test_no_token_counts():
    """Targets all outside: losses and gradients of 0, lse all the same."""
    x, w, _, gl, _ = case(2, 40, 300, 64, BF16, torch.int64, None)
    t = torch.full((2, 40), -100)
    lse = torch.empty(2, 40, device=DEV)
    loss = g.vocab_loss(x.to(DEV), w.to(DEV), t.to(DEV), lse=lse)
    assert not loss.any()
    check_bound(lse, torch.logsumexp(x.double() @ w.double().T, -1), errors(x, w, None)[0] * 1.1, "lse")
    got = g.vocab_loss_backward(x.to(DEV), w.to(DEV), t.to(DEV), lse, gl.to(DEV))
    assert not got["x"].any() and not got["weight"].any()


def test_logits_far_from_zero():
    """Logits in the hundreds: the maximum is taken out before exponentials."""
    c = (1, 20, 300, 64, F32, torch.int64, None)
    x, w, t, gl, lens = case(*c, seed=3)
    check(c, x * 40, w * 3, t, gl, lens)


def test_one_target_in_many_tokens():
    """Runs of one target over many chunks of sorted tokens, and rows of x that
    nothing but the target's own weight moves."""
    c = (1, 700, 260, 72, BF16, torch.int64, None)
    x, w, t, gl, lens = case(*c, seed=4)
    t[:] = 259
    t[0, :40] = 0
    t[0, 100:133] = 17
    check(c, x, w, t, gl, lens)


def test_pieces_of_the_vocabulary_and_parts_of_dx():
    """Enough tokens and vocabulary that the backward pass takes several pieces
    (a piece's G is at most half a GiB), the last of another length."""
    T, V, D = 8192, 66_000, 24
    gen = torch.Generator().manual_seed(6)
    x = torch.randn(1, T, D, generator=gen).to(BF16)
    w = (torch.randn(V, D, generator=gen) * 0.4).to(BF16)
    t = torch.randint(0, V, (1, T), generator=gen)
    gl = torch.rand(1, T, generator=gen) + 0.5
    xd, wd, td, gd = x.to(DEV), w.to(DEV), t.to(DEV), gl.to(DEV)
    lse = torch.empty(1, T, device=DEV)
    loss = g.vocab_loss(xd, wd, td, lse=lse)
    got = g.vocab_loss_backward(xd, wd, td, lse, gd)
    x64, w64 = xd[0].double(), wd.double()
    dw, ref_loss, dx = torch.zeros_like(w64), [], []
    for i in range(0, T, 2048):
        z = x64[i:i + 2048] @ w64.T
        l = torch.logsumexp(z, 1)
        tt = td[0, i:i + 2048, None]
        ref_loss.append(l - z.gather(1, tt)[:, 0])
        p = torch.exp(z - l[:, None])
        p.scatter_add_(1, tt, torch.full_like(tt, -1, dtype=torch.float64))
        p *= gd[0, i:i + 2048, None]
        dx.append(p @ w64)
        dw += p.T @ x64[i:i + 2048]
    ref_loss, dx = torch.cat(ref_loss), torch.cat(dx)
    assert float((loss[0].double() - ref_loss).abs().max()) <= 1e-4
    for name, a, b in (("x", got["x"][0], dx), ("weight", got["weight"], dw)):
        own = float((b.to(BF16).double() - b).norm())
        # the operand's rounding beside the result's own: at most a fifth more
        assert float((a.double() - b).norm()) <= 1.2 * own, name


@pytest.mark.parametrize("V,D", [(2000, 256), (5000, 72)])
def test_gradients_keep_the_targets_precision(V, D):
    """With bf16 operands a gradient is hardly further from 64 bits than its own
    rounding; with the targets' entries rounded too it would be 1.4 times."""
    x, w, t, gl, _ = case(2, 500, V, D, BF16, torch.int64, None, seed=9, drop=False)
    d = [v.to(DEV) for v in (x, w, t, gl)]
    lse = torch.empty(2, 500, device=DEV)
    g.vocab_loss(*d[:3], lse=lse)
    got = g.vocab_loss_backward(*d[:3], lse, d[3])
    xs, ws = (v.double().to(DEV).requires_grad_() for v in (x, w))
    z = xs @ ws.T
    loss = torch.logsumexp(z, -1) - z.gather(2, d[2][..., None])[..., 0]
    for k, ref in zip(("x", "weight"), torch.autograd.grad((loss * d[3].double()).sum(), (xs, ws))):
        own = float((ref.to(BF16).double() - ref).norm())
        assert float((got[k].double() - ref).norm()) <= 1.2 * own, k


def test_large_batch_score():
    """More tokens than tokens that count: 3 x 3000, two thirds of them padding."""
    x, w, t, _, _ = case(3, 3000, 700, 64, BF16, torch.int64, None, seed=11, drop=False)
    lens = torch.tensor([10, 2990, 0], dtype=torch.int32)
    lse = torch.empty(3, 3000, device=DEV)
    loss = g.vocab_loss(x.to(DEV), w.to(DEV), t.to(DEV), lens=lens.to(DEV), lse=lse).cpu()
    z = x.double() @ w.double().T
    ref = torch.logsumexp(z, -1)
    live = torch.arange(3000)[None] < lens[:, None]
    e = errors(x, w, None)[0]
    check_bound(lse.cpu()[live], ref[live], e[live] + S * ref[live].abs(), "lse")
    check_bound(loss[live], (ref - z.gather(2, t[..., None])[..., 0])[live], 2 * e[live] + S * 20, "loss")
    assert not loss[~live].any() and not lse.cpu()[~live].any()


def test_streams_replays_and_supplied_outputs():
    x, w, t, gl, _ = case(2, 130, 700, 136, BF16, torch.int64, None, seed=12)
    d = [v.to(DEV) for v in (x, w, t, gl)]

    def both(stream=None, **kw):
        lse = torch.empty(2, 130, device=DEV)
        loss = g.vocab_loss(*d[:3], lse=lse, stream=stream)
        return [loss, lse, *g.vocab_loss_backward(*d[:3], lse, d[3], stream=stream, **kw).values()]

    want = both()
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    rounds = [both(s) for _ in range(3) for s in (s1, s2)]
    grads = {"x": torch.full_like(d[0], NAN), "weight": torch.full_like(d[1], NAN)}
    torch.cuda.synchronize()
    rounds.append(both(grads=grads))
    for r in rounds:
        for a, b in zip(want, r):
            assert torch.equal(a, b)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kept = both()
    for _ in range(3):
        d[0].normal_()
        d[2].random_(-1, 701)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(kept, both()):
            assert torch.equal(a, b)


def test_binding_refuses():
    x = torch.zeros(2, 3, 16, device=DEV)
    w, t = torch.zeros(5, 16, device=DEV), torch.zeros(2, 3, dtype=torch.int64, device=DEV)
    lse = torch.zeros(2, 3, device=DEV)
    for bad in (lambda: g.vocab_loss(x, w[:, :8], t), lambda: g.vocab_loss(x, w.bfloat16(), t),
                lambda: g.vocab_loss(x, w, t.float()), lambda: g.vocab_loss(x, w, t[:1]),
                lambda: g.vocab_loss(x, w, t, lse=lse[:1]), lambda: g.vocab_loss(x, w, t, out=lse.bfloat16()),
                lambda: g.vocab_loss(x[0], w, t), lambda: g.vocab_loss_backward(x, w, t, lse, lse[:, :2])):
        with pytest.raises(ValueError):
            bad()
    off = torch.zeros(5 * 16 + 1, device=DEV)[1:].view(5, 16)
    for bad, name in ((lambda: g.vocab_loss(x, off, t), "GSPN_E_ALIGN"),
                      (lambda: g.vocab_loss(x, w, t, out=lse, lse=lse), "GSPN_E_ALIAS"),
                      (lambda: g.vocab_loss(x, w, t, workspace=torch.empty(256, dtype=torch.uint8, device=DEV)),
                       "GSPN_E_WORKSPACE")):
        with pytest.raises(g.GspnError) as e:
            bad()
        assert e.value.name == name


@pytest.mark.parametrize("T,V,D,dtype,ragged", [
    (300, 13_000, 1032, BF16, False),      # whole tiles of 256 in the gradients, none whole at the edges
    (300, 13_001, 1031, F32, True),        # the same in fp32, rows of no whole pieces
    (1000, 5000, 520, BF16, True),         # tiles of 128
    (999, 3001, 517, F32, False),
    (4097, 700, 200, BF16, True),          # many tokens, few rows
    (65, 9000, 264, BF16, False),          # one token past the kernel for few
    (2100, 6001, 72, BF16, False),         # logits in tiles of 256
    (2100, 6000, 40, F32, True),
    (64, 16_384, 72, BF16, False),         # few tokens, the last vocabulary in tiles of 64 rows
    (33, 16_385, 40, F32, True),           # the first in tiles of 128
    (64, 20_001, 136, BF16, True),
])
def test_tiles_of_every_size(T, V, D, dtype, ragged):
    """Tiles that run off every edge, against 64 bits on the GPU, in the norm: the
    rounding of results and operands (see above) for bf16; for fp32 a sum of n
    products has at most n roundings of 2^-24 of its size, their root as they fall."""
    gen = torch.Generator(device=DEV).manual_seed(T + V)
    B = 2
    L = (T + 1) // 2
    x = torch.randn(B, L, D, generator=gen, device=DEV).to(dtype)
    w = (torch.randn(V, D, generator=gen, device=DEV) * 2 * D ** -0.5).to(dtype)
    t = torch.randint(-1, V, (B, L), generator=gen, device=DEV)
    gl = torch.rand(B, L, generator=gen, device=DEV) + 0.5
    lens = torch.tensor([L, L // 3], dtype=torch.int32, device=DEV) if ragged else None
    live = torch.ones(B, L, dtype=torch.bool, device=DEV)
    if ragged:
        live = torch.arange(L, device=DEV)[None] < lens[:, None]
        x = x.masked_fill(~live[..., None], NAN)
    lse = torch.empty(B, L, device=DEV)
    loss = g.vocab_loss(x, w, t, lens=lens, lse=lse)
    got = g.vocab_loss_backward(x, w, t, lse, gl, lens=lens)
    on = live & (t >= 0)
    xs = x.double().nan_to_num().masked_fill(~live[..., None], 0.0).requires_grad_()
    ws = w.double().requires_grad_()
    z = xs @ ws.T
    ref_lse = torch.logsumexp(z, -1)
    ref = (ref_lse - z.gather(2, t.clamp(min=0)[..., None])[..., 0]) * on
    dx, dw = torch.autograd.grad((ref * gl.double()).sum(), (xs, ws))
    for name, a, b in (("lse", lse, (ref_lse * live).detach()), ("loss", loss, ref.detach())):
        assert float((a.double() - b).norm() / b.norm()) <= 2 * (D ** 0.5 + 30) * S, name
    for name, a, b, n in (("x", got["x"], dx, V), ("weight", got["weight"], dw, T)):
        own = float((b.to(dtype).double() - b).norm() / b.norm())
        bound = 1.2 * own if dtype == BF16 else own + (n ** 0.5 + 2 * D ** 0.5 + 60) * S
        assert float((a.double() - b).norm() / b.norm()) <= bound, name
        assert torch.isfinite(a).all()
    assert not got["x"][~on].any()


def test_offsets_past_32_bits():
    """A vocabulary of more than 2^31 weights, targets in its last rows. In the
    norm, with the bounds of the tests above."""
    V, D, T = 950_000, 2304, 40
    gen = torch.Generator(device=DEV).manual_seed(10)
    w = torch.empty(V, D, dtype=BF16, device=DEV).normal_(0.0, 2 * D ** -0.5, generator=gen)
    x = torch.randn(1, T, D, generator=gen, device=DEV).to(BF16)
    t = V - 1 - torch.arange(T, device=DEV)[None]
    gl = torch.rand(1, T, generator=gen, device=DEV) + 0.5
    lse = torch.empty(1, T, device=DEV)
    loss = g.vocab_loss(x, w, t, lse=lse)
    got = g.vocab_loss_backward(x, w, t, lse, gl)
    x64, step = x[0].double(), 50_000
    z = torch.cat([x64 @ w[v:v + step].double().T for v in range(0, V, step)], 1)
    ref_lse = torch.logsumexp(z, 1)
    ref = ref_lse - z.gather(1, t.T)[:, 0]
    for name, a, b in (("lse", lse[0], ref_lse), ("loss", loss[0], ref)):
        assert float((a.double() - b).norm() / b.norm()) <= 2 * (D ** 0.5 + 30) * S, name
    G = torch.exp(z - ref_lse[:, None]).scatter_add_(1, t.T, torch.full((T, 1), -1.0, dtype=torch.float64, device=DEV))
    G *= gl[0].double()[:, None]
    dx = sum(G[:, v:v + step] @ w[v:v + step].double() for v in range(0, V, step))
    dw = G[:, V - T:].T @ x64
    for name, a, b in (("x", got["x"][0], dx), ("weight", got["weight"][V - T:], dw)):
        own = float((b.to(BF16).double() - b).norm())
        assert float((a.double() - b).norm()) <= 1.2 * own, name
    for v in range(0, V, step):
        assert torch.isfinite(got["weight"][v:v + step]).all()
