"""The token-sequence operators on the GPU against their plain 64-bit forms
(plain_tokens.py), at the sizes, strides and masks where they can go wrong.

Bound per element: |got - ref| <= rtol (|ref| + rms(ref) + floor). The result is
rounded once to its storage type, which alone is 2^-9 |ref| for bf16 and
2^-24 |ref| for fp32; on top come
  fp32: a recurrence or sum over n tokens rounds each step by at most about
        two units of 2^-24, so rtol = max(1e-5, n 2^-23);
  bf16: attention rounds each probability and score gradient to bf16
        (2^-9), independent errors that add in the root of their squares, as
        the terms of the sum do, so they stay a multiple of 2^-9 of the rms:
        five standard deviations (0.58 2^-9 each) of two such roundings and
        the result's own are 0.011; rtol = 2e-2. The other operators round
        once: rtol = 1e-2.
A gradient that vanishes identically has no scale of its own: floor is 1e-3
of the largest rms among the call's gradients (0 for single results)."""
from __future__ import annotations

import math

import pytest
import torch

import linear_spatial_propagation_line_amd as g
import plain_tokens as plain

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
F32, BF16 = torch.float32, torch.bfloat16


def rms(t):
    return float(t.double().pow(2).mean().sqrt()) if t.numel() else 0.0


def close(got, ref, rtol, what, floor=0.0):
    assert tuple(got.shape) == tuple(ref.shape), (what, got.shape, ref.shape)
    got, ref = got.detach().double().cpu(), ref.detach().double()
    assert torch.isfinite(got).all(), f"{what}: non-finite"
    if not ref.numel():
        return
    err = float(((got - ref).abs() / (ref.abs() + rms(ref) + floor + 1e-300)).max())
    assert err <= rtol, f"{what}: scaled error {err:.3e} > {rtol:.1e}"


def close_all(got, ref, rtol, what):
    floor = 1e-3 * max(rms(t) for t in ref.values())
    assert set(got) == set(ref), (what, set(got), set(ref))
    for n in ref:
        close(got[n], ref[n], rtol, f"{what} d{n}", floor)


def normal(gen, *shape, dtype=F32, std=1.0):
    return (torch.randn(shape, generator=gen) * std).to(dtype)


def dev(d):
    return {k: (v.to(DEV) if isinstance(v, torch.Tensor) else v) for k, v in d.items()}


def strided(t, extra=3, offset=1):
    """The same values as a slice of rows that are `extra` longer, starting
    at element `offset` (an unaligned view)."""
    wide = torch.full(t.shape[:-1] + (t.shape[-1] + extra,), float("nan"), dtype=t.dtype, device=t.device)
    wide[..., offset:offset + t.shape[-1]] = t
    return wide[..., offset:offset + t.shape[-1]]


def lens_of(spec):
    return None if spec is None else torch.tensor(spec, dtype=torch.int32)


def poison(t, lens):
    """NaN in the padding."""
    if lens is not None:
        t = t.clone()
        for b, n in enumerate(lens):
            t[b, max(int(n), 0):] = float("nan")
    return t


# --------------------------------------------------------------------------
# convolution
# --------------------------------------------------------------------------
CONV = [
    # B, L, C, K, dtype, lens, state, bias, silu
    (1, 1, 1, 1, F32, None, False, False, True),
    (2, 1, 64, 4, BF16, None, True, True, True),
    (3, 2, 130, 4, F32, None, True, True, True),          # shorter than the taps
    (2, 33, 96, 4, BF16, None, False, True, True),        # just past one run
    (4, 70, 129, 3, F32, (70, 0, 1, 37), True, True, True),
    (4, 200, 520, 4, BF16, (200, 0, 2, 129), True, True, True),
    (2, 130, 257, 2, BF16, None, True, False, False),
    (1, 300, 7, 4, F32, None, False, True, False),
    (3, 40, 8, 1, BF16, (40, 7, 0), False, True, True),
    (3, 0, 16, 4, F32, None, True, True, True),           # no tokens: the state passes through
]


def conv_case(B, L, C, K, dtype, lens, state, bias, silu, seed=0):
    gen = torch.Generator().manual_seed(100 + seed)
    lens = lens_of(lens)
    return dict(x=poison(normal(gen, B, L, C, dtype=dtype), lens), w=normal(gen, C, K, dtype=dtype, std=K ** -0.5),
                bias=normal(gen, C, dtype=dtype, std=0.3) if bias else None,
                state=normal(gen, B, K - 1, C, dtype=dtype) if state else None, lens=lens,
                silu=silu), poison(normal(gen, B, L, C, dtype=dtype), lens)


def conv_call(d, **kw):
    return g.causal_conv(d["x"], d["w"], d["bias"], state=d["state"], lens=d["lens"], silu=d["silu"], **kw)


@pytest.mark.parametrize("case", CONV)
@pytest.mark.parametrize("view", [False, True])
def test_conv(case, view):
    inp, gy = conv_case(*case)
    dtype = case[4]
    rtol = 1e-5 if dtype == F32 else 1e-2
    d, gyd = dev(inp), gy.to(DEV)
    if view:
        d["x"], gyd = strided(d["x"]), strided(gyd, 5, 2)
    B, L, C = inp["x"].shape
    K = inp["w"].shape[1]
    end = torch.full((B, K - 1, C), float("nan"), dtype=dtype, device=DEV)
    out = conv_call(d, state_out=end)
    ref, ref_end = plain.conv(**inp)
    close(out, ref, rtol, "out")
    assert torch.equal(end.cpu().double(), ref_end)       # moved, not computed
    wrt = [n for n in ("x", "w", "bias", "state") if inp[n] is not None]
    got = g.causal_conv_backward(d["x"], d["w"], d["bias"], gyd, state=d["state"], lens=d["lens"],
                                 silu=d["silu"])
    got["w"] = got.pop("weight")
    rg = plain.gradients(plain.conv, inp, wrt, torch.nan_to_num(gy))
    rg["x"] = torch.nan_to_num(rg["x"])
    close_all(got, rg, max(rtol, B * L * 2.0 ** -23) if dtype == F32 else rtol, "conv")


def test_conv_in_steps_and_in_place():
    """A prompt in pieces, the state carried in place, equals the whole."""
    inp, _ = conv_case(2, 50, 96, 4, BF16, None, True, True, True)
    d = dev(inp)
    whole = conv_call(d)
    st, parts, t = d["state"].clone(), [], 0
    for n in (1, 2, 30, 0, 16, 1):
        piece = dict(d, x=d["x"][:, t:t + n], state=st)
        parts.append(conv_call(piece, state_out=st))
        t += n
    assert torch.equal(torch.cat(parts, 1), whole)
    assert torch.equal(st, d["x"][:, -3:])


# --------------------------------------------------------------------------
# scan
# --------------------------------------------------------------------------
SCAN = [
    # B, L, C, N, G, dtype, lens, state, D, z, bias, softplus
    (1, 1, 1, 1, 1, F32, None, False, False, False, False, True),
    (2, 1, 66, 16, 1, BF16, None, True, True, True, True, True),
    (3, 4, 130, 9, 1, F32, (4, 0, 2), True, True, False, True, True),
    (2, 5, 64, 4, 2, F32, None, True, True, True, True, True),
    (2, 33, 70, 16, 1, BF16, None, False, True, True, True, True),
    (4, 100, 96, 16, 1, F32, (100, 0, 1, 65), True, True, True, True, True),
    (2, 64, 132, 8, 2, F32, (64, 31), True, False, True, False, True),
    (1, 40, 100, 32, 1, BF16, None, True, True, True, True, True),
    (3, 37, 30, 24, 3, F32, (37, 32, 5), True, True, True, True, True),
    (2, 70, 64, 3, 1, F32, None, False, True, True, False, False),
    (1, 257, 64, 16, 1, F32, None, True, True, True, True, True),   # more than one segment
    (2, 0, 20, 5, 1, F32, None, True, True, True, True, True),
]


def scan_case(B, L, C, N, G, dtype, lens, state, D, z, bias, softplus, seed=0):
    gen = torch.Generator().manual_seed(200 + seed)
    lens = lens_of(lens)
    dt = normal(gen, B, L, C, dtype=dtype, std=0.5)
    if not softplus:
        dt = dt.abs() * 0.2
    d = dict(x=normal(gen, B, L, C, dtype=dtype), dt=dt,
             A=-torch.rand((C, N), generator=gen) * 3 - 0.05,
             Bm=normal(gen, B, L, G, N, dtype=dtype), Cm=normal(gen, B, L, G, N, dtype=dtype),
             D=normal(gen, C) if D else None, z=normal(gen, B, L, C, dtype=dtype) if z else None,
             dt_bias=normal(gen, C) - 2 if bias else None,
             state=normal(gen, B, C, N) if state else None, lens=lens, softplus=softplus)
    for k in ("x", "dt", "z", "Bm", "Cm"):
        if d[k] is not None:
            d[k] = poison(d[k], lens)
    return d, poison(normal(gen, B, L, C, dtype=dtype), lens)


def scan_args(d):
    return ((d["x"], d["dt"], d["A"], d["Bm"], d["Cm"]),
            dict(D=d["D"], z=d["z"], dt_bias=d["dt_bias"], state=d["state"], lens=d["lens"],
                 softplus=d["softplus"]))


def scan_tol(dtype, L):
    return max(1e-5, L * 2.0 ** -23) if dtype == F32 else 1e-2


@pytest.mark.parametrize("case", SCAN)
@pytest.mark.parametrize("view", [False, True])
def test_scan(case, view):
    inp, _ = scan_case(*case)
    dtype, L = case[5], case[1]
    d = dev(inp)
    if view:
        for k, (extra, off) in dict(x=(3, 1), dt=(8, 8), z=(1, 0), Bm=(5, 2), Cm=(4, 1)).items():
            if d[k] is not None:
                d[k] = strided(d[k], extra, off)
    args, par = scan_args(d)
    end = torch.full(inp["A"].shape, float("nan"), device=DEV).expand(case[0], -1, -1).contiguous()
    out = g.selective_scan(*args, **par, state_out=end)
    ref, ref_end = plain.scan(**inp)
    close(out, ref, scan_tol(dtype, L), "out")
    close(end, ref_end, max(1e-5, L * 2.0 ** -23), "state")


@pytest.mark.parametrize("case", SCAN)
@pytest.mark.parametrize("keep", [False, True])
def test_scan_gradients(case, keep):
    inp, gy = scan_case(*case)
    B, L, dtype = case[0], case[1], case[5]
    d = dev(inp)
    args, par = scan_args(d)
    gen = torch.Generator().manual_seed(7)
    gs = torch.randn(B, inp["A"].shape[0], inp["A"].shape[1], generator=gen) if keep else None
    saved = None
    if keep:
        saved = g.selective_scan_saved(*args)
        saved.fill_(255)
        g.selective_scan(*args, **par, saved=saved)
    got = g.selective_scan_backward(*args, gy.to(DEV), **par, saved=saved,
                                    grad_state=None if gs is None else gs.to(DEV))
    got["Bm"], got["Cm"] = got.pop("B"), got.pop("C")
    wrt = [n for n in ("x", "dt", "A", "Bm", "Cm", "D", "z", "dt_bias", "state") if inp[n] is not None]
    ref = plain.gradients(plain.scan, inp, wrt, torch.nan_to_num(gy), gs)
    ref = {n: torch.nan_to_num(t) for n, t in ref.items()}
    # sums over all tokens of all entries
    tol = max(1e-5, B * L * 2.0 ** -23) if dtype == F32 else 1e-2
    close_all(got, ref, tol, "scan")


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_scan_in_steps_and_in_place(dtype):
    """A prompt in pieces of every length class, the state carried in place."""
    inp, _ = scan_case(2, 120, 70, 16, 1, dtype, None, True, True, True, True, True, seed=3)
    d = dev(inp)
    ref, ref_end = plain.scan(**inp)
    st, parts, t = d["state"].clone(), [], 0
    for n in (1, 1, 4, 5, 64, 0, 41, 4):
        piece = dict(d, state=st, **{k: d[k][:, t:t + n] for k in ("x", "dt", "z", "Bm", "Cm")})
        args, par = scan_args(piece)
        parts.append(g.selective_scan(*args, **par, state_out=st))
        t += n
    assert t == 120
    close(torch.cat(parts, 1), ref, scan_tol(dtype, 120), "out")
    close(st, ref_end, max(1e-5, 120 * 2.0 ** -23), "state")


def test_scan_small_steps_keep_precision():
    """softplus far below zero, where log(1 + e) alone would lose digits, and
    far above, where it must not overflow."""
    gen = torch.Generator().manual_seed(5)
    inp, _ = scan_case(1, 48, 64, 4, 1, F32, None, False, False, False, True, True, seed=9)
    inp["dt_bias"] = torch.linspace(-14, 60, 64)
    inp["A"] = -torch.rand((64, 4), generator=gen) * 0.1
    inp["x"] = inp["x"].abs()
    inp["Bm"], inp["Cm"] = inp["Bm"].abs(), inp["Cm"].abs()
    d = dev(inp)
    args, par = scan_args(d)
    out = g.selective_scan(*args, **par).cpu().double()
    ref, _ = plain.scan(**inp)
    # all terms positive: nothing cancels, so the bound is purely relative
    assert float(((out - ref).abs() / ref).max()) <= 48 * 2.0 ** -22


# --------------------------------------------------------------------------
# cross attention
# --------------------------------------------------------------------------
ATTN = [
    # B, Lq, Lk, Hq, Hkv, E, dtype, mask
    (1, 1, 1, 1, 1, 1, F32, None),
    (1, 1, 1, 1, 1, 64, BF16, None),
    (2, 3, 5, 4, 2, 40, F32, "random"),
    (2, 1, 300, 8, 2, 128, BF16, "random"),              # one query, keys split and joined
    (1, 1, 1111, 4, 4, 72, F32, "random"),
    (2, 33, 77, 3, 3, 64, BF16, "right"),
    (3, 130, 129, 6, 2, 96, BF16, "empty"),
    (2, 200, 65, 5, 5, 32, F32, "left"),
    (1, 140, 257, 2, 1, 128, F32, "random"),
    (1, 97, 64, 4, 1, 24, BF16, "one"),
    (2, 50, 90, 2, 2, 7, BF16, "random"),                # E odd: values one by one
    (1, 65, 40, 3, 1, 13, F32, None),
    (2, 64, 0, 2, 1, 32, F32, None),                     # no keys
    (2, 0, 16, 2, 1, 32, F32, None),                     # no queries
]


def attn_mask(kind, B, Lk, gen):
    if kind is None:
        return None
    m = torch.rand((B, Lk), generator=gen) > 0.3
    if kind == "right":
        m = torch.arange(Lk)[None] < torch.tensor([[Lk], [Lk // 3]])[:B]
    elif kind == "left":
        m = torch.arange(Lk)[None] >= torch.tensor([[Lk // 2], [Lk - 1]])[:B]
    elif kind == "empty":
        m[1] = False
    elif kind == "one":
        m[:] = False
        m[:, Lk - 1] = True
    return m


def attn_case(B, Lq, Lk, Hq, Hkv, E, dtype, mask, seed=0):
    gen = torch.Generator().manual_seed(300 + seed)
    q = normal(gen, B, Lq, Hq, E, dtype=dtype)
    k, v = normal(gen, B, Lk, Hkv, E, dtype=dtype), normal(gen, B, Lk, Hkv, E, dtype=dtype)
    m = attn_mask(mask, B, Lk, gen)
    return dict(q=q, k=k, v=v, mask=m), normal(gen, B, Lq, Hq, E, dtype=dtype)


@pytest.mark.parametrize("case", ATTN)
@pytest.mark.parametrize("view", [False, True])
def test_attention(case, view):
    inp, gy = attn_case(*case)
    B, Lq, Lk, Hq, Hkv, E, dtype, _ = case
    d, gyd = dev(inp), gy.to(DEV)
    if d["mask"] is not None:       # dropped keys may hold anything
        bad = ~d["mask"][:, :, None, None]
        d["k"] = d["k"].masked_fill(bad, float("nan"))
        d["v"] = torch.where(bad & (torch.arange(E, device=DEV) % 2 == 0), float("inf"), d["v"]).to(dtype)
    if view:
        d["q"], gyd = strided(d["q"], 3, 1), strided(gyd, 8, 8)
        d["k"], d["v"] = strided(d["k"], 5, 2), strided(d["v"], 1, 0)
        if d["mask"] is not None:
            d["mask"] = torch.cat([d["mask"], d["mask"]], 1)[:, :Lk]
    lse = torch.full((B, Hq, Lq), float("nan"), device=DEV)
    out = g.cross_attention(d["q"], d["k"], d["v"], mask=d["mask"], lse=lse)
    ref, ref_lse = plain.attention(**inp)
    rtol = 1e-5 if dtype == F32 else 2e-2
    close(out, ref, rtol, "out")
    dead = torch.isinf(ref_lse)
    assert torch.equal(torch.isinf(lse.cpu()), dead) and bool((lse.cpu()[dead] < 0).all())
    # the scores' rounding (fp32 accumulation of E products) is absolute
    assert float((lse.cpu().double() - ref_lse)[~dead].abs().max() if (~dead).any() else 0) <= 1e-5
    got = g.cross_attention_backward(d["q"], d["k"], d["v"], out, lse, gyd, mask=d["mask"])
    rg = plain.gradients(plain.attention, inp, ["q", "k", "v"], gy)
    if Lq and Lk:
        close_all(got, rg, max(rtol, Lq * Hq * 2.0 ** -23), "attn")
    else:
        for n in "qkv":
            assert got[n].shape == inp[n].shape and not got[n].any()
    if d["mask"] is not None:
        assert not got["k"][~d["mask"]].any() and not got["v"][~d["mask"]].any()


# rows enough for the kernels that fill the chip (128 rows, up to E = 64 256 rows, per workgroup)
MANY = [
    # B, Lq, Lk, Hq, Hkv, E, dtype, mask
    (2, 1570, 200, 16, 8, 128, BF16, "left"),
    (2, 1600, 333, 8, 8, 96, BF16, "random"),
    (2, 3200, 150, 8, 8, 64, BF16, "empty"),
    (2, 3210, 129, 8, 8, 32, BF16, "one"),
    (1, 3100, 257, 8, 8, 64, BF16, None),
    (1, 2100, 33, 4, 2, 64, BF16, "random"),      # short key axis, several row tiles per wavefront
    (1, 1300, 128, 8, 4, 72, BF16, "random"),
    (1, 2050, 70, 3, 3, 64, F32, "random"),
    (1, 70, 128, 2, 2, 128, F32, "random"),       # keys that LDS does not hold as a whole
    (1, 70, 97, 2, 1, 128, F32, None),
    (1, 70, 65, 2, 2, 100, F32, "random"),
    (1, 70, 100, 2, 1, 96, F32, "left"),
    (16, 300, 128, 16, 16, 96, BF16, "random"),   # keys that LDS holds only once per compute unit
]


@pytest.mark.parametrize("case", MANY)
def test_attention_many_rows(case):
    inp, gy = attn_case(*case, seed=5)
    B, Lq, Lk, Hq, Hkv, E, dtype, _ = case
    d = dev(inp)
    if d["mask"] is not None:
        bad = ~d["mask"][:, :, None, None]
        d["k"], d["v"] = d["k"].masked_fill(bad, float("nan")), d["v"].masked_fill(bad, float("inf"))
    lse = torch.full((B, Hq, Lq), float("nan"), device=DEV)
    out = g.cross_attention(d["q"], d["k"], d["v"], mask=d["mask"], lse=lse)
    ref, ref_lse = plain.attention(**inp)
    rtol = 1e-5 if dtype == F32 else 2e-2
    close(out, ref, rtol, "out")
    assert torch.equal(torch.isinf(lse.cpu()), torch.isinf(ref_lse))
    got = g.cross_attention_backward(d["q"], d["k"], d["v"], out, lse, gy.to(DEV), mask=d["mask"])
    rg = plain.gradients(plain.attention, inp, ["q", "k", "v"], gy)
    close_all(got, rg, max(rtol, Lq * Hq * 2.0 ** -23), "attn")


@pytest.mark.parametrize("shape", [(1, 1, 600, 1, 1, 64), (1, 4, 100, 1, 1, 64), (1, 200, 300, 1, 1, 64),
                                   (1, 3100, 300, 8, 8, 128)])
@pytest.mark.parametrize("order", [1, -1])
def test_attention_moving_maximum(shape, order):
    """Scores that grow (or fall) by far along the key axis, in every kernel:
    a result so far has to be rescaled, or later keys have to vanish."""
    B, Lq, Lk, Hq, Hkv, E = shape
    inp, _ = attn_case(B, Lq, Lk, Hq, Hkv, E, BF16, None, seed=6)
    grow = torch.linspace(0, 40, Lk)
    grow = grow if order > 0 else grow.flip(0)
    inp["k"] = (inp["q"][:, :1, :1].float() * grow[None, :, None, None]).to(BF16).expand(-1, -1, Hkv, -1).contiguous()
    d = dev(inp)
    out = g.cross_attention(d["q"], d["k"], d["v"])
    ref, _ = plain.attention(**inp)
    close(out, ref, 2e-2, "out")


def test_results_do_not_depend_on_the_neighbours():
    """What a call chooses by its size (runs, segments) changes no token's
    result beyond rounding: slices of a large call equal the calls on the
    slices, convolution outputs bit for bit."""
    gen = torch.Generator(device=DEV).manual_seed(3)
    x = torch.randn((16, 517, 4096), generator=gen, device=DEV).to(BF16)
    gy = torch.randn((16, 517, 4096), generator=gen, device=DEV).to(BF16)
    w, b = torch.randn((4096, 4), generator=gen, device=DEV).to(BF16), torch.randn(4096, generator=gen, device=DEV).to(BF16)
    out = g.causal_conv(x, w, b)
    big = g.causal_conv_backward(x, w, b, gy)
    for sl in (slice(0, 128), slice(3000, 3128)):
        part = g.causal_conv_backward(x[..., sl], w[sl].contiguous(), b[sl].contiguous(), gy[..., sl])
        assert torch.equal(g.causal_conv(x[..., sl], w[sl].contiguous(), b[sl].contiguous()), out[..., sl])
        assert torch.equal(part["x"], big["x"][..., sl])
        # the same terms in another order, then one rounding to bf16
        close(part["weight"], big["weight"][sl].cpu(), 2.0 ** -7, "dw")
        close(part["bias"], big["bias"][sl].cpu(), 2.0 ** -7, "db")
    inp, gy = scan_case(24, 300, 256, 16, 1, F32, tuple(range(300, 0, -13))[:24], True, True, True, True, True, seed=8)
    d = dev(inp)
    args, par = scan_args(d)
    out = g.selective_scan(*args, **par)
    big = g.selective_scan_backward(*args, gy.to(DEV), **par)
    for e in (0, 7, 23):
        one = {k: (v[e:e + 1] if isinstance(v, torch.Tensor) and v.shape[:1] == (24,) else v) for k, v in d.items()}
        args, par = scan_args(one)
        close(g.selective_scan(*args, **par), out[e:e + 1].cpu(), 300 * 2.0 ** -23, "out")
        part = g.selective_scan_backward(*args, gy[e:e + 1].to(DEV), **par)
        for k in ("x", "dt", "B", "C", "z", "state"):
            close(part[k], big[k][e:e + 1].cpu(), 300 * 2.0 ** -23, k, 1e-3 * rms(big["x"]))


def test_attention_scale_and_large_scores():
    """Scores far apart: the running maximum has to move, also late, and a
    row's probabilities underflow without harm."""
    inp, _ = attn_case(1, 70, 200, 2, 1, 64, F32, None, seed=4)
    inp["k"] = inp["k"] * torch.linspace(0.01, 30, 200)[None, :, None, None]
    d = dev(inp)
    for scale in (0.125, 1.0):
        out = g.cross_attention(d["q"], d["k"], d["v"], scale=scale)
        ref, _ = plain.attention(**inp, scale=scale)
        # a score of size s is off by E 2^-24 s, which the exponential makes
        # a relative error of its probability
        s = scale * float((inp["q"].double().norm(dim=-1).max() * inp["k"].double().norm(dim=-1).max()))
        close(out, ref, max(1e-5, 8 * s * 2.0 ** -24), f"scale {scale}")


# --------------------------------------------------------------------------
# gradients against differences, streams, graphs, determinism, the C ABI's view
# --------------------------------------------------------------------------
def test_gradients_against_differences():
    gen = torch.Generator().manual_seed(11)

    def check(fn, inp, name, gy, grad):
        v = torch.randn(inp[name].shape, generator=gen, dtype=torch.float64)
        want = plain.difference(fn, inp, name, v, gy)
        have = float((grad.double().cpu() * v).sum())
        # fp32 gradients of size |grad| |v| each, central difference error 1e-8
        scale = float(grad.double().norm()) * float(v.norm()) + 1e-6
        assert abs(have - want) <= 2e-5 * scale, (fn.__name__, name, have, want)

    inp, gy = conv_case(2, 40, 33, 4, F32, None, True, True, True, seed=1)
    d = dev(inp)
    got = g.causal_conv_backward(d["x"], d["w"], d["bias"], gy.to(DEV), state=d["state"])
    for n, k in (("x", "x"), ("w", "weight"), ("bias", "bias"), ("state", "state")):
        check(plain.conv, inp, n, gy, got[k])
    inp, gy = scan_case(2, 40, 34, 5, 2, F32, None, True, True, True, True, True, seed=1)
    d = dev(inp)
    args, par = scan_args(d)
    got = g.selective_scan_backward(*args, gy.to(DEV), **par)
    for n, k in (("x", "x"), ("dt", "dt"), ("A", "A"), ("Bm", "B"), ("Cm", "C"), ("D", "D"), ("z", "z"),
                 ("dt_bias", "dt_bias"), ("state", "state")):
        check(plain.scan, inp, n, gy, got[k])
    inp, gy = attn_case(2, 20, 30, 4, 2, 16, F32, "random", seed=1)
    d = dev(inp)
    lse = torch.empty((2, 4, 20), device=DEV)
    out = g.cross_attention(d["q"], d["k"], d["v"], mask=d["mask"], lse=lse)
    got = g.cross_attention_backward(d["q"], d["k"], d["v"], out, lse, gy.to(DEV), mask=d["mask"])
    for n in "qkv":
        check(plain.attention, inp, n, gy, got[n])


def everything(seed=0, stream=None):
    """One call of each operator and its gradients, as a flat list."""
    r = []
    inp, gy = conv_case(3, 90, 136, 4, BF16, (90, 0, 41), True, True, True, seed=seed)
    d = dev(inp)
    r.append(conv_call(d, stream=stream))
    r += g.causal_conv_backward(d["x"], d["w"], d["bias"], gy.to(DEV), state=d["state"], lens=d["lens"],
                                stream=stream).values()
    inp, gy = scan_case(2, 200, 136, 16, 1, BF16, (200, 77), True, True, True, True, True, seed=seed)
    d = dev(inp)
    args, par = scan_args(d)
    r.append(g.selective_scan(*args, **par, stream=stream))
    r += g.selective_scan_backward(*args, gy.to(DEV), **par, stream=stream).values()
    inp, gy = attn_case(2, 100, 150, 4, 2, 64, BF16, "random", seed=seed)
    d = dev(inp)
    lse = torch.empty((2, 4, 100), device=DEV)
    out = g.cross_attention(d["q"], d["k"], d["v"], mask=d["mask"], lse=lse, stream=stream)
    r.append(out)
    r += g.cross_attention_backward(d["q"], d["k"], d["v"], out, lse, gy.to(DEV), mask=d["mask"],
                                    stream=stream).values()
    r.append(g.cross_attention(d["q"][:, :1], d["k"], d["v"], mask=d["mask"], stream=stream))
    return r


def test_repeatable_and_on_another_stream():
    first = everything()
    again = everything()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    torch.cuda.synchronize()
    other = everything(stream=side)
    raw = everything(stream=side.cuda_stream)
    side.synchronize()
    for a, b, c, e in zip(first, again, other, raw):
        assert torch.equal(a, b) and torch.equal(a, c) and torch.equal(a, e)


def test_captured_graph_replays():
    """Forward, backward and single-token calls captured once; every replay on
    new inputs equals the eager result."""
    inp, gy = scan_case(2, 96, 72, 16, 1, BF16, None, True, True, True, True, True, seed=2)
    d = dev(inp)
    gyd = gy.to(DEV)
    cin, cgy = conv_case(2, 50, 72, 4, BF16, None, True, True, True, seed=2)
    cd, cg = dev(cin), cgy.to(DEV)
    ain, agy = attn_case(2, 40, 300, 4, 2, 64, BF16, "random", seed=2)
    ad, ag = dev(ain), agy.to(DEV)
    lse = torch.empty((2, 4, 40), device=DEV)

    def work():
        args, par = scan_args(d)
        r = [g.selective_scan(*args, **par)]
        r += g.selective_scan_backward(*args, gyd, **par).values()
        r.append(conv_call(cd))
        r += g.causal_conv_backward(cd["x"], cd["w"], cd["bias"], cg, state=cd["state"]).values()
        out = g.cross_attention(ad["q"], ad["k"], ad["v"], mask=ad["mask"], lse=lse)
        r.append(out)
        r += g.cross_attention_backward(ad["q"], ad["k"], ad["v"], out, lse, ag, mask=ad["mask"]).values()
        r.append(g.cross_attention(ad["q"][:, :1], ad["k"], ad["v"], mask=ad["mask"]))
        return r

    work()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = work()
    for k in range(3):
        for t in (d["x"], cd["x"], ad["q"], ad["v"], gyd):
            t.mul_(-0.5 if k % 2 else 1.75)
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in captured]
        want = work()
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b), k


def test_offsets_past_32_bits():
    """Inputs whose last element lies more than 2^32 elements from the first,
    as strided views (nothing of that size is read)."""
    rows, wide = 5, (1 << 30) + 8
    big = torch.empty((rows, wide), dtype=BF16, device=DEV)      # 10 GiB, only the views written
    x = big[None, :, 8:8 + 128]
    gen = torch.Generator().manual_seed(21)
    val = normal(gen, 1, rows, 128, dtype=BF16)
    x.copy_(val)
    w = normal(gen, 128, 4, dtype=BF16)
    ref, _ = plain.conv(val, w)
    close(g.causal_conv(x, w.to(DEV)), ref, 1e-2, "conv")
    inp, _ = scan_case(1, rows, 128, 16, 1, BF16, None, False, True, False, True, True)
    d = dev(inp)
    d["x"] = x
    inp["x"] = val
    args, par = scan_args(d)
    close(g.selective_scan(*args, **par), plain.scan(**inp)[0], 1e-2, "scan")
    kv = x.unflatten(-1, (2, 64))
    q = normal(gen, 1, 40, 2, 64, dtype=BF16)
    ref, _ = plain.attention(q, val.unflatten(-1, (2, 64)), val.unflatten(-1, (2, 64)))
    close(g.cross_attention(q.to(DEV), kv, kv), ref, 2e-2, "attention")


def test_refusals():
    """Wrong tensors raise before anything is launched."""
    inp, gy = scan_case(2, 6, 16, 4, 2, F32, None, True, True, True, True, True)
    d = dev(inp)
    args, par = scan_args(d)
    x, dt, A, Bm, Cm = args
    bad = [
        ((x.cpu(), dt, A, Bm, Cm), {}, TypeError),
        ((x.half(), dt, A, Bm, Cm), {}, TypeError),
        ((x, dt.to(BF16), A, Bm, Cm), {}, ValueError),
        ((x, dt[:, :5], A, Bm, Cm), {}, ValueError),
        ((x, dt, A.double(), Bm, Cm), {}, ValueError),
        ((x, dt, A, Bm, Cm[:, :, :1]), {}, ValueError),
        ((x.transpose(1, 2).contiguous().transpose(1, 2), dt, A, Bm, Cm), {}, ValueError),
        (args, dict(D=d["D"].to(BF16)), ValueError),
        (args, dict(lens=torch.zeros(2, dtype=torch.int64, device=DEV)), ValueError),
        (args, dict(out=torch.empty_like(x)[:, :5]), ValueError),
        (args, dict(state_out=torch.empty((2, 16, 4))), TypeError),
        (args, dict(saved=torch.empty(8, dtype=torch.uint8, device=DEV)), ValueError),
    ]
    for a, k, exc in bad:
        with pytest.raises(exc):
            g.selective_scan(*a, **k)
    with pytest.raises(g.GspnError) as e:       # 33 states
        g.selective_scan(x, dt, torch.zeros(16, 33, device=DEV), torch.zeros(2, 6, 2, 33, device=DEV),
                         torch.zeros(2, 6, 2, 33, device=DEV))
    assert e.value.name == "GSPN_E_SHAPE"
    with pytest.raises(g.GspnError) as e:       # out over an input
        g.selective_scan(*args, out=x)
    assert e.value.name == "GSPN_E_ALIAS"
    with pytest.raises(g.GspnError) as e:
        g.selective_scan(*args, workspace=torch.empty(16, dtype=torch.uint8, device=DEV))
    assert e.value.name == "GSPN_E_WORKSPACE"
    w = torch.zeros(16, 4, device=DEV)
    for a, k, exc in [((x, w[:, :, None]), {}, ValueError), ((x, w[:8]), {}, ValueError),
                      ((x, w.to(BF16)), {}, ValueError), ((x[0], w), {}, ValueError),
                      ((x, w), dict(state=torch.zeros(2, 4, 16, device=DEV)), ValueError)]:
        with pytest.raises(exc):
            g.causal_conv(*a, **k)
    with pytest.raises(g.GspnError) as e:       # five taps
        g.causal_conv(x, torch.zeros(16, 5, device=DEV))
    assert e.value.name == "GSPN_E_SHAPE"
    q = torch.zeros(2, 3, 4, 8, device=DEV)
    kv = torch.zeros(2, 5, 2, 8, device=DEV)
    for a, k, exc in [((q[0], kv, kv), {}, ValueError), ((q, kv, kv[:, :4]), {}, ValueError),
                      ((q, kv[..., :4], kv), {}, ValueError),
                      ((q, kv, kv), dict(mask=torch.ones(2, 4, dtype=torch.bool, device=DEV)), ValueError),
                      ((q, kv, kv), dict(mask=torch.ones(2, 5, device=DEV)), ValueError),
                      ((q, kv, kv), dict(lse=torch.zeros(2, 3, 4, device=DEV)), ValueError)]:
        with pytest.raises(exc):
            g.cross_attention(*a, **k)
    for a, k in [((q[:, :, :3], kv, kv), {}), ((q, kv, kv), dict(scale=0.0)),
                 ((q, kv, kv), dict(scale=math.inf))]:
        with pytest.raises(g.GspnError) as e:
            g.cross_attention(*(t.contiguous() for t in a), **k)
        assert e.value.name == "GSPN_E_SHAPE"
