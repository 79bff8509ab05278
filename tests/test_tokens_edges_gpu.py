"""The token-sequence operators on the GPU where a call can go wrong without
looking wrong: precision of the operands, memory that is input and output,
infinities beside masks, launches of many workgroups, states handed from chunk
to chunk. References are the plain 64-bit forms (plain_tokens.py)."""
from __future__ import annotations

import pytest
import torch

import linear_spatial_propagation_line_amd as g
import plain_tokens as plain
from test_tokens_gpu import (BF16, CONV, DEV, F32, MANY, attn_case, close, close_all, conv_call, conv_case, dev, rms,
                             scan_args, scan_case)

pytestmark = pytest.mark.gpu


# --------------------------------------------------------------------------
# attention in bf16: the operands of the second products
# --------------------------------------------------------------------------
PRECISE = [
    # B, Lq, Lk, Hq, Hkv, E, mask: one for each kernel, split and whole
    (2, 300, 128, 4, 4, 64, "random"),       # short key axis
    (2, 3, 900, 8, 2, 128, "random"),        # few rows, keys split
    (1, 4, 180, 2, 2, 72, None),             # few rows
    (1, 300, 700, 4, 2, 96, "random"),       # many rows, keys split
    (2, 3200, 300, 8, 8, 32, "left"),        # many rows
]


@pytest.mark.parametrize("case", PRECISE)
def test_attention_operands_add_no_error_of_their_own(case):
    """A bf16 result differs from 64 bits by its own rounding, whose rms over
    these values is that of the exact result's rounding. Operands with 16 bits
    of mantissa add 2^-8 of that in the root of the squares, fp32 sums less:
    out and dv stay within 1.05 of it. dq and dk also take grad_out . out from
    the rounded out, which is one error per row against a sum over the kept
    keys: about 1 / sqrt(kept / e) of the rounding, under a fifth here, or two
    hundredths in the root of the squares; 1.1. (Operands in bf16 alone, as
    large an error as the result's rounding, give 1.3 to 1.4.)"""
    inp, gy = attn_case(*case[:6], BF16, case[6], seed=12)
    B, Lq, Lk, Hq, Hkv, E, _ = case
    d = dev(inp)
    lse = torch.empty((B, Hq, Lq), device=DEV)
    out = g.cross_attention(d["q"], d["k"], d["v"], mask=d["mask"], lse=lse)
    got = g.cross_attention_backward(d["q"], d["k"], d["v"], out, lse, gy.to(DEV), mask=d["mask"])
    ref = plain.gradients(plain.attention, inp, ["q", "k", "v"], gy)
    got["out"], ref["out"] = out, plain.attention(**inp)[0]
    for n, most in (("out", 1.05), ("v", 1.05), ("q", 1.1), ("k", 1.1)):
        own = rms(ref[n].to(BF16).double() - ref[n])
        err = rms(got[n].cpu().double() - ref[n])
        assert err <= most * own, f"{n}: {err / own:.3f} of the result's own rounding"


@pytest.mark.parametrize("case", [
    (2, 300, 2, 4, 2, 64, None), (2, 70, 5, 4, 4, 128, "random"), (1, 700, 8, 6, 3, 32, None),
    (2, 200, 32, 2, 2, 96, None), (2, 90, 900, 4, 2, 64, "few"), (2, 90, 900, 2, 2, 40, "across"),
    (2, 300, 77, 5, 5, 64, "sharp"),
])
def test_attention_gradients_with_few_keys(case):
    """Few kept keys: a row's probabilities are large and its score gradients
    small differences, which the rounding of out (grad_out . out) would change
    by more than their own rounding. Taken from the probabilities themselves
    they leave the result's own rounding, as above: 1.1 of it."""
    B, Lq, Lk, Hq, Hkv, E, kind = case
    inp, gy = attn_case(B, Lq, Lk, Hq, Hkv, E, BF16, "random" if kind == "random" else None, seed=25)
    key = torch.arange(Lk)[None]
    if kind == "few":         # right padding down to 17 and 4 keys
        inp["mask"] = key < torch.tensor([[17], [4]])
    elif kind == "across":    # a few keys in two tiles
        inp["mask"] = (key >= torch.tensor([[30], [445]])) & (key < torch.tensor([[34], [450]]))
    elif kind == "random":
        inp["mask"][:, 0] = True
    scale = inp["scale"] = 1.0 if kind == "sharp" else E ** -0.5    # scores of 8: one key or two count
    d = dev(inp)
    lse = torch.empty((B, Hq, Lq), device=DEV)
    out = g.cross_attention(d["q"], d["k"], d["v"], mask=d["mask"], scale=scale, lse=lse)
    got = g.cross_attention_backward(d["q"], d["k"], d["v"], out, lse, gy.to(DEV), mask=d["mask"], scale=scale)
    ref = plain.gradients(plain.attention, inp, ["q", "k", "v"], gy)
    for n in "qkv":
        own = rms(ref[n].to(BF16).double() - ref[n])
        err = rms(got[n].cpu().double() - ref[n])
        assert err <= 1.1 * own, f"{n}: {err / own:.3f} of the result's own rounding"


@pytest.mark.parametrize("case", MANY)
def test_attention_lse_of_many_rows(case):
    """The values of lse, row by row, in the kernels that fill the chip. The
    scores' rounding (fp32 sums of E products) is absolute, a few 2^-24 of a
    score; scores stay below 8 here."""
    inp, _ = attn_case(*case, seed=5)
    B, Lq, Lk, Hq, Hkv, E, _, _ = case
    d = dev(inp)
    lse = torch.full((B, Hq, Lq), float("nan"), device=DEV)
    g.cross_attention(d["q"], d["k"], d["v"], mask=d["mask"], lse=lse)
    ref = plain.attention(**inp)[1]
    dead = torch.isinf(ref)
    assert torch.equal(lse.cpu() == -float("inf"), dead)
    assert float((lse.cpu().double() - ref)[~dead].abs().max()) <= 1e-5


# --------------------------------------------------------------------------
# attention: what dropped keys may not do
# --------------------------------------------------------------------------
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("shape", [(3, 70, 77, 4, 2, 64), (3, 2, 700, 4, 2, 64), (3, 300, 700, 4, 2, 64)])
def test_attention_without_keys_whatever_the_query_holds(shape, dtype):
    """An entry that keeps no key gives 0, lse = -inf and gradients of 0, also
    for queries and gradients that hold infinities or NaN; and in entries that
    keep some such a row spoils no other row."""
    inp, gy = attn_case(*shape, dtype, "empty", seed=18)
    B, Lq, Lk, Hq, Hkv, E = shape
    bad = [float("nan"), float("inf"), -float("inf")]
    q, gyb = inp["q"].clone(), gy.clone()
    for t in (q, gyb):
        t[:, 0, 0, :3] = torch.tensor(bad)
        t[1] = torch.tensor(bad)[torch.arange(t[1].numel()) % 3].reshape(t[1].shape)
    d = dev(inp)
    lse = torch.full((B, Hq, Lq), 7.0, device=DEV)
    out = g.cross_attention(q.to(DEV), d["k"], d["v"], mask=d["mask"], lse=lse)
    assert not out[1].any() and bool((lse[1] == -float("inf")).all())
    assert bool(out[0, 0, 0].isnan().all()) and bool(lse[0, 0, 0].isnan())
    keep = torch.ones((B, Lq, Hq), dtype=torch.bool)
    keep[:, 0, 0] = keep[1] = False
    ref, ref_lse = plain.attention(**inp)
    close(out.cpu()[keep], ref[keep], 1e-5 if dtype == F32 else 2e-2, "out")
    alive = keep.transpose(1, 2)
    assert float((lse.cpu().double() - ref_lse)[alive].abs().max()) <= 1e-5
    got = g.cross_attention_backward(q.to(DEV), d["k"], d["v"], out, lse, gyb.to(DEV), mask=d["mask"])
    for n in "qkv":
        assert not got[n][1].any(), n
    for n in "kv":      # dropped keys take no part in any entry
        assert not got[n].cpu()[~inp["mask"]].any(), n


@pytest.mark.parametrize("scale", [3e38, 1e39, float("nan"), 1e-50])
def test_attention_scales_that_no_float_holds(scale):
    """The kernels take scale * log2(e): it has to be finite too (zeros times
    an infinity would be NaN)."""
    q = torch.zeros(1, 3, 2, 8, device=DEV)
    with pytest.raises(g.GspnError) as e:
        g.cross_attention(q, q, q, scale=scale)
    assert e.value.name == "GSPN_E_SHAPE"
    assert not g.cross_attention(q, q, q, scale=1e38).any()


# --------------------------------------------------------------------------
# silu far below zero
# --------------------------------------------------------------------------
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("L", [1, 40])
def test_silu_at_the_lowest_values(dtype, L):
    """silu(v) and its slope vanish far below zero, down to the type's lowest
    value, as a gate and as the convolution's activation. In 32 bits what is
    left at v = -80 is below 1e-32."""
    low = torch.finfo(dtype).min
    vals = torch.tensor([low, low / 2, -1e30, -1e4, -200.0, -80.0, 0.0, 80.0]).to(dtype)
    inp, gy = scan_case(1, L, 8, 4, 1, dtype, None, True, True, True, True, True, seed=19)
    inp["z"] = vals.expand(1, L, 8).contiguous()
    d = dev(inp)
    args, par = scan_args(d)
    out = g.selective_scan(*args, **par)
    assert bool((out[..., :6].abs() <= 1e-30).all())
    close(out[..., 6:], plain.scan(**inp)[0][..., 6:], 1e-5 if dtype == F32 else 1e-2, "out")
    got = g.selective_scan_backward(*args, gy.to(DEV), **par)
    assert all(bool(t.isfinite().all()) for t in got.values())
    for n in ("x", "dt", "z"):
        assert bool((got[n][..., :6].abs() <= 1e-30).all()), n
    x = vals.expand(1, L, 8).contiguous().to(DEV)
    w = torch.ones((8, 1), dtype=dtype, device=DEV)
    out = g.causal_conv(x, w)
    assert bool((out[..., :6].abs() <= 1e-30).all()) and torch.equal(out[..., 6:], x[..., 6:])
    dx = g.causal_conv_backward(x, w, None, torch.ones_like(x))["x"]
    want = torch.tensor([0, 0, 0, 0, 0, 0, 0.5, 1.0])
    assert float((dx.float().cpu() - want).abs().max()) <= 1e-6


# --------------------------------------------------------------------------
# states moved on in place
# --------------------------------------------------------------------------
def launches(fn):
    """fn's result and the names of the kernels that it launched."""
    import bench
    L = g.lib()
    hip = bench.Hip()
    evs = hip.events(32)
    L.gspn_trace_events(evs, 16)
    r = fn()
    torch.cuda.synchronize()
    L.gspn_trace_events(None, 0)
    names = [L.gspn_trace_kernel(i, None).decode() for i in range(L.gspn_trace_count())]
    hip.destroy(evs)
    return r, names


@pytest.mark.parametrize("shape", [
    # B, L, C, N, G, dtype, lens: calls whose token axis is cut into segments
    (1, 512, 2304, 16, 1, BF16, None),
    (16, 2048, 2304, 16, 1, BF16, (2048, 0, 1, 2047, 1500, 16, 17, 900, 64, 65, 1024, 3, 2000, 333, 700, 5)),
    (4, 700, 520, 9, 2, F32, (700, 150, 0, 431)),
    (2, 1000, 96, 24, 1, F32, None),
])
def test_scan_in_place_over_several_segments(shape):
    """state_out = state: the end state may not be stored over the initial one
    before every segment has taken it. Bit for bit the call with two buffers."""
    inp, _ = scan_case(*shape, True, True, True, True, True, seed=13)
    d = dev(inp)
    args, par = scan_args(d)
    end = torch.full_like(d["state"], float("nan"))
    saved = g.selective_scan_saved(*args)
    saved.zero_()
    out, names = launches(lambda: g.selective_scan(*args, **par, state_out=end, saved=saved))
    assert "scan_local" in names, names
    for _ in range(3):
        st, kept = d["state"].clone(), torch.zeros_like(saved)
        got = g.selective_scan(*args, **dict(par, state=st), state_out=st, saved=kept)
        assert torch.equal(got, out) and torch.equal(st, end) and torch.equal(kept, saved)


def test_scan_in_place_over_several_segments_is_right():
    inp, _ = scan_case(3, 300, 100, 5, 1, F32, (300, 40, 0), True, True, False, True, True, seed=14)
    d = dev(inp)
    args, par = scan_args(d)
    st = d["state"]
    out, names = launches(lambda: g.selective_scan(*args, **par, state_out=st))
    assert "scan_local" in names, names
    ref, ref_end = plain.scan(**inp)
    close(out, ref, 300 * 2.0 ** -23, "out")
    close(st, ref_end, 300 * 2.0 ** -23, "state")


def test_scan_states_that_grow_over_several_segments():
    """Steps below zero (no softplus) make states grow, here by exp(96) and more
    over 16 tokens. A channel without input before its last tokens stays at 0
    until then, and its gradient at 0 behind the first ones; a tiny state that
    grows and shrinks in turn is found again. 64-bit references; an exponent of
    size s is off by s 2^-23, and every token adds two units of 2^-23."""
    L, C, N = 512, 64, 2
    gen = torch.Generator().manual_seed(24)
    normal = lambda *s: torch.randn(s, generator=gen)    # noqa: E731
    inp = dict(x=normal(1, L, C), dt=-torch.ones(1, L, C), A=torch.tensor([[-8.0, -6.0]]).repeat(C, 1),
               Bm=normal(1, L, 1, N), Cm=normal(1, L, 1, N), D=normal(C), z=None, dt_bias=None, state=None,
               lens=None, softplus=False)
    inp["x"][:, :-8] = 0
    gy = normal(1, L, C)
    gy[:, 8:] = 0
    d = dev(inp)
    args, par = scan_args(d)
    end = torch.empty((1, C, N), device=DEV)
    out, names = launches(lambda: g.selective_scan(*args, **par, state_out=end))
    assert "scan_local" in names, names
    tol = 64 * 2.0 ** -23 + 16 * 2.0 ** -23
    ref, ref_end = plain.scan(**inp)
    close(out, ref, tol, "out")
    close(end, ref_end, tol, "state")
    got = g.selective_scan_backward(*args, gy.to(DEV), **par)
    got["Bm"], got["Cm"] = got.pop("B"), got.pop("C")
    rg = plain.gradients(plain.scan, inp, list(got), gy)
    close_all(got, rg, 2 * tol, "scan")
    inp["x"][:] = 0
    inp["dt"] = inp["dt"].unflatten(1, (L // 32, 2, 16)) * torch.tensor([1.0, -1.0])[:, None, None]
    inp["dt"] = inp["dt"].flatten(1, 3)
    inp["state"] = torch.full((1, C, N), 1e-30)
    d = dev(inp)
    args, par = scan_args(d)
    out = g.selective_scan(*args, **par, state_out=end)
    ref, ref_end = plain.scan(**inp)
    tol = L * 2.0 ** -22 + 128 * 2.0 ** -23
    close(out, ref, tol, "out")
    close(end, ref_end, tol, "state")


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_conv_in_place_over_several_runs(dtype):
    inp, _ = conv_case(4, 300, 200, 4, dtype, (300, 0, 2, 129), True, True, True, seed=13)
    d = dev(inp)
    end, st = torch.empty_like(d["state"]), d["state"].clone()
    out = conv_call(d, state_out=end)
    assert torch.equal(conv_call(dict(d, state=st), state_out=st), out) and torch.equal(st, end)


# --------------------------------------------------------------------------
# gradients handed from chunk to chunk
# --------------------------------------------------------------------------
@pytest.mark.parametrize("case", [c for c in CONV if c[3] > 1])
def test_conv_gradient_of_the_state_handed_on(case):
    """dL/dstate_out reaches x, and state where the entry is shorter than the
    window (also with no tokens at all). One term more in the sums, so the
    bounds of the plain gradients hold."""
    inp, gy = conv_case(*case, seed=15)
    B, L, C, K, dtype = case[:5]
    gs = torch.randn((B, K - 1, C), generator=torch.Generator().manual_seed(16)).to(dtype)
    d = dev(inp)
    got = g.causal_conv_backward(d["x"], d["w"], d["bias"], gy.to(DEV), state=d["state"], lens=d["lens"],
                                 silu=d["silu"], grad_state=gs.to(DEV))
    got["w"] = got.pop("weight")
    ref = plain.gradients(plain.conv, inp, list(got), torch.nan_to_num(gy), gs)
    ref["x"] = torch.nan_to_num(ref["x"])
    close_all(got, ref, max(1e-5, B * L * 2.0 ** -23) if dtype == F32 else 1e-2, "conv")


def test_conv_gradients_in_chunks():
    """A sequence trained in chunks, one shorter than the window, gives the
    gradients of the whole."""
    inp, gy = conv_case(2, 60, 70, 4, F32, None, True, True, True, seed=17)
    d, gyd = dev(inp), gy.to(DEV)
    whole = g.causal_conv_backward(d["x"], d["w"], d["bias"], gyd, state=d["state"])
    cuts, states, t = [], [d["state"]], 0
    for n in (1, 30, 2, 27):
        cuts.append((t, t + n))
        states.append(torch.empty_like(d["state"]))
        conv_call(dict(d, x=d["x"][:, t:t + n], state=states[-2]), state_out=states[-1])
        t += n
    gs, parts = None, []
    for (a, b), st in reversed(list(zip(cuts, states))):
        parts.append(g.causal_conv_backward(d["x"][:, a:b], d["w"], d["bias"], gyd[:, a:b], state=st,
                                            grad_state=gs))
        gs = parts[-1]["state"]
    # as many fp32 operations, in another order
    close(torch.cat([p["x"] for p in reversed(parts)], 1), whole["x"].cpu(), 1e-5, "dx")
    close(gs, whole["state"].cpu(), 1e-5, "dstate")
    for n in ("weight", "bias"):
        close(sum(p[n] for p in parts), whole[n].cpu(), 120 * 2.0 ** -23, n)


def test_conv_grad_state_refusals():
    x, w = torch.zeros(2, 6, 16, device=DEV), torch.zeros(16, 4, device=DEV)
    for bad in (torch.zeros(2, 4, 16, device=DEV), torch.zeros(2, 3, 16, device=DEV, dtype=BF16),
                torch.zeros(2, 3, 32, device=DEV)[..., ::2]):
        with pytest.raises(ValueError):
            g.causal_conv_backward(x, w, None, x.clone(), grad_state=bad)
    gs = torch.zeros(2, 3, 16, device=DEV)
    with pytest.raises(g.GspnError) as e:       # a gradient over an input
        g.causal_conv_backward(x, w, None, x.clone(), state=torch.zeros_like(gs), grad_state=gs,
                               grads=dict(x=None, weight=None, state=gs))
    assert e.value.name == "GSPN_E_ALIAS"


@pytest.mark.parametrize("shape", [(2, 40, 0, 4, 2), (2, 3, 0, 9, 1), (0, 40, 6, 4, 2), (2, 0, 6, 4, 2)])
def test_scan_gradients_of_nothing_are_zeros(shape):
    """No channels, no entries, no tokens: sums of nothing are written too."""
    B, L, C, N, G = shape
    zeros = lambda *s: torch.zeros(s, device=DEV)    # noqa: E731
    x, bc, state = zeros(B, L, C), zeros(B, L, G, N) + 1, zeros(B, C, N) + 1
    like = dict(x=x, dt=x, A=zeros(C, N), B=bc, C=bc, D=zeros(C), dt_bias=zeros(C), state=state)
    grads = {n: torch.full_like(t, float("nan")) for n, t in like.items()}
    out = g.selective_scan(x, x, like["A"], bc, bc, D=like["D"], dt_bias=like["dt_bias"], state=state)
    assert out.shape == x.shape
    got = g.selective_scan_backward(x, x, like["A"], bc, bc, x, D=like["D"], dt_bias=like["dt_bias"], state=state,
                                    grads=grads)
    for n, t in got.items():
        assert not t.any(), n


# --------------------------------------------------------------------------
# more workgroups than one launch takes (2^32 threads)
# --------------------------------------------------------------------------
def big(gen, *shape, std=1.0, dtype=BF16):
    return torch.empty(shape, dtype=dtype, device=DEV).normal_(0.0, std, generator=gen)


def test_conv_of_many_sequences():
    """One token each of 2^23 sequences, 65 channels: 2^24 workgroups."""
    gen = torch.Generator(device=DEV).manual_seed(20)
    B, C, K = (1 << 23) + 5, 65, 2
    x, st, gy = big(gen, B, 1, C), big(gen, B, K - 1, C), big(gen, B, 1, C)
    w, b = big(gen, C, K), big(gen, C)
    out = g.causal_conv(x, w, b, state=st, state_out=st)
    assert torch.equal(st, x)
    got = g.causal_conv_backward(x, w, b, gy, state=st)
    for e in (0, 1 << 22, B - 3):
        sl = slice(e, e + 3)
        old = st[sl].clone()
        want = g.causal_conv_backward(x[sl], w, b, gy[sl], state=old)
        assert torch.equal(got["x"][sl], want["x"]) and torch.equal(got["state"][sl], want["state"])
    last = g.causal_conv(x[-3:], w, b, state=out.new_zeros(3, K - 1, C))
    first = g.causal_conv(x[-3:], w, b, state=st[-3:])
    assert not torch.equal(last, first)
    assert all(bool(t.isfinite().all()) for t in got.values())


def test_scan_of_many_tokens():
    """2^26 tokens of 32 states: 2^32 values of B and C, read from one row."""
    gen = torch.Generator(device=DEV).manual_seed(21)
    B, L, N = (1 << 16) + 3, 1024, 32
    x, dt, gy = (big(gen, B, L, 1) for _ in range(3))
    Bm, Cm = (big(gen, 1, L, 1, N).expand(B, -1, -1, -1) for _ in range(2))
    A = -torch.arange(1, N + 1, device=DEV, dtype=F32)[None]
    out = g.selective_scan(x, dt, A, Bm, Cm)
    got = g.selective_scan_backward(x, dt, A, Bm, Cm, gy)
    for e in (0, 1 << 15, B - 2):
        sl = slice(e, e + 2)
        part = (x[sl], dt[sl], A, Bm[sl], Cm[sl])
        close(out[sl], g.selective_scan(*part).cpu(), 1e-2, "out")
        want = g.selective_scan_backward(*part, gy[sl])
        for n in ("x", "dt", "B", "C"):
            close(got[n][sl], want[n].cpu(), 1e-2, n)
    assert bool(got["A"].isfinite().all())


def test_scan_of_many_short_sequences():
    """2^24 sequences of five tokens: as many workgroups."""
    gen = torch.Generator(device=DEV).manual_seed(22)
    B, L, N = (1 << 24) + 3, 5, 2
    x, dt = big(gen, B, L, 1), big(gen, B, L, 1)
    Bm, Cm = (big(gen, 1, L, 1, N).expand(B, -1, -1, -1) for _ in range(2))
    A = -torch.arange(1, N + 1, device=DEV, dtype=F32)[None]
    for t in (L, 1):
        out = g.selective_scan(x[:, :t], dt[:, :t], A, Bm[:, :t], Cm[:, :t])
        for e in (0, 1 << 23, B - 3):
            sl = slice(e, e + 3)
            close(out[sl], g.selective_scan(x[sl, :t], dt[sl, :t], A, Bm[sl, :t], Cm[sl, :t]).cpu(), 1e-2, "out")


def test_attention_of_many_rows_backward():
    """2^28 rows: sixteen lanes each for grad_out . out."""
    gen = torch.Generator(device=DEV).manual_seed(23)
    Lq, Lk = (1 << 28) + 100, 3
    q, gy = big(gen, 1, Lq, 1, 1), big(gen, 1, Lq, 1, 1)
    k, v = big(gen, 1, Lk, 1, 1), big(gen, 1, Lk, 1, 1)
    lse = torch.empty((1, 1, Lq), device=DEV)
    out = g.cross_attention(q, k, v, lse=lse)
    got = g.cross_attention_backward(q, k, v, out, lse, gy)
    for e in (0, 1 << 27, Lq - 64):
        sl = slice(e, e + 64)
        one = torch.empty((1, 1, 64), device=DEV)
        o = g.cross_attention(q[:, sl], k, v, lse=one)
        assert torch.equal(out[:, sl], o) and torch.equal(lse[..., sl], one)
        want = g.cross_attention_backward(q[:, sl], k, v, o, one, gy[:, sl].contiguous())
        assert torch.equal(got["q"][:, sl], want["q"])
    assert bool(got["k"].isfinite().all()) and bool(got["v"].isfinite().all())


def test_attention_without_keys_of_many_values():
    Lq = (1 << 26) + 1
    q = torch.ones((1, Lq, 1, 64), dtype=BF16, device=DEV)
    none = q[:, :0]
    out, lse = torch.ones_like(q), torch.zeros((1, 1, Lq), device=DEV)
    g.cross_attention(q, none, none, out=out, lse=lse)
    assert not bool(out.any()) and bool((lse == -float("inf")).all())
