"""The gated recurrence and its gradients on the GPU against their plain
64-bit forms, at the lengths, masks and strides where they can go wrong.

Counts of roundings. The decay a = exp(A s): s is off by at most 3 steps
(exponential, sum, reciprocal), the product, its product with log2(e) and the
exponential by 1 each, so a by 6 steps for |log a| <= 1 (the cases' |A| are
below 1, where the error in log a is no larger than itself), and 8 for the
widest |A| used, whose a is small. beta u: 1 - a^2 by 10, its root by half of
that and one more, the gate by 3, products by 3: 12. A step of the recurrence
adds a's 8 and one rounding to what the state before is off, relative to the
recurrence of absolute values: a state is off by at most 9 t + 13 after t
tokens, and a product of chunks' decays and the fold by as much again: 18 t + 26.
Gradients take g (as many), the state (as many), the slope a^2 / beta (20) and
up to 8 products and gates: 36 L + 80, and dA a sum over all tokens more."""
from __future__ import annotations

import pytest
import torch

import linear_spatial_propagation_line_amd as g
import plain_prompt as plain

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
F32, BF16 = torch.float32, torch.bfloat16
NAN = float("nan")


def rows_of(t, extra=3, offset=1):
    wide = torch.full(t.shape[:-1] + (t.shape[-1] + extra,), NAN, dtype=t.dtype, device=t.device)
    wide[..., offset:offset + t.shape[-1]] = t
    return wide[..., offset:offset + t.shape[-1]]


CASES = [
    # B, L, C, dtype, lens, state
    (1, 1, 1, F32, None, False),
    (2, 1, 66, BF16, None, True),
    (3, 4, 130, F32, (4, 0, 2), True),
    (2, 8, 7, F32, None, True),                        # a lane walks all tokens
    (2, 9, 64, BF16, (9, 3), True),
    (2, 12, 64, BF16, (12, 3), True),                  # the last length of that with few channels
    (2, 13, 31, F32, (13, 12), True),                  # the first of the other
    (2, 17, 33, BF16, None, False),
    (4, 64, 96, F32, (64, 0, 1, 37), True),            # one whole chunk
    (3, 65, 128, BF16, (65, 64, 63), True),            # one token past it
    (2, 200, 129, F32, (200, 129), True),              # odd channels
    (1, 1100, 70, F32, None, True),                    # more chunks than are looked back
    (5, 300, 258, BF16, (300, 0, 128, 65, 192), False),
    (2, 0, 20, F32, None, True),                       # no tokens: the state passes through
    (0, 70, 20, F32, None, False),
]


def case(B, L, C, dtype, lens, state, seed=0):
    gen = torch.Generator().manual_seed(400 + seed)
    d = dict(x=torch.randn(B, L, C, generator=gen).to(dtype), r=torch.randn(B, L, C, generator=gen).to(dtype),
             i=torch.randn(B, L, C, generator=gen).to(dtype), A=-torch.rand(C, generator=gen) * 0.8 - 0.005,
             state=torch.randn(B, C, generator=gen) if state else None,
             lens=None if lens is None else torch.tensor(lens, dtype=torch.int32))
    gy = torch.randn(B, L, C, generator=gen).to(dtype)
    for b, n in enumerate(plain.lengths(lens, B, L)):
        for t in (d["x"], d["r"], d["i"], gy):
            t[b, n:] = NAN
    return d, gy


def dev(d):
    return {k: (v.to(DEV) if isinstance(v, torch.Tensor) else v) for k, v in d.items()}


def split(d):
    return (d["x"], d["r"], d["i"], d["A"]), dict(state=d["state"], lens=d["lens"])


@pytest.mark.parametrize("c", CASES)
@pytest.mark.parametrize("view", [False, True])
def test_gated(c, view):
    inp, _ = case(*c)
    B, L, C, dtype = c[:4]
    d = dev(inp)
    if view:
        for k, (extra, off) in dict(x=(3, 1), r=(C, 0), i=(C, C)).items():
            d[k] = rows_of(d[k], extra, off)
    args, par = split(d)
    end = torch.full((B, C), NAN, device=DEV)
    out = g.gated_recurrence(*args, **par, state_out=end)
    ref, ref_end = plain.gated(**inp) if B else (torch.zeros(0, L, C), torch.zeros(0, C))
    size, size_end = plain.gated(**inp, absolute=True) if B else (ref, ref_end)
    plain.within(out, ref, size, 18 * L + 26, "out")
    plain.within(end, ref_end, size_end, 18 * L + 26, "state")
    assert torch.equal(out, g.gated_recurrence(*args, **par))       # the same bits again


@pytest.mark.parametrize("c", CASES)
@pytest.mark.parametrize("keep", [False, True])
def test_gated_gradients(c, keep):
    inp, gy = case(*c)
    B, L, C, dtype = c[:4]
    d, gyd = dev(inp), gy.to(DEV)
    args, par = split(d)
    gs = torch.randn(B, C, generator=torch.Generator().manual_seed(3)) if keep else None
    saved = None
    if keep:
        saved = g.gated_recurrence_saved(d["x"])
        saved.fill_(255)
        g.gated_recurrence(*args, **par, saved=saved)
        gyd = rows_of(gyd, 5, 2)
    got = g.gated_recurrence_backward(*args, gyd, **par, saved=saved,
                                      grad_state=None if gs is None else gs.to(DEV))
    clean = dict(inp, gy=torch.nan_to_num(gy), r=torch.nan_to_num(inp["r"]), i=torch.nan_to_num(inp["i"]))
    ref = plain.gated_grads(**clean, grad_state=gs)
    size = plain.gated_grads(**clean, grad_state=gs, absolute=True)
    assert set(got) == set(ref)
    for k in ref:
        plain.within(got[k], ref[k], size[k], 36 * L + 80 + (B * L if k == "A" else 0), "d" + k)


@pytest.mark.parametrize("B,L,C,dtype", [(70, 13, 1001, F32), (130, 32, 1010, BF16), (129, 33, 1010, BF16)])
def test_many_channels_short(B, L, C, dtype):
    """So many channels that a lane walks all of up to 32 tokens."""
    lens = tuple((7 * b) % (L + 1) for b in range(B))
    inp, gy = case(B, L, C, dtype, lens, True, seed=21)
    args, par = split(dev(inp))
    end = torch.full((B, C), NAN, device=DEV)
    saved = g.gated_recurrence_saved(args[0])
    out = g.gated_recurrence(*args, **par, state_out=end, saved=saved)
    ref, ref_end = plain.gated(**inp)
    size, size_end = plain.gated(**inp, absolute=True)
    plain.within(out, ref, size, 18 * L + 26, "out")
    plain.within(end, ref_end, size_end, 18 * L + 26, "state")
    a = g.gated_recurrence_backward(*args, gy.to(DEV), **par, saved=saved)
    b = g.gated_recurrence_backward(*args, gy.to(DEV), **par)
    for k in a:
        assert torch.equal(a[k], b[k]), k


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_in_steps_and_in_place(dtype):
    """A prompt in pieces of every path, the state carried in place."""
    inp, _ = case(2, 333, 70, dtype, None, True, seed=3)
    d = dev(inp)
    ref, ref_end = plain.gated(**inp)
    size, size_end = plain.gated(**inp, absolute=True)
    st, parts, t = d["state"].clone(), [], 0
    for n in (1, 1, 8, 9, 0, 64, 200, 50):
        piece = dict(d, state=st, **{k: d[k][:, t:t + n] for k in "xri"})
        args, par = split(piece)
        parts.append(g.gated_recurrence(*args, **par, state_out=st))
        t += n
    assert t == 333
    plain.within(torch.cat(parts, 1), ref, size, 18 * 333 + 26, "out")
    plain.within(st, ref_end, size_end, 18 * 333 + 26, "state")


def test_gradients_handed_from_chunk_to_chunk():
    """Two calls, the second's state gradient handed to the first, give the
    gradients of one call."""
    inp, gy = case(2, 150, 64, F32, None, True, seed=5)
    d, gyd = dev(inp), gy.to(DEV)
    args, par = split(d)
    whole = g.gated_recurrence_backward(*args, gyd, **par)
    cut = 70
    mid = torch.empty_like(d["state"])
    first = [t[:, :cut] for t in args[:3]] + [d["A"]]
    second = [t[:, cut:] for t in args[:3]] + [d["A"]]
    g.gated_recurrence(*first, state=d["state"], state_out=mid)
    b = g.gated_recurrence_backward(*second, gyd[:, cut:], state=mid)
    a = g.gated_recurrence_backward(*first, gyd[:, :cut], state=d["state"], grad_state=b["state"])
    size = plain.gated_grads(**inp, gy=gy, absolute=True)
    for k in "xri":
        plain.within(torch.cat([a[k], b[k]], 1), whole[k], size[k], 2 * (36 * 150 + 80), "d" + k)
    plain.within(a["A"] + b["A"], whole["A"], size["A"], 2 * (36 * 150 + 80 + 300), "dA")
    plain.within(a["state"], whole["state"], size["state"], 2 * (36 * 150 + 80), "dstate")


def test_gates_at_their_ends():
    """Gates shut and open to the type's limits: a = 1 (no input, no slope), a
    next to 1 and a = 0, all finite."""
    C = 8
    top = torch.finfo(F32).max
    r = torch.tensor([-top, -1e4, -90.0, -20.0, 0.0, 20.0, 1e4, top]).repeat(1, 70, 1)
    i = torch.tensor([-top, -100.0, top, 0.0, -3.0, 100.0, 1.0, -1.0]).repeat(1, 70, 1)
    gen = torch.Generator().manual_seed(1)
    x, gy = torch.randn(2, 1, 70, C, generator=gen)
    for A in (torch.full((C,), -0.5), torch.full((C,), -300.0), torch.zeros(C)):
        inp = dict(x=x, r=r, i=i, A=A, state=torch.randn(1, C, generator=gen), lens=None)
        d = dev(inp)
        args, par = split(d)
        out = g.gated_recurrence(*args, **par)
        ref, _ = plain.gated(**inp)
        size, _ = plain.gated(**inp, absolute=True)
        plain.within(out, ref, size + 1e-18, 18 * 70 + 26, "out")
        got = g.gated_recurrence_backward(*args, gy.to(DEV), **par)
        ref = plain.gated_grads(**inp, gy=gy)
        size = plain.gated_grads(**inp, gy=gy, absolute=True)
        for k in ref:
            # beta below 1e-19 is taken as 0; dA has a pole where a goes to 1
            fine = (r[0, 0] > -50) & (A < 0) if k == "A" else slice(None)
            plain.within(got[k][..., fine], ref[k][..., fine], size[k][..., fine] + 1e-10, 36 * 70 + 200, "d" + k)
            assert torch.isfinite(got[k]).all()


def test_a_long_axis_keeps_its_precision():
    """20000 tokens, slow decay: relative to the recurrence of absolute values
    the state stays within its last thousand tokens' roundings."""
    gen = torch.Generator().manual_seed(4)
    B, L, C = 1, 20000, 64
    x, r, i = torch.randn(3, B, L, C, generator=gen).to(BF16)
    A = -torch.rand(C, generator=gen) * 0.3 - 0.02
    out = torch.empty(B, L, C, dtype=BF16, device=DEV)
    end = torch.empty(B, C, device=DEV)
    g.gated_recurrence(x.to(DEV), r.to(DEV), i.to(DEV), A.to(DEV), out=out, state_out=end)
    la = A.double() * torch.sigmoid(r.double())
    a, b = torch.exp(la)[0], (torch.sqrt(-torch.expm1(2 * la)) * torch.sigmoid(i.double()) * x.double())[0]
    h, m, hs, ms = torch.zeros(C, dtype=torch.float64), torch.zeros(C, dtype=torch.float64), [], []
    for t in range(L):
        h, m = a[t] * h + b[t], a[t] * m + b[t].abs()
        hs.append(h)
        ms.append(m)
    # a is below exp(-0.02 / 50): what is 18 000 tokens back counts for nothing
    plain.within(end, h[None], m[None], 18 * 1000 + 26, "state")
    plain.within(out, torch.stack(hs)[None], torch.stack(ms)[None], 18 * 1000 + 26, "out")


def test_two_streams_at_once_and_replays():
    """Calls that run at the same time hand their states on apart; a captured
    call gives the eager bits at every replay."""
    d1, gy1 = case(3, 900, 256, BF16, (900, 500, 64), True, seed=7)
    d2, gy2 = case(2, 1300, 130, F32, None, False, seed=8)
    sets = []
    for d, gy in ((d1, gy1), (d2, gy2)):
        args, par = split(dev(d))
        sets.append((args, par, gy.to(DEV)))

    def both(args, par, gy, stream=None):
        out = g.gated_recurrence(*args, **par, stream=stream)
        return [out, *g.gated_recurrence_backward(*args, gy, **par, stream=stream).values()]

    want = [both(*s) for s in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    got = [[both(*s, stream=st) for s, st in zip(sets, streams)] for _ in range(4)]
    torch.cuda.synchronize()
    for rnd in got:
        for w, r in zip(want, rnd):
            for a, b in zip(w, r):
                assert torch.equal(a.nan_to_num(), b.nan_to_num())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kept = both(*sets[0])
    for _ in range(3):
        sets[0][0][0].normal_()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(kept, both(*sets[0])):
            assert torch.equal(a, b)


def test_binding_refuses():
    x = torch.zeros(2, 70, 8, device=DEV)
    A = torch.zeros(8, device=DEV)
    st = torch.zeros(2, 8, device=DEV)
    for bad in (lambda: g.gated_recurrence(x, x[:, :3], x, A), lambda: g.gated_recurrence(x, x, x.bfloat16(), A),
                lambda: g.gated_recurrence(x, x, x, A[:7]), lambda: g.gated_recurrence(x, x, x, A.bfloat16()),
                lambda: g.gated_recurrence(x, x, x, A, state=st.bfloat16()),
                lambda: g.gated_recurrence(x, x, x, A, saved=torch.empty(3, dtype=torch.uint8, device=DEV)),
                lambda: g.gated_recurrence(x.transpose(1, 2), x, x, A),
                lambda: g.gated_recurrence_backward(x, x, x, A, x[:1])):
        with pytest.raises(ValueError):
            bad()
    for kw, name in ((dict(out=x), "GSPN_E_ALIAS"), (dict(state_out=A.expand(2, 8).contiguous(), state=st,
                                                          workspace=torch.empty(64, dtype=torch.uint8, device=DEV)),
                                                     "GSPN_E_WORKSPACE")):
        with pytest.raises(g.GspnError) as e:
            g.gated_recurrence(x, x, x, A, **kw)
        assert e.value.name == name


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_broadcast_gates(dtype):
    """Gates, inputs and grad_out that are one row for all tokens or entries
    (stride 0): the results and gradients of the written-out ones, bit for bit."""
    gen = torch.Generator().manual_seed(31)
    B, L, C = 3, 150, 70
    x = torch.randn(1, L, C, generator=gen).to(dtype).to(DEV).expand(B, L, C)
    r = torch.randn(B, 1, C, generator=gen).to(dtype).to(DEV).expand(B, L, C)
    i = torch.randn(1, 1, C, generator=gen).to(dtype).to(DEV).expand(B, L, C)
    gy = torch.randn(1, 1, C, generator=gen).to(dtype).to(DEV).expand(B, L, C)
    A = (-torch.rand(C, generator=gen)).to(DEV)
    own = [t.contiguous() for t in (x, r, i)]
    assert torch.equal(g.gated_recurrence(x, r, i, A), g.gated_recurrence(*own, A))
    a = g.gated_recurrence_backward(x, r, i, A, gy)
    b = g.gated_recurrence_backward(*own, A, gy.contiguous())
    for k in a:
        assert torch.equal(a[k], b[k]), k


def test_offsets_past_32_bits():
    """One prompt of more than 2^31 values. The decay is below 2^-9 a token, so the
    last 100 tokens hang on the 100 before them alone (2^-900): those 200 tokens'
    roundings bound them."""
    L, C, n = 950_000, 2304, 200
    gen = torch.Generator(device=DEV).manual_seed(9)
    x = torch.empty(1, L, C, dtype=BF16, device=DEV).normal_(generator=gen)
    r = (2 + torch.rand(1, 1, C, generator=gen, device=DEV)).to(BF16).expand(1, L, C)
    i = torch.randn(1, 1, C, generator=gen, device=DEV).to(BF16).expand(1, L, C)
    gy = torch.randn(1, 1, C, generator=gen, device=DEV).to(BF16).expand(1, L, C)
    A = torch.full((C,), -8.0, device=DEV)
    out = g.gated_recurrence(x, r, i, A)
    tail = dict(x=x[:, -n:].cpu(), r=r[:, -n:].cpu(), i=i[:, -n:].cpu(), A=A.cpu())
    ref, size = plain.gated(**tail)[0], plain.gated(**tail, absolute=True)[0]
    plain.within(out[:, -100:], ref[:, -100:], size[:, -100:], 18 * n + 26, "out")
    got = g.gated_recurrence_backward(x, r, i, A, gy)
    gyt = gy[:, -n:].cpu()
    ref, size = plain.gated_grads(**tail, gy=gyt), plain.gated_grads(**tail, gy=gyt, absolute=True)
    for k in "xri":
        plain.within(got[k][:, -100:], ref[k][:, -100:], size[k][:, -100:], 36 * n + 80, "d" + k)
