"""The token embedding, the gated recurrence and the vocabulary loss on the GPU
where a call can go wrong without looking wrong. References are the plain 64-bit forms
(plain_prompt.py)."""
from __future__ import annotations

import pytest
import torch

import linear_spatial_propagation_line_amd as g
import plain_prompt as plain
from linear_spatial_propagation_line_amd import tokens
from test_tokens_edges_gpu import launches
from test_vocab_loss_gpu import case as loss_case, check

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
F32, BF16 = torch.float32, torch.bfloat16


# --------------------------------------------------------------------------
# vocabulary loss: G as an operand in bf16, from diffuse to peaked softmaxes
# --------------------------------------------------------------------------
@pytest.mark.parametrize("std", [2, 4, 8, 16, 64])
def test_peaked_softmax_in_bf16(std):
    """Logits of a standard deviation of up to 64: a token's softmax is then one
    entry, which is not its target. Entries off the target are rounded to bf16 as
    operands. They sum to 1 - p(target), so the sum of their squares is at most the
    square of the target's entry, which is not rounded: at most half of G's squares are
    rounded, and over rows of one length and of no relation the gradients' squares stand
    to their errors as G's. Values of one distribution (g and the results are normal)
    have the same mean square of a rounding, so the operand adds at most half of the
    result's own: a root of 1.5. Over 1000 tokens that share of squares is known to
    some 7 % (the fourth moment of a normal value is 3, and a rounding's square varies
    as much again), three times which gives the root of 1.61, 1.27."""
    x, w, t, gl, _ = loss_case(2, 500, 4000, 256, BF16, torch.int64, None, seed=31, drop=False)
    d = [x.to(DEV), (w * (std / 2)).to(DEV), t.to(DEV), gl.to(DEV)]
    lse = torch.empty(2, 500, device=DEV)
    g.vocab_loss(*d[:3], lse=lse)
    got = g.vocab_loss_backward(*d[:3], lse, d[3])
    xs, ws = (v.double().requires_grad_() for v in d[:2])
    z = xs @ ws.T
    loss = torch.logsumexp(z, -1) - z.gather(2, d[2][..., None])[..., 0]
    for k, ref in zip(("x", "weight"), torch.autograd.grad((loss * d[3].double()).sum(), (xs, ws))):
        own = float((ref.to(BF16).double() - ref).norm())
        assert float((got[k].double() - ref).norm()) <= 1.27 * own, k


def test_peaked_softmax_value_by_value():
    """The same with logits of a standard deviation of 32, each value against the
    bound of its products' sizes."""
    c = (2, 20, 300, 64, BF16, torch.int64, (20, 13))
    x, w, t, gl, lens = loss_case(*c, seed=32)
    check(c, x, w * 16, t, gl, lens)


# --------------------------------------------------------------------------
# gated recurrence: decays from next to 1 to next to 0
# --------------------------------------------------------------------------
def steps_of_decay(rmax, vmax):
    """By how many steps of 2^-24 the decay exp(A s) is off, relative to itself,
    for |r| <= rmax and |A s| <= vmax. exp(-r): r log2(e) is rounded (the product and
    the constant: 2 |r|, in the exponent) and the exponential is off by 2; the sum
    by 1, the reciprocal by 2: s by 2 rmax + 5. v = A s by 1 more, so exp(v) by
    vmax (2 rmax + 6), the product with log2(e) 2 vmax, the exponential 2."""
    return vmax * (2 * rmax + 8) + 2


FLUSH = 1000 * torch.finfo(F32).tiny
STRONG = [
    # B, L, C, lens
    (1, 1, 64, None),
    (2, 4, 130, (4, 3)),
    (2, 13, 66, None),         # chunks
    (1, 13, 7, None),          # single channels a lane
    (3, 70, 128, (70, 64, 65)),
    (1, 300, 70, None),
]


def strong_case(B, L, C, lens, dtype=F32):
    """|A s| between 0.1 and 17, over the channels; every third channel's input gate
    is shut, so that its state is nothing but a product of decays."""
    gen = torch.Generator().manual_seed(700 + L)
    r = torch.rand(B, L, C, generator=gen) * 2 - 1                   # s between 0.27 and 0.73
    A = -torch.exp(torch.linspace(-1.0, 3.14, C)) if C > 1 else torch.full((1,), -16.0)
    i = torch.randn(B, L, C, generator=gen)
    i[..., ::3] = -100.0
    d = dict(x=torch.randn(B, L, C, generator=gen).to(dtype), r=r.to(dtype), i=i.to(dtype), A=A,
             state=torch.randn(B, C, generator=gen),
             lens=None if lens is None else torch.tensor(lens, dtype=torch.int32))
    return d, torch.randn(B, L, C, generator=gen).to(dtype), torch.randn(B, C, generator=gen)


def on(d):
    return {k: (v.to(DEV) if isinstance(v, torch.Tensor) else v) for k, v in d.items()}


def split(d):
    return (d["x"], d["r"], d["i"], d["A"]), dict(state=d["state"], lens=d["lens"])


@pytest.mark.parametrize("c", STRONG)
@pytest.mark.parametrize("keep", [False, True])
def test_strong_decays(c, keep):
    """A decay of exp(-17) is off by no more than its exponent's roundings, so
    states, gradients of A, r and the state keep the digits that products of such decays
    have. A token adds a decay's steps and 3 (a product, a sum, the input's own
    roundings are counted below) to what the state before is off; chunks fold once more.
    beta sigmoid(i) x by 12 and half of the decay's steps (1 - a^2 = -e (2 + e), and e is
    off by at most as much as a). The gradients take g and a state (as many each), the
    decay twice, its slope and up to 8 products: three times as many and 80.
    What is below the normal range is taken as 0, and enters results times factors (g,
    A, sums over tokens) below 1000: FLUSH."""
    B, L, C, lens = c
    inp, gy, gs = strong_case(*c)
    d = on(inp)
    args, par = split(d)
    n = steps_of_decay(1.0, 17.0)
    count = 2 * L * (n + 3) + n + 12
    end = torch.empty(B, C, device=DEV)
    saved = g.gated_recurrence_saved(args[0]) if keep else None
    out = g.gated_recurrence(*args, **par, state_out=end, saved=saved)
    (ref, ref_end), (size, size_end) = plain.gated(**inp), plain.gated(**inp, absolute=True)
    small = FLUSH / (count * plain.F32_STEP)
    plain.within(out, ref, size + small, count, "out")
    plain.within(end, ref_end, size_end + small, count, "state")
    got = g.gated_recurrence_backward(*args, gy.to(DEV), **par, saved=saved, grad_state=gs.to(DEV))
    ref = plain.gated_grads(**inp, gy=gy, grad_state=gs)
    size = plain.gated_grads(**inp, gy=gy, grad_state=gs, absolute=True)
    for k in ref:
        plain.within(got[k], ref[k], size[k] + small, 3 * count + 80 + (B * L if k == "A" else 0), "d" + k)


@pytest.mark.parametrize("A", [-0.5, -8.0, -16.0, -32.0])
@pytest.mark.parametrize("C", [64, 63])
def test_strong_decays_in_the_norm(A, C):
    """Errors of r's and A's gradients in the norm. Where |A s| is v, the decay is off
    by some v sqrt(6) + 2 steps as its exponent's roundings fall, and a value's
    weight falls with the decay, exp(-v): v exp(-v) has its largest value at 1, so the
    decay's part is below 6 steps whatever A is; 12 products and sums of state
    and slope fall as 4 more, and the sums of A's gradient over 256 tokens 16: 2^-24 times
    16 and 32."""
    gen = torch.Generator().manual_seed(40)
    B, L = 1, 256
    x, r, i, gy = torch.randn(4, B, L, C, generator=gen)
    inp = dict(x=x, r=r, i=i, A=torch.full((C,), A))
    got = g.gated_recurrence_backward(*(v.to(DEV) for v in inp.values()), gy.to(DEV))
    ref = plain.gated_grads(**inp, gy=gy)
    for k, steps in (("r", 16), ("A", 32), ("x", 16), ("i", 16)):
        err = float((got[k].double().cpu() - ref[k]).norm() / ref[k].norm())
        assert err <= steps * plain.F32_STEP, (k, err)


# --------------------------------------------------------------------------
# gated recurrence: infinities beside padding
# --------------------------------------------------------------------------
@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
@pytest.mark.parametrize("B,L,C,dtype,lens", [
    (2, 70, 66, BF16, (59, 3)),       # the last token within a run of eight and of sixteen
    (2, 70, 7, F32, (1, 64)),
    (2, 20, 130, F32, (13, 9)),
    (3, 200, 64, BF16, (129, 0, 130)),
])
def test_padding_beside_a_last_token_that_is_not_finite(B, L, C, dtype, lens, bad):
    """The last token's x, its gates and the state's gradient not finite: padding has
    zeros all the same, in results and gradients."""
    gen = torch.Generator().manual_seed(41)
    x, r, i, gy = (torch.randn(B, L, C, generator=gen).to(dtype) for _ in range(4))
    A, gs = -torch.rand(C, generator=gen) - 0.1, torch.randn(B, C, generator=gen)
    pad = torch.arange(L)[None] >= torch.tensor(lens)[:, None]
    for name in ("x", "r", "i", "gy", "gs", "state"):
        v = {"x": x.clone(), "r": r.clone(), "i": i.clone(), "gy": gy.clone(), "gs": gs.clone(),
             "state": torch.randn(B, C, generator=gen)}
        for b, n in enumerate(lens):
            if name in ("gs", "state"):
                v[name][b] = bad
            elif n:
                v[name][b, n - 1] = bad
        d = {k: t.to(DEV) for k, t in v.items()}
        args = (d["x"], d["r"], d["i"], A.to(DEV))
        par = dict(state=d["state"], lens=torch.tensor(lens, dtype=torch.int32, device=DEV))
        assert not g.gated_recurrence(*args, **par).cpu()[pad].any(), name
        got = g.gated_recurrence_backward(*args, d["gy"], **par, grad_state=d["gs"])
        for k in "xri":
            assert not got[k].cpu()[pad].any(), (name, k)      # NaN counts as any


# --------------------------------------------------------------------------
# vocabulary loss: no tokens
# --------------------------------------------------------------------------
@pytest.mark.parametrize("D,dtype", [(15, F32), (7, BF16), (16, F32), (16, BF16)])
@pytest.mark.parametrize("B,L", [(0, 4), (3, 0)])
def test_empty_batch_does_not_read_the_weight(B, L, D, dtype):
    """Rows of whole pieces and of none, with a weight and without one: the weight's
    gradient is zeros, and nothing is packed."""
    V = 700
    x, w = torch.empty(B, L, D, dtype=dtype, device=DEV), torch.ones(V, D, dtype=dtype, device=DEV)
    t, no = torch.empty(B, L, dtype=torch.int64, device=DEV), torch.empty(B, L, device=DEV)
    got, names = launches(lambda: g.vocab_loss_backward(x, w, t, no, no))
    assert got["x"].shape == (B, L, D) and not got["weight"].any()
    assert "loss_pack" not in names, names
    L_ = tokens._lib()
    code = tokens._CODE[dtype]
    need = L_.gspn_vocab_loss_backward_workspace_bytes(B, L, V, D, code)
    ws = torch.empty(need, dtype=torch.uint8, device=DEV)
    dw = torch.full((V, D), float("nan"), dtype=dtype, device=DEV)
    a = tokens._LOSS.pack(B, L, V, D, code, 1, 0, 0, 0, 0, 0, 0, 0, 0, 0)
    stream = torch.cuda.current_stream().cuda_stream
    assert L_.gspn_vocab_loss_backward_ws(a, tokens._LOSS_GRADS.pack(0, 0, 0, dw.data_ptr()), ws.data_ptr(), need,
                                          stream) == 0
    torch.cuda.synchronize()
    assert not dw.any()


# --------------------------------------------------------------------------
# gated recurrence: up to how many tokens a lane walks them all
# --------------------------------------------------------------------------
@pytest.mark.parametrize("B,C,dtype,last", [
    (16, 130, BF16, 12),        # few lanes
    (64, 2304, BF16, 28),       # 73728 lanes of two channels
    (64, 2304, F32, 28),
    (80, 1001, BF16, 24),       # 80080 of one
    (80, 2304, BF16, 32),       # 92160 of two
    (128, 1001, F32, 32),
])
def test_a_lane_walks_all_tokens_only_where_chunks_take_longer(B, C, dtype, last):
    gen = torch.Generator().manual_seed(50)
    A, state = -torch.rand(C, generator=gen), torch.randn(B, C, generator=gen)
    for L, want in ((last, "gated_short"), (last + 1, "gated")):
        x, r, i = (torch.randn(B, L, C, generator=gen).to(dtype) for _ in range(3))
        end = torch.empty(B, C, device=DEV)
        out, names = launches(lambda: g.gated_recurrence(x.to(DEV), r.to(DEV), i.to(DEV), A.to(DEV),
                                                         state=state.to(DEV), state_out=end))
        assert names[-1] == want, (L, names)
        few = slice(B - 2, B)
        inp = dict(x=x[few], r=r[few], i=i[few], A=A, state=state[few])
        (ref, ref_end), (size, size_end) = plain.gated(**inp), plain.gated(**inp, absolute=True)
        plain.within(out[few], ref, size, 18 * L + 26, "out")          # |A| <= 1: as in test_gated_gpu.py
        plain.within(end[few], ref_end, size_end, 18 * L + 26, "state")
