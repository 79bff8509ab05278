"""The token embedding, the gated recurrence and the vocabulary loss on the GPU
where a call can go wrong without looking wrong. References are the plain 64-bit forms
(plain_prompt.py)."""
from __future__ import annotations

import pytest
import torch

import linear_spatial_propagation_line_amd as g
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
