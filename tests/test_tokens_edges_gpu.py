"""The token-sequence operators on the GPU where a call can go wrong without
looking wrong: precision of the operands, memory that is input and output,
infinities beside masks, launches of many workgroups, states handed from chunk
to chunk. References are the plain 64-bit forms (plain_tokens.py)."""
from __future__ import annotations

import pytest
import torch

import linear_spatial_propagation_line_amd as g
import plain_tokens as plain
from test_tokens_gpu import BF16, DEV, F32, attn_case, dev, rms

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
