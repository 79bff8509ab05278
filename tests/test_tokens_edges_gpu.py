"""The token-sequence operators on the GPU where a call can go wrong without
looking wrong: precision of the operands, memory that is input and output,
infinities beside masks, launches of many workgroups, states handed from chunk
to chunk. References are the plain 64-bit forms (plain_tokens.py)."""
from __future__ import annotations

import pytest
import torch

import linear_spatial_propagation_line_amd as g
import plain_tokens as plain
from test_tokens_gpu import BF16, DEV, F32, attn_case, close, conv_call, conv_case, dev, rms, scan_args, scan_case

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


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_conv_in_place_over_several_runs(dtype):
    inp, _ = conv_case(4, 300, 200, 4, dtype, (300, 0, 2, 129), True, True, True, seed=13)
    d = dev(inp)
    end, st = torch.empty_like(d["state"]), d["state"].clone()
    out = conv_call(d, state_out=end)
    assert torch.equal(conv_call(dict(d, state=st), state_out=st), out) and torch.equal(st, end)
