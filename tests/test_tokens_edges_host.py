"""Host-only checks of the token operators' C ABI beyond the documented
refusals: what may and may not be the same memory. No call here reaches a HIP
API."""
from __future__ import annotations

import linear_spatial_propagation_line_amd as g
from test_tokens_host import L, at, conv, scan  # noqa: F401  (L is a fixture)


def test_only_the_state_may_be_moved_on_in_place(L):
    """state_out may be state, and nothing else that happens to span the same
    bytes: here x of three tokens for four taps, and dt of as many tokens as
    there are states."""
    # so that a call that gets past the alias checks stops at the workspace
    one = dict(B=1, T=3, C=16, K=4, xs=(48, 16), bias=0, lens=0)
    assert conv(L, **one, x=at(3), state_out=at(3)) == g.STATUS["GSPN_E_ALIAS"]
    assert conv(L, **one, x=at(3), state=0, state_out=at(3)) == g.STATUS["GSPN_E_ALIAS"]
    eight = dict(B=1, T=8, C=16, N=8, G=1, ws=None)
    assert scan(L, **eight, d=at(8), state_out=at(8)) == g.STATUS["GSPN_E_ALIAS"]
    assert scan(L, **eight, D=at(8), state=at(8), state_out=at(8)) == g.STATUS["GSPN_E_ALIAS"]
    assert scan(L, **eight, state_out=at(8)) == g.STATUS["GSPN_E_WORKSPACE"]
    assert scan(L, **eight, state_out=at(8) + 64) == g.STATUS["GSPN_E_ALIAS"]
