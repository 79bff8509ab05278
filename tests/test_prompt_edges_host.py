"""Host-only checks of the token embedding, the gated recurrence and the vocabulary
loss where a plan, not an argument, can be wrong (no call here reaches a HIP API)."""
from __future__ import annotations

import pytest

from test_tokens_host import L  # noqa: F401  (a fixture)


@pytest.mark.parametrize("B,T", [(0, 4), (3, 0)])
@pytest.mark.parametrize("dt,D", [(0, 15), (1, 15), (0, 1), (1, 2049)])
def test_an_empty_batch_packs_no_weight(L, B, T, dt, D):  # noqa: F811
    """Rows of no whole pieces are packed, V of them, into the workspace; without a
    token the weight may be NULL, and no copy of it is planned."""
    V = 1 << 20
    need = L.gspn_vocab_loss_backward_workspace_bytes
    row = -(-D * (4, 2)[dt] // 128) * 128
    # 4096 for lists of one token
    assert need(B, T, V, D, dt) < need(1, 1, V, D, dt) - V * row + 4096
