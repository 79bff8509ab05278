"""Host-only checks of the C ABI of the token embedding, the gated recurrence and
the vocabulary loss (no call here reaches a HIP API) and of their plain forms: argument structs laid
out as the header's, refusals with the documented status before anything is
enqueued, workspace sizes; the plain gradients against differences."""
from __future__ import annotations

import os
import subprocess

import pytest
import torch

import linear_spatial_propagation_line_amd as g
import plain_prompt as plain
import plain_tokens
from linear_spatial_propagation_line_amd import tokens
from test_tokens_host import L, ROOT, at  # noqa: F401  (L is a fixture)


def test_struct_layouts_match_the_header(tmp_path):
    src = tmp_path / "sizes.c"
    names = ("embed_args", "embed_grads", "gated_args", "gated_grads", "loss_args", "loss_grads")
    src.write_text('#include <stdio.h>\n#include "gspn_tokens.h"\nint main(void) {\n'
                   + "".join(f'  printf("%zu\\n", sizeof(gspn_{n}));\n' for n in names)
                   + '  printf("%zu %zu %zu\\n", offsetof(gspn_embed_args, scale), offsetof(gspn_embed_args, ids),'
                     " offsetof(gspn_gated_args, A));\n  return 0;\n}\n")
    exe = tmp_path / "sizes"
    subprocess.run(["gcc", "-D__HIP_PLATFORM_AMD__", "-I", os.path.join(ROOT, "include"), "-I",
                    "/opt/rocm/include", str(src), "-o", str(exe)], check=True)
    got = subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()
    structs = (tokens._EMBED, tokens._EMBED_GRADS, tokens._GATED, tokens._GATED_GRADS, tokens._LOSS,
               tokens._LOSS_GRADS)
    assert [int(v) for v in got[:6]] == [s.size for s in structs]
    assert [int(v) for v in got[6:]] == [40, 48, 3 * 8 + 8 + 9 * 8]


# ---- embedding ----------------------------------------------------------------
def embed(L, B=2, T=8, V=50, D=16, dt=0, wide=1, scale=1.0, ids=at(0), ib=8, lens=at(1), w=at(2), out=at(3),
          null=False):
    a = tokens._EMBED.pack(B, T, V, D, dt, wide, scale, ids, ib, lens, w, out)
    return L.gspn_token_embedding(None if null else a, None)


@pytest.mark.parametrize("kw,status", [
    (dict(null=True), "GSPN_E_NULL"), (dict(ids=0), "GSPN_E_NULL"), (dict(w=0), "GSPN_E_NULL"),
    (dict(out=0), "GSPN_E_NULL"), (dict(dt=2), "GSPN_E_DTYPE"), (dict(B=-1), "GSPN_E_SHAPE"),
    (dict(T=-1), "GSPN_E_SHAPE"), (dict(V=0), "GSPN_E_SHAPE"), (dict(D=0), "GSPN_E_SHAPE"),
    (dict(V=1 << 31), "GSPN_E_SHAPE"), (dict(B=1 << 16, T=1 << 15), "GSPN_E_SHAPE"),
    (dict(B=1 << 15, T=1 << 15, D=1 << 23), "GSPN_E_SHAPE"), (dict(ib=-1), "GSPN_E_SHAPE"),
    (dict(scale=float("nan")), "GSPN_E_SHAPE"), (dict(scale=float("inf")), "GSPN_E_SHAPE"),
    (dict(ids=at(0) + 4), "GSPN_E_ALIGN"), (dict(ids=at(0) + 2, wide=0), "GSPN_E_ALIGN"),
    (dict(w=at(2) + 2), "GSPN_E_ALIGN"), (dict(lens=at(1) + 2), "GSPN_E_ALIGN"),
    (dict(out=at(2) + 64), "GSPN_E_ALIAS"), (dict(out=at(0)), "GSPN_E_ALIAS"),
])
def test_embedding_refusals(L, kw, status):  # noqa: F811
    assert embed(L, **kw) == g.STATUS[status]


def embed_grad(L, B=2, T=8, V=50, D=16, dt=0, ids=at(0), gy=at(1), rows=(128, 16), dw=at(2), ws=at(3),
               ws_bytes=1 << 30):
    a = tokens._EMBED.pack(B, T, V, D, dt, 1, 1.0, ids, 8, 0, 0, 0)
    return L.gspn_token_embedding_backward_ws(a, tokens._EMBED_GRADS.pack(gy, *rows, dw), ws, ws_bytes, None)


@pytest.mark.parametrize("kw,status", [
    (dict(ids=0), "GSPN_E_NULL"), (dict(gy=0), "GSPN_E_NULL"), (dict(dw=0), "GSPN_E_NULL"),
    (dict(rows=(128, -16)), "GSPN_E_SHAPE"), (dict(dw=at(1)), "GSPN_E_ALIAS"), (dict(ws=at(1)), "GSPN_E_ALIAS"),
    (dict(ws=at(2)), "GSPN_E_ALIAS"), (dict(ws=at(3) + 64), "GSPN_E_ALIGN"), (dict(ws=None), "GSPN_E_WORKSPACE"),
    (dict(ws_bytes=100), "GSPN_E_WORKSPACE"),
])
def test_embedding_backward_refusals(L, kw, status):  # noqa: F811
    assert embed_grad(L, **kw) == g.STATUS[status]


# ---- gated recurrence ---------------------------------------------------------
def gated(L, B=2, T=80, C=16, dt=0, x=at(0), r=at(1), i=at(2), A=at(3), state=at(4), lens=at(5), out=at(6),
          state_out=at(7), saved=at(8), ws=at(9), ws_bytes=1 << 30, row=16, null=False):
    a = tokens._GATED.pack(B, T, C, dt, x, 1280, row, r, 1280, 16, i, 1280, 16, A, state, lens, out, state_out, saved)
    return L.gspn_gated_recurrence_ws(None if null else a, ws, ws_bytes, None)


@pytest.mark.parametrize("kw,status", [
    (dict(null=True), "GSPN_E_NULL"), (dict(x=0), "GSPN_E_NULL"), (dict(r=0), "GSPN_E_NULL"),
    (dict(i=0), "GSPN_E_NULL"), (dict(A=0), "GSPN_E_NULL"), (dict(out=0), "GSPN_E_NULL"),
    (dict(dt=-1), "GSPN_E_DTYPE"), (dict(B=-1), "GSPN_E_SHAPE"), (dict(C=-2), "GSPN_E_SHAPE"),
    (dict(T=1 << 31), "GSPN_E_SHAPE"), (dict(C=1 << 30), "GSPN_E_SHAPE"), (dict(row=-1), "GSPN_E_SHAPE"),
    (dict(B=1 << 20, T=1 << 20, C=1 << 20), "GSPN_E_SHAPE"),
    (dict(x=at(0) + 2), "GSPN_E_ALIGN"), (dict(A=at(3) + 2), "GSPN_E_ALIGN"), (dict(saved=at(8) + 16), "GSPN_E_ALIGN"),
    (dict(ws=at(9) + 8), "GSPN_E_ALIGN"), (dict(out=at(0)), "GSPN_E_ALIAS"), (dict(state_out=at(3)), "GSPN_E_ALIAS"),
    (dict(state_out=at(4) + 64), "GSPN_E_ALIAS"), (dict(saved=at(2)), "GSPN_E_ALIAS"), (dict(ws=at(6)), "GSPN_E_ALIAS"),
    (dict(ws=None), "GSPN_E_WORKSPACE"), (dict(ws_bytes=64), "GSPN_E_WORKSPACE"),
    (dict(state_out=at(4), ws=None), "GSPN_E_WORKSPACE"),      # in place: past the alias checks
])
def test_gated_refusals(L, kw, status):  # noqa: F811
    assert gated(L, **kw) == g.STATUS[status]


def test_gated_backward_refusals(L):  # noqa: F811
    def call(dx=at(20), ws=at(9), saved=at(8), dA=at(23)):
        a = tokens._GATED.pack(2, 80, 16, 0, at(0), 1280, 16, at(1), 1280, 16, at(2), 1280, 16, at(3), 0, 0, 0, 0, saved)
        gr = tokens._GATED_GRADS.pack(at(10), 1280, 16, 0, dx, at(21), at(22), dA, 0)
        return L.gspn_gated_recurrence_backward_ws(a, gr, ws, 0, None)
    assert call() == g.STATUS["GSPN_E_WORKSPACE"]
    assert call(dx=0) == call(dA=0) == g.STATUS["GSPN_E_NULL"]
    assert call(dx=at(10)) == call(dx=at(8)) == call(dx=at(21)) == g.STATUS["GSPN_E_ALIAS"]
    assert call(saved=at(8) + 4) == g.STATUS["GSPN_E_ALIGN"]


# ---- vocabulary loss ----------------------------------------------------------
def loss(L, B=2, T=8, V=50, D=16, dt=0, wide=1, x=at(0), row=16, w=at(1), t=at(2), tb=8, lens=at(3), out=at(4),
         lse=at(5), ws=at(6), ws_bytes=1 << 30, null=False):
    a = tokens._LOSS.pack(B, T, V, D, dt, wide, x, 128, row, w, t, tb, lens, out, lse)
    return L.gspn_vocab_loss_ws(None if null else a, ws, ws_bytes, None)


@pytest.mark.parametrize("kw,status", [
    (dict(null=True), "GSPN_E_NULL"), (dict(x=0), "GSPN_E_NULL"), (dict(w=0), "GSPN_E_NULL"),
    (dict(t=0), "GSPN_E_NULL"), (dict(out=0), "GSPN_E_NULL"), (dict(dt=3), "GSPN_E_DTYPE"),
    (dict(B=-1), "GSPN_E_SHAPE"), (dict(V=0), "GSPN_E_SHAPE"), (dict(D=0), "GSPN_E_SHAPE"),
    (dict(D=1 << 20), "GSPN_E_SHAPE"), (dict(V=1 << 31), "GSPN_E_SHAPE"), (dict(B=1 << 14, T=1 << 14), "GSPN_E_SHAPE"),
    (dict(B=1 << 13, T=1 << 14, V=1 << 30), "GSPN_E_SHAPE"), (dict(row=-1), "GSPN_E_SHAPE"), (dict(tb=-8), "GSPN_E_SHAPE"),
    (dict(x=at(0) + 2), "GSPN_E_ALIGN"), (dict(w=at(1) + 4), "GSPN_E_ALIGN"), (dict(w=at(1) + 2, D=15), "GSPN_E_ALIGN"),
    (dict(t=at(2) + 4), "GSPN_E_ALIGN"), (dict(lse=at(5) + 2), "GSPN_E_ALIGN"), (dict(ws=at(6) + 16), "GSPN_E_ALIGN"),
    (dict(out=at(5)), "GSPN_E_ALIAS"), (dict(lse=at(2)), "GSPN_E_ALIAS"), (dict(ws=at(1)), "GSPN_E_ALIAS"),
    (dict(ws=None), "GSPN_E_WORKSPACE"), (dict(ws_bytes=512), "GSPN_E_WORKSPACE"),
    (dict(w=at(1) + 4, D=15, ws=None), "GSPN_E_WORKSPACE"),     # rows of no whole pieces may begin anywhere
])
def test_loss_refusals(L, kw, status):  # noqa: F811
    assert loss(L, **kw) == g.STATUS[status]


def test_loss_backward_refusals(L):  # noqa: F811
    def call(lse=at(5), gl=at(7), dx=at(8), dw=at(9), ws=at(6), n=0):
        a = tokens._LOSS.pack(2, 8, 50, 16, 0, 1, at(0), 128, 16, at(1), at(2), 8, 0, 0, 0)
        return L.gspn_vocab_loss_backward_ws(a, tokens._LOSS_GRADS.pack(lse, gl, dx, dw), ws, n, None)
    assert call() == g.STATUS["GSPN_E_WORKSPACE"]
    for kw in (dict(lse=0), dict(gl=0), dict(dx=0), dict(dw=0)):
        assert call(**kw) == g.STATUS["GSPN_E_NULL"]
    for kw in (dict(dx=at(0)), dict(dw=at(1)), dict(dw=at(8)), dict(dx=at(5)), dict(ws=at(9), n=1 << 30)):
        assert call(**kw) == g.STATUS["GSPN_E_ALIAS"]


def test_empty_batches_enqueue_nothing(L):  # noqa: F811
    assert embed(L, B=0) == 0 and embed(L, T=0) == 0
    assert gated(L, B=0) == 0 and gated(L, C=0) == 0
    assert loss(L, B=0, ws=None) == 0 and loss(L, T=0, ws=None) == 0


def test_workspace_sizes(L):  # noqa: F811
    w = L.gspn_gated_recurrence_workspace_bytes
    assert w(4, 64, 256, 1) == 0 and w(4, 65, 256, 1) > 0 and w(4, 65, -1, 1) == 0
    s = L.gspn_gated_recurrence_saved_bytes
    assert s(2, 64, 10) == 2 * 10 * 4 and s(2, 65, 10) == 2 * 2 * 10 * 4
    e = L.gspn_token_embedding_backward_workspace_bytes
    assert e(2, 10, 50, 16, 0) > 0 and e(2, 10, 0, 16, 0) == 0
    f, b = L.gspn_vocab_loss_workspace_bytes, L.gspn_vocab_loss_backward_workspace_bytes
    assert f(2, 0, 50, 16, 0) == 0 and f(2, 8, 50, 16, 0) > 0 and f(2, 8, 0, 16, 0) == 0
    assert b(2, 0, 50, 16, 0) > 0 and b(2, 8, 50, 16, 2) == 0
    # pieces: the logits of 8192 tokens over 131072 rows would take 2 GiB
    assert b(1, 8192, 131072, 64, 1) < (1 << 30)


# ---- the plain forms ----------------------------------------------------------
def test_plain_gated_gradients_against_differences():
    gen = torch.Generator().manual_seed(0)
    B, T, C = 2, 9, 3
    lens = torch.tensor([9, 4])
    d = dict(x=torch.randn(B, T, C, generator=gen), r=torch.randn(B, T, C, generator=gen),
             i=torch.randn(B, T, C, generator=gen), A=-torch.rand(C, generator=gen) - 0.05,
             state=torch.randn(B, C, generator=gen), lens=lens)
    gy = torch.randn(B, T, C, generator=gen)
    got = plain.gated_grads(**d, gy=gy)
    for k in ("x", "r", "i", "A", "state"):
        way = torch.randn(d[k].shape, generator=gen)
        want = plain_tokens.difference(plain.gated, d, k, way, gy)
        # the difference's own error is O(1e-8) of third derivatives of order 1
        assert abs(float((got[k] * way.double()).sum()) - want) <= 1e-6, k


def test_plain_loss_gradients_against_differences():
    gen = torch.Generator().manual_seed(1)
    x, w = torch.randn(2, 5, 4, generator=gen), torch.randn(7, 4, generator=gen)
    t = torch.tensor([[0, 6, -100, 3, 3], [1, 7, 2, 5, 4]])
    lens, gl = torch.tensor([5, 3]), torch.randn(2, 5, generator=gen)
    d = dict(x=x, weight=w, targets=t, lens=lens)
    got, _ = plain.vocab_loss_grads(x, w, t, gl, lens)
    for k in ("x", "weight"):
        way = torch.randn(d[k].shape, generator=gen)
        want = plain_tokens.difference(plain.vocab_loss, d, k, way, gl)
        assert abs(float((got[k] * way.double()).sum()) - want) <= 1e-6, k
