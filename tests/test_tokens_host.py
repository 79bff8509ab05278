"""Host-only checks of the token operators' C ABI (no call here reaches a HIP
API): argument structs laid out as the header's, refusals with the documented
status before anything is enqueued, workspace sizes."""
from __future__ import annotations

import os
import subprocess

import pytest

import linear_spatial_propagation_line_amd as g
from linear_spatial_propagation_line_amd import tokens

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
# fake, well-aligned device addresses: validation never dereferences them
BASE, SZ = 1 << 40, 1 << 36


def at(i):
    return BASE + i * SZ


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(g.LIB_PATH):
        from linear_spatial_propagation_line_amd import build
        build.build()
    return tokens._lib()


def test_struct_layouts_match_the_header(tmp_path):
    src = tmp_path / "sizes.c"
    names = ("conv_args", "conv_grads", "scan_args", "scan_grads", "attn_args", "attn_grads")
    src.write_text('#include <stdio.h>\n#include "gspn_tokens.h"\nint main(void) {\n'
                   + "".join(f'  printf("%zu\\n", sizeof(gspn_{n}));\n' for n in names)
                   + '  printf("%zu %zu %zu\\n", offsetof(gspn_scan_args, A), offsetof(gspn_scan_args, saved),'
                     " offsetof(gspn_attn_args, mask));\n  return 0;\n}\n")
    exe = tmp_path / "sizes"
    subprocess.run(["gcc", "-D__HIP_PLATFORM_AMD__", "-I", os.path.join(ROOT, "include"), "-I",
                    "/opt/rocm/include", str(src), "-o", str(exe)], check=True)
    got = subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()
    structs = (tokens._CONV, tokens._CONV_GRADS, tokens._SCAN, tokens._SCAN_GRADS, tokens._ATTN,
               tokens._ATTN_GRADS)
    assert [int(v) for v in got[:6]] == [s.size for s in structs]
    assert [int(v) for v in got[6:]] == [5 * 8 + 8 + 9 * 8, 248 - 8, 6 * 8 + 8 + 12 * 8]


def conv(L, B=2, T=8, C=16, K=4, dt=0, x=at(0), xs=(128, 16), w=at(1), bias=at(2), state=at(3), lens=at(4),
         out=at(5), state_out=at(6), null=False):
    a = tokens._CONV.pack(B, T, C, K, dt, 1, x, *xs, w, bias, state, lens, out, state_out)
    return L.gspn_causal_conv(None if null else a, None)


@pytest.mark.parametrize("kw,status", [
    (dict(null=True), "GSPN_E_NULL"), (dict(x=0), "GSPN_E_NULL"), (dict(w=0), "GSPN_E_NULL"),
    (dict(out=0), "GSPN_E_NULL"),
    (dict(dt=2), "GSPN_E_DTYPE"), (dict(B=-1), "GSPN_E_SHAPE"), (dict(T=-1), "GSPN_E_SHAPE"),
    (dict(K=0), "GSPN_E_SHAPE"), (dict(K=5), "GSPN_E_SHAPE"), (dict(C=1 << 31), "GSPN_E_SHAPE"),
    (dict(B=1 << 30, T=1 << 30, C=1 << 20), "GSPN_E_SHAPE"), (dict(xs=(-1, 16)), "GSPN_E_SHAPE"),
    (dict(xs=(1 << 62, 16)), "GSPN_E_SHAPE"),
    (dict(x=at(0) + 2), "GSPN_E_ALIGN"), (dict(lens=at(4) + 1), "GSPN_E_ALIGN"),
    (dict(out=at(0) + 64), "GSPN_E_ALIAS"), (dict(out=at(3)), "GSPN_E_ALIAS"),
    (dict(state_out=at(3) + 64), "GSPN_E_ALIAS"), (dict(state_out=at(5) + 4), "GSPN_E_ALIAS"),
    (dict(xs=(1 << 34, 16), out=at(0) + (1 << 36)), "GSPN_E_ALIAS"),      # reaches into the view's span
])
def test_conv_refusals(L, kw, status):
    assert conv(L, **kw) == g.STATUS[status]
    assert L.gspn_last_error().decode() != "" or status == "GSPN_E_NOMEM"


def test_empty_batches_enqueue_nothing(L):
    assert conv(L, B=0) == 0 and conv(L, C=0) == 0
    assert scan(L, B=0) == 0 and scan(L, C=0) == 0
    assert attn(L, B=0) == 0 and attn(L, Lq=0) == 0


def scan(L, B=2, T=8, C=16, N=4, G=2, dt=0, x=at(0), d=at(1), z=at(2), A=at(3), Bm=at(4), Cm=at(5), D=at(6),
         bias=at(7), state=at(8), lens=at(9), out=at(10), state_out=at(11), saved=at(12), ws=at(13),
         ws_bytes=1 << 30, head=4):
    a = tokens._SCAN.pack(B, T, C, N, G, dt, 1, x, 128, 16, d, 128, 16, z, 128, 16, A, Bm, 64, 8, head, Cm, 64,
                          8, 4, D, bias, state, lens, out, state_out, saved)
    return L.gspn_selective_scan_ws(a, ws, ws_bytes, None)


@pytest.mark.parametrize("kw,status", [
    (dict(x=0), "GSPN_E_NULL"), (dict(A=0), "GSPN_E_NULL"), (dict(Bm=0), "GSPN_E_NULL"), (dict(out=0), "GSPN_E_NULL"),
    (dict(dt=-1), "GSPN_E_DTYPE"), (dict(N=0), "GSPN_E_SHAPE"), (dict(N=33), "GSPN_E_SHAPE"),
    (dict(G=3), "GSPN_E_SHAPE"), (dict(G=0), "GSPN_E_SHAPE"), (dict(head=-4), "GSPN_E_SHAPE"),
    (dict(A=at(3) + 2), "GSPN_E_ALIGN"), (dict(saved=at(12) + 16), "GSPN_E_ALIGN"), (dict(ws=at(13) + 8), "GSPN_E_ALIGN"),
    (dict(out=at(2)), "GSPN_E_ALIAS"), (dict(state_out=at(10)), "GSPN_E_ALIAS"), (dict(state_out=at(6)), "GSPN_E_ALIAS"),
    (dict(saved=at(0)), "GSPN_E_ALIAS"), (dict(ws=at(5)), "GSPN_E_ALIAS"), (dict(ws=at(10)), "GSPN_E_ALIAS"),
    (dict(ws=None), "GSPN_E_WORKSPACE"), (dict(ws_bytes=100), "GSPN_E_WORKSPACE"),
])
def test_scan_refusals(L, kw, status):
    assert scan(L, **kw) == g.STATUS[status]


def test_scan_backward_wants_the_gate_gradient_with_a_gate(L):
    def call(z, dz):
        a = tokens._SCAN.pack(2, 8, 16, 4, 1, 0, 1, at(0), 128, 16, at(1), 128, 16, z, 128, 16, at(3), at(4), 32, 4,
                              4, at(5), 32, 4, 4, 0, 0, 0, 0, 0, 0, 0)
        gr = tokens._SCAN_GRADS.pack(at(14), 128, 16, 0, at(15), at(16), dz, at(17), at(18), at(19), 0, 0, 0)
        return L.gspn_selective_scan_backward_ws(a, gr, None, 0, None)
    assert call(at(2), 0) == g.STATUS["GSPN_E_NULL"]
    assert call(0, at(20)) == g.STATUS["GSPN_E_NULL"]
    assert call(at(2), at(20)) == g.STATUS["GSPN_E_WORKSPACE"]     # past the gate check


def attn(L, B=2, Lq=8, Lk=12, Hq=4, Hkv=2, E=16, dt=0, scale=0.25, q=at(0), k=at(1), v=at(2), mask=at(3), out=at(4),
         lse=at(5), ws=at(6), ws_bytes=1 << 34, row=64):
    a = tokens._ATTN.pack(B, Lq, Lk, Hq, Hkv, E, dt, scale, q, 512, row, 16, k, 384, 32, 16, v, 384, 32, 16, mask, 12,
                          out, lse)
    return L.gspn_cross_attention_ws(a, ws, ws_bytes, None)


@pytest.mark.parametrize("kw,status", [
    (dict(q=0), "GSPN_E_NULL"), (dict(k=0), "GSPN_E_NULL"), (dict(out=0), "GSPN_E_NULL"),
    (dict(dt=7), "GSPN_E_DTYPE"), (dict(E=0), "GSPN_E_SHAPE"), (dict(E=129), "GSPN_E_SHAPE"),
    (dict(Hq=3), "GSPN_E_SHAPE"), (dict(Hkv=0), "GSPN_E_SHAPE"), (dict(Lk=-1), "GSPN_E_SHAPE"),
    (dict(scale=0.0), "GSPN_E_SHAPE"), (dict(scale=-1.0), "GSPN_E_SHAPE"), (dict(scale=float("nan")), "GSPN_E_SHAPE"),
    (dict(scale=float("inf")), "GSPN_E_SHAPE"), (dict(row=-64), "GSPN_E_SHAPE"), (dict(Lq=1 << 31), "GSPN_E_SHAPE"),
    (dict(q=at(0) + 2), "GSPN_E_ALIGN"), (dict(lse=at(5) + 2), "GSPN_E_ALIGN"),
    (dict(out=at(1)), "GSPN_E_ALIAS"), (dict(out=at(3)), "GSPN_E_ALIAS"), (dict(lse=at(4)), "GSPN_E_ALIAS"),
    # few queries over a long key axis: partial results need scratch memory
    (dict(Lq=1, Lk=8192, ws=None), "GSPN_E_WORKSPACE"), (dict(Lq=1, Lk=8192, ws=at(6) + 128), "GSPN_E_ALIGN"),
    (dict(Lq=1, Lk=8192, ws=at(2)), "GSPN_E_ALIAS"),
])
def test_attention_refusals(L, kw, status):
    assert attn(L, **kw) == g.STATUS[status]


def test_workspace_sizes(L):
    w = L.gspn_selective_scan_workspace_bytes
    assert w(4, 1, 256, 16, 1, 1) == 0 and w(4, 4, 256, 16, 1, 1) == 0      # single tokens
    assert w(4, 64, 256, 16, 1, 1) > 0 and w(4, 64, 256, 40, 1, 1) == 0     # 0 for what the call refuses
    s = L.gspn_selective_scan_saved_bytes
    assert s(2, 64, 10, 16) == 2 * 4 * 16 * 10 * 4 and s(2, 65, 10, 9) == 2 * 5 * 16 * 10 * 4
    a = L.gspn_cross_attention_workspace_bytes
    assert a(2, 1 << 20, 77, 4, 4, 64, 1) == 0                               # rows enough: nothing split
    assert a(2, 1, 8192, 4, 4, 64, 1) > 0
    assert L.gspn_causal_conv_backward_workspace_bytes(2, 100, 64, 9, 0) == 0
