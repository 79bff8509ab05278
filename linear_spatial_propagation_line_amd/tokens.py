"""The token-sequence operators of ``libgspn.so`` (include/gspn_tokens.h):
the short causal convolution and the selective scan of a state space block,
and cross attention to an encoder's states, each with its gradients.

Like the rest of the binding this module only checks and marshals arguments.
Tensors are token-major device tensors of float32 or bfloat16, the last
dimension contiguous; inputs may otherwise be strided views. Work is enqueued
on ``stream`` (default: torch's current stream of the inputs' device), and
what a call allocates belongs to that stream."""
from __future__ import annotations

import ctypes
import struct

import torch

from . import GSPN_BF16, GSPN_F32, GspnError, lib

_CODE = {torch.float32: GSPN_F32, torch.bfloat16: GSPN_BF16}

# the argument structs of gspn_tokens.h, in native layout
_CONV = struct.Struct("@4qii PqqPPPPPP".replace(" ", ""))
_CONV_GRADS = struct.Struct("@PqqPPPPP")
_SCAN = struct.Struct("@5qii PqqPqqPqq P PqqqPqqq PPPP PPP".replace(" ", ""))
_SCAN_GRADS = struct.Struct("@PqqPPPPPPPPPP")
_ATTN = struct.Struct("@6qif PqqqPqqqPqqq Pq PP".replace(" ", ""))
_ATTN_GRADS = struct.Struct("@PqqqPPP")

_Tensor = torch.Tensor
# the current stream's handle and the current device, without the objects
# around them where torch offers that
_stream_of = getattr(torch._C, "_cuda_getCurrentRawStream",
                     lambda i: torch.cuda.current_stream(i).cuda_stream)
_device_now = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)

_tok = None


def _lib():
    """The library with the token operators' prototypes set."""
    global _tok
    if _tok is None:
        L = lib()
        a, vp, sz, i64 = ctypes.c_char_p, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int64
        for name, args, res in (
                ("gspn_causal_conv", [a, vp], ctypes.c_int),
                ("gspn_causal_conv_backward_ws", [a, a, vp, sz, vp], ctypes.c_int),
                ("gspn_causal_conv_backward_workspace_bytes", [i64] * 4 + [ctypes.c_int], sz),
                ("gspn_selective_scan_ws", [a, vp, sz, vp], ctypes.c_int),
                ("gspn_selective_scan_workspace_bytes", [i64] * 5 + [ctypes.c_int], sz),
                ("gspn_selective_scan_saved_bytes", [i64] * 4, sz),
                ("gspn_selective_scan_backward_ws", [a, a, vp, sz, vp], ctypes.c_int),
                ("gspn_selective_scan_backward_workspace_bytes", [i64] * 5 + [ctypes.c_int], sz),
                ("gspn_cross_attention_ws", [a, vp, sz, vp], ctypes.c_int),
                ("gspn_cross_attention_workspace_bytes", [i64] * 6 + [ctypes.c_int], sz),
                ("gspn_cross_attention_backward_ws", [a, a, vp, sz, vp], ctypes.c_int),
                ("gspn_cross_attention_backward_workspace_bytes", [i64] * 6 + [ctypes.c_int], sz)):
            f = getattr(L, name)
            f.argtypes, f.restype = args, res
        _tok = L
    return _tok


class _Call:
    """Checks tensors against the first one's device, allocates for the
    call's stream and runs one entry point on it."""

    def __init__(self, first, what, stream, dtype=None):
        if not isinstance(first, torch.Tensor) or first.device.type != "cuda":
            raise TypeError(f"{what} must be a torch tensor on a GPU")
        if first.dtype not in _CODE:
            raise TypeError(f"unsupported dtype {first.dtype} (float32 or bfloat16)")
        self.device, self.dtype, self.code = first.device, first.dtype, _CODE[first.dtype]
        self.index = first.get_device()
        if stream is None:
            self.ptr, self.own = _stream_of(self.index), None
        elif hasattr(stream, "cuda_stream"):
            self.ptr, self.own = stream.cuda_stream, stream
        else:
            self.ptr = int(stream)
            self.own = torch.cuda.ExternalStream(self.ptr, device=first.device)

    def tensor(self, t, shape, what, dtype=None, contiguous=False):
        """An input of the given shape, in the call's dtype (or ``dtype``)."""
        if not isinstance(t, torch.Tensor) or t.get_device() != self.index:
            raise TypeError(f"{what} must be a torch tensor on {self.device}")
        if t.dtype is not (dtype or self.dtype):
            raise ValueError(f"{what} must be {dtype or self.dtype}, not {t.dtype}")
        if t.shape != shape:
            raise ValueError(f"{what} must have shape {tuple(shape)}, not {tuple(t.shape)}")
        if contiguous and not t.is_contiguous():
            raise ValueError(f"{what} must be contiguous")
        return t

    def view(self, t, shape, what):
        """(address, strides) of an input whose last dimension is contiguous."""
        if not (type(t) is _Tensor and t.get_device() == self.index and t.dtype is self.dtype
                and t.shape == shape):
            self.tensor(t, shape, what)
        s = t.stride()
        if s[-1] != 1 and shape[-1] > 1:
            raise ValueError(f"{what} must be contiguous in its last dimension")
        return (t.data_ptr(),) + s[:-1]

    def data(self, t, shape, what, dtype=None):
        """Address of a contiguous input, 0 for None."""
        if t is None:
            return 0
        if not (type(t) is _Tensor and t.get_device() == self.index
                and t.dtype is (dtype or self.dtype) and t.shape == shape and t.is_contiguous()):
            self.tensor(t, shape, what, dtype, True)
        return t.data_ptr()

    def empty(self, shape, dtype=None):
        if self.own is None:
            return torch.empty(shape, dtype=dtype or self.dtype, device=self.device)
        with torch.cuda.stream(self.own):
            return torch.empty(shape, dtype=dtype or self.dtype, device=self.device)

    def out(self, t, shape, what, dtype=None):
        """A caller's output, checked, or a new one."""
        if t is None:
            return self.empty(shape, dtype)
        return self.tensor(t, shape, what, dtype, True)

    def workspace(self, ws, need):
        if ws is None:
            if need == 0:
                return None, 0, 0
            ws = self.empty((need,), torch.uint8)
        else:
            if not isinstance(ws, torch.Tensor) or ws.device != self.device:
                raise TypeError(f"workspace must be a torch tensor on {self.device}")
            if ws.dtype != torch.uint8 or not ws.is_contiguous():
                raise ValueError("workspace must be a contiguous uint8 tensor")
        return ws, ws.data_ptr(), ws.numel()

    def run(self, f, *args):
        if _device_now() == self.index:
            status = f(*args, self.ptr)
        else:
            with torch.cuda.device(self.device):
                status = f(*args, self.ptr)
        if status != 0:
            raise GspnError(status, _tok.gspn_last_error().decode())


def _shape3(x, what):
    if not isinstance(x, torch.Tensor) or x.dim() != 3:
        raise ValueError(f"{what} must be a [B, L, C] tensor")
    return tuple(x.shape)


# --------------------------------------------------------------------------
# causal convolution
# --------------------------------------------------------------------------
def _conv_args(c, x, weight, bias, state, lens, silu, out, state_out):
    B, L, C = x.shape
    if not isinstance(weight, torch.Tensor) or weight.dim() != 2:
        raise ValueError("weight must be a [C, K] tensor")
    K = weight.shape[1]
    xp, xb, xr = c.view(x, (B, L, C), "x")
    st = (B, max(K - 1, 0), C)
    return _CONV.pack(B, L, C, K, c.code, int(bool(silu)), xp, xb, xr,
                      c.data(weight, (C, K), "weight"), c.data(bias, (C,), "bias"),
                      c.data(state, st, "state"), c.data(lens, (B,), "lens", torch.int32),
                      0 if out is None else out.data_ptr(),
                      c.data(state_out, st, "state_out")), K


def causal_conv(x, weight, bias=None, state=None, lens=None, silu: bool = True, out=None,
                state_out=None, stream=None):
    """out[b, t, c] = act(bias[c] + sum_j weight[c, j] xx[b, t + j, c]) with
    xx = ``state`` (the K - 1 tokens before, [B, K-1, C]; zeros when None)
    followed by ``x`` [B, L, C], and act = silu, or none. ``weight`` [C, K],
    K <= 4; ``lens`` int32 [B]: tokens past an entry's length are padding
    (out = 0). ``state_out`` [B, K-1, C] (may be ``state`` itself) receives
    the K - 1 tokens before the next one; with L = 1 this is one step of a
    serving loop."""
    shape = _shape3(x, "x")
    c = _Call(x, "x", stream)
    out = c.out(out, shape, "out")
    args, _ = _conv_args(c, x, weight, bias, state, lens, silu, out, state_out)
    c.run(_lib().gspn_causal_conv, args)
    return out


def causal_conv_backward(x, weight, bias, grad_out, state=None, lens=None, silu: bool = True,
                         grads=None, workspace=None, stream=None, grad_state=None) -> dict:
    """Gradients of causal_conv() given ``grad_out`` = dL/dout [B, L, C] and
    optionally ``grad_state`` = dL/dstate_out [B, K-1, C], which the next chunk
    of a sequence hands back: a dict with "x", "weight", "bias" (when there is
    one) and "state" (when there is one), shaped and typed like the inputs
    (``grads`` may supply them)."""
    B, L, C = _shape3(x, "x")
    c = _Call(x, "x", stream)
    args, K = _conv_args(c, x, weight, bias, state, lens, silu, None, None)
    shapes = {"x": (B, L, C), "weight": (C, K)}
    if bias is not None:
        shapes["bias"] = (C,)
    if state is not None:
        shapes["state"] = (B, K - 1, C)
    g = {k: c.out(None if grads is None else grads[k], s, f"grads[{k!r}]") for k, s in shapes.items()}
    packed = _CONV_GRADS.pack(*c.view(grad_out, (B, L, C), "grad_out"), g["x"].data_ptr(),
                              g["weight"].data_ptr(), *(g[k].data_ptr() if k in g else 0
                                                        for k in ("bias", "state")),
                              c.data(grad_state, (B, K - 1, C), "grad_state"))
    L_ = _lib()
    ws, wp, wn = c.workspace(workspace, L_.gspn_causal_conv_backward_workspace_bytes(B, L, C, K, c.code))
    c.run(L_.gspn_causal_conv_backward_ws, args, packed, wp, wn)
    return g


# --------------------------------------------------------------------------
# selective scan
# --------------------------------------------------------------------------
def _scan_sizes(x, A, Bm):
    B, L, C = _shape3(x, "x")
    if not isinstance(A, torch.Tensor) or A.dim() != 2:
        raise ValueError("A must be a [C, N] tensor")
    if not isinstance(Bm, torch.Tensor) or Bm.dim() not in (3, 4):
        raise ValueError("B and C must be [B, L, G, N] (or [B, L, N]) tensors")
    return B, L, C, A.shape[1], Bm.shape[2] if Bm.dim() == 4 else 1


def _scan_args(c, sizes, x, dt, A, Bm, Cm, D, z, dt_bias, state, lens, softplus, out, state_out, saved):
    B, L, C, N, G = sizes
    f32, rows = torch.float32, (B, L, C)
    if Bm.dim() == 3:
        Bm, Cm = Bm.unsqueeze(2), (Cm.unsqueeze(2) if isinstance(Cm, torch.Tensor) and Cm.dim() == 3 else Cm)
    if saved is not None:
        need = _lib().gspn_selective_scan_saved_bytes(B, L, C, N)
        c.tensor(saved, (need,), "saved", torch.uint8, True)
    return _SCAN.pack(
        B, L, C, N, G, c.code, int(bool(softplus)), *c.view(x, rows, "x"), *c.view(dt, rows, "dt"),
        *((0, 0, 0) if z is None else c.view(z, rows, "z")), c.data(A, (C, N), "A", f32),
        *c.view(Bm, (B, L, G, N), "B"), *c.view(Cm, (B, L, G, N), "C"), c.data(D, (C,), "D", f32),
        c.data(dt_bias, (C,), "dt_bias", f32), c.data(state, (B, C, N), "state", f32),
        c.data(lens, (B,), "lens", torch.int32), 0 if out is None else out.data_ptr(),
        c.data(state_out, (B, C, N), "state_out", f32), 0 if saved is None else saved.data_ptr())


def selective_scan_saved(x, dt, A, Bm, Cm, stream=None):
    """An uninitialised buffer for selective_scan()'s ``saved``."""
    B, L, C, N, _ = _scan_sizes(x, A, Bm)
    need = _lib().gspn_selective_scan_saved_bytes(B, L, C, N)
    return _Call(x, "x", stream).empty((need,), torch.uint8)


def selective_scan(x, dt, A, Bm, Cm, D=None, z=None, dt_bias=None, state=None, lens=None,
                   softplus: bool = True, out=None, state_out=None, saved=None, workspace=None,
                   stream=None):
    """The selective scan, per channel with N <= 32 states:
        d_t = softplus(dt_t + dt_bias),  h_t = exp(d_t A) h_{t-1} + d_t x_t B_t,
        out_t = (C_t . h_t + D x_t) * silu(z_t).
    ``x``, ``dt``, ``z`` [B, L, C]; ``Bm``, ``Cm`` [B, L, G, N] or [B, L, N]
    (channel c reads group c // (C / G)) in x's dtype; ``A`` [C, N], ``D``,
    ``dt_bias`` [C], ``state`` and ``state_out`` [B, C, N] in float32.
    ``lens`` int32 [B]: tokens past an entry's length are padding (out = 0,
    the state stays). ``state_out`` may be ``state`` itself: with L = 1 that
    is one step of a serving loop. ``saved`` (selective_scan_saved()) keeps
    what the backward pass of the same arguments needs."""
    sizes = _scan_sizes(x, A, Bm)
    c = _Call(x, "x", stream)
    out = c.out(out, sizes[:3], "out")
    args = _scan_args(c, sizes, x, dt, A, Bm, Cm, D, z, dt_bias, state, lens, softplus, out,
                      state_out, saved)
    L_ = _lib()
    ws, wp, wn = c.workspace(workspace, L_.gspn_selective_scan_workspace_bytes(*sizes, c.code))
    c.run(L_.gspn_selective_scan_ws, args, wp, wn)
    return out


def selective_scan_backward(x, dt, A, Bm, Cm, grad_out, D=None, z=None, dt_bias=None, state=None,
                            lens=None, softplus: bool = True, grad_state=None, saved=None,
                            grads=None, workspace=None, stream=None) -> dict:
    """Gradients of selective_scan() given ``grad_out`` = dL/dout [B, L, C]
    and optionally ``grad_state`` = dL/dstate_out: a dict with "x", "dt", "A",
    "B", "C", and, for the inputs given, "D", "z", "dt_bias", "state", shaped
    and typed like the inputs (``grads`` may supply them). ``saved`` is what
    the forward call of the same arguments kept; without it the states are
    found again."""
    sizes = _scan_sizes(x, A, Bm)
    B, L, C, N, G = sizes
    c = _Call(x, "x", stream)
    args = _scan_args(c, sizes, x, dt, A, Bm, Cm, D, z, dt_bias, state, lens, softplus, None, None, saved)
    f32, bc = torch.float32, tuple(Bm.shape)
    want = {"x": ((B, L, C), None), "dt": ((B, L, C), None), "A": ((C, N), f32), "B": (bc, None),
            "C": (bc, None)}
    if z is not None:
        want["z"] = ((B, L, C), None)
    for k, t, s in (("D", D, (C,)), ("dt_bias", dt_bias, (C,)), ("state", state, (B, C, N))):
        if t is not None:
            want[k] = (s, f32)
    g = {k: c.out(None if grads is None else grads[k], s, f"grads[{k!r}]", d)
         for k, (s, d) in want.items()}
    packed = _SCAN_GRADS.pack(*c.view(grad_out, (B, L, C), "grad_out"),
                              c.data(grad_state, (B, C, N), "grad_state", f32),
                              *(g[k].data_ptr() if k in g else 0 for k in (
                                  "x", "dt", "z", "B", "C", "A", "D", "dt_bias", "state")))
    L_ = _lib()
    ws, wp, wn = c.workspace(workspace, L_.gspn_selective_scan_backward_workspace_bytes(*sizes, c.code))
    c.run(L_.gspn_selective_scan_backward_ws, args, packed, wp, wn)
    return g


# --------------------------------------------------------------------------
# cross attention
# --------------------------------------------------------------------------
def _attn_args(c, q, k, v, mask, scale, out, lse):
    for t, what in ((q, "q"), (k, "k"), (v, "v")):
        if not isinstance(t, torch.Tensor) or t.dim() != 4:
            raise ValueError(f"{what} must be a [B, L, H, E] tensor")
    B, Lq, Hq, E = q.shape
    Lk, Hkv = k.shape[1], k.shape[2]
    if scale is None:
        scale = E ** -0.5 if E > 0 else 1.0
    mp, mb = 0, 0
    if mask is not None:
        c.tensor(mask, (B, Lk), "mask", torch.bool)
        if mask.stride(1) != 1 and Lk > 1:
            raise ValueError("mask must be contiguous in its last dimension")
        mp, mb = mask.data_ptr(), mask.stride(0)
    sizes = (B, Lq, Lk, Hq, Hkv, E)
    return _ATTN.pack(*sizes, c.code, scale, *c.view(q, (B, Lq, Hq, E), "q"),
                      *c.view(k, (B, Lk, Hkv, E), "k"), *c.view(v, (B, Lk, Hkv, E), "v"), mp, mb,
                      out.data_ptr(), 0 if lse is None else lse.data_ptr()), sizes


def cross_attention(q, k, v, mask=None, scale=None, out=None, lse=None, workspace=None, stream=None):
    """Attention of ``q`` [B, Lq, Hq, E] to an encoder's states ``k``, ``v``
    [B, Lk, Hkv, E] (query head h reads key head h // (Hq / Hkv); E <= 128):
    out = softmax(scale q k^T) v over the keys that ``mask`` (bool [B, Lk],
    True = keep; None = all) keeps. Dropped keys take no part, whatever they
    hold; an entry that keeps none gives 0. ``scale`` defaults to E ** -0.5.
    ``lse`` (float32 [B, Hq, Lq]) receives the log of the softmax's sum, which
    the backward pass needs."""
    c = _Call(q, "q", stream)
    if q.dim() != 4:
        raise ValueError("q must be a [B, L, H, E] tensor")
    B, Lq, Hq, E = q.shape
    out = c.out(out, (B, Lq, Hq, E), "out")
    if lse is not None:
        c.tensor(lse, (B, Hq, Lq), "lse", torch.float32, True)
    args, sizes = _attn_args(c, q, k, v, mask, scale, out, lse)
    L_ = _lib()
    ws, wp, wn = c.workspace(workspace, L_.gspn_cross_attention_workspace_bytes(*sizes, c.code))
    c.run(L_.gspn_cross_attention_ws, args, wp, wn)
    return out


def cross_attention_backward(q, k, v, out, lse, grad_out, mask=None, scale=None, grads=None,
                             workspace=None, stream=None) -> dict:
    """Gradients of cross_attention() given its results ``out`` and ``lse``
    and ``grad_out`` = dL/dout: a dict with "q", "k", "v", contiguous, shaped
    and typed like the inputs (``grads`` may supply them)."""
    c = _Call(q, "q", stream)
    if q.dim() != 4:
        raise ValueError("q must be a [B, L, H, E] tensor")
    B, Lq, Hq, E = q.shape
    c.tensor(out, (B, Lq, Hq, E), "out", None, True)
    c.tensor(lse, (B, Hq, Lq), "lse", torch.float32, True)
    args, sizes = _attn_args(c, q, k, v, mask, scale, out, lse)
    g = {n: c.out(None if grads is None else grads[n], tuple(t.shape), f"grads[{n!r}]")
         for n, t in (("q", q), ("k", k), ("v", v))}
    packed = _ATTN_GRADS.pack(*c.view(grad_out, (B, Lq, Hq, E), "grad_out"),
                              *(g[n].data_ptr() for n in "qkv"))
    L_ = _lib()
    ws, wp, wn = c.workspace(workspace, L_.gspn_cross_attention_backward_workspace_bytes(*sizes, c.code))
    c.run(L_.gspn_cross_attention_backward_ws, args, packed, wp, wn)
    return g
