"""A text-conditioned image block from the library's operators, trained for a
few steps, with its prompt encoder also run token by token.

    python examples/prompt_conditioned.py

The prompt is encoded by a state space block (causal convolution, selective
scan, gate); the image latent is mixed by the 2D propagation and then reads
the prompt's states by cross attention. Every mixing step is a call into
libgspn.so, forward and backward; projections are plain matrix products."""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import linear_spatial_propagation_line_amd as g  # noqa: E402


class Conv(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, w, b, lens):
        ctx.save_for_backward(x, w, b, lens)
        return g.causal_conv(x, w, b, lens=lens)

    @staticmethod
    def backward(ctx, gy):
        x, w, b, lens = ctx.saved_tensors
        d = g.causal_conv_backward(x, w, b, gy.contiguous(), lens=lens)
        return d["x"], d["weight"], d["bias"], None


class Scan(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, dt, A, B, C, D, z, dt_bias, lens):
        saved = g.selective_scan_saved(x, dt, A, B, C)
        out = g.selective_scan(x, dt, A, B, C, D=D, z=z, dt_bias=dt_bias, lens=lens, saved=saved)
        ctx.save_for_backward(x, dt, A, B, C, D, z, dt_bias, lens, saved)
        return out

    @staticmethod
    def backward(ctx, gy):
        x, dt, A, B, C, D, z, dt_bias, lens, saved = ctx.saved_tensors
        d = g.selective_scan_backward(x, dt, A, B, C, gy.contiguous(), D=D, z=z, dt_bias=dt_bias,
                                      lens=lens, saved=saved)
        return (*(d[k] for k in ("x", "dt", "A", "B", "C", "D", "z", "dt_bias")), None)


class Propagate(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, l0, l1, l2, lam, u):
        ctx.save_for_backward(x, l0, l1, l2, lam, u)
        return g.propagate(x, (l0, l1, l2), lam, u)

    @staticmethod
    def backward(ctx, gy):
        x, l0, l1, l2, lam, u = ctx.saved_tensors
        d = g.propagate_backward(x, (l0, l1, l2), lam, u, gy.contiguous())
        return tuple(d[k] for k in g.GRAD_NAMES)


class Attend(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, mask):
        B, Lq, H, _ = q.shape
        lse = torch.empty((B, H, Lq), dtype=torch.float32, device=q.device)
        out = g.cross_attention(q, k, v, mask=mask, lse=lse)
        ctx.save_for_backward(q, k, v, mask, out, lse)
        return out

    @staticmethod
    def backward(ctx, gy):
        q, k, v, mask, out, lse = ctx.saved_tensors
        d = g.cross_attention_backward(q, k, v, out, lse, gy.contiguous(), mask=mask)
        return d["q"], d["k"], d["v"], None


class PromptEncoder(torch.nn.Module):
    """A state space block over token embeddings."""

    def __init__(self, width, inner, states=16, taps=4):
        super().__init__()
        self.inner, self.states = inner, states
        self.w_in = torch.nn.Linear(width, 2 * inner, bias=False)
        self.conv_w = torch.nn.Parameter(torch.randn(inner, taps) * taps ** -0.5)
        self.conv_b = torch.nn.Parameter(torch.zeros(inner))
        self.w_sel = torch.nn.Linear(inner, inner + 2 * states, bias=False)
        self.A_log = torch.nn.Parameter(torch.arange(1, states + 1).float().log().repeat(inner, 1))
        self.D = torch.nn.Parameter(torch.ones(inner))
        self.dt_bias = torch.nn.Parameter(torch.full((inner,), -3.0))
        self.w_out = torch.nn.Linear(inner, width, bias=False)

    def split(self, t):
        return t.split((self.inner, self.states, self.states), -1)

    def forward(self, tokens, lens):
        x, z = self.w_in(tokens).chunk(2, -1)
        x = Conv.apply(x, self.conv_w, self.conv_b, lens)
        dt, B, C = self.split(self.w_sel(x))
        y = Scan.apply(x, dt, -self.A_log.exp(), B, C, self.D, z, self.dt_bias, lens)
        return tokens + self.w_out(y)

    @torch.no_grad()
    def state(self, batch):
        dev = self.D.device
        return (torch.zeros(batch, self.conv_w.shape[1] - 1, self.inner, device=dev),
                torch.zeros(batch, self.inner, self.states, device=dev))

    @torch.no_grad()
    def step(self, token, state):
        """One token [B, 1, width]; the state moves on in place."""
        window, h = state
        x, z = self.w_in(token).chunk(2, -1)
        x = g.causal_conv(x, self.conv_w.detach(), self.conv_b.detach(), state=window, state_out=window)
        dt, B, C = self.split(self.w_sel(x))
        y = g.selective_scan(x, dt, -self.A_log.exp(), B, C, D=self.D.detach(), z=z,
                             dt_bias=self.dt_bias.detach(), state=h, state_out=h)
        return token + self.w_out(y)


class ImageBlock(torch.nn.Module):
    """2D propagation of the latent, then cross attention to the prompt."""

    def __init__(self, channels, heads, width):
        super().__init__()
        self.heads = heads
        self.params = torch.nn.Conv2d(channels, 5 * channels, 1)
        self.w_q = torch.nn.Linear(channels, channels, bias=False)
        self.w_kv = torch.nn.Linear(width, 2 * channels, bias=False)
        self.w_o = torch.nn.Linear(channels, channels, bias=False)

    def forward(self, latent, prompt, mask):
        l0, l1, l2, lam, u = (t.contiguous() for t in self.params(latent).chunk(5, 1))
        latent = latent + Propagate.apply(latent, l0, l1, l2, lam, u)
        B, C, H, W = latent.shape
        rows = latent.flatten(2).transpose(1, 2)                    # [B, H W, C]
        q = self.w_q(rows).unflatten(-1, (self.heads, -1))
        k, v = self.w_kv(prompt).unflatten(-1, (2, self.heads, -1)).unbind(2)   # views of one projection
        rows = rows + self.w_o(Attend.apply(q, k, v, mask).flatten(2))
        return rows.transpose(1, 2).reshape(B, C, H, W)


def main(steps: int = 5, device: str = "cuda:0") -> dict:
    torch.manual_seed(0)
    B, L, width, channels, side = 3, 40, 96, 64, 32
    lens = torch.tensor([40, 17, 0], dtype=torch.int32, device=device)     # the last prompt is empty
    mask = torch.arange(L, device=device)[None] < lens[:, None]
    encoder, block = PromptEncoder(width, 2 * width).to(device), ImageBlock(channels, 4, width).to(device)
    tokens = torch.randn(B, L, width, device=device)
    latent, target = torch.randn(2, B, channels, side, side, device=device)
    opt = torch.optim.Adam([*encoder.parameters(), *block.parameters()], lr=3e-3)
    losses = []
    for _ in range(steps):
        opt.zero_grad()
        loss = (block(latent, encoder(tokens, lens), mask) - target).square().mean()
        loss.backward()
        opt.step()
        losses.append(float(loss.detach()))
    # the encoder again, one token at a time, as a serving loop runs it
    with torch.no_grad():
        whole = encoder(tokens, torch.full((B,), L, dtype=torch.int32, device=device))
    state = encoder.state(B)
    steps_out = torch.cat([encoder.step(tokens[:, t:t + 1].contiguous(), state) for t in range(L)], 1)
    gap = float((steps_out - whole).abs().max() / whole.abs().max())
    return {"losses": losses, "token_by_token_gap": gap}


if __name__ == "__main__":
    r = main()
    print("loss by step:", " ".join(f"{x:.4f}" for x in r["losses"]))
    print(f"whole prompt against token by token: {r['token_by_token_gap']:.1e}")
