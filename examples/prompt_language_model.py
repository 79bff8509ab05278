"""A prompt encoder trained on its own prompts: token ids to the loss of the next
token through the library's operators, then run token by token.

    python examples/prompt_language_model.py

Ids are looked up in a table (token embedding), mixed along the prompt by a
gated linear recurrence between two projections, and scored against the same
table (vocabulary loss), whose gradient is the sum of both uses. Projections are
plain matrix products."""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import linear_spatial_propagation_line_amd as g  # noqa: E402


class Embed(torch.autograd.Function):
    @staticmethod
    def forward(ctx, ids, table, scale, lens):
        ctx.save_for_backward(ids, lens)
        ctx.vocab, ctx.scale = table.shape[0], scale
        return g.token_embedding(ids, table, scale=scale, lens=lens)

    @staticmethod
    def backward(ctx, gy):
        ids, lens = ctx.saved_tensors
        d = g.token_embedding_backward(ids, gy.contiguous(), ctx.vocab, scale=ctx.scale, lens=lens)
        return None, d["weight"], None, None


class Recur(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, r, i, A, lens):
        saved = g.gated_recurrence_saved(x)
        out = g.gated_recurrence(x, r, i, A, lens=lens, saved=saved)
        ctx.save_for_backward(x, r, i, A, lens, saved)
        return out

    @staticmethod
    def backward(ctx, gy):
        x, r, i, A, lens, saved = ctx.saved_tensors
        d = g.gated_recurrence_backward(x, r, i, A, gy.contiguous(), lens=lens, saved=saved)
        return d["x"], d["r"], d["i"], d["A"], None


class Loss(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, table, targets, lens):
        lse = torch.empty(targets.shape, dtype=torch.float32, device=x.device)
        out = g.vocab_loss(x, table, targets, lens=lens, lse=lse)
        ctx.save_for_backward(x, table, targets, lse, lens)
        return out

    @staticmethod
    def backward(ctx, gl):
        x, table, targets, lse, lens = ctx.saved_tensors
        d = g.vocab_loss_backward(x, table, targets, lse, gl.contiguous(), lens=lens)
        return d["x"], d["weight"], None, None


class PromptModel(torch.nn.Module):
    def __init__(self, vocab, width, inner, device="cpu"):
        super().__init__()
        kw = dict(device=device)
        self.inner, self.scale = inner, width ** 0.5
        self.table = torch.nn.Parameter(torch.randn(vocab, width, **kw) * width ** -0.5)
        self.w_in = torch.nn.Linear(width, 3 * inner, bias=False, **kw)
        self.decay = torch.nn.Parameter(torch.rand(inner, **kw) * 2 - 2)
        self.w_out = torch.nn.Linear(inner, width, bias=False, **kw)

    def rate(self):
        return -torch.nn.functional.softplus(self.decay)

    def hidden(self, ids, lens):
        tokens = Embed.apply(ids, self.table, self.scale, lens)
        x, r, i = self.w_in(tokens).chunk(3, -1)          # views of one projection
        return tokens + self.w_out(Recur.apply(x, r, i, self.rate(), lens))

    def forward(self, ids, targets, lens):
        """Loss of every token's target, [B, L]."""
        return Loss.apply(self.hidden(ids, lens), self.table, targets, lens)

    @torch.no_grad()
    def step(self, ids, state):
        """Hidden states of one token per sequence [B, 1]; the state moves on in place."""
        table = self.table.detach()
        tokens = g.token_embedding(ids, table, scale=self.scale)
        x, r, i = self.w_in(tokens).chunk(3, -1)
        return tokens + self.w_out(g.gated_recurrence(x, r, i, self.rate(), state=state, state_out=state))


def batch(device, vocab=500, B=4, L=70):
    """Prompts of different lengths that count upwards from a first token, the
    last one empty; each token's target is the next one of its prompt."""
    gen = torch.Generator().manual_seed(1)
    first = torch.randint(0, vocab, (B, 1), generator=gen)
    ids = (first + torch.arange(L + 1)) % vocab
    lens = torch.tensor([L, L // 2, 3, 0], dtype=torch.int32)
    targets = ids[:, 1:].clone()
    targets[torch.arange(L)[None] == lens[:, None] - 1] = -100      # nothing follows a prompt's last token
    return ids[:, :-1].contiguous().to(device), targets.to(device), lens.to(device)


def main(steps: int = 5, device: str = "cuda:0") -> dict:
    torch.manual_seed(0)
    model = PromptModel(500, 64, 96, device)
    ids, targets, lens = batch(device)
    opt = torch.optim.Adam(model.parameters(), lr=1e-2)
    losses = []
    for _ in range(steps):
        opt.zero_grad()
        loss = model(ids, targets, lens).sum() / (targets >= 0).sum()
        loss.backward()
        opt.step()
        losses.append(float(loss.detach()))
    # a prompt's hidden states again, one token at a time
    with torch.no_grad():
        whole = model.hidden(ids, torch.full_like(lens, ids.shape[1]))
    state = torch.zeros(ids.shape[0], model.inner, device=device)
    steps_out = torch.cat([model.step(ids[:, t:t + 1].contiguous(), state) for t in range(ids.shape[1])], 1)
    gap = float((steps_out - whole).abs().max() / whole.abs().max())
    return {"losses": losses, "token_by_token_gap": gap}


if __name__ == "__main__":
    r = main()
    print("loss by step:", " ".join(f"{x:.4f}" for x in r["losses"]))
    print(f"whole prompt against token by token: {r['token_by_token_gap']:.1e}")
