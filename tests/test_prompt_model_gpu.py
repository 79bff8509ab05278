"""The token embedding, the gated recurrence and the vocabulary loss as a prompt
model uses them: every gradient through the three against the same model in 64
bits, the table's being the sum of its two uses; the example's run, and the same
hidden states token by token.

Everything is fp32. An operator's result is off by some 10 roundings (2^-24 each)
of the sizes its sums have, a product's over at most 96 values by 96 at the
most and by their root, 10, as rounding goes; eight operators and products lie
between the table and the loss and eight back, so a gradient is off by at most
16 x 20 x 2^-24 = 2e-5 of its own size where sums do not cancel: 2e-4 leaves them
a factor of ten for cancelling."""
from __future__ import annotations

import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                    "prompt_language_model.py")


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("prompt_language_model", PATH)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def plain_loss(m, p, ids, targets, lens):
    """The model's summed loss in 64 bits, from parameters p, sequence by sequence."""
    total = 0
    for b in range(ids.shape[0]):
        n = int(lens[b])
        if n == 0:
            continue
        tokens = p["table"][ids[b, :n]] * m.scale
        x, r, i = (tokens @ p["w_in.weight"].T).chunk(3, -1)
        log_a = -torch.nn.functional.softplus(p["decay"]) * torch.sigmoid(r)
        h, hs = torch.zeros(m.inner, dtype=torch.float64), []
        for t in range(n):
            h = torch.exp(log_a[t]) * h + torch.sqrt(-torch.expm1(2 * log_a[t])) * torch.sigmoid(i[t]) * x[t]
            hs.append(h)
        z = (tokens + torch.stack(hs) @ p["w_out.weight"].T) @ p["table"].T
        on = targets[b, :n] >= 0
        total = total + torch.nn.functional.cross_entropy(z[on], targets[b, :n][on], reduction="sum")
    return total


def test_gradients_through_all_three(example):
    torch.manual_seed(3)
    model = example.PromptModel(500, 64, 96, DEV)
    ids, targets, lens = example.batch(DEV)
    loss = model(ids, targets, lens)
    assert not loss[3].any() and not loss[1, 35:].any()
    loss.sum().backward()
    p = {n: q.detach().cpu().double().requires_grad_() for n, q in model.named_parameters()}
    ref = plain_loss(model, p, ids.cpu(), targets.cpu(), lens.cpu())
    assert abs(float(loss.detach().sum()) - float(ref.detach())) <= 2e-4 * float(ref.detach())
    for (n, q), r in zip(model.named_parameters(), torch.autograd.grad(ref, list(p.values()))):
        off = float((q.grad.cpu().double() - r).norm() / r.norm())
        assert off <= 2e-4, (n, off)


def test_example_runs(example):
    r = example.main(steps=3)
    assert len(r["losses"]) == 3 and all(x == x and abs(x) < 1e3 for x in r["losses"])
    # the two ways differ by the roundings of products and of at most 70 steps of a decay
    assert r["token_by_token_gap"] <= 1e-5
