"""The token embedding and its gradient on the GPU against their plain 64-bit
forms, at the sizes, ids and lengths where they can go wrong. The lookup rounds
one product, twice (to 32 bits, to the storage type); a gradient's row of n
tokens takes n sums and a product: n + 1 roundings."""
from __future__ import annotations

import pytest
import torch

import linear_spatial_propagation_line_amd as g
import plain_prompt as plain

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
F32, BF16 = torch.float32, torch.bfloat16
NAN = float("nan")


def rows_of(t, extra=5, offset=3):
    """The same values as an unaligned slice of longer rows."""
    wide = torch.full(t.shape[:-1] + (t.shape[-1] + extra,), NAN, dtype=t.dtype, device=t.device)
    wide[..., offset:offset + t.shape[-1]] = t
    return wide[..., offset:offset + t.shape[-1]]


CASES = [
    # B, L, V, D, dtype, ids, lens, scale
    (1, 1, 1, 1, F32, torch.int64, None, 1.0),
    (2, 1, 50, 64, BF16, torch.int32, None, 8.0),
    (3, 7, 5, 33, F32, torch.int64, (7, 0, 3), 0.37),          # odd rows; few rows, each with many tokens
    (4, 70, 300, 136, BF16, torch.int64, (70, 0, 1, 37), 11.6),
    (2, 500, 3, 24, F32, torch.int64, None, 1.0),              # long runs over many chunks
    (1, 33, 1, 16, BF16, torch.int64, None, 1.0),              # one row, one token past a chunk
    (1, 64, 1, 9, F32, torch.int32, None, -2.0),
    (2, 96, 70000, 8, F32, torch.int64, None, 1.0),            # most of the table without a token
    (5, 0, 20, 12, F32, torch.int64, None, 1.0),               # no tokens
    (0, 4, 20, 12, BF16, torch.int64, None, 1.0),
    (2, 9, 40, 520, BF16, torch.int64, (-3, 99), 1.0),         # lengths are clamped
    (2, 50, 60, 70, BF16, torch.int64, (50, 44), 3.0),         # rows of whole pairs
    (1, 40, 7, 131, BF16, torch.int32, None, 1.0),             # of none
]


def case(B, L, V, D, dtype, idt, lens, scale, seed=0):
    gen = torch.Generator().manual_seed(seed)
    ids = torch.randint(0, V, (B, L), generator=gen)
    if ids.numel() > 8:        # ids that are no row
        ids.view(-1)[1::7] = -1
        ids.view(-1)[5::11] = V
        if idt is torch.int64:
            ids.view(-1)[6::13] = (1 << 32) + 1
        ids.view(-1)[3::13] = -100
    w = torch.randn(V, D, generator=gen).to(dtype)
    gy = torch.randn(B, L, D, generator=gen).to(dtype)
    for b, n in enumerate(plain.lengths(lens, B, L)):
        gy[b, n:] = NAN
    return ids.to(idt), w, gy, None if lens is None else torch.tensor(lens, dtype=torch.int32)


@pytest.mark.parametrize("c", CASES)
@pytest.mark.parametrize("view", [False, True])
def test_embedding(c, view):
    ids, w, gy, lens = case(*c)
    V, scale = c[2], c[7]
    di = ids.to(DEV)
    if view:                    # a column of ids among others
        wide = torch.full((ids.shape[0], ids.shape[1] + 3), 1, dtype=ids.dtype, device=DEV)
        wide[:, 2:2 + ids.shape[1]] = di
        di = wide[:, 2:2 + ids.shape[1]]
    dl = None if lens is None else lens.to(DEV)
    out = g.token_embedding(di, w.to(DEV), scale=scale, lens=dl)
    ref = plain.embedding(ids, w, scale, lens)
    plain.within(out, ref, ref.abs(), 1, "out")
    gd = gy.to(DEV)
    got = g.token_embedding_backward(di, rows_of(gd) if view else gd, V, scale=scale, lens=dl)
    dw, size, count = plain.embedding_grad(ids, torch.nan_to_num(gy), V, scale, lens)
    plain.within(got["weight"], dw, size * (count + 1), 1, "weight")
    assert set(got) == {"weight"}


@pytest.mark.parametrize("idt", [torch.int32, torch.int64])
def test_gradient_of_many_tokens_is_exact_for_whole_numbers(idt):
    """30000 tokens over 3000 rows, one row in a third of them, in wavefronts'
    shares that end inside a batch: sums of small whole numbers have no
    rounding, so every token is counted once and in its row."""
    gen = torch.Generator().manual_seed(2)
    B, L, V, D = 3, 10007, 3001, 40
    ids = torch.randint(0, V, (B, L), generator=gen)
    ids[torch.rand(B, L, generator=gen) < 0.33] = 1234
    gy = torch.randint(-8, 9, (B, L, D), generator=gen).float()
    lens = torch.tensor([L, 9001, 77], dtype=torch.int32)
    ref = torch.zeros(V, D)
    for b in range(B):
        ref.index_add_(0, ids[b, :lens[b]], gy[b, :lens[b]])
    got = g.token_embedding_backward(ids.to(idt).to(DEV), gy.to(DEV), V, lens=lens.to(DEV))["weight"]
    assert torch.equal(got.cpu(), ref)


def test_large_table_of_many_ranges():
    """More rows than 256 ranges of 1024, the last range in part."""
    V, D, T = 300_001, 8, 5000
    gen = torch.Generator().manual_seed(3)
    ids = torch.randint(0, V, (1, T), generator=gen)
    ids[0, :3] = torch.tensor([0, V - 1, V - 2])
    gy = torch.randint(-8, 9, (1, T, D), generator=gen).to(BF16)
    ref = torch.zeros(V, D).index_add_(0, ids[0], gy[0].float())
    got = g.token_embedding_backward(ids.to(DEV), gy.to(DEV), V)["weight"]
    assert torch.equal(got.cpu().float(), ref)


def test_supplied_outputs_workspaces_and_streams():
    ids, w, gy, _ = case(4, 70, 300, 136, BF16, torch.int64, None, 1.0, seed=5)
    gy = torch.nan_to_num(gy)
    di, dw, dg = ids.to(DEV), w.to(DEV), gy.to(DEV)
    base = g.token_embedding(di, dw)
    base_g = g.token_embedding_backward(di, dg, 300)["weight"]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    out = torch.full_like(base, NAN)
    grads = {"weight": torch.full_like(dw, NAN)}
    ws = torch.full((1 << 20,), 255, dtype=torch.uint8, device=DEV)
    s.wait_stream(torch.cuda.current_stream())
    assert g.token_embedding(di, dw, out=out, stream=s) is out
    got = g.token_embedding_backward(di, dg, 300, grads=grads, workspace=ws, stream=s)
    assert got["weight"] is grads["weight"]
    s.synchronize()
    assert torch.equal(out, base) and torch.equal(got["weight"], base_g)


def test_captured_and_replayed():
    """A graph replayed on new ids, other work between the replays."""
    ids, w, gy, _ = case(4, 70, 300, 136, F32, torch.int64, None, 1.0, seed=6)
    gy = torch.nan_to_num(gy).to(DEV)
    di, dw = ids.to(DEV), w.to(DEV)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        g.token_embedding(di, dw)
        g.token_embedding_backward(di, gy, 300)
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = g.token_embedding(di, dw)
        grad = g.token_embedding_backward(di, gy, 300)["weight"]
    gen = torch.Generator().manual_seed(8)
    for _ in range(3):
        di.copy_(torch.randint(-1, 301, di.shape, generator=gen))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, g.token_embedding(di, dw))
        assert torch.equal(grad, g.token_embedding_backward(di, gy, 300)["weight"])


def test_binding_refuses():
    ids = torch.zeros(2, 3, dtype=torch.int64, device=DEV)
    w = torch.zeros(4, 8, device=DEV)
    gy = torch.zeros(2, 3, 8, device=DEV)
    for bad in (lambda: g.token_embedding(ids.float(), w), lambda: g.token_embedding(ids[0], w),
                lambda: g.token_embedding(ids, w[:, ::2]), lambda: g.token_embedding(ids, w[0]),
                lambda: g.token_embedding(ids.t(), w),
                lambda: g.token_embedding(ids, w, lens=torch.ones(2, device=DEV)),
                lambda: g.token_embedding(ids, w, out=torch.empty(2, 3, 7, device=DEV)),
                lambda: g.token_embedding_backward(ids, gy[:, :2], 4),
                lambda: g.token_embedding_backward(ids, gy.transpose(0, 2), 4)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(TypeError):
        g.token_embedding(ids.cpu(), w)
    for bad in (lambda: g.token_embedding(ids, w, scale=float("inf")),
                lambda: g.token_embedding_backward(ids, gy, 0)):
        with pytest.raises(g.GspnError) as e:
            bad()
        assert e.value.name == "GSPN_E_SHAPE"


@pytest.mark.parametrize("T,V", [(8192, 900), (8193, 70), (16384, 5000), (16385, 2), (40000, 300_000)])
def test_sorts_of_every_size(T, V):
    """One turn of the sort, the first token past it, two parts, the first past
    them, more than one turn a part: every token once and in its row (whole
    numbers), and the same bits whatever the ids' type."""
    gen = torch.Generator().manual_seed(T)
    ids = (torch.rand(1, T, generator=gen) ** 3 * V).long().clamp(max=V - 1)
    ids[0, 5::9] = -1
    whole = torch.randint(-8, 9, (1, T, 4), generator=gen).float()
    ref = torch.zeros(V + 1, 4).index_add_(0, ids[0].where(ids[0] >= 0, torch.tensor(V)), whole[0])[:V]
    assert torch.equal(g.token_embedding_backward(ids.to(DEV), whole.to(DEV), V)["weight"].cpu(), ref)
    gy = torch.randn(1, T, 4, generator=gen).to(DEV)
    a = g.token_embedding_backward(ids.to(DEV), gy, V)["weight"]
    assert torch.equal(a, g.token_embedding_backward(ids.int().to(DEV), gy, V)["weight"])
    dw, size, count = torch.zeros(3, V, 4, dtype=torch.float64)
    on = ids[0] >= 0
    dw.index_add_(0, ids[0][on], gy[0].cpu().double()[on])
    size.index_add_(0, ids[0][on], gy[0].cpu().double().abs()[on])
    count.index_add_(0, ids[0][on], torch.ones(int(on.sum()), 4, dtype=torch.float64))
    plain.within(a, dw, size * (count + 1), 1, "weight")


def test_offsets_past_32_bits():
    """A table, tokens and a gradient of more than 2^31 values each. One row of whole
    numbers as every token's gradient: a table row's is that row times its tokens, at
    most 4 x 64, which bf16 holds."""
    V = T = 950_000
    D = 2304
    gen = torch.Generator(device=DEV).manual_seed(8)
    w = torch.empty(V, D, dtype=BF16, device=DEV).normal_(generator=gen)
    ids = torch.randint(0, V, (1, T), generator=gen, device=DEV)
    ids[0, -3:] = torch.tensor([V - 1, 0, V - 1], device=DEV)
    out = g.token_embedding(ids, w)
    for t in (slice(0, 2000), slice(T // 2, T // 2 + 2000), slice(T - 2000, T)):
        assert torch.equal(out[0, t], w[ids[0, t]])
    row = torch.randint(-4, 5, (1, 1, D), generator=gen, device=DEV).to(BF16)
    count = torch.bincount(ids[0], minlength=V)
    assert int(count.max()) <= 64
    got = g.token_embedding_backward(ids, row.expand(1, T, D), V)["weight"]
    for v in range(0, V, 50_000):
        assert torch.equal(got[v:v + 50_000].float(), count[v:v + 50_000, None] * row[0].float())
