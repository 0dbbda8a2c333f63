"""The embedding whose rows are dealt out to the ranks (Comm.embedding and its
gradient) on the GPU against the formulas in 64 bits.

Bounds: the lookup is one product, rounded to 32 bits and then to its type.
The gradient of an id with m tokens adds them one after another in chunks of
8 to 64 and then the chunks (in calls of up to 1024 tokens all of them, or
quarters of them and then these): below m + 2 additions, one product with
scale and one addition where it accumulates: m + 4 roundings.
"""
import pytest
import torch

import allreduce_reduction_amd as hc
import rankops_ref as ref

pytestmark = pytest.mark.gpu

TYPES = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16}


def make_ids(n, vocab, seed, kind="skew", dtype=torch.int64):
    g = torch.Generator().manual_seed(seed)
    if kind == "skew":  # a few ids are frequent
        ids = torch.exp(torch.rand(n, generator=g).double() * torch.log(torch.tensor(vocab + 1.0).double())).long() - 1
    elif kind == "one":
        ids = torch.full((n,), vocab - 1)
    elif kind == "none":
        ids = torch.full((n,), -1)
    elif kind == "runs":  # runs of 31 to 33 tokens: ends on both sides of chunks
        ids = torch.arange(n) // (31 + torch.arange(n) // 200 % 3) % vocab
        ids = ids[torch.randperm(n, generator=g)]
    else:
        ids = torch.randint(0, vocab, (n,), generator=g)
    ids = ids.clamp(-1, vocab - 1)
    if kind in ("skew", "even") and n > 3:
        ids[torch.rand(n, generator=g) < 0.05] = -1
        ids[n // 2] = vocab
        ids[n // 3] = -(2 ** 31)
    return ids.to(dtype)


def lookup(P, counts, vocab, H, dtype, id_dtype=torch.int64, scale=3.0, shift=0, kind="skew"):
    g = torch.Generator().manual_seed(H)
    table = torch.randn(vocab, H, generator=g).to(TYPES[dtype])
    ids = make_ids(sum(counts), vocab, 3, kind, id_dtype)
    flat = [torch.empty(x.numel() + shift, dtype=x.dtype, device="cuda")[shift:].copy_(x.reshape(-1)).view(x.shape)
            for x in ref.split_rows(table, P)]
    out = [torch.full((n, H), 7.0, dtype=table.dtype, device="cuda") for n in counts]
    with hc.Comm(P, "ring") as comm:
        comm.embedding(flat, [t.cuda() for t in ids.split(counts)], out, scale=scale)
    ref.check(torch.cat(out), ref.embed_forward(table, ids, scale), 1, "rows")


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("P,counts,vocab,H", [
    (8, [1] * 8, 1000, 4096), (4, [3, 0, 700, 1], 333, 1001), (1, [17], 5, 1), (3, [5, 5, 5], 2, 7), (64, [2] * 64, 50, 65),
    (2, [100, 33], 70000, 136), (16, [9] * 16, 40, 16384), (5, [0, 0, 1, 0, 0], 7, 2500), (2, [40, 2], 90, 20003),
])
def test_lookup(P, counts, vocab, H, dtype):
    lookup(P, counts, vocab, H, dtype)


@pytest.mark.parametrize("id_dtype", [torch.int32, torch.int64])
@pytest.mark.parametrize("shift", [0, 1])
def test_lookup_ids_and_alignment(id_dtype, shift):
    lookup(3, [50, 60, 70], 999, 264, "bf16", id_dtype, -0.3, shift, "even")


def test_lookup_past_the_cache():
    """96 MiB of rows and more are stored past the caches."""
    lookup(3, [9000, 1, 8000], 5000, 2997, "bf16", shift=1)


def test_lookup_nothing():
    lookup(3, [0, 0, 0], 10, 16, "bf16")


def test_shared_ids():
    """All ranks may look up the same tokens, from one buffer."""
    table = torch.randn(100, 72).bfloat16()
    ids = make_ids(40, 100, 1).cuda()
    out = torch.empty(4, 40, 72, dtype=torch.bfloat16, device="cuda")
    with hc.Comm(4, "ring") as comm:
        comm.embedding(table.cuda().view(4, 25, 72), [ids] * 4, out)
    for p in range(4):
        assert torch.equal(out[p].cpu(), torch.where((ids.cpu() >= 0)[:, None] & (ids.cpu() < 100)[:, None],
                                                     table[ids.cpu().clamp(0, 99)], 0))


def gradient(P, counts, vocab, H, dtype, gdtype, accumulate, kind="skew", id_dtype=torch.int64, scale=0.5, shift=0):
    g = torch.Generator().manual_seed(vocab)
    N = sum(counts)
    ids = make_ids(N, vocab, 11, kind, id_dtype)
    grads = torch.randn(N, H, generator=g).to(TYPES[dtype])
    base = torch.randn(vocab, H, generator=g).to(TYPES[gdtype]) if accumulate else None
    start = torch.full((vocab, H), 7.0).to(TYPES[gdtype]) if base is None else base
    with hc.Comm(P, "ring") as comm:
        results = []
        for _ in range(2):
            flat = [torch.empty(x.numel() + shift, dtype=x.dtype, device="cuda")[shift:].copy_(x.reshape(-1)).view(x.shape)
                    for x in ref.split_rows(start, P)]
            comm.embedding_grad([t.cuda() for t in grads.split(counts)], [t.cuda() for t in ids.split(counts)], flat,
                                scale=scale, accumulate=accumulate)
            results.append(torch.cat(flat))
    assert torch.equal(results[0].view(torch.uint8), results[1].view(torch.uint8))
    inside = ids[(ids >= 0) & (ids < vocab)]
    most = int(torch.bincount(inside.long()).max()) if inside.numel() else 0
    ref.check(results[0], ref.embed_backward(grads, ids, vocab, scale, base), most + 4, "table")
    if accumulate:
        rest = torch.ones(vocab, dtype=torch.bool).index_fill_(0, inside.long(), False)
        assert torch.equal(results[0].cpu()[rest], base[rest])


@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("dtype,gdtype", [("bf16", "fp32"), ("bf16", "bf16"), ("fp16", "fp16"), ("fp16", "fp32"), ("fp32", "fp32")])
@pytest.mark.parametrize("P,counts,vocab,H", [
    (4, [1, 0, 0, 0], 100, 64), (3, [20, 0, 300], 77, 1001), (2, [500, 600], 3000, 136), (1, [9], 3, 3), (5, [7] * 5, 4, 520),
    (64, [1] * 64, 1025, 40),
])
def test_gradient(P, counts, vocab, H, dtype, gdtype, accumulate):
    gradient(P, counts, vocab, H, dtype, gdtype, accumulate)


@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("kind", ["skew", "one", "none", "runs", "even"])
@pytest.mark.parametrize("N,vocab,H", [(15, 900, 24), (1024, 1024, 24), (1025, 50001, 24), (8192, 1, 16), (8193, 70000, 16),
                                       (40000, 2_000_000, 8), (70001, 1000, 16), (33000, 1048576, 9), (540_001, 5000, 8)])
def test_sorting(N, vocab, H, kind, accumulate):
    """One to three digits, one to 64 sorting workgroups, ids that fill whole
    chunks, cross them, and do not occur at all."""
    counts = [N // 3, N // 2, N - N // 3 - N // 2]
    gradient(3, counts, vocab, H, "bf16", "fp32", accumulate, kind, torch.int32)


@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("kind", ["skew", "one", "none", "runs", "even"])
@pytest.mark.parametrize("N,vocab,H", [(1, 1, 1), (2, 3, 600), (9, 1, 520), (63, 20, 24), (64, 1000, 7), (65, 65, 1001), (255, 9, 2050),
                                       (256, 70000, 4), (257, 3, 4099), (512, 300, 24), (513, 31, 6000), (768, 40, 2048), (1024, 77, 2600),
                                       (1024, 30000, 64), (3000, 500, 136)])
def test_few_tokens(N, vocab, H, kind, accumulate):
    """Up to 1024 tokens take one launch without sorting: one, two and four
    tokens a lane, one piece of a row a workgroup and four, ids of one wave and
    of all four."""
    counts = [N // 4, 0, N - N // 4 - N // 8, N // 8, 0]
    gradient(5, counts, vocab, H, "bf16", "fp32", accumulate, kind, torch.int32)
    gradient(5, counts, vocab, H, "fp16", "fp16", accumulate, kind, scale=-1.5, shift=1)


@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("H", [1048576, 1048577])
def test_few_wide_rows(H, accumulate):
    """Rows of up to 4096 pieces are added without sorting, wider ones with."""
    gradient(2, [2, 1], 3, H, "fp32", "fp32", accumulate, "even")


def test_gradient_alignment():
    gradient(3, [100, 90, 80], 211, 72, "bf16", "bf16", True, "runs", shift=1)
    gradient(3, [100, 90, 80], 211, 72, "bf16", "fp32", False, "runs", shift=1)


@pytest.mark.parametrize("accumulate", [False, True])
def test_gradient_without_tokens(accumulate):
    gradient(3, [0, 0, 0], 1000, 40, "bf16", "fp32", accumulate)


def test_gradient_is_the_lookups():
    """sum(weights * lookup(table)) moves along a direction as the gradient
    says: the lookup is linear, so the difference over any step is exact but
    for fp32 rounding: 2 + 1 roundings a term here and m + 4 there."""
    g = torch.Generator().manual_seed(0)
    vocab, H, counts = 50, 40, [30, 41]
    table, way = torch.randn(vocab, H, generator=g), torch.randn(vocab, H, generator=g)
    ids, w = make_ids(71, vocab, 2), torch.randn(71, H, generator=g)
    with hc.Comm(2, "ring") as comm:
        def loss(t):
            out = [torch.empty(n, H, device="cuda") for n in counts]
            comm.embedding([x.cuda() for x in ref.split_rows(t, 2)], [x.cuda() for x in ids.split(counts)], out, scale=1.5)
            return (torch.cat(out).double().cpu() * w.double()).sum()
        grad = [torch.empty(25, H, device="cuda") for _ in range(2)]
        comm.embedding_grad([x.cuda() for x in w.split(counts)], [x.cuda() for x in ids.split(counts)], grad, scale=1.5)
        along = (torch.cat(grad).double().cpu() * way.double()).sum()
        diff = loss(table + way) - loss(table)
    size = (w.double().abs().sum() * 1.5 * (table.abs() + way.abs()).max()).item()
    assert abs((diff - along).item()) <= 80 * 2.0 ** -24 * size
