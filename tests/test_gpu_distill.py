"""Distillation from a teacher's top logits (Comm.distill_loss and its
gradient) on the GPU against the formulas in 64 bits.

Bounds, in roundings to 32 bits of the magnitudes that rankops_ref gives
(which hold the size of logits / temperature and of the log-sum-exp, each
rounded once before their differences are raised):
- the log-sum-exp: exponentials of rounded arguments (2 roundings of the
  argument, 2 units of the hardware's exponential), sums of 64 terms a lane,
  6 steps a wave and the pieces' sums; in the logarithm these relative errors
  are absolute ones: 2 + 2 + 64 + 6 + 22 below 100, scaled by 1 <= |lse| + max
  |z| in every test here;
- the loss adds K <= 1024 terms by 64 lanes (16 + 6) with some 10 products: 140;
- the gradient: 4 for the argument, 2 for the exponential, 30 for q: below 40.
"""
import pytest
import torch

import allreduce_reduction_amd as hc
import rankops_ref as ref

pytestmark = pytest.mark.gpu

TYPES = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16}


def case(n, vocab, k, dtype, tdtype="fp32", seed=0):
    g = torch.Generator().manual_seed(seed * 31 + n * 7 + vocab + k)
    z = (3 * torch.randn(n, vocab, generator=g)).to(TYPES[dtype])
    ids = torch.stack([torch.randperm(vocab, generator=g)[:k] if k <= vocab else torch.randint(0, vocab, (k,), generator=g)
                       for _ in range(n)]) if n else torch.empty(0, k, dtype=torch.int64)
    t = (4 + 2 * torch.randn(n, k, generator=g)).to(TYPES[tdtype])
    return z, t, ids, torch.randn(n, generator=g)


def shards(z, P, shift=0):
    out = []
    for lo, hi in ref.segments(z.shape[1], P):
        x = z[:, lo:hi].contiguous()
        out.append(torch.empty(x.numel() + shift, dtype=x.dtype, device="cuda")[shift:].copy_(x.reshape(-1)).view(x.shape))
    return out


def run(z, t, ids, dl, P, tau=1.0, shift=0, lse_exact=False):
    n = z.shape[0]
    loss, lse = torch.full((n,), 7.0, device="cuda"), torch.full((n,), 7.0, device="cuda")
    with hc.Comm(P, "ring") as comm:
        parts = shards(z, P, shift)
        comm.distill_loss(parts, t.cuda(), ids.cuda(), loss, lse, temperature=tau)
        grads = [torch.full_like(x, 7.0) for x in parts]
        given = lse
        comm.distill_loss_grad(parts, t.cuda(), ids.cuda(), given, dl.cuda(), grads, temperature=tau)
        inplace = [x.clone() for x in parts]
        comm.distill_loss_grad(inplace, t.cuda(), ids.cuda(), given, dl.cuda(), inplace, temperature=tau)
        for a, b in zip(grads, inplace):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    return loss, lse, torch.cat(grads, 1)


def check(z, t, ids, dl, P, tau=1.0, shift=0):
    loss, lse, grads = run(z, t, ids, dl, P, tau, shift)
    want = ref.distill_forward(z, t, ids, tau)
    ref.check(lse, want["lse"], 100, "lse")
    ref.check(loss, want["loss"], 140, "loss")
    ref.check(grads, ref.distill_backward(z, t, ids, tau, dl, lse.cpu()), 40, "grads")


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("P,n,vocab,k", [
    (8, 1, 32768, 64), (4, 7, 50001, 20), (1, 3, 1, 1), (3, 5, 2, 2), (5, 33, 1003, 64), (16, 2, 100, 100), (2, 2, 8192, 1024),
    (1, 4, 4096, 65), (1, 4, 4097, 1), (1, 2, 20000, 1000), (64, 3, 640, 8), (7, 129, 333, 3), (2, 3, 16, 40),
    # pieces and their joining in two launches: many rows, or long ones
    (5, 600, 1003, 64), (3, 513, 9001, 300), (1, 600, 4097, 7), (64, 513, 100, 2), (2, 3, 140001, 1000), (3, 1, 270000, 260),
])
def test_shapes(P, n, vocab, k, dtype):
    check(*case(n, vocab, k, dtype), P, 2.0 if k > 1 else 1.0)


@pytest.mark.parametrize("tdtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("id_dtype", [torch.int32, torch.int64])
@pytest.mark.parametrize("tau", [0.5, 1.0, 7.0])
def test_teacher_types(tdtype, id_dtype, tau):
    z, t, ids, dl = case(10, 5000, 31, "bf16", tdtype)
    check(z, t, ids.to(id_dtype), dl, 3, tau, shift=1)


def test_past_the_cache():
    """Logits of 96 MiB and more are read and their gradients stored past the caches."""
    check(*case(260, 200001, 130, "bf16"), 3, 2.0)


def test_no_rows():
    run(*case(0, 100, 4, "bf16"), 3)


@pytest.mark.parametrize("rows", [12, 600])
def test_masks(rows):
    """Entries that do not count, rows in which none does, padding rows whose
    logits hold anything, masked logits, the same column twice."""
    z, t, ids, dl = case(rows, 9000, 16, "bf16", seed=4)
    ids[0, 3:] = -1
    ids[1] = -1
    ids[2, 5], ids[2, 6] = 9000, 2 ** 40
    t[3, :] = -torch.inf
    t[4, 1:] = -torch.inf
    ids[5, 8:] = ids[5, :8]
    ids[6] = ids[6, 0]
    z[7, :4000] = -torch.inf
    ids[7] = torch.arange(16) + 8000
    ids[8, :8] = -(2 ** 63)
    z[9] = torch.finfo(torch.bfloat16).min  # masked by the type's lowest value
    z[9, ids[9]] = 1.0
    z[11] = torch.finfo(torch.bfloat16).min  # in every column
    check(z, t, ids, dl, 4, 1.5)
    check(z, t, ids, dl, 4, 1.0)
    loss, lse, grads = run(z, t, ids, dl, 4)
    assert torch.isfinite(loss).all() and torch.isfinite(lse).all() and torch.isfinite(grads).all()
    dl[10] = 0
    z[10] = float("nan")
    ids[1] = -1
    z[1] = float("nan")
    loss, lse, grads = run(z, t, ids, dl, 4, 1.5)
    assert not grads[10].any() and not grads[1].any() and not grads[3].any() and loss[1] == 0 and loss[3] == 0
    assert torch.isnan(loss[10]) and not torch.isnan(loss[:10]).any() and torch.isnan(lse[10])
    assert not torch.isnan(grads).any()


@pytest.mark.parametrize("rows", [3, 513])
def test_nothing_left(rows):
    """A masked teacher column: infinite loss, and a gradient without NaN; a
    row of -infinity alone has no distribution and p counts as zero."""
    z, t, ids, dl = case(rows, 600, 8, "fp32", seed=2)
    z[0, ids[0, 2]] = -torch.inf
    z[1] = -torch.inf
    loss, lse, grads = run(z, t, ids, dl, 3)
    assert loss[0] == torch.inf and loss[1] == torch.inf and torch.isfinite(loss[2])
    assert lse[1] == -torch.inf
    ref.check(grads, ref.distill_backward(z, t, ids, 1.0, dl, lse.cpu()), 40, "grads")


@pytest.mark.parametrize("rows", [2, 520])
def test_large_values(rows):
    """Logits of the size of fp32's and fp16's ends do not overflow."""
    for dtype, big in (("fp16", 60000.0), ("fp32", 1e30)):
        z, t, ids, dl = case(rows, 3000, 5, dtype)
        z[0, 100], z[0, 200] = big, -big
        ids[0, 0] = 100
        loss, lse, grads = run(z, t, ids, dl, 2)
        assert torch.isfinite(loss).all() and torch.isfinite(lse).all() and torch.isfinite(grads).all()
        assert lse[0] == torch.tensor(big)


def test_gradient_against_differences():
    """Along random directions: fp32 gradients against central differences of
    the loss in 64 bits (step 1e-5: differences are off by 1e-10 of the third
    derivative and 2^-52 / step of the loss)."""
    z, t, ids, dl = case(4, 300, 12, "fp32", seed=9)
    _, _, grads = run(z, t, ids, dl, 3, 1.3)
    way = torch.randn(z.shape, generator=torch.Generator().manual_seed(1)).double()
    f = lambda x: (ref.distill_forward(x, t, ids, 1.3)["loss"][0] * dl.double()).sum()  # noqa: E731
    diff = (f(z.double() + 1e-5 * way) - f(z.double() - 1e-5 * way)) / 2e-5
    along = (grads.double().cpu() * way).sum()
    size = (grads.double().cpu() * way).abs().sum()
    assert abs((diff - along).item()) <= 1e-4 * size.item() + 1e-6


def check_far(z, t, ids, dl, P, tau):
    """Teacher rows of any size: q follows from differences to the row's
    largest counting entry, and one that is not zero lies within 104 / 1 of it
    (exp(-104) is below fp32's smallest number), so its roundings count 104 in
    the place of the entries' own size."""
    loss, lse, grads = run(z, t, ids, dl, P, tau)
    zz = z.double() / tau
    want_lse = torch.logsumexp(zz, 1)
    ref.check(lse, (want_lse, want_lse.abs() + zz.abs().max(1).values), 100, "lse")
    q, log_q, some = ref.teacher(t, ids, z.shape[1], tau)
    at = ids.long().clamp(0, z.shape[1] - 1)
    log_p = zz.gather(1, at) - want_lse[:, None]
    size = zz.abs().max(1).values + want_lse.abs()
    on = q > 1e-44
    terms = torch.where(on, q * (log_q - log_p), 0.0)
    mag = torch.where(on, q * (log_q.abs() + log_p.abs() + 104 + size[:, None]), 0.0)
    ref.check(loss, (tau * tau * terms.sum(1), tau * tau * mag.sum(1)), 140, "loss")
    p = (zz - lse.double().cpu()[:, None]).exp()
    by = (dl.double() * tau)[:, None]
    value = p.scatter_add(1, at, -q) * by * some[:, None]
    # p and q below fp32's normal range are multiples of 2^-149, each off by up
    # to 2^-150, before the product with `by` is rounded there once more
    small = 2 * 2.0 ** -150 / (40 * 2.0 ** -24)
    mag = (small + p * (1 + size[:, None]) + torch.zeros_like(p).scatter_add(1, at, q * 105)) * by.abs() * some[:, None]
    ref.check(grads, (value, mag), 40, "grads")


@pytest.mark.parametrize("tau", [0.25, 0.5, 1.0, 3.0])
@pytest.mark.parametrize("tdtype", ["bf16", "fp32", "fp16"])
@pytest.mark.parametrize("rows,k", [(12, 16), (12, 300), (600, 16)])
def test_teacher_rows_of_any_size(rows, k, tdtype, tau):
    """Entries masked by the type's lowest value count, alone in their row or
    beside others, and so do entries near its largest one; their quotients by
    a temperature below 1 lie past the type's range."""
    z, t, ids, dl = case(rows, 9000, k, "fp32", tdtype, seed=6)
    top, low = torch.finfo(TYPES[tdtype]).max, torch.finfo(TYPES[tdtype]).min
    t[0] = low
    t[1, 1:] = low
    t[2] = top
    t[3, :k // 2] = top
    t[4, 3] = 0.8 * top
    t[5] = low
    ids[5, 1:] = -1  # one counting entry
    t[6] = low
    ids[6] = ids[6, 0]  # one column
    t[7, ::2], t[7, 1::2] = low, -torch.inf
    t[8] = 0.9 * low
    t[8, k - 1] = low
    t[9] = top
    t[9, 0] = low
    check_far(z, t, ids, dl, 4, tau)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("rows", [4, 520])
def test_student_rows_past_the_range(rows, dtype):
    """Logits whose quotient by a temperature below 1 lies past fp32's range:
    the log-sum-exp is then an infinity (and p zero in the gradient), but the
    loss comes from differences.  8 entries, q known to 140 roundings of
    magnitudes below 16."""
    z, t, ids, dl = case(rows, 3000, 8, dtype, seed=3)
    info = torch.finfo(TYPES[dtype])
    z[0] = info.min  # uniform
    z[1, ids[1]] = info.max  # uniform over the teacher's columns
    tau = 0.5
    loss, lse, grads = run(z, t, ids, dl, 3, tau)
    q, log_q, _ = ref.teacher(t, ids, 3000, tau)
    entropy = (q * log_q).sum(1)
    for row, log_n in ((0, torch.tensor(3000.0).log()), (1, torch.tensor(8.0).log())):
        want = tau * tau * (entropy[row] + log_n)
        assert abs(loss[row].item() - want.item()) <= 140 * 2.0 ** -24 * 16, row
    assert lse[0] == -torch.inf and lse[1] == torch.inf and torch.isfinite(lse[2:]).all()
    assert torch.isfinite(loss).all() and not torch.isnan(grads).any()
    want = torch.zeros(2, 3000).double().scatter_add(1, ids[:2], -q[:2]) * (dl[:2].double() * tau)[:, None]
    mag = torch.zeros(2, 3000).double().scatter_add(1, ids[:2], 105 * q[:2]) * (dl[:2].double().abs() * tau)[:, None]
    ref.check(grads[:2], (want, mag), 40, "grads")


@pytest.mark.parametrize("tau", [0.7, 1.0, 1.3, 3.0])
@pytest.mark.parametrize("dtype,size", [("fp32", 1e4), ("fp32", 1e9), ("fp32", 1e30), ("bf16", 1e4), ("bf16", 1e30), ("fp16", 1e4)])
@pytest.mark.parametrize("rows,vocab", [(7, 300), (5, 20001), (600, 4097)])
def test_large_logits_at_any_temperature(rows, vocab, dtype, size, tau):
    """A column above the others by more than exp resolves has p = 1 and they
    have 0, whatever its quotient by the temperature rounds to: the gradient's
    rounding of it is the log-sum-exp's.  (The 64-bit value is taken from exact
    quotients, not from the 32-bit log-sum-exp.)"""
    z, t, ids, dl = case(rows, vocab, 6, dtype, seed=8)
    z = (z.double() / 20 * size).to(TYPES[dtype])  # below size
    best = torch.arange(rows) * 7919 % vocab
    z[torch.arange(rows), best] = 4 * size
    z[:, 5] = -size
    z[0, 5] = -torch.inf
    ids[1] = -1
    loss, lse, grads = run(z, t, ids, dl, 3, tau)
    want, _ = ref.distill_backward(z, t, ids, tau, dl)
    q, _, some = ref.teacher(t, ids, vocab, tau)
    p = torch.zeros(rows, vocab).double()
    p[torch.arange(rows), best] = 1.0
    by = (dl.double() * tau)[:, None] * some[:, None]
    at = ids.long().clamp(0, vocab - 1)
    ref.check(grads, (p.scatter_add(1, at, -q) * by, p.scatter_add(1, at, 105 * q) * by.abs()), 40, "grads")
    assert (want - p.scatter_add(1, at, -q) * by).abs().max() < 1e-12
    assert torch.isfinite(lse).all() and not torch.isnan(loss).any()
