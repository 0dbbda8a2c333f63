"""The norms at a block's end (Comm.reduce_norm and its gradient) on the GPU
against the formulas in 64 bits.

Bounds: `steps` roundings to 32 bits.  Forward: P - 1 for the ranks' sum, at
most 16 + 6 + 16 + 1 in each of the two row sums (a lane's terms, the wave, the
waves, the mean), counted once for the value and half for the square root of
each, and about 12 products: P + 16 + 39 + 12 < P + 80.  Gradient: two row sums
one inside the other and up to 30 products: P + 2 * 39 + 30 < P + 120; the
weights' gradients add the rows: at most 9 rows a chunk and eight slots, 256
chunks by 16 waves: 9 + 8 + 16 + 16 more, below 60.
"""
import pytest
import torch

import allreduce_reduction_amd as hc
import rankops_ref as ref

pytestmark = pytest.mark.gpu

TYPES = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16}


def case(P, T, H, dtype, post=True, gates=1, seed=0):
    g = torch.Generator().manual_seed(seed * 7919 + P * 1000003 + T * 101 + H)
    dt = TYPES[dtype]
    c = {"parts": (torch.randn(P, T, H, generator=g) / P ** 0.5).to(dt), "residual": (2 * torch.randn(T, H, generator=g)).to(dt),
         "pre": (1 + 0.2 * torch.randn(H, generator=g)).to(dt),
         "post": (1 + 0.2 * torch.randn(H, generator=g)).to(dt) if post else None,
         "gate": torch.randn(gates, H, generator=g).to(dt) if gates else None,
         "out_grads": (0.3 * torch.randn(P, T, H, generator=g)).to(dt), "residual_in": torch.randn(T, H, generator=g).to(dt)}
    c["gate_rows"] = max(1, T // gates) if gates else 1
    return c


def dev(x, shift=0):
    """On the GPU, `shift` elements past a 256-byte boundary."""
    if x is None:
        return None
    if shift == 0:
        return x.cuda()
    flat = torch.empty(x.numel() + shift, dtype=x.dtype, device="cuda")
    return flat[shift:].copy_(x.reshape(-1)).view(x.shape)


def forward(c, comm, scale=0.75, save=True, shift=0, **kw):
    P, T, H = c["parts"].shape
    res = [dev(x, shift) for x in ref.split_rows(c["residual"], P)]
    out = [torch.full((T, H), 7.0, dtype=x.dtype, device="cuda") for x in c["parts"]]
    res_out = [torch.full_like(x, 7.0) for x in res]
    sums = [torch.full_like(x, 7.0) for x in res] if save else None
    comm.reduce_norm([dev(x, shift) for x in c["parts"]], res, out, dev(c["pre"], shift), residual_out=res_out, sums=sums,
                     post_weight=dev(c["post"], shift), gate=dev(c["gate"], shift), scale=scale, **kw)
    return out, res_out, sums


def backward(c, comm, scale=0.75, has_in=True, shift=0, **kw):
    P, T, H = c["parts"].shape
    x = c["parts"].double().sum(0).to(c["parts"].dtype)
    hidden = [dev(t, shift) for t in ref.split_rows(c["residual"], P)]
    sums = [dev(t, shift) for t in ref.split_rows(x, P)] if c["post"] is not None or c["gate"] is not None else None
    res_in = [dev(t, shift) for t in ref.split_rows(c["residual_in"], P)] if has_in else None
    parts = [torch.full((T, H), 7.0, dtype=x.dtype, device="cuda") for _ in range(P)]
    res = [torch.full_like(t, 7.0) for t in hidden]
    wide = dict(dtype=torch.float32, device="cuda")
    pre = torch.full((H,), 7.0, **wide)
    post = torch.full((H,), 7.0, **wide) if c["post"] is not None else None
    gate = torch.full(c["gate"].shape, 7.0, **wide) if c["gate"] is not None else None
    comm.reduce_norm_grad([dev(t, shift) for t in c["out_grads"]], hidden, parts, res, dev(c["pre"], shift), pre, sums=sums,
                          residual_grad_in=res_in, post_weight=dev(c["post"], shift), post_weight_grad=post,
                          gate=dev(c["gate"], shift), gate_grad=gate, scale=scale, **kw)
    want = ref.norm_backward(c["out_grads"], c["residual"], c["pre"], x, c["residual_in"] if has_in else None, c["post"],
                             c["gate"], c["gate_rows"], scale, **kw)
    return {"parts": parts, "residual": res, "pre": pre, "post": post, "gate": gate}, want


def check_forward(got, c, scale=0.75, save=True, **kw):
    P = c["parts"].shape[0]
    want = ref.norm_forward(c["parts"], c["residual"], c["pre"], c["post"], c["gate"], c["gate_rows"], scale, **kw)
    out, res, sums = got
    for p in range(P):
        ref.check(out[p], want["out"], P + 80, f"out[{p}]")
        assert torch.equal(out[p], out[0])
    ref.check(torch.cat(res), want["residual"], P + 80, "residual")
    if save:
        ref.check(torch.cat(sums), want["sums"], P, "sums")


def check_backward(got, want):
    P = len(got["parts"])
    for p in range(P):
        ref.check(got["parts"][p], want["parts"], P + 120, f"parts[{p}]")
        assert torch.equal(got["parts"][p], got["parts"][0])
    ref.check(torch.cat(got["residual"]), want["residual"], P + 120, "residual")
    for n in ("pre", "post", "gate"):
        if got[n] is not None:
            ref.check(got[n], want[n], P + 180, n)


SHAPES = [
    # P, T, H: every lane form (a wave to 16, 1 to 4 vectors a lane), odd
    # widths, widths below a vector, more ranks than rows, one rank
    (8, 1, 4096), (4, 3, 512), (5, 7, 1001), (3, 5, 2049), (2, 9, 7), (1, 4, 1), (16, 2, 130), (64, 3, 72),
    (8, 65, 256), (7, 33, 1024), (2, 3, 8192), (3, 2, 16384), (9, 2, 16383), (2, 5, 8193), (12, 700, 64), (1, 600, 40),
    (2, 513, 1000), (2, 512, 1999), (2, 520, 4095), (1, 512, 8190),
]


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("P,T,H", SHAPES)
def test_forward(P, T, H, dtype):
    c = case(P, T, H, dtype)
    with hc.Comm(P, "ring") as comm:
        check_forward(forward(c, comm), c)


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("P,T,H", SHAPES)
def test_backward(P, T, H, dtype):
    c = case(P, T, H, dtype)
    with hc.Comm(P, "ring") as comm:
        check_backward(*backward(c, comm))


@pytest.mark.parametrize("post", [False, True])
@pytest.mark.parametrize("T,H,gates", [(1800, 48, g) for g in (0, 1, 2, 3, 12, 60, 900, 1800)]
                         + [(60, H, g) for H in (1000, 16384) for g in (0, 1, 2, 3, 12, 60)])
def test_variants(post, T, H, gates):
    """Without the norm after the block, without a gate, gate rows for long
    groups of rows, short ones and single rows."""
    c = case(3, T, H, "bf16", post, gates)
    with hc.Comm(3, "rhd") as comm:
        check_forward(forward(c, comm, save=gates != 2), c, save=gates != 2)
        check_backward(*backward(c, comm, has_in=gates != 1))


def test_stores_past_the_cache():
    """96 MiB of outputs and more are stored past the caches."""
    c = case(4, 2049, 6400, "bf16", True, 3)
    with hc.Comm(4, "ring") as comm:
        check_forward(forward(c, comm), c)
        check_backward(*backward(c, comm))


@pytest.mark.parametrize("H", [64, 1001])
def test_more_rows_than_one_round(H):
    c = case(2, 2048, H, "fp16", True, 16)
    with hc.Comm(2, "ring") as comm:
        check_forward(forward(c, comm, eps=1e-3, post_eps=1e-2), c, eps=1e-3, post_eps=1e-2)
        check_backward(*backward(c, comm, eps=1e-3, post_eps=1e-2))


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_unaligned_buffers(dtype):
    c = case(5, 6, 520, dtype)
    with hc.Comm(5, "ring") as comm:
        check_forward(forward(c, comm, shift=3), c)
        check_backward(*backward(c, comm, shift=1))


def test_ranks_as_one_tensor():
    c = case(4, 6, 256, "bf16")
    with hc.Comm(4, "ring") as comm:
        want, res, _ = forward(c, comm)
        out = torch.empty(4, 6, 256, dtype=torch.bfloat16, device="cuda")
        seg = [t.cuda() for t in ref.split_rows(c["residual"], 4)]
        comm.reduce_norm(c["parts"].cuda(), seg, out, c["pre"].cuda(), post_weight=c["post"].cuda(), gate=c["gate"].cuda(),
                         scale=0.75)  # residual in place
        for p in range(4):
            assert torch.equal(out[p], want[p])
        assert all(torch.equal(a, b) for a, b in zip(seg, res))


@pytest.mark.parametrize("H", [7, 129, 1001, 4099, 16383])
def test_in_place(H):
    """Outputs over their inputs give the same bits."""
    c = case(3, 5, H, "bf16")
    with hc.Comm(3, "ring") as comm:
        want, res, _ = forward(c, comm)
        bufs = [x.cuda() for x in c["parts"]]
        seg = [x.cuda() for x in ref.split_rows(c["residual"], 3)]
        kw = dict(post_weight=c["post"].cuda(), gate=c["gate"].cuda(), scale=0.75)
        comm.reduce_norm(bufs, seg, bufs, c["pre"].cuda(), **kw)
        assert all(torch.equal(a, b) for a, b in zip(bufs, want))
        assert all(torch.equal(a, b) for a, b in zip(seg, res))
        got, _ = backward(c, comm)
        grads = [x.cuda() for x in c["out_grads"]]
        rin = [x.cuda() for x in ref.split_rows(c["residual_in"], 3)]
        x = c["parts"].double().sum(0).to(torch.bfloat16)
        wide = dict(dtype=torch.float32, device="cuda")
        pre, post, gate = torch.empty(H, **wide), torch.empty(H, **wide), torch.empty(1, H, **wide)
        comm.reduce_norm_grad(grads, [t.cuda() for t in ref.split_rows(c["residual"], 3)], grads, rin, c["pre"].cuda(), pre,
                              sums=[t.cuda() for t in ref.split_rows(x, 3)], residual_grad_in=rin, post_weight_grad=post,
                              gate_grad=gate, **kw)
        assert all(torch.equal(a, b) for a, b in zip(grads, got["parts"]))
        assert all(torch.equal(a, b) for a, b in zip(rin, got["residual"]))
        assert torch.equal(pre, got["pre"]) and torch.equal(post, got["post"]) and torch.equal(gate, got["gate"])


def test_no_rows():
    c = case(4, 0, 96, "bf16", True, 0)
    with hc.Comm(4, "ring") as comm:
        forward(c, comm)
        got, _ = backward(c, comm)
        assert not got["pre"].any() and not got["post"].any()


def test_zero_and_special_rows():
    """Rows of zeros give zeros; a NaN or an infinity stays in its own row."""
    c = case(3, 6, 300, "fp16")
    for t in (c["parts"], c["out_grads"]):
        t[:, 1] = 0
    c["residual"][1] = 0
    c["residual_in"][1] = 0
    clean = {k: v.clone() if torch.is_tensor(v) else v for k, v in c.items()}
    c["parts"][1, 3, 17] = float("nan")
    c["parts"][2, 4, 299] = float("inf")
    with hc.Comm(3, "ring") as comm:
        out, res, _ = forward(c, comm)
        want, wres, _ = forward(clean, comm)
        for row in (0, 1, 2, 5):
            assert torch.equal(out[0][row], want[0][row]) and torch.equal(torch.cat(res)[row], torch.cat(wres)[row])
        assert not want[0][1].any() and not torch.cat(wres)[1].any()
        assert torch.isnan(out[0][3]).all() and torch.isnan(out[0][4]).any()
        got, _ = backward(clean, comm)
        assert not torch.isnan(got["pre"]).any() and not got["parts"][0][1].any()


def test_gradient_against_differences():
    """fp32 gradients along random directions against central differences of
    the loss sum(out * weights) + sum(residual_out * weights), the forward in
    64 bits (its own formula against which the kernels are checked above)."""
    c = case(3, 4, 40, "fp32", True, 2, seed=5)
    scale = 0.75
    with hc.Comm(3, "ring") as comm:
        out, res, sums = forward(c, comm, scale)
        g = torch.Generator().manual_seed(3)
        wo = torch.randn(3, 4, 40, generator=g)
        wr = torch.randn(4, 40, generator=g)
        c2 = dict(c, out_grads=wo, residual_in=wr, residual=torch.cat(res).cpu())
        got, _ = backward(c2, comm, scale)

    def loss(v):
        r = ref.norm_forward(v["parts"], v["residual"], v["pre"], v["post"], v["gate"], 2, scale)
        return ((r["out"][0] * wo.double().sum(0)).sum() + (r["residual"][0] * wr.double()).sum()).item()

    for name in ("parts", "residual", "pre", "post", "gate"):
        base = {k: v.double() if torch.is_tensor(v) else v for k, v in c.items()}
        way = torch.randn(c[name].shape, generator=g).double()
        step = 1e-5
        lo, hi = dict(base), dict(base)
        lo[name], hi[name] = base[name] - step * way, base[name] + step * way
        diff = (loss(hi) - loss(lo)) / (2 * step)
        grad = {"parts": lambda: torch.stack(got["parts"]), "residual": lambda: torch.cat(got["residual"])}.get(name, lambda: got[name])()
        along = (grad.double().cpu() * way).sum().item()
        size = (grad.double().cpu() * way).abs().sum().item()
        # differences: step^2 of the third derivative and 2^-52 / step of the
        # loss; gradient: 123 + 56 roundings of terms up to a few times its own
        assert abs(diff - along) <= 1e-4 * size + 1e-6, name


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("H", [64, 1000, 16384])
@pytest.mark.parametrize("hidden,sums,eps", [(1e15, 1.0, 1e-6), (1.0, 1e15, 1e-6), (1e16, 1e16, 1e-6), (1e-14, 1e-14, 0.0),
                                             (1e-17, 1.0, 0.0), (1.0, 1e-17, 0.0), (1e-14, 1e-14, 1e-30)])
def test_rows_of_any_size(hidden, sums, eps, H, dtype):
    """Rows whose size's cube, or its inverse, leaves fp32's range: the
    gradient is bounded as everywhere else.  (Squares of 1e16 add up to 2e36
    over 16384 columns; gradients stay between 1e-33 and 1e35.)  A tiny eps
    takes a row of zeros too, whose gradient is the incoming one over its
    root."""
    c = case(3, 6, H, dtype, True, 2)
    x = c["parts"].double().sum(0)
    c["residual"] = (c["residual"].double() / 2 * hidden).to(TYPES[dtype])
    # the gradient's sums are the rounded sum over the ranks of `parts`
    c["parts"] = torch.stack([(x * sums).to(TYPES[dtype]), torch.zeros_like(c["parts"][0]), torch.zeros_like(c["parts"][0])])
    if eps == 1e-30:
        c["residual"][2], c["parts"][:, 2] = 0, 0
    with hc.Comm(3, "ring") as comm:
        got, want = backward(c, comm, has_in=False, eps=eps)
        assert all(bool(torch.isfinite(v).all()) for v, _ in want.values())
        check_backward(got, want)
        check_forward(forward(c, comm, eps=eps), c, eps=eps)
