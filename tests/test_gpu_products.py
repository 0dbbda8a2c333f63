"""Products of 8-bit codes over the ranks on the GPU, against 64 bits.

The sums are whole numbers and exact; rounding one to 32 bits and the two scales
take three roundings, then half a step of the result's type.  Codes and scales
are defined by their 32-bit steps and have to be equal.
"""
import pytest
import torch

import allreduce_reduction_amd as hc
import rankops_ref as ref
import stepops_ref as step
from test_gpu_rank_ops import guarded, same

pytestmark = pytest.mark.gpu

F32, F16, BF = torch.float32, torch.float16, torch.bfloat16


def split(x, P):
    return [x[:, lo:hi].contiguous() for lo, hi in ref.segments(x.shape[1], P)]


class Layer:
    def __init__(self, rows, inner, channels, dtype, seed=0):
        g = torch.Generator().manual_seed(seed + rows + 3 * inner + 7 * channels)
        self.dtype = dtype
        self.q = torch.randint(-128, 128, (rows, inner), generator=g).to(torch.int8)
        self.w = torch.randint(-128, 128, (channels, inner), generator=g).to(torch.int8)
        self.xs, self.ws = torch.rand(rows, generator=g) / 1000, torch.rand(channels, generator=g) / 100 + 1e-3
        self.want = step.product(self.q, self.xs, self.w, self.ws)

    def run(self, form, P):
        rows, channels = len(self.xs), len(self.ws)
        xs = guarded(self.xs)
        zeros = lambda *s: guarded(torch.zeros(*s, dtype=self.dtype))  # noqa: E731
        if form == "channels":
            x = [guarded(self.q)] * P
            w, ws = [guarded(t) for t in ref.split_rows(self.w, P)], [guarded(t) for t in ref.split_rows(self.ws, P)]
            out = [zeros(rows, len(t)) for t, _ in w]
        else:
            x, w, ws = [guarded(t) for t in split(self.q, P)], [guarded(t) for t in split(self.w, P)], [guarded(self.ws)]
            out = [zeros(len(t), channels) for t in ref.split_rows(self.xs, P)] if form == "scatter" else [zeros(rows, channels) for _ in range(P)]
        f = lambda pairs: [t for t, _ in pairs]  # noqa: E731
        with hc.Comm(P, "ring") as c:
            if form in ("reduce", "scatter"):
                c.reduce_product(f(x), xs[0], f(w), ws[0][0], f(out), scatter=form == "scatter")
            else:
                c.product(f(x), xs[0], f(w), f(ws) if form == "channels" else ws[0][0], f(out))
        value, mag = self.want
        if form == "channels":
            ref.check(torch.cat(f(out), 1), self.want, 3, form)
        elif form == "partial":
            for (lo, hi), o in zip(ref.segments(self.q.shape[1], P), f(out)):
                ref.check(o, step.product(self.q[:, lo:hi], self.xs, self.w[:, lo:hi], self.ws), 3, form)
        elif form == "reduce":
            for o in f(out):
                ref.check(o, self.want, 3, form)
        else:
            ref.check(torch.cat(f(out)), self.want, 3, form)
        assert all(ok() for _, ok in x + w + ws + out + [xs])


FORMS = ["channels", "partial", "reduce", "scatter"]
SIZES = [(1, 1, 1), (1, 64, 64), (3, 100, 70), (5, 16, 5), (17, 1001, 131), (33, 257, 1000), (64, 64, 64), (65, 129, 257),
         (130, 2048, 300), (300, 96, 515), (257, 1024, 513)]


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("rows,inner,channels", SIZES)
@pytest.mark.parametrize("P", [1, 3, 8])
def test_against_64_bits(form, rows, inner, channels, P):
    Layer(rows, inner, channels, BF).run(form, P)


@pytest.mark.parametrize("dtype", [F32, F16])
@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("rows,inner,channels", [(1, 256, 64), (7, 1003, 65), (129, 512, 258)])
def test_types(form, dtype, rows, inner, channels):
    Layer(rows, inner, channels, dtype).run(form, 4)


@pytest.mark.parametrize("rows", [1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 100, 128, 129, 255, 256, 257, 400])
@pytest.mark.parametrize("form,inner,channels", [("reduce", 2048, 256), ("channels", 1024, 1040), ("scatter", 2056, 200)])
def test_rows(rows, form, inner, channels):
    Layer(rows, inner, channels, BF).run(form, 8)


@pytest.mark.parametrize("form", ["reduce", "scatter"])
@pytest.mark.parametrize("rows,inner,channels,P", [(1024, 2048, 768, 8), (513, 4096, 1025, 2), (2048, 1280, 512, 5)])
def test_larger(form, rows, inner, channels, P):
    Layer(rows, inner, channels, BF).run(form, P)


def aligned(rows, inner, channels, P, form, dtype=BF, seed=0):
    """Buffers as an allocator hands them out."""
    x = Layer(rows, inner, channels, dtype, seed)
    cols = form == "channels"
    q = [x.q.cuda()] * P if cols else [t.cuda() for t in split(x.q, P)]
    w = [t.cuda() for t in (ref.split_rows(x.w, P) if cols else split(x.w, P))]
    ws = [t.cuda() for t in ref.split_rows(x.ws, P)] if cols else x.ws.cuda()
    out = ([torch.zeros(rows, len(t), dtype=dtype, device="cuda") for t in w] if cols else
           [torch.zeros(len(t), channels, dtype=dtype, device="cuda") for t in ref.split_rows(x.xs, P)] if form == "scatter" else
           [torch.zeros(rows, channels, dtype=dtype, device="cuda") for _ in range(P)])

    def call(c):
        if form in ("channels", "partial"):
            c.product(q, xs, w, ws, out)
        else:
            c.reduce_product(q, xs, w, ws, out, scatter=form == "scatter")

    xs = x.xs.cuda()
    return x, out, call


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("rows,inner,channels,P", [(1, 4096, 512, 4), (3, 8192, 1024, 8), (40, 2048, 2048, 2), (200, 1024, 1024, 2),
                                                   (512, 2048, 1024, 1), (700, 1152, 640, 3)])
def test_aligned_buffers(form, rows, inner, channels, P):
    x, out, call = aligned(rows, inner, channels, P, form)
    with hc.Comm(P, "ring") as c:
        call(c)
    if form == "partial":
        for (lo, hi), o in zip(ref.segments(inner, P), out):
            ref.check(o, step.product(x.q[:, lo:hi], x.xs, x.w[:, lo:hi], x.ws), 3, form)
    else:
        for got in out if form == "reduce" else [torch.cat(out, 1 if form == "channels" else 0)]:
            ref.check(got, x.want, 3, form)


def test_the_widest_sum():
    """Every product 2^14, 131071 of them: the largest sum, and its negative."""
    n = 131071
    q = torch.full((2, n), -128, dtype=torch.int8)
    w = torch.stack([torch.full((n,), v, dtype=torch.int8) for v in (-128, 127, 0)])
    out = torch.zeros(2, 3, device="cuda")
    with hc.Comm(1, "ring") as c:
        c.product([q.cuda()], torch.ones(2, device="cuda"), [w.cuda()], [torch.ones(3, device="cuda")], [out])
        ref.check(out, step.product(q, torch.ones(2), w, torch.ones(3)), 1, "widest")
        with pytest.raises(hc.HbmcError):
            big = torch.zeros(1, n + 1, dtype=torch.int8, device="cuda")
            c.product([big], torch.ones(1, device="cuda"), [big], [torch.ones(1, device="cuda")], [torch.zeros(1, 1, device="cuda")])


def test_a_token_without_a_scale():
    """NaN for a token whose scale is NaN, nothing else touched by it."""
    x = Layer(70, 96, 80, BF)
    x.xs[[3, 69]] = torch.nan
    out = [torch.zeros(70, 80, dtype=BF, device="cuda")]
    with hc.Comm(1, "ring") as c:
        c.product([x.q.cuda()], x.xs.cuda(), [x.w.cuda()], x.ws.cuda(), out)
    bad = out[0].isnan().cpu()
    assert bool(bad[[3, 69]].all()) and int(bad.sum()) == 160


def test_no_rows():
    with hc.Comm(2, "ring") as c:
        e = lambda *s, dt=torch.int8: torch.zeros(*s, dtype=dt, device="cuda")  # noqa: E731
        c.quantize_rows([e(0, 5, dt=BF), e(0, 4, dt=BF)], [e(0, 5), e(0, 4)], e(0, dt=F32))
        c.reduce_product([e(0, 5), e(0, 4)], e(0, dt=F32), [e(6, 5), e(6, 4)], e(6, dt=F32), [e(0, 6, dt=BF)] * 2)


@pytest.mark.parametrize("dtype", [F32, F16, BF])
@pytest.mark.parametrize("rows,width,P", [(1, 1, 1), (1, 5, 8), (3, 4096, 8), (17, 1001, 3), (5, 8192, 1), (2, 16384, 4),
                                          (3, 40003, 2), (300, 64, 5), (2, 131071, 8), (70, 129, 16)])
def test_rounding_to_codes(dtype, rows, width, P):
    g = torch.Generator().manual_seed(width)
    x = (torch.randn(rows, width, generator=g) * torch.rand(rows, 1, generator=g).exp() * 7).to(dtype)
    if rows > 2:
        x[1] = 0
        x[2, width // 2] = -x.abs().max()
    want, scale = step.codes(x)
    dev = [guarded(t) for t in split(x, P)]
    q = [guarded(torch.zeros_like(t, dtype=torch.int8)) for t, _ in dev]
    s = guarded(torch.zeros(rows))
    with hc.Comm(P, "ring") as c:
        c.quantize_rows([t for t, _ in dev], [t for t, _ in q], s[0])
    assert torch.equal(torch.cat([t.cpu() for t, _ in q], 1), want)
    assert torch.equal(s[0].cpu(), scale)
    assert all(ok() for _, ok in dev + q + [s])
    # half a step of the scale, and the 32-bit steps' rounding of codes up to 127
    off = (x.double() - want.double() * scale.double()[:, None]).abs()
    assert bool((off <= scale.double()[:, None] * (0.5 + 127 * 4 * 2.0 ** -24)).all())


def test_rows_without_a_finite_scale():
    x = torch.ones(6, 300)
    x[0, 7], x[1, 299], x[2, 0] = torch.nan, torch.inf, -torch.inf
    x[3] *= 1e-38   # below the least size that has codes
    x[4] *= 3e38
    q, s = torch.full((6, 300), 9, dtype=torch.int8, device="cuda"), torch.full((6,), 9.0, device="cuda")
    with hc.Comm(1, "ring") as c:
        c.quantize_rows([x.cuda()], [q], s)
    q, s = q.cpu(), s.cpu()
    assert bool((q[:4] == 0).all()) and bool(s[:3].isnan().all()) and float(s[3]) == 0.0
    assert bool((q[4:] == 127).all()) and torch.equal(s[4:], torch.div(x[4:, 0], torch.full((2,), 127.0)))


@pytest.mark.parametrize("form", FORMS)
def test_captured_and_on_several_streams(form):
    sets = [aligned(rows, 1024, 512, 4, form, seed=rows) for rows in (2, 50, 300)]
    with hc.Comm(4, "ring") as c:
        for _, _, call in sets:
            call(c)
        torch.cuda.synchronize()
        want = [[t.clone() for t in out] for _, out, _ in sets]
        graphs = []
        for _, _, call in sets[:2]:
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                call(c)
            graphs.append(graph)
        for rep in range(3):
            for _, out, _ in sets:
                for t in out:
                    t.fill_(rep)
            torch.cuda.synchronize()
            for graph in graphs:
                graph.replay()
            sets[2][2](c)
            torch.cuda.synchronize()
            assert all(same(out, w) for (_, out, _), w in zip(sets, want))
        for _, out, _ in sets:
            for t in out:
                t.fill_(5)
        streams = [torch.cuda.Stream() for _ in sets]
        torch.cuda.synchronize()
        for _ in range(3):
            for (_, _, call), q in zip(sets, streams):
                with torch.cuda.stream(q):
                    call(c)
        torch.cuda.synchronize()
        assert all(same(out, w) for (_, out, _), w in zip(sets, want))


def test_past_32_bit_offsets():
    """Weights of 4.3 GB, a result of 4.4 GB: ones and twos."""
    n, k = 70001, 61440
    w = torch.ones(n, k, dtype=torch.int8, device="cuda")
    w[n - 1] = 2
    one = lambda m: torch.ones(m, device="cuda")  # noqa: E731
    out = torch.zeros(3, n, device="cuda")
    with hc.Comm(1, "ring") as c:
        c.product([torch.ones(3, k, dtype=torch.int8, device="cuda")], one(3), [w], [one(n)], [out])
        assert bool((out[:, :n - 1] == k).all()) and bool((out[:, n - 1] == 2 * k).all())
        del w
        t = 34000
        big = torch.zeros(t, 65536, dtype=BF, device="cuda")
        c.product([torch.ones(t, 64, dtype=torch.int8, device="cuda")], one(t), [torch.ones(65536, 64, dtype=torch.int8, device="cuda")],
                  [one(65536)], [big])
        assert bool((big == 64).all())


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("rows", [5, 200, 1100])
@pytest.mark.parametrize("inner,channels,P", [(48, 64, 3), (1376, 528, 1), (3 * 208, 300, 3), (16, 1030, 1), (2000, 272, 5)])
def test_inner_widths_that_end_inside_a_stage(form, rows, inner, channels, P):
    """Whole chunks of 16 codes, but no whole stages of them; neighbouring memory is not zero."""
    x, out, call = aligned(rows, inner, channels, P, form, seed=5)
    with hc.Comm(P, "ring") as c:
        call(c)
    if form == "partial":
        for (lo, hi), o in zip(ref.segments(inner, P), out):
            ref.check(o, step.product(x.q[:, lo:hi], x.xs, x.w[:, lo:hi], x.ws), 3, form)
    else:
        for got in out if form == "reduce" else [torch.cat(out, 1 if form == "channels" else 0)]:
            ref.check(got, x.want, 3, form)


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("rows,inner,channels,P", [(20, 512, 33000, 1), (64, 256, 66000, 2), (64, 272, 16400, 1), (300, 4096, 4096, 2),
                                                   (2000, 640, 3000, 5), (1500, 333, 5000, 3), (9, 2000, 20000, 2), (9, 2001, 20000, 2)])
def test_each_kind_of_tile(form, rows, inner, channels, P):
    """Sizes between which the tile's shape changes."""
    Layer(rows, inner, channels, BF).run(form, P)
    x, out, call = aligned(rows, inner, channels, P, form)
    with hc.Comm(P, "ring") as c:
        call(c)
    if form == "partial":
        for (lo, hi), o in zip(ref.segments(inner, P), out):
            ref.check(o, step.product(x.q[:, lo:hi], x.xs, x.w[:, lo:hi], x.ws), 3, form)
    else:
        for got in out if form == "reduce" else [torch.cat(out, 1 if form == "channels" else 0)]:
            ref.check(got, x.want, 3, form)


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("rows", [3, 40, 300])
@pytest.mark.parametrize("inner,P", [(304, 20), (48, 16), (9, 8), (16, 3), (1, 2)])
def test_ranks_that_hold_none_of_the_inner_width(form, rows, inner, P):
    """304 over 20 ranks: 16 each, the last one none."""
    Layer(rows, inner, 70, BF).run(form, P)
    x, out, call = aligned(rows, inner, 80, P, form)
    with hc.Comm(P, "ring") as c:
        call(c)
    if form == "partial":
        for (lo, hi), o in zip(ref.segments(inner, P), out):
            ref.check(o, step.product(x.q[:, lo:hi], x.xs, x.w[:, lo:hi], x.ws), 3, form)
    else:
        for got in out if form == "reduce" else [torch.cat(out, 1 if form == "channels" else 0)]:
            ref.check(got, x.want, 3, form)


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("rows,inner,channels,P", [(3, 91, 517, 12), (300, 67, 200, 8), (129, 180, 130, 12), (40, 15, 70, 16), (5, 240, 33, 16)])
def test_ranks_with_fewer_than_16_codes(form, dtype, rows, inner, channels, P):
    Layer(rows, inner, channels, dtype).run(form, P)


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("rows,inner,channels,P", [(2304, 256, 4096, 2), (1500, 100, 6000, 8), (1, 333, 5003, 3), (1, 90, 8170, 3),
                                                   (2, 333, 4090, 1), (2, 333, 4100, 1), (30, 256, 12288, 1), (30, 256, 12200, 1)])
def test_each_side_of_a_kind_of_tile(form, rows, inner, channels, P):
    Layer(rows, inner, channels, BF).run(form, P)
    x, out, call = aligned(rows, inner, channels, P, form)
    with hc.Comm(P, "ring") as c:
        call(c)
    if form == "partial":
        for (lo, hi), o in zip(ref.segments(inner, P), out):
            ref.check(o, step.product(x.q[:, lo:hi], x.xs, x.w[:, lo:hi], x.ws), 3, form)
    else:
        for got in out if form == "reduce" else [torch.cat(out, 1 if form == "channels" else 0)]:
            ref.check(got, x.want, 3, form)


def fenced(t, pad=64):
    """A copy of t on the GPU, aligned as an allocator's, between guard zones, and their check."""
    flat = torch.full((t.numel() + 2 * pad,), 7, dtype=t.dtype, device="cuda")
    view = flat[pad:pad + t.numel()].view(t.shape)
    view.copy_(t)
    return view, lambda: bool((flat[:pad] == 7).all()) and bool((flat[pad + t.numel():] == 7).all())


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("dtype", [F32, F16])
@pytest.mark.parametrize("rows,inner,channels,P", [
    (20, 512, 12301, 1),    # 32 by 64 of aligned rows
    (30, 256, 12201, 1),    # 32 by 32
    (50, 272, 8101, 1),     # 64 by 32
    (64, 256, 65381, 1),    # 64 by 256
    (64, 272, 16401, 1),    # 64 by 64
    (2000, 640, 3001, 5),   # 128 by 128
    (2304, 256, 4097, 2),   # 256 by 256, the ranks' own parts 128 by 128
    (300, 333, 517, 3),     # 64 by 64 at any alignment
    (1500, 333, 5001, 3),   # 128 by 128
    (300, 67, 201, 8),      # 64 by 64 of ranks with fewer than 16 codes
    (1500, 100, 6001, 8),   # 128 by 128
])
def test_types_in_each_kind_of_tile(form, dtype, rows, inner, channels, P):
    """Whose results end inside 16 bytes, rows of them at odd addresses."""
    x = Layer(rows, inner, channels, dtype)
    cols = form == "channels"
    q = [x.q.cuda()] * P if cols else [t.cuda() for t in split(x.q, P)]
    w = [t.cuda() for t in (ref.split_rows(x.w, P) if cols else split(x.w, P))]
    ws = [t.cuda() for t in ref.split_rows(x.ws, P)] if cols else x.ws.cuda()
    zeros = lambda *s: fenced(torch.zeros(*s, dtype=dtype))  # noqa: E731
    out = ([zeros(rows, len(t)) for t in w] if cols else
           [zeros(len(t), channels) for t in ref.split_rows(x.xs, P)] if form == "scatter" else [zeros(rows, channels) for _ in range(P)])
    with hc.Comm(P, "ring") as c:
        if form in ("channels", "partial"):
            c.product(q, x.xs.cuda(), w, ws, [t for t, _ in out])
        else:
            c.reduce_product(q, x.xs.cuda(), w, ws, [t for t, _ in out], scatter=form == "scatter")
    if form == "partial":
        for (lo, hi), (o, _) in zip(ref.segments(inner, P), out):
            ref.check(o, step.product(x.q[:, lo:hi], x.xs, x.w[:, lo:hi], x.ws), 3, form)
    elif form == "reduce":
        ref.check(out[0][0], x.want, 3, form)
        assert all(same([o], [out[0][0]]) for o, _ in out)
    else:
        ref.check(torch.cat([o for o, _ in out], 1 if cols else 0), x.want, 3, form)
    assert all(ok() for _, ok in out)
