"""Penalties, biases and masks on logits on the GPU, against 64 bits.

A column takes at most one rounding to 32 bits each for the repetition, the
frequency's product, the two differences, the biases' sum (one a bias more) and
its addition: 6 + its biases, relative to the terms' sizes; then half a step of
its type.
"""
import pytest
import torch

import allreduce_reduction_amd as hc
import rankops_ref as ref
import stepops_ref as step
from test_gpu_rank_ops import guarded, same

pytestmark = pytest.mark.gpu

F32, F16, BF = torch.float32, torch.float16, torch.bfloat16


class Rows:
    """One call's inputs: on the host, and the ranks' columns on the GPU."""

    def __init__(self, rows, vocab, dtype, history=0, biases=0, masked=False, seed=0, ids=torch.int64, lengths=torch.int32):
        g = torch.Generator().manual_seed(seed + rows * 7 + vocab)
        self.z = (torch.randn(rows, vocab, generator=g) * 3).to(dtype)
        self.kw = {}
        if history:
            t = torch.randint(-2, vocab + 2, (rows, history), generator=g)
            t[:, ::3] = torch.randint(0, min(vocab, 5), (rows, len(range(0, history, 3))), generator=g)  # some often
            n = torch.randint(0, history + 1, (rows,), generator=g)
            n[0] = history
            p = (n * torch.rand(rows, generator=g)).long()
            self.kw.update(tokens=t.to(ids), prompt_lengths=p.to(lengths), lengths=n.to(lengths),
                           repetition=torch.rand(rows, generator=g) + 0.5, frequency=torch.rand(rows, generator=g) - 0.3,
                           presence=torch.rand(rows, generator=g) - 0.5)
        if biases:
            b = torch.randint(-2, vocab + 2, (rows, biases), generator=g)
            b[:, 1::4] = b[:, :1]  # one column named often
            self.kw.update(bias_ids=b.to(ids), bias=torch.randn(rows, biases, generator=g) * 2)
        if masked:
            on = torch.rand(rows, vocab, generator=g) < torch.tensor([0.5, 0.02, 1.0, 0.0])[torch.arange(rows) % 4][:, None]
            self.kw.update(mask=step.bits(on))

    def device(self, P):
        self.dev = {k: guarded(v) for k, v in self.kw.items()}
        return [guarded(self.z[:, lo:hi].contiguous()) for lo, hi in ref.segments(self.z.shape[1], P)]

    def check(self, got, most=0):
        want, mag = step.adjust(self.z, **self.kw)
        steps = 6 + most + (self.kw["bias_ids"].shape[1] if "bias_ids" in self.kw else 0)
        got = torch.cat([t.cpu() for t in got], 1)
        finite = torch.isfinite(want)
        assert bool((got.double() == want)[~finite].all())
        ref.check(got[finite], (want[finite], mag[finite]), steps, "logits")
        named = torch.zeros_like(finite)
        for r in range(named.shape[0]):
            for k in ("tokens", "bias_ids"):
                if k in self.kw:
                    at = self.kw[k][r].long()
                    named[r, at[(at >= 0) & (at < named.shape[1])]] = True
        kept = finite & ~named
        assert same([got[kept].contiguous()], [self.z[kept].contiguous()])

    def run(self, P, in_place):
        z = self.device(P)
        out = z if in_place else [guarded(torch.zeros_like(t)) for t, _ in z]
        with hc.Comm(P, "ring") as c:
            c.adjust_logits([t for t, _ in z], None if in_place else [t for t, _ in out], **{k: v for k, (v, _) in self.dev.items()})
        self.check([t for t, _ in out])
        assert all(ok() for _, ok in z + out + list(self.dev.values()))


SHAPES = [(1, 1), (1, 33), (3, 500), (5, 4099), (2, 50001), (9, 1000), (1, 131072)]


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("dtype", [F32, F16, BF])
@pytest.mark.parametrize("rows,vocab", SHAPES)
@pytest.mark.parametrize("P,history,biases,masked", [(1, 300, 0, False), (3, 41, 9, True), (4, 0, 5, False), (8, 0, 0, True),
                                                     (7, 1, 1, False), (2, 5000, 300, True)])
def test_against_64_bits(rows, vocab, dtype, in_place, P, history, biases, masked):
    Rows(rows, vocab, dtype, history, biases, masked).run(P, in_place)


@pytest.mark.parametrize("ids", [torch.int32, torch.int64])
@pytest.mark.parametrize("lengths", [torch.int32, torch.int64])
def test_types_of_ids_and_lengths(ids, lengths):
    Rows(4, 3001, BF, 77, 6, True, ids=ids, lengths=lengths).run(3, True)


@pytest.mark.parametrize("rows,vocab,P", [(300, 5003, 3), (700, 64, 8), (70, 131072, 8)])
def test_many_rows(rows, vocab, P):
    Rows(rows, vocab, BF, 100, 4, True).run(P, True)


@pytest.mark.parametrize("history,biases", [(200000, 0), (524287, 3), (3, 4095)])
def test_the_longest_lists(history, biases):
    """Nearly every third place of the history holds one of five tokens."""
    Rows(1, 20011, F32, history, biases).run(2, False)


def test_each_penalty_alone_and_defaults():
    """Without prompt lengths all is output; without lengths rows are full."""
    x = Rows(5, 2000, F32, 64, 0)
    full = dict(x.kw)
    for keep in (("repetition",), ("frequency",), ("presence",), ("repetition", "presence"), ()):
        for lists in (("prompt_lengths",), ("lengths",), (), ("prompt_lengths", "lengths")):
            x.kw = {k: full[k] for k in ("tokens",) + keep + lists}
            x.run(3, True)
            x.run(3, False)


def test_nothing_asked_copies():
    z = [torch.randn(3, 7, device="cuda"), torch.randn(3, 6, device="cuda")]
    out = [torch.zeros_like(t) for t in z]
    with hc.Comm(2, "ring") as c:
        c.adjust_logits(z, out)
        assert same(z, out)
        before = [t.clone() for t in z]
        c.adjust_logits(z)
        c.adjust_logits(z, tokens=torch.zeros(3, 0, dtype=torch.int32, device="cuda"), presence=torch.ones(3, device="cuda"),
                        bias_ids=torch.zeros(3, 0, dtype=torch.int64, device="cuda"), bias=torch.zeros(3, 0, device="cuda"))
        assert same(z, before)
        c.adjust_logits([t[:0] for t in z], [t[:0] for t in out])


def test_lengths_out_of_range_are_taken_into_it():
    x = Rows(4, 300, F32, 20)
    x.kw["lengths"] = torch.tensor([-5, 99, 2 ** 31 - 1, 7], dtype=torch.int32)
    x.kw["prompt_lengths"] = torch.tensor([3, -9, 500, 9], dtype=torch.int32)
    x.run(3, True)


@pytest.mark.parametrize("dtype", [F32, F16, BF])
@pytest.mark.parametrize("in_place", [False, True])
def test_values_that_are_no_numbers(dtype, in_place):
    """A NaN or an infinity stays where nothing touches it and goes where the
    mask forbids it; the lowest value stays finite under a penalty of 1."""
    low = torch.finfo(dtype).min
    z = torch.tensor([[torch.nan, torch.inf, -torch.inf, low, torch.nan, torch.inf, -torch.inf, low] * 5]).to(dtype)
    on = torch.tensor([[True, True, True, True, False, False, False, False] * 5])
    dev = z.cuda()
    out = dev if in_place else torch.zeros_like(dev)
    with hc.Comm(1, "ring") as c:
        c.adjust_logits([dev], [out], mask=step.bits(on).cuda(), tokens=torch.tensor([[3, 11]]).cuda(),
                        repetition=torch.ones(1, device="cuda"), bias_ids=torch.tensor([[0, 1, 9]]).cuda(),
                        bias=torch.tensor([[1.0, -torch.inf, -torch.inf]]).cuda())
    got = out.cpu()[0]
    assert bool((got[~on[0]] == -torch.inf).all())
    assert bool(got[0].isnan()) and bool(got[1].isnan()) and bool(got[9].isnan())  # infinity - infinity
    assert float(got[2]) == -torch.inf and float(got[3]) == low and float(got[11]) == low and float(got[17]) == torch.inf
    assert bool(got[8].isnan())


def test_banned_by_a_bias():
    z = torch.zeros(2, 10, device="cuda")
    with hc.Comm(1, "ring") as c:
        c.adjust_logits([z], bias_ids=torch.tensor([[4, -1, 4], [9, 10, 0]]).cuda(),
                        bias=torch.tensor([[-torch.inf, 5.0, 2.0], [1.0, 5.0, -torch.inf]]).cuda())
    want = torch.zeros(2, 10)
    want[0, 4], want[1, 9], want[1, 0] = -torch.inf, 1.0, -torch.inf
    assert torch.equal(z.cpu(), want)


def test_captured_and_on_several_streams():
    xs = [Rows(5 + k, 4001, BF, 60, 8, True, seed=k) for k in range(3)]
    P = 4
    with hc.Comm(P, "ring") as c:
        zs = [x.device(P) for x in xs]
        outs = [[torch.zeros_like(t) for t, _ in z] for z in zs]

        def call(k):
            c.adjust_logits([t for t, _ in zs[k]], outs[k], **{n: v for n, (v, _) in xs[k].dev.items()})

        graphs = []
        for k in range(2):
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                call(k)
            graphs.append(graph)
        for rep in range(3):
            for o in outs:
                for t in o:
                    t.fill_(rep)
            torch.cuda.synchronize()
            graphs[0].replay()
            graphs[1].replay()
            call(2)
            torch.cuda.synchronize()
            for x, o in zip(xs, outs):
                x.check(o)
        for o in outs:
            for t in o:
                t.fill_(5)
        streams = [torch.cuda.Stream() for _ in xs]
        torch.cuda.synchronize()
        for k, q in enumerate(streams):
            with torch.cuda.stream(q):
                call(k)
        torch.cuda.synchronize()
        for x, o in zip(xs, outs):
            x.check(o)


def test_past_32_bit_offsets():
    rows, vocab = 4500, 500000
    z = torch.zeros(rows, vocab, dtype=BF, device="cuda")
    tokens = torch.full((rows, 2), vocab - 1, device="cuda")
    mask = torch.full((rows, vocab // 32), -1, dtype=torch.int32, device="cuda")
    mask[rows - 1, 7] = 0
    with hc.Comm(1, "ring") as c:
        c.adjust_logits([z], tokens=tokens, frequency=torch.ones(rows, device="cuda"), mask=mask)
    assert bool((z[:, vocab - 1] == -2).all()) and bool((z[rows - 1, 7 * 32:8 * 32] == -torch.inf).all())
    assert int((z != 0).sum()) == rows + 32


@pytest.mark.parametrize("ids", [torch.int32, torch.int64])
@pytest.mark.parametrize("history", [1, 2, 3, 4, 5, 2047, 2048, 2049, 4095, 4097, 8193])
@pytest.mark.parametrize("masked", [False, True])
def test_histories_that_end_inside_a_load(history, ids, masked):
    for in_place in (False, True):
        Rows(3, 9001, BF, history, 2, masked, ids=ids).run(1, in_place)


@pytest.mark.parametrize("rows,vocab,P", [(1, 16385, 1), (40, 16385, 2), (700, 8193, 1), (130, 20000, 2), (520, 16384, 1)])
def test_each_length_of_tile(rows, vocab, P):
    """Tiles of 2048, 4096 and 8192 columns, the last of a rank a few columns short or long."""
    for in_place in (False, True):
        Rows(rows, vocab, F16, 30, 3, True).run(P, in_place)


@pytest.mark.parametrize("in_place", [False, True])
def test_every_bias_names_one_column(in_place):
    x = Rows(2, 500, F32, 9, 700)
    x.kw["bias_ids"][:] = 77
    x.kw["bias_ids"][1, ::2] = 76
    x.run(3, in_place)


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("masked", [False, True])
def test_most_biases_over_the_longest_tile(in_place, masked):
    Rows(190, 20000, BF, 12, 4095, masked).run(1, in_place)


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("masked", [False, True])
@pytest.mark.parametrize("dtype", [F32, F16, BF])
def test_bits_beside_a_named_column(dtype, masked, in_place):
    """Every other column a signalling NaN, whose quiet bit a conversion would
    set, beside columns that tokens and biases name."""
    rows, vocab, P = 5, 3001, 3
    x = Rows(rows, vocab, dtype, 40, 6, masked)
    ints, low, quiet = {F32: (torch.int32, 0x7f800000, 1 << 22), F16: (torch.int16, 0x7c00, 1 << 9), BF: (torch.int16, 0x7f80, 1 << 6)}[dtype]
    g = torch.Generator().manual_seed(1)
    nan = low + torch.randint(1, quiet, (rows, vocab), generator=g)
    nan = nan - torch.where(torch.rand(rows, vocab, generator=g) < 0.5, 2 ** (8 * x.z.element_size() - 1), 0)  # either sign
    named = torch.zeros(rows, vocab, dtype=torch.bool)
    for r in range(rows):
        for k in ("tokens", "bias_ids"):
            at = x.kw[k][r]
            named[r, at[(at >= 0) & (at < vocab)]] = True
    bits = torch.where(named, x.z.view(ints).long(), nan).to(ints)
    z = [guarded(bits[:, lo:hi].contiguous()) for lo, hi in ref.segments(vocab, P)]
    out = z if in_place else [guarded(torch.zeros_like(t)) for t, _ in z]
    with hc.Comm(P, "ring") as c:
        c.adjust_logits([t.view(dtype) for t, _ in z], [t.view(dtype) for t, _ in out], **{k: v.cuda() for k, v in x.kw.items()})
    got = torch.cat([t.cpu() for t, _ in out], 1)
    kept = ~named & (step.allowed(x.kw["mask"], vocab) if masked else True)
    assert int(kept.sum()) > 100
    assert torch.equal(got[kept], bits[kept])
    assert all(ok() for _, ok in z + out)


def joined(ids, bias, vocab):
    """The biases of each column added up in 32 bits, in list order."""
    z = torch.zeros(ids.shape[0], vocab)
    for r in range(ids.shape[0]):
        seen = set()
        for v, b in zip(ids[r].tolist(), bias[r]):
            if 0 <= v < vocab:
                z[r, v] = z[r, v] + b if v in seen else b
                seen.add(v)
    return z


def repeated(kind, n, vocab, g):
    """Places of a list of n biases that name columns again."""
    ids = torch.randperm(vocab, generator=g)[:n]
    if kind == "one":
        ids[-1] = ids[0]
    elif kind == "pairs":
        ids[n // 2:2 * (n // 2)] = ids[:n // 2]
    elif kind == "all":
        ids[:] = ids[0]
    elif kind == "few":
        ids = ids[torch.randint(0, min(n, 7), (n,), generator=g)]
    elif kind == "wrapping":  # places 5, 1000 and 3096, whose sum's low twelve bits are the first's; the last place of all
        ids[999], ids[3095], ids[4094] = ids[4], ids[4], ids[7]
    elif kind == "cancelling":  # the sums' low bits are none at all
        ids[4094] = ids[0]
    return ids


@pytest.mark.parametrize("kind,n", [(k, n) for k in ("one", "pairs", "all", "few") for n in (2, 3, 65, 513, 1000)] +
                         [(k, 4095) for k in ("one", "pairs", "all", "few", "wrapping", "cancelling")])
@pytest.mark.parametrize("masked,in_place", [(False, True), (True, True), (False, False)])
def test_repeated_biases_add_up_in_their_order(kind, n, masked, in_place):
    """To zeros, so that the sums' bits are the results'; values whose order matters, in one tile and over several."""
    g = torch.Generator().manual_seed(n)
    rows, vocab, P = 3, 9000, 2
    ids = torch.stack([repeated(kind, n, vocab, g), repeated(kind, n, vocab, g), torch.randint(-1, vocab, (n,), generator=g)])
    bias = torch.randn(rows, n, generator=g) * torch.tensor([1.0, 1e4, 1e8])[torch.randint(0, 3, (rows, n), generator=g)]
    on = torch.rand(rows, vocab, generator=g) < 0.7
    want = joined(ids, bias, vocab)
    if masked:
        want[~on] = -torch.inf
    z = [guarded(torch.zeros(rows, hi - lo)) for lo, hi in ref.segments(vocab, P)]
    out = z if in_place else [guarded(torch.ones(rows, hi - lo)) for lo, hi in ref.segments(vocab, P)]
    with hc.Comm(P, "ring") as c:
        c.adjust_logits([t for t, _ in z], [t for t, _ in out], bias_ids=ids.cuda(), bias=bias.cuda(),
                        mask=step.bits(on).cuda() if masked else None)
    assert torch.equal(torch.cat([t.cpu() for t, _ in out], 1), want)
    assert all(ok() for _, ok in z + out)


def test_a_repeated_bias_costs_little():
    """Once every bias of a tile with one repeated was compared with all others, which
    took 250 times as long as distinct ones; twenty times is far from both."""
    rows, n, vocab = 1, 4095, 8192
    ids = torch.randperm(vocab, generator=torch.Generator().manual_seed(1))[None, :n]
    again = ids.clone()
    again[0, -1] = again[0, 0]
    z, bias, took = [torch.zeros(rows, vocab, device="cuda")], torch.zeros(rows, n, device="cuda"), []
    with hc.Comm(1, "ring") as c:
        for names in (ids.cuda(), again.cuda()):
            best = float("inf")
            for _ in range(5):
                start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
                c.adjust_logits(z, bias_ids=names, bias=bias)
                start.record()
                for _ in range(20):
                    c.adjust_logits(z, bias_ids=names, bias=bias)
                end.record()
                torch.cuda.synchronize()
                best = min(best, start.elapsed_time(end))
            took.append(best)
    assert took[1] < 20 * took[0], took
