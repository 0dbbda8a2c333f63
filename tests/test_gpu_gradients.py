"""The global norm of gradients and their clipping on the GPU, against 64 bits.

The norm is taken in 64 bits and rounded once: half a step, 2^-24.  A gradient
is multiplied by a factor rounded to 32 bits and rounded to 32 bits and then to
its type: two roundings to 32 bits and half a step of the type.
"""
import ctypes
import math

import pytest
import torch

import allreduce_reduction_amd as hc
import rankops_ref as ref
import stepops_ref as step
from test_gpu_rank_ops import guarded, same

pytestmark = pytest.mark.gpu

F32, F16, BF = torch.float32, torch.float16, torch.bfloat16
INF = math.inf


def number(x=7.0):
    return torch.full((1,), x, device="cuda")


def near(got, want):
    assert abs(float(got) - float(want)) <= 1.01 * 2.0 ** -24 * abs(float(want)), (float(got), float(want))


def made(lengths, dtypes, seed, by=1.0):
    g = torch.Generator().manual_seed(seed)
    return [(torch.randn(n, generator=g) * by).to(dtypes[i % len(dtypes)]) for i, n in enumerate(lengths)]


LENGTHS = [[1], [3, 0, 5], [4095, 4097, 8192, 8193], [100003, 17, 1, 0, 33333], [1 << 20, 999999, 7] * 3, list(range(1, 700, 3))]


@pytest.mark.parametrize("dtypes", [(F32,), (F16,), (BF,), (BF, F32, F16)])
@pytest.mark.parametrize("lengths", LENGTHS)
@pytest.mark.parametrize("norm_type", [1.0, 2.0, INF])
def test_dealt(lengths, dtypes, norm_type):
    """Each rank its own tensors, every one past alignment between guard zones."""
    P = 3
    host = made(lengths, dtypes, len(lengths))
    held = [guarded(t) for t in host]
    out = number()
    size = step.norm(host, norm_type, 0.5)
    with hc.Comm(P, "ring") as c, c.gradients(dealt=[[t for t, _ in held[r::P]] for r in range(P)]) as g:
        g.norm(out, norm_type=norm_type, scale=-0.5)
        near(out, size)
        assert all(torch.equal(t.cpu(), h) for (t, _), h in zip(held, host))
        out.zero_()
        most = float(size) / 3 + 1e-30
        g.clip(most, out, norm_type=norm_type, scale=-0.5, eps=0.0)
        near(out, size)
    by = step.factor(size, most, -0.5, 0.0)
    for (t, ok), h in zip(held, host):
        v = h.double() * by
        ref.check(t, (v, v.abs()), 2, "gradient")
        assert ok()


@pytest.mark.parametrize("dtype", [F32, F16, BF])
@pytest.mark.parametrize("lengths", [[5], [4097, 12, 1], [300007, 64, 70001]])
@pytest.mark.parametrize("P", [1, 2, 8])
def test_same_on_every_rank(P, lengths, dtype):
    """Counted once; the copies, which lie at other alignments, written from the first rank's."""
    host = made(lengths, (dtype,), P)
    copies = [[guarded(t, 40 + r) for t in host] for r in range(P)]
    for r in range(1, P):
        for t, _ in copies[r]:
            t.zero_()  # never read
    out = number()
    size = step.norm(host, 2.0, 1.0 / P)
    with hc.Comm(P, "rhd") as c, c.gradients(same=[[t for t, _ in mine] for mine in copies]) as g:
        g.clip(0.1 * float(size), out, scale=1.0 / P)
    near(out, size)
    by = step.factor(size, 0.1 * float(size), 1.0 / P)
    for mine in copies:
        for (t, ok), h in zip(mine, host):
            ref.check(t, (h.double() * by, h.double().abs() * by), 2, "gradient")
            assert ok()
    for mine in copies[1:]:
        assert same([t for t, _ in mine], [t for t, _ in copies[0]])


def test_dealt_and_same_together():
    """As tensor parallelism leaves them: dealt-out weights and replicated norms."""
    P = 4
    own, all_ = made([5000, 70000, 3, 123], (BF,), 1), made([64, 4096], (F32,), 2)
    d = [[t.cuda()] for t in own]
    s = [[t.cuda() for t in all_] for _ in range(P)]
    out = number()
    with hc.Comm(P, "ring") as c, c.gradients(dealt=d, same=s) as g:
        g.clip(1.0, out)
    size = step.norm(own + all_, 2.0)
    near(out, size)
    by = step.factor(size, 1.0)
    for got, h in zip([t for m in d for t in m] + s[3], own + all_):
        ref.check(got, (h.double() * by, h.double().abs() * by), 2, "gradient")


@pytest.mark.parametrize("n", [2, 700000])
@pytest.mark.parametrize("by", [1e30, 1e-30])
@pytest.mark.parametrize("dtype", [F32, BF])
def test_sizes_whose_squares_32_bits_do_not_hold(dtype, by, n):
    host = made([n], (dtype,), 5, by)
    t, out = host[0].cuda(), number()
    size = step.norm(host, 2.0)
    with hc.Comm(1, "ring") as c, c.gradients(dealt=[[t]]) as g:
        g.clip(float(size) / 4, out, eps=0.0)
    near(out, size)
    ref.check(t, (host[0].double() / 4, host[0].double().abs() / 4), 3, "gradient")


@pytest.mark.parametrize("n", [9, 300000])
@pytest.mark.parametrize("norm_type", [1.0, 2.0, INF])
def test_nothing_to_clip_leaves_the_bits(norm_type, n):
    host = made([n], (BF,), 3)[0]
    host[0] = -0.0
    for most in (1e9, INF, float(step.norm([host], norm_type)) * (1 + 1e-12)):
        t, out = host.cuda(), number()
        with hc.Comm(1, "ring") as c, c.gradients(dealt=[[t]]) as g:
            g.clip(most, out, norm_type=norm_type, eps=0.0)
        assert same([t.cpu()], [host])
        near(out, step.norm([host], norm_type))


@pytest.mark.parametrize("n", [9, 300000])
@pytest.mark.parametrize("norm_type", [1.0, 2.0, INF])
def test_infinity_and_nan(norm_type, n):
    with hc.Comm(1, "ring") as c:
        t, out = torch.ones(n, device="cuda"), number()
        t[n // 2] = -INF
        with c.gradients(dealt=[[t]]) as g:
            g.clip(1.0, out, norm_type=norm_type)
        assert float(out) == INF and float(t[0]) == 0.0 and bool(t[n // 2].isnan()) and int(t.isnan().sum()) == 1
        t = torch.ones(n, device="cuda")
        t[n - 1] = math.nan
        with c.gradients(dealt=[[t]]) as g:
            g.norm(out, norm_type=norm_type)
            assert bool(out.isnan())
            g.clip(1.0, out, norm_type=norm_type)
        assert bool(out.isnan()) and bool(t.isnan().all())


def test_nothing_and_zeros():
    with hc.Comm(2, "ring") as c:
        out = number()
        with c.gradients(dealt=[[], [torch.empty(0, device="cuda")]]) as g:
            g.clip(1.0, out)
        assert float(out) == 0.0
        t = torch.zeros(5, device="cuda")
        with c.gradients(dealt=[[t], []]) as g:
            for most, eps in ((1.0, 1e-6), (0.0, 0.0), (0.0, 1e-6)):
                out.fill_(7)
                g.clip(most, out, eps=eps)
                assert float(out) == 0.0 and bool((t == 0).all())
        t.fill_(1)
        with c.gradients(dealt=[[t], []]) as g:
            g.clip(0.0, out)
            assert bool((t == 0).all())


@pytest.mark.parametrize("lengths", [[1000, 33], [500001, 4097]])
def test_captured_and_on_several_streams(lengths):
    """Two graphs over one handle's kept table, their own workspaces, with eager
    calls between the replays; then several handles at once."""
    host = made(lengths, (F32, BF), 9)
    size = step.norm(host, 2.0)

    def fresh():
        return [t.cuda() for t in host]

    def check(tensors, out, by):
        near(out, size)
        for t, h in zip(tensors, host):
            ref.check(t, (h.double() * by, h.double().abs() * by), 2, "gradient")

    with hc.Comm(1, "ring") as c:
        t, outs = fresh(), [number(), number()]
        g = c.gradients(dealt=[t])
        graphs = [torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()]
        with torch.cuda.graph(graphs[0]):
            g.norm(outs[0])
        with torch.cuda.graph(graphs[1]):
            g.clip(1.0, outs[1])
        for rep in range(4):
            for x, h in zip(t, host):
                x.copy_(h)
            torch.cuda.synchronize()
            graphs[0].replay()
            graphs[1].replay()
            other = fresh()
            with c.gradients(dealt=[other]) as e:
                out = number()
                e.clip(2.0, out)
                torch.cuda.synchronize()
            check(other, out, step.factor(size, 2.0))
            near(outs[0], size)
            check(t, outs[1], step.factor(size, 1.0))
            for o in outs:
                o.fill_(rep)
        torch.cuda.synchronize()
        g.close()
        many = [fresh() for _ in range(4)]
        handles = [c.gradients(dealt=[x]) for x in many]
        streams, outs = [torch.cuda.Stream() for _ in many], [number() for _ in many]
        torch.cuda.synchronize()
        for k, (h, q) in enumerate(zip(handles, streams)):
            with torch.cuda.stream(q):
                h.clip(1.0 + k, outs[k])
        torch.cuda.synchronize()
        for k, (x, h) in enumerate(zip(many, handles)):
            check(x, outs[k], step.factor(size, 1.0 + k))
            h.close()


def test_two_norms_of_one_handle_at_once():
    host = made([700001], (F32,), 4)
    with hc.Comm(1, "ring") as c, c.gradients(dealt=[[host[0].cuda()]]) as g:
        streams, outs = [torch.cuda.Stream() for _ in range(4)], [number() for _ in range(4)]
        torch.cuda.synchronize()
        for _ in range(5):
            for q, o in zip(streams, outs):
                g.norm(o, stream=q)
        torch.cuda.synchronize()
    for o in outs:
        near(o, step.norm(host, 2.0))
    assert same(outs, [outs[0]] * 4)


def test_an_exact_workspace_and_what_is_refused():
    L = hc.load_library()
    t, out = torch.ones(300000, device="cuda"), number()
    with hc.Comm(1, "ring") as c, c.gradients(dealt=[[t]]) as g:
        need = ctypes.c_size_t()
        assert L.hbmc_gradients_workspace(g._h, ctypes.byref(need)) == 0 and need.value > 0
        flat = torch.full((need.value + 512,), 0xa5, dtype=torch.uint8, device="cuda")
        ws = flat.data_ptr() + 256
        q = torch.cuda.current_stream().cuda_stream
        call = lambda norm, ws, n: L.hbmc_gradients_clip(g._h, 2.0, 1.0, 1.0, 1e-6, norm, ws, n, q)  # noqa: E731
        assert call(out.data_ptr(), ws, need.value) == 0
        torch.cuda.synchronize()
        assert bool((flat[:256] == 0xa5).all()) and bool((flat[256 + need.value:] == 0xa5).all())
        near(out, math.sqrt(300000))
        before = t.clone()
        for norm, w, n in ((out.data_ptr(), ws, need.value - 1), (out.data_ptr(), ws + 8, need.value), (out.data_ptr(), None, need.value),
                           (None, ws, need.value), (t.data_ptr() + 40, ws, need.value), (out.data_ptr(), t.data_ptr() + 1600, need.value),
                           (ws, ws, need.value)):
            assert call(norm, w, n) == 1
        torch.cuda.synchronize()
        assert torch.equal(t, before)
        with pytest.raises(ValueError):
            g.norm(torch.zeros(1))
        with pytest.raises(ValueError):
            g.norm(torch.zeros(2, device="cuda"))
        for kw in (dict(norm_type=3.0), dict(scale=math.nan), dict(eps=-1.0), dict(eps=INF)):
            with pytest.raises(hc.HbmcError):
                g.clip(1.0, out, **kw)
        for most in (-1.0, math.nan):
            with pytest.raises(hc.HbmcError):
                g.clip(most, out)
        with pytest.raises(hc.HbmcError):  # the same memory twice
            c.gradients(dealt=[[t, t[5:9]]])
        with pytest.raises(ValueError):
            c.gradients(dealt=[[t[::2]]])
        with pytest.raises(TypeError):
            c.gradients(dealt=[[t.double()]])
    with pytest.raises(hc.HbmcError):
        g.norm(out)  # closed
    with hc.Comm(2, "ring") as c:
        with pytest.raises(ValueError):
            c.gradients(same=[[t], [out]])
        with pytest.raises(ValueError):
            c.gradients(same=[[t], []])
        with pytest.raises(ValueError):
            c.gradients(dealt=[[t]])


def test_past_32_bit_offsets():
    """A tensor of 4.3 GB: zeros but for a few values."""
    n = (1 << 31) + 12345
    t = torch.zeros(n, dtype=BF, device="cuda")
    t[5], t[n - 1], t[1 << 30] = 3.0, 4.0, 12.0
    out = number()
    with hc.Comm(1, "ring") as c, c.gradients(dealt=[[t]]) as g:
        g.clip(6.5, out, eps=0.0)
    assert float(out) == 13.0 and float(t[n - 1]) == 2.0 and float(t[1 << 30]) == 6.0 and float(t[5]) == 1.5
    assert int((t != 0).sum()) == 3


@pytest.mark.parametrize("dtype", [F32, F16, BF])
@pytest.mark.parametrize("P", [2, 3, 12])
@pytest.mark.parametrize("lengths", [[1 << 18, 65537, 3, 0, 129], [33, 1]])
def test_copies_at_every_phase(P, lengths, dtype):
    """Copy after copy one element further from 128 bytes, packed tensor behind tensor, with guards."""
    host = made(lengths, (dtype,), P)
    total = sum(lengths)
    flats = [torch.full((total + 300,), 7, dtype=dtype, device="cuda") for _ in range(P)]
    copies = []
    for r, flat in enumerate(flats):
        at = 100 + 5 * r
        copies.append(list(flat[at:at + total].split(lengths)))
        if r == 0:
            for t, h in zip(copies[0], host):
                t.copy_(h)
    out = number()
    size = step.norm(host, 2.0, 0.25)
    with hc.Comm(P, "ring") as c, c.gradients(same=copies) as g:
        g.clip(float(size) / 2, out, scale=0.25, eps=0.0)
    near(out, size)
    by = step.factor(size, float(size) / 2, 0.25, 0.0)
    for r, flat in enumerate(flats):
        for t, h in zip(copies[r], host):
            ref.check(t, (h.double() * by, h.double().abs() * by), 2, "gradient")
        at = 100 + 5 * r
        assert bool((flat[:at] == 7).all()) and bool((flat[at + total:] == 7).all())


@pytest.mark.parametrize("pieces", [1, 4, 5, 8, 9, 1023, 1024, 1025, 2048, 2049, 5000])
def test_each_way_of_launching(pieces):
    n = pieces * 4096 - 3
    t, out = torch.full((n,), 0.5, device="cuda"), number()
    host = torch.full((n,), 0.5)
    with hc.Comm(1, "ring") as c, c.gradients(dealt=[[t]]) as g:
        size = step.norm([host], 2.0)
        g.norm(out)
        near(out, size)
        g.clip(float(size) / 8, out, eps=0.0)
        near(out, size)
    ref.check(t.cpu(), (torch.full((n,), 0.0625).double(), torch.full((n,), 0.0625).double()), 2, "gradient")


@pytest.mark.parametrize("norm_type", [1.0, 2.0, INF])
def test_a_norm_of_more_than_the_caches_hold(norm_type):
    """300 MB in three types, the norm alone and before clipping: the same bits."""
    lengths = [40000001, 30000000, 29999999, 5]
    held = []
    for i, n in enumerate(lengths):
        t = torch.randn(n, generator=torch.Generator("cuda").manual_seed(i), device="cuda")
        held.append(t.to((F32, BF, F16, F32)[i]))
    alone, before = number(), number()
    size = step.norm([t.cpu() for t in held], norm_type)
    with hc.Comm(4, "ring") as c, c.gradients(dealt=[[t] for t in held]) as g:
        g.norm(alone, norm_type=norm_type)
        near(alone, size)
        g.clip(INF, before, norm_type=norm_type)
    assert torch.equal(alone, before)


def phased(host, rank, whole):
    """One rank's tensors of `host`, type by type packed in a buffer at a place of
    the rank's own in 128 bytes (every third rank's is rank 0's); `whole`: with
    their values.  The tensors, and the check of what lies around them."""
    out, checks = [None] * len(host), []
    for dt in sorted({t.dtype for t in host}, key=str):
        mine = [i for i, t in enumerate(host) if t.dtype == dt]
        total = sum(host[i].numel() for i in mine)
        at = 64 + (5 * rank if rank % 3 else 0)
        flat = torch.full((total + at + 70,), 7, dtype=dt, device="cuda")
        for i, t in zip(mine, flat[at:at + total].split([host[i].numel() for i in mine])):
            t.copy_(host[i]) if whole else t.zero_()
            out[i] = t
        checks.append(lambda flat=flat, at=at, total=total: bool((flat[:at] == 7).all()) and bool((flat[at + total:] == 7).all()))
    return out, lambda: all(ok() for ok in checks)


@pytest.mark.parametrize("norm_type", [2.0, INF])
@pytest.mark.parametrize("P,times", [(1, 1), (2, 1), (2, 2), (11, 1)])
def test_copies_of_thousands_of_pieces(P, times, norm_type):
    """2260 pieces of 16 KiB and twice as many, whose scaling takes the factor from
    a launch of its own; 74 MB written within the caches, 148 and 407 past them; more
    than eight other copies."""
    lengths = [n * times for n in (5000001, 2999999, 1, 2000003, 1500007, 1000, 1499993, 77)]
    host = made(lengths, (BF, F32, F16), 10 * P + times)
    held = [phased(host, r, r == 0) for r in range(P)]
    assert sum(t.numel() * t.element_size() for t in host) > 2048 * 16384 * times
    out = number()
    size = step.norm(host, norm_type, 1.0 / P)
    with hc.Comm(P, "ring") as c, c.gradients(same=[mine for mine, _ in held]) as g:
        g.clip(0.3 * float(size), out, norm_type=norm_type, scale=1.0 / P, eps=0.0)
    near(out, size)
    by = step.factor(size, 0.3 * float(size), 1.0 / P, 0.0)
    for t, h in zip(held[0][0], host):
        v = h.double() * by
        ref.check(t, (v, v.abs()), 2, "gradient")
    for mine, ok in held:
        assert all(torch.equal(a, b) for a, b in zip(mine, held[0][0])) and ok()


@pytest.mark.parametrize("times", [1, 3])
def test_dealt_shares_of_thousands_of_pieces(times):
    """40 MB and 120 MB of random values dealt out, each rank's at a place of its own in 128 bytes."""
    P = 3
    host = made([n * times for n in (4000001, 2222221, 3000000, 1777, 2000003, 1111111)], (F32, BF, F16), times)
    held = [phased(host[r::P], r, True) for r in range(P)]
    out = number()
    size = step.norm(host, 2.0)
    with hc.Comm(P, "ring") as c, c.gradients(dealt=[mine for mine, _ in held]) as g:
        g.clip(0.3 * float(size), out, eps=0.0)
    near(out, size)
    by = step.factor(size, 0.3 * float(size), 1.0, 0.0)
    for r, (mine, ok) in enumerate(held):
        for t, h in zip(mine, host[r::P]):
            v = h.double() * by
            ref.check(t, (v, v.abs()), 2, "gradient")
        assert ok()
