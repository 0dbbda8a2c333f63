"""The operators of a training and a decoding step on the CPU: every refusal of
the C ABI (nothing is launched: each call is refused, or has nothing to do,
before any device work) and of the Python binding, and the test references.
"""
import ctypes
import math
import os
import subprocess
import sys

import pytest
import torch

import allreduce_reduction_amd as hc
import stepops_ref as step

OK, BAD, UNSUPPORTED = 0, 1, 2
L = hc.load_library()
BASE = 1 << 40  # addresses that no call may touch


def ptrs(P, first, step=1 << 20):
    return (ctypes.c_void_p * P)(*[first + r * step for r in range(P)])


@pytest.fixture()
def comm():
    with hc.Comm(4, "ring") as c:
        yield c


# ------------------------------------------------------------------- logits

LISTS = dict(history=10, id_bytes=8, tokens=BASE, length_bytes=4, prompt_lengths=BASE + 4096, lengths=BASE + 8192,
             repetition=BASE + 12288, frequency=BASE + 16384, presence=BASE + 20480, biases=3, bias_id_bytes=8,
             bias_ids=BASE + 24576, bias=BASE + 28672, mask=BASE + 32768)


def logits_call(c, rows=16, vocab=1000, dtype=2, z=None, out=None, **kw):
    m = hc.Logits(rows=rows, vocab=vocab, dtype=dtype, **kw)
    z = ptrs(4, BASE + (1 << 20)) if z is None else z
    return L.hbmc_adjust_logits(c._h, m, z, z if out is None else out, None)


@pytest.mark.parametrize("kw,code", [
    (dict(vocab=0), BAD), (dict(vocab=2 ** 30 + 1), BAD), (dict(rows=2 ** 31), BAD), (dict(rows=2 ** 31 - 1, vocab=2 ** 30), UNSUPPORTED),
    (dict(dtype=3), UNSUPPORTED), (dict(dtype=4), UNSUPPORTED), (dict(dtype=9), BAD), (dict(history=2 ** 19), UNSUPPORTED),
    (dict(biases=4096), UNSUPPORTED), (dict(id_bytes=2), BAD), (dict(length_bytes=1), BAD), (dict(bias_id_bytes=0), BAD),
    (dict(tokens=None), BAD), (dict(tokens=BASE + 4), BAD), (dict(lengths=BASE + 2), BAD), (dict(repetition=BASE + 1), BAD),
    (dict(bias=None), BAD), (dict(bias_ids=None), BAD), (dict(bias_ids=BASE + 4), BAD), (dict(mask=BASE + 1), BAD),
    (dict(history=0), BAD),  # lengths and penalties without tokens
    (dict(rows=2 ** 21), UNSUPPORTED),
])
def test_logits_descriptor(comm, kw, code):
    args = {**LISTS, **kw}
    far = ptrs(4, 1 << 50, 1 << 46)
    assert logits_call(comm, z=far, **args) == code


def test_logits_buffers(comm):
    assert logits_call(comm, rows=0, **LISTS) == OK
    assert logits_call(comm) == OK  # in place, nothing asked
    assert logits_call(comm, history=10, id_bytes=4, tokens=BASE) == OK  # tokens without a penalty
    assert L.hbmc_adjust_logits(None, hc.Logits(rows=1, vocab=1), None, None, None) == BAD
    assert L.hbmc_adjust_logits(comm._h, None, ptrs(4, BASE), ptrs(4, BASE), None) == BAD
    assert L.hbmc_adjust_logits(comm._h, hc.Logits(rows=1, vocab=4, dtype=0), None, ptrs(4, BASE), None) == BAD
    z = ptrs(4, BASE + (1 << 20))
    mixed = ptrs(4, BASE + (1 << 20))
    mixed[2] = BASE + (30 << 20)  # in place on some ranks alone
    assert logits_call(comm, z=z, out=mixed, **LISTS) == BAD
    assert logits_call(comm, z=z, out=ptrs(4, BASE + (1 << 20) + 2), **LISTS) == BAD
    assert logits_call(comm, z=z, out=ptrs(4, BASE + (10 << 20), 64), **LISTS) == BAD
    null = ptrs(4, BASE + (1 << 20))
    null[1] = None
    assert logits_call(comm, z=null, out=ptrs(4, BASE + (10 << 20)), **LISTS) == BAD
    for name, size in (("tokens", 16 * 80), ("lengths", 64), ("repetition", 64), ("bias", 192), ("mask", 16 * 128)):
        assert logits_call(comm, z=ptrs(4, BASE + (1 << 20) - size + 8), **{**LISTS, name: BASE + (1 << 20) - size + 16}) == BAD


# ----------------------------------------------------------------- products


def product_call(c, rows=16, inner=64, channels=32, dtype=2, form=0, **kw):
    a = dict(x=ptrs(4, BASE), xs=BASE + (8 << 20), w=ptrs(4, BASE + (10 << 20)), ws=ptrs(4, BASE + (20 << 20)),
             out=ptrs(4, BASE + (30 << 20)))
    a.update(kw)
    return L.hbmc_product(c._h, hc.Product(rows, inner, channels, dtype, form), a["x"], a["xs"], a["w"], a["ws"], a["out"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(inner=0), BAD), (dict(channels=0), BAD), (dict(rows=2 ** 31), BAD), (dict(channels=2 ** 31), BAD),
    (dict(inner=131072), UNSUPPORTED), (dict(dtype=3), UNSUPPORTED), (dict(dtype=4), UNSUPPORTED), (dict(dtype=7), BAD),
    (dict(form=-1), BAD), (dict(form=4), BAD), (dict(x=None), BAD), (dict(w=None), BAD), (dict(ws=None), BAD), (dict(out=None), BAD),
    (dict(xs=None), BAD), (dict(xs=BASE + (8 << 20) + 1), BAD), (dict(out=ptrs(4, BASE + (30 << 20) + 1)), BAD),
    (dict(out=ptrs(4, BASE)), BAD), (dict(out=ptrs(4, BASE + (30 << 20), 16)), BAD), (dict(ws=ptrs(4, BASE + (20 << 20) + 2)), BAD),
])
def test_product_refusals(comm, kw, code):
    assert product_call(comm, **kw) == code


def test_product_sizes_past_a_launch(comm):
    far = dict(x=ptrs(4, 1 << 50, 1 << 46), w=ptrs(4, 1 << 51, 1 << 46), ws=ptrs(4, 1 << 52, 1 << 46), out=ptrs(4, 1 << 53, 1 << 48),
               xs=1 << 54)
    assert product_call(comm, rows=2 ** 20, channels=2 ** 20, form=2, **far) == UNSUPPORTED
    assert product_call(comm, rows=0) == OK
    assert L.hbmc_product(None, hc.Product(1, 1, 1, 2, 0), None, None, None, None, None, None) == BAD
    assert L.hbmc_product(comm._h, None, None, None, None, None, None, None) == BAD


def test_quantize_refusals(comm):
    call = lambda rows=4, width=64, dtype=2, x=ptrs(4, BASE), q=ptrs(4, BASE + (8 << 20)), s=BASE + (16 << 20), c=comm: (  # noqa: E731
        L.hbmc_quantize_rows(c._h if c else None, rows, width, dtype, x, q, s, None))
    assert call(rows=0) == OK
    assert call(c=None) == BAD
    for kw in (dict(width=0), dict(rows=2 ** 31), dict(width=2 ** 31), dict(x=None), dict(q=None), dict(s=None), dict(s=BASE + (16 << 20) + 2),
               dict(x=ptrs(4, BASE + 1)), dict(q=ptrs(4, BASE + 2)), dict(q=ptrs(4, BASE + (8 << 20), 8)), dict(dtype=-3)):
        assert call(**kw) == BAD, kw
    assert call(dtype=3) == UNSUPPORTED and call(dtype=4) == UNSUPPORTED


# ---------------------------------------------------------------- gradients


def gradient(count=16, dtype=0, copies=1, first=BASE, step=1 << 20):
    return hc.Gradient(count, dtype, copies, ptrs(max(copies, 1), first, step))


@pytest.mark.parametrize("tensors,code", [
    ([gradient(dtype=3)], UNSUPPORTED), ([gradient(dtype=4)], UNSUPPORTED), ([gradient(dtype=9)], BAD), ([gradient(copies=2)], BAD),
    ([gradient(copies=0)], BAD), ([gradient(count=2 ** 62)], BAD), ([gradient(first=BASE + 2)], BAD), ([gradient(first=0)], BAD),
    ([gradient(), gradient(first=BASE + 60)], BAD), ([gradient(copies=4, step=32)], BAD), ([gradient(), gradient()], BAD),
    ([hc.Gradient(4, 0, 1, None)], BAD),
])
def test_gradient_tables(comm, tensors, code):
    out = ctypes.c_void_p(1)
    assert L.hbmc_gradients_create(comm._h, len(tensors), (hc.Gradient * len(tensors))(*tensors), ctypes.byref(out)) == code
    assert out.value is None


def test_gradient_handles(comm):
    out = ctypes.c_void_p()
    assert L.hbmc_gradients_create(None, 0, None, ctypes.byref(out)) == BAD
    assert L.hbmc_gradients_create(comm._h, 1, None, ctypes.byref(out)) == BAD
    assert L.hbmc_gradients_create(comm._h, 0, None, None) == BAD
    assert L.hbmc_gradients_destroy(None) == BAD
    n = ctypes.c_size_t()
    assert L.hbmc_gradients_workspace(None, ctypes.byref(n)) == BAD
    assert L.hbmc_gradients_norm(None, 2.0, 1.0, BASE, None, 0, None) == BAD
    assert L.hbmc_gradients_clip(None, 2.0, 1.0, 1.0, 0.0, BASE, None, 0, None) == BAD


# ------------------------------------------------------------------- Python


def test_python_refuses_host_tensors(comm):
    z = [torch.zeros(2, 3) for _ in range(4)]
    q = [t.to(torch.int8) for t in z]
    s = torch.zeros(2)
    with pytest.raises((ValueError, RuntimeError, AssertionError)):
        comm.adjust_logits(z)
    with pytest.raises((ValueError, RuntimeError, AssertionError)):
        comm.quantize_rows(z, q, s)
    with pytest.raises((ValueError, RuntimeError, AssertionError)):
        comm.product(q, s, q, [s] * 4, z)
    with pytest.raises((ValueError, RuntimeError, AssertionError)):
        comm.gradients(dealt=[[t] for t in z])


# --------------------------------------------------------------- references


def test_reference_masks_round_trip():
    on = torch.rand(5, 77) < 0.5
    assert torch.equal(step.allowed(step.bits(on), 77), on)


def test_reference_penalties_by_hand():
    z, _ = step.adjust(torch.tensor([[2.0, -2.0, 1.0, 0.0]]), tokens=torch.tensor([[0, 1, 1, 3, 9]]), prompt_lengths=[1], lengths=[4],
                       repetition=[2.0], frequency=[0.5], presence=[0.25], bias_ids=torch.tensor([[2, 2, -1]]),
                       bias=torch.tensor([[1.0, 2.0, 9.0]]), mask=torch.tensor([[0b0111]], dtype=torch.int32))
    assert z.tolist() == [[1.0, -4.0 - 1.0 - 0.25, 4.0, -math.inf]]


def test_reference_norms_by_hand():
    t = [torch.tensor([3.0, -4.0]), torch.tensor([12.0])]
    assert [float(step.norm(t, p, -2.0)) for p in (1.0, 2.0, math.inf)] == [38.0, 26.0, 24.0]
    assert step.factor(10.0, 5.0, 3.0, 0.0) == 1.5 and step.factor(1.0, 5.0, 3.0) == 3.0


def test_reference_codes_by_hand():
    q, s = step.codes(torch.tensor([[127.0, -63.0, 0.4], [0.0, 0.0, 0.0], [1.0, math.nan, 0.0]]))
    assert q.tolist() == [[127, -63, 0], [0, 0, 0], [0, 0, 0]] and s[:2].tolist() == [1.0, 0.0] and bool(s[2].isnan())


# ------------------------------------------- limits met before memory is used

LIMIT = """
import ctypes, resource, sys
import allreduce_reduction_amd as hc
L = hc.load_library()
comm = hc.Comm(4, "ring")
used = int(open("/proc/self/statm").read().split()[0]) * resource.getpagesize()
resource.setrlimit(resource.RLIMIT_AS, (used + (64 << 20), -1))
table = (hc.Gradient * 2)()
counts = [int(n) for n in sys.argv[1].split(",")]
for i, n in enumerate(counts):
    table[i] = hc.Gradient(n, 0, 1, (ctypes.c_void_p * 1)((i + 1) << 50))
out = ctypes.c_void_p()
print(L.hbmc_gradients_create(comm._h, len(counts), table, ctypes.byref(out)), out.value)
"""


@pytest.mark.parametrize("counts", [[2 ** 45], [2 ** 35 + 1], [4096, 2 ** 35 - 4095], [2 ** 47, 1]])
def test_too_many_pieces_are_refused_before_they_are_made(counts):
    """2^35 fp32 elements are the 2^23 pieces of 16 KiB that a handle holds; with 64
    MiB more of memory than the library needs there is no room for their table."""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", LIMIT, ",".join(map(str, counts))], cwd=root, capture_output=True, text=True, timeout=100)
    assert r.stdout.split() == [str(UNSUPPORTED), "None"], (r.stdout, r.stderr)
