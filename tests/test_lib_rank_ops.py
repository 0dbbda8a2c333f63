"""The row operators over the ranks on the CPU: every refusal of the C ABI
(nothing is launched: each call is refused, or has nothing to do, before any
device work), of the Python binding, and the test references' gradients
against differences.
"""
import ctypes

import pytest
import torch

import allreduce_reduction_amd as hc
import rankops_ref as ref

OK, BAD, UNSUPPORTED = 0, 1, 2
L = hc.load_library()
BASE = 1 << 40  # addresses that no call may touch


def ptrs(P, first, step):
    return (ctypes.c_void_p * P)(*[first + r * step for r in range(P)])


@pytest.fixture()
def comm():
    with hc.Comm(4, "ring") as c:
        yield c


def norm_args(rows=16, width=64, **kw):
    d = dict(rows=rows, width=width, gate_rows=1, dtype=2, scale=1.0, pre_eps=1e-6, post_eps=1e-6, pre_weight=BASE,
             post_weight=BASE + 4096, gate=None)
    d.update(kw)
    return hc.Norm(**d)


def norm_call(c, n, **kw):
    a = dict(parts=ptrs(4, BASE + (1 << 20), 1 << 20), residual=ptrs(4, BASE + (8 << 20), 1 << 20),
             residual_out=ptrs(4, BASE + (16 << 20), 1 << 20), out=ptrs(4, BASE + (24 << 20), 1 << 20), sums=None)
    a.update(kw)
    return L.hbmc_reduce_norm(c._h, n, a["parts"], a["residual"], a["residual_out"], a["out"], a["sums"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(width=0), BAD), (dict(width=16385), UNSUPPORTED), (dict(rows=2 ** 31), BAD), (dict(rows=2 ** 62, width=8), BAD),
    (dict(dtype=3), UNSUPPORTED), (dict(dtype=4), UNSUPPORTED), (dict(dtype=5), BAD), (dict(dtype=-1), BAD),
    (dict(scale=float("nan")), BAD), (dict(scale=float("inf")), BAD), (dict(pre_eps=-1.0), BAD),
    (dict(post_eps=float("nan")), BAD), (dict(pre_weight=None), BAD), (dict(gate=BASE + 8192, gate_rows=0), BAD),
    (dict(pre_weight=BASE + 1), BAD), (dict(gate=BASE + 8193), BAD),
])
def test_norm_descriptor(comm, kw, code):
    assert norm_call(comm, norm_args(**kw)) == code
    n = ctypes.c_size_t()
    if kw.get("pre_weight") != BASE + 1 and kw.get("gate") != BASE + 8193:  # the workspace call reads no address
        assert L.hbmc_reduce_norm_grad_workspace(comm._h, norm_args(**kw), ctypes.byref(n)) == code


def test_norm_buffers(comm):
    n = norm_args()
    assert norm_call(comm, norm_args(rows=0)) == OK
    assert L.hbmc_reduce_norm(None, n, None, None, None, None, None, None) == BAD
    assert norm_call(comm, None) == BAD
    for name in ("parts", "residual", "residual_out", "out"):
        assert norm_call(comm, n, **{name: None}) == BAD
        null = ptrs(4, BASE + (40 << 20), 1 << 20)
        null[2] = None
        assert norm_call(comm, n, **{name: null}) == BAD
        odd = ptrs(4, BASE + (40 << 20) + 1, 1 << 20)
        assert norm_call(comm, n, **{name: odd}) == BAD
    parts = ptrs(4, BASE + (1 << 20), 1 << 20)
    assert norm_call(comm, n, out=ptrs(4, BASE + (1 << 20) + 2, 1 << 20)) == BAD       # overlaps parts partly
    swapped = (ctypes.c_void_p * 4)(parts[1], parts[0], parts[2], parts[3])
    assert norm_call(comm, n, out=swapped) == BAD                                     # another rank's input
    assert norm_call(comm, n, residual_out=ptrs(4, BASE + (24 << 20), 1 << 20)) == BAD  # an output
    assert norm_call(comm, n, sums=ptrs(4, BASE + (16 << 20) + 64, 1 << 20)) == BAD
    assert norm_call(comm, n, out=ptrs(4, BASE + (24 << 20), 64)) == BAD              # outputs of two ranks
    wrap = ptrs(4, BASE + (24 << 20), 1 << 20)
    wrap[3] = 2 ** 64 - 64
    assert norm_call(comm, n, out=wrap) == BAD


def grad_call(c, n, bytes_=1 << 30, **kw):
    a = dict(out_grads=ptrs(4, BASE + (1 << 20), 1 << 20), hidden=ptrs(4, BASE + (8 << 20), 1 << 20),
             sums=ptrs(4, BASE + (16 << 20), 1 << 20), rin=None, parts=ptrs(4, BASE + (24 << 20), 1 << 20),
             res=ptrs(4, BASE + (32 << 20), 1 << 20), pre=BASE + (40 << 20), post=BASE + (41 << 20), gate=None,
             ws=BASE + (1 << 31))
    a.update(kw)
    return L.hbmc_reduce_norm_grad(c._h, n, a["out_grads"], a["hidden"], a["sums"], a["rin"], a["parts"], a["res"], a["pre"],
                                   a["post"], a["gate"], a["ws"], bytes_, None)


def test_norm_gradient_buffers(comm):
    n, need = norm_args(), ctypes.c_size_t()
    assert L.hbmc_reduce_norm_grad_workspace(comm._h, n, None) == BAD
    assert L.hbmc_reduce_norm_grad_workspace(comm._h, n, ctypes.byref(need)) == OK and need.value > 0
    assert grad_call(comm, n, need.value - 1) == BAD
    assert grad_call(comm, n, ws=None) == BAD
    assert grad_call(comm, n, ws=BASE + (1 << 31) + 4) == BAD
    assert grad_call(comm, n, ws=BASE + (1 << 20)) == BAD
    for name in ("out_grads", "hidden", "sums", "parts", "res", "pre", "post"):
        assert grad_call(comm, n, **{name: None}) == BAD
    assert grad_call(comm, n, gate=BASE + (42 << 20)) == BAD            # no gate
    assert grad_call(comm, norm_args(gate=BASE + 8192)) == BAD          # no gate_grad
    assert grad_call(comm, norm_args(post_weight=None)) == BAD          # post_weight_grad without one
    assert grad_call(comm, n, pre=BASE + (41 << 20) + 64) == BAD        # pre and post overlap
    assert grad_call(comm, n, rin=ptrs(4, BASE + (32 << 20) + 2, 1 << 20)) == BAD
    assert grad_call(comm, n, parts=ptrs(4, BASE + (8 << 20), 1 << 20)) == BAD


def emb_args(**kw):
    d = dict(vocab=100, width=64, dtype=2, id_bytes=8, scale=1.0)
    d.update(kw)
    return hc.Embedding(**d)


def emb_call(c, e, tokens=(4, 4, 4, 4), **kw):
    a = dict(tables=ptrs(4, BASE + (1 << 20), 1 << 20), ids=ptrs(4, BASE + (8 << 20), 1 << 20),
             out=ptrs(4, BASE + (16 << 20), 1 << 20))
    a.update(kw)
    t = (ctypes.c_size_t * 4)(*tokens) if tokens else None
    return L.hbmc_embedding(c._h, e, a["tables"], a["ids"], t, a["out"], None)


def emb_grad_call(c, e, tokens=(4, 4, 4, 4), gd=0, acc=0, ws=BASE + (1 << 31), bytes_=1 << 30, **kw):
    a = dict(grads=ptrs(4, BASE + (1 << 20), 1 << 20), ids=ptrs(4, BASE + (8 << 20), 1 << 20),
             table=ptrs(4, BASE + (16 << 20), 1 << 20))
    a.update(kw)
    t = (ctypes.c_size_t * 4)(*tokens) if tokens else None
    return L.hbmc_embedding_grad(c._h, e, a["grads"], a["ids"], t, a["table"], gd, acc, ws, bytes_, None)


@pytest.mark.parametrize("kw,code", [
    (dict(vocab=0), BAD), (dict(vocab=2 ** 30 + 1), BAD), (dict(width=0), BAD), (dict(width=2 ** 24 + 1), BAD),
    (dict(dtype=3), UNSUPPORTED), (dict(dtype=9), BAD), (dict(id_bytes=2), BAD), (dict(scale=float("nan")), BAD),
])
def test_embedding_descriptor(comm, kw, code):
    assert emb_call(comm, emb_args(**kw)) == code
    assert emb_grad_call(comm, emb_args(**kw)) == code


def test_embedding_buffers(comm):
    e = emb_args()
    assert emb_call(comm, e, (0, 0, 0, 0), ids=ptrs(4, 0, 0), out=ptrs(4, 0, 0)) == OK
    assert emb_call(comm, e, None) == BAD and emb_call(comm, None) == BAD
    assert emb_call(comm, e, (4, 4, 4, 2 ** 26)) == BAD
    for name in ("tables", "ids", "out"):
        assert emb_call(comm, e, **{name: None}) == BAD
        assert emb_call(comm, e, **{name: ptrs(4, BASE + (40 << 20) + 1, 1 << 20)}) == BAD
        assert emb_call(comm, e, **{name: ptrs(4, 0, 0)}) == BAD
    assert emb_call(comm, e, ids=ptrs(4, BASE + (8 << 20) + 4, 1 << 20)) == BAD  # 8-byte ids
    assert emb_call(comm, e, out=ptrs(4, BASE + (1 << 20), 1 << 20)) == BAD
    assert emb_call(comm, e, out=ptrs(4, BASE + (16 << 20), 256)) == BAD
    for name in ("grads", "ids", "table"):
        assert emb_grad_call(comm, e, **{name: None}) == BAD
        assert emb_grad_call(comm, e, **{name: ptrs(4, BASE + (40 << 20) + 1, 1 << 20)}) == BAD
    assert emb_grad_call(comm, e, gd=1) == BAD and emb_grad_call(comm, e, gd=3) == BAD
    assert emb_grad_call(comm, e, table=ptrs(4, BASE + (1 << 20), 1 << 20)) == BAD
    assert emb_grad_call(comm, e, table=ptrs(4, BASE + (16 << 20), 25 * 64 * 2)) == BAD  # overlap in fp32
    need = ctypes.c_size_t()
    few = (ctypes.c_size_t * 4)(256, 256, 256, 256)  # needs none
    assert L.hbmc_embedding_grad_workspace(comm._h, e, few, ctypes.byref(need)) == OK and need.value == 0
    many = (400, 0, 400, 400)
    t = (ctypes.c_size_t * 4)(*many)
    assert L.hbmc_embedding_grad_workspace(comm._h, e, t, ctypes.byref(need)) == OK and need.value > 0
    assert L.hbmc_embedding_grad_workspace(comm._h, e, t, None) == BAD
    assert L.hbmc_embedding_grad_workspace(comm._h, e, None, ctypes.byref(need)) == BAD
    assert emb_grad_call(comm, e, many, bytes_=need.value - 1) == BAD
    assert emb_grad_call(comm, e, many, ws=None) == BAD and emb_grad_call(comm, e, many, ws=BASE + (1 << 31) + 8) == BAD
    assert emb_grad_call(comm, e, (0, 0, 0, 0), acc=1, table=ptrs(4, BASE + (16 << 20), 1 << 20)) == OK  # nothing to add


@pytest.mark.parametrize("width,dtype,pieces", [(1, 2, 1), (7, 1, 1), (512, 2, 1), (513, 2, 2), (1200, 1, 3), (1024, 0, 4),
                                                (4096, 2, 8)])
def test_embedding_gradient_limit(width, dtype, pieces):
    """A launch takes fewer than 2^32 threads, and the joining one has 256 for
    each 64 tokens and piece of a row (64 vectors of 16 bytes): tokens times
    pieces past 2^30 are refused, before anything is launched."""
    limit, need = 2 ** 30 // pieces, ctypes.c_size_t()
    none = ptrs(64, 0, 0)
    with hc.Comm(64, "ring") as c:
        def counts(total):
            return (ctypes.c_size_t * 64)(*[total // 64 + (r < total % 64) for r in range(64)])
        e = emb_args(width=width, dtype=dtype)
        assert L.hbmc_embedding_grad_workspace(c._h, e, counts(limit), ctypes.byref(need)) == OK and need.value > 16 * limit
        assert (-(-limit // 64) - 1) * pieces < 2 ** 24
        for total in (limit + 1, min(2 * limit, 2 ** 31 - 1)):
            assert L.hbmc_embedding_grad_workspace(c._h, e, counts(total), ctypes.byref(need)) == UNSUPPORTED, total
            assert L.hbmc_embedding_grad(c._h, e, none, none, counts(total), none, 0, 0, None, 0, None) == UNSUPPORTED, total
            assert L.hbmc_embedding(c._h, e, none, none, counts(total), none, None) == BAD  # the lookup takes them: NULLs


def distill_args(**kw):
    d = dict(rows=4, vocab=100, top=8, dtype=2, teacher_dtype=0, id_bytes=8, temperature=1.0, teacher_logits=BASE,
             teacher_ids=BASE + 65536)
    d.update(kw)
    return hc.Distill(**d)


def distill_call(c, d, loss=BASE + (40 << 20), lse=BASE + (41 << 20), ws=BASE + (1 << 31), bytes_=1 << 30, **kw):
    logits = kw.get("logits", ptrs(4, BASE + (1 << 20), 1 << 20))
    return L.hbmc_distill_loss(c._h, d, logits, loss, lse, ws, bytes_, None)


def distill_grad_call(c, d, lse=BASE + (40 << 20), dl=BASE + (41 << 20), **kw):
    logits = kw.get("logits", ptrs(4, BASE + (1 << 20), 1 << 20))
    return L.hbmc_distill_loss_grad(c._h, d, logits, lse, dl, kw.get("grads", ptrs(4, BASE + (8 << 20), 1 << 20)), None)


@pytest.mark.parametrize("kw,code", [
    (dict(vocab=0), BAD), (dict(vocab=2 ** 30 + 1), BAD), (dict(top=0), BAD), (dict(top=1025), UNSUPPORTED),
    (dict(dtype=3), UNSUPPORTED), (dict(teacher_dtype=4), UNSUPPORTED), (dict(dtype=7), BAD), (dict(teacher_dtype=-1), BAD),
    (dict(id_bytes=1), BAD), (dict(temperature=0.0), BAD), (dict(temperature=-1.0), BAD),
    (dict(temperature=1e-39), BAD), (dict(temperature=1e20), BAD), (dict(temperature=float("nan")), BAD), (dict(temperature=float("inf")), BAD), (dict(rows=2 ** 31), BAD),
    (dict(teacher_logits=None), BAD), (dict(teacher_ids=None), BAD), (dict(teacher_ids=BASE + 65540), BAD),
    (dict(teacher_logits=BASE + 2), BAD),
])
def test_distill_descriptor(comm, kw, code):
    assert distill_call(comm, distill_args(**kw)) == code
    assert distill_grad_call(comm, distill_args(**kw)) == code


@pytest.mark.parametrize("temperature,code", [(1e-39, BAD), (2.95e-39, BAD), (4.2e-39, BAD), (4.3e-39, OK), (1e-30, OK), (1e19, OK),
                                              (1.9e19, BAD)])
def test_distill_temperatures(comm, temperature, code):
    """The kernels multiply by log2(e) / temperature, which has to be finite."""
    d = distill_args(rows=0, teacher_logits=None, teacher_ids=None, temperature=temperature)
    assert distill_call(comm, d, loss=None, lse=None, ws=None, bytes_=0, logits=ptrs(4, 0, 0)) == code
    assert distill_grad_call(comm, d, lse=None, dl=None, logits=ptrs(4, 0, 0), grads=ptrs(4, 0, 0)) == code
    assert L.hbmc_distill_loss_workspace(comm._h, d, ctypes.byref(ctypes.c_size_t())) == code


def test_distill_buffers(comm):
    d = distill_args()
    assert distill_call(comm, distill_args(rows=0, teacher_logits=None, teacher_ids=None), loss=None, lse=None, ws=None,
                        bytes_=0, logits=ptrs(4, 0, 0)) == OK
    assert distill_call(comm, None) == BAD and distill_grad_call(comm, None) == BAD
    for kw in (dict(loss=None), dict(lse=None), dict(logits=None), dict(logits=ptrs(4, 0, 0)),
               dict(lse=BASE + (40 << 20) + 4), dict(loss=BASE + (1 << 20)), dict(loss=BASE + (39 << 20) + 2)):
        assert distill_call(comm, d, **kw) == BAD, kw
    need = ctypes.c_size_t(1)
    assert L.hbmc_distill_loss_workspace(comm._h, d, ctypes.byref(need)) == OK and need.value == 0  # one launch
    assert L.hbmc_distill_loss_workspace(comm._h, d, None) == BAD
    many = distill_args(rows=5000, teacher_logits=BASE + (50 << 20), teacher_ids=BASE + (60 << 20))
    assert L.hbmc_distill_loss_workspace(comm._h, many, ctypes.byref(need)) == OK and need.value > 0
    for kw in (dict(bytes_=need.value - 1), dict(ws=None), dict(ws=BASE + (1 << 31) + 4), dict(ws=BASE + (1 << 20))):
        assert distill_call(comm, many, **kw) == BAD, kw
    for kw in (dict(lse=None), dict(dl=None), dict(grads=None), dict(logits=None), dict(grads=ptrs(4, 0, 0)),
               dict(grads=ptrs(4, BASE + (1 << 20) + 2, 1 << 20)), dict(grads=ptrs(4, BASE + (8 << 20), 64)),
               dict(dl=BASE + (8 << 20))):
        assert distill_grad_call(comm, d, **kw) == BAD, kw


def test_more_ranks_than_columns():
    """Ranks that own nothing pass NULL."""
    with hc.Comm(4, "ring") as c:
        d = distill_args(vocab=2, rows=0)
        assert distill_grad_call(c, d, logits=ptrs(4, 0, 0), grads=ptrs(4, 0, 0)) == OK


# ------------------------------------------------------- the Python binding


@pytest.fixture()
def on_device(monkeypatch):
    """Host tensors stand in for device ones; calls that pass the checks must
    not be made, except where the library itself refuses them."""
    monkeypatch.setattr(hc, "_current_device", lambda: -1)
    monkeypatch.setattr(hc, "_stream", lambda stream: 0)


def one(shape, dtype=torch.bfloat16, contiguous=True):
    if not contiguous:
        return torch.zeros(shape[:-1] + (2 * shape[-1],), dtype=dtype)[..., ::2]
    return torch.zeros(shape, dtype=dtype)


Fake = one


def fakes(n, shape, at=1, **kw):
    return [one(shape, **kw) for _ in range(n)]


def norm_binding(c, **kw):
    a = dict(parts=fakes(4, (8, 16)), residual=fakes(4, (2, 16), 10), out=fakes(4, (8, 16), 20), pre_weight=Fake((16,)))
    a.update(kw)
    c.reduce_norm(a.pop("parts"), a.pop("residual"), a.pop("out"), a.pop("pre_weight"), **a)


@pytest.mark.parametrize("kw", [
    dict(parts=fakes(3, (8, 16))), dict(parts=fakes(4, (8, 16), contiguous=False)),
    dict(parts=fakes(4, (8, 16, 1))), dict(parts=[]), dict(residual=fakes(4, (8, 16), 10)),
    dict(residual=fakes(4, (2, 16), 10, dtype=torch.float16)), dict(out=fakes(4, (8, 15), 20)), dict(pre_weight=Fake((15,))),
    dict(pre_weight=Fake((16,), torch.float32)), dict(gate=Fake((3, 16))), dict(gate=Fake((0, 16))), dict(gate=Fake((16,))), dict(gate=Fake((2, 8))),
    dict(post_weight=Fake((16,), contiguous=False)), dict(sums=fakes(4, (8, 16), 30)), dict(residual_out=fakes(2, (2, 16), 30)),
])
def test_norm_binding_refuses(comm, on_device, kw):
    with pytest.raises(ValueError):
        norm_binding(comm, **kw)


def test_binding_types(comm, on_device):
    for dt in (torch.int32, torch.float64):
        with pytest.raises(TypeError):
            norm_binding(comm, parts=fakes(4, (8, 16), dtype=dt))
    for bad in (3, "abcd", None, [1, 2, 3, 4], iter(())):
        with pytest.raises(TypeError):
            norm_binding(comm, parts=bad)
    with pytest.raises(TypeError):
        norm_binding(comm, scale="x")
    with pytest.raises(ValueError):
        norm_binding(comm, parts=Fake((3, 8, 16)))
    with pytest.raises(TypeError):  # one tensor cannot hold segments of unequal length
        norm_binding(comm, parts=fakes(4, (7, 16)), out=fakes(4, (7, 16)), residual=Fake((4, 2, 16)))
    parts = fakes(4, (8, 16))
    with pytest.raises(hc.HbmcError) as e:  # out over the ranks' inputs in another order
        norm_binding(comm, parts=parts, out=parts[::-1])
    assert e.value.code == BAD


def test_closed_communicator(on_device):
    """As with the collectives: the library's refusal, not a conversion's."""
    c = hc.Comm(4, "ring")
    c.close()
    for call in (lambda: norm_binding(c), lambda: c.embedding(fakes(4, (5, 16)), fakes(4, (3,), dtype=torch.int64), fakes(4, (3, 16)))):
        with pytest.raises(hc.HbmcError) as e:
            call()
        assert e.value.code == BAD


def test_norm_gradient_binding_refuses(comm, on_device):
    def call(**kw):
        a = dict(out_grads=fakes(4, (8, 16)), hidden=fakes(4, (2, 16), 10), part_grads=fakes(4, (8, 16), 20),
                 residual_grad=fakes(4, (2, 16), 30), pre_weight=Fake((16,)),
                 pre_weight_grad=Fake((16,), torch.float32))
        a.update(kw)
        comm.reduce_norm_grad(*[a.pop(n) for n in ("out_grads", "hidden", "part_grads", "residual_grad", "pre_weight",
                                                   "pre_weight_grad")], **a)
    w, wg = Fake((16,)), Fake((16,), torch.float32)
    for kw in (dict(post_weight=w), dict(post_weight_grad=wg), dict(post_weight=w, post_weight_grad=wg),
               dict(gate=Fake((1, 16))), dict(pre_weight_grad=Fake((16,))), dict(hidden=fakes(4, (3, 16), 10)),
               dict(residual_grad_in=fakes(4, (2, 15), 40)), dict(part_grads=fakes(4, (7, 16), 20))):
        with pytest.raises(ValueError):
            call(**kw)


def test_embedding_binding_refuses(comm, on_device):
    def call(fn="embedding", **kw):
        a = dict(tables=fakes(4, (5, 16)), ids=fakes(4, (3,), 10, dtype=torch.int64), out=fakes(4, (3, 16), 20))
        a.update(kw)
        if fn == "embedding":
            comm.embedding(a["tables"], a["ids"], a["out"])
        else:
            comm.embedding_grad(a["out"], a["ids"], a["tables"])
    for fn in ("embedding", "embedding_grad"):
        for kw in (dict(tables=fakes(4, (5,))), dict(tables=fakes(3, (5, 16)) + fakes(1, (6, 16), 5)), dict(tables=[]),
                   dict(ids=fakes(3, (3,), 10, dtype=torch.int64)), dict(ids=fakes(4, (3, 1), 10, dtype=torch.int64)),
                   dict(out=fakes(4, (4, 16), 20)), dict(out=fakes(4, (3, 17), 20))):
            with pytest.raises(ValueError):
                call(fn, **kw)
        with pytest.raises(TypeError):
            call(fn, ids=fakes(4, (3,), 10, dtype=torch.int16))
    with pytest.raises(ValueError):
        call(out=fakes(4, (3, 16), 20, dtype=torch.float16))
    with pytest.raises(TypeError):
        call("embedding_grad", tables=fakes(4, (5, 16), dtype=torch.float16))


def test_distill_binding_refuses(comm, on_device):
    f32 = torch.float32

    def call(fn="loss", **kw):
        a = dict(logits=fakes(4, (3, 5)), t=Fake((3, 2), f32), ids=Fake((3, 2), torch.int64), one=Fake((3,), f32),
                 two=Fake((3,), f32), grads=fakes(4, (3, 5), 10), temperature=1.0)
        a.update(kw)
        if fn == "loss":
            comm.distill_loss(a["logits"], a["t"], a["ids"], a["one"], a["two"], temperature=a["temperature"])
        else:
            comm.distill_loss_grad(a["logits"], a["t"], a["ids"], a["one"], a["two"], a["grads"], temperature=a["temperature"])
    for fn in ("loss", "grad"):
        for kw in (dict(logits=fakes(4, (4, 5))), dict(logits=fakes(3, (3, 5)) + fakes(1, (3, 6), 9)), dict(logits=fakes(4, (3,))),
                   dict(t=Fake((3,), f32)), dict(t=Fake((3, 3), f32)), dict(ids=Fake((4, 2), torch.int64)),
                   dict(one=Fake((4,), f32)), dict(two=Fake((3,), torch.bfloat16)), dict(one=Fake((3,), f32, contiguous=False))):
            with pytest.raises(ValueError):
                call(fn, **kw)
        for kw in (dict(t=Fake((3, 2), torch.int32)), dict(ids=Fake((3, 2), f32))):
            with pytest.raises(TypeError):
                call(fn, **kw)
    with pytest.raises(ValueError):
        call("grad", grads=fakes(4, (3, 4), 10))
    with pytest.raises(hc.HbmcError):
        call("grad", temperature=0.0)


def test_host_tensors_never_reach_the_library(comm, monkeypatch):
    monkeypatch.setattr(hc, "_current_device", lambda: 0)
    monkeypatch.setattr(hc, "_stream", lambda stream: 0)
    host = fakes(4, (8, 16))
    with pytest.raises(ValueError, match="on device 0 is needed"):
        comm.reduce_norm(host, [t[:2] for t in host], host, torch.ones(16, dtype=torch.bfloat16))
    with pytest.raises(ValueError, match="on device 0 is needed"):
        comm.embedding(host, [torch.zeros(1, dtype=torch.int64)] * 4, [t[:1] for t in host])
    with pytest.raises(ValueError, match="on device 0 is needed"):
        comm.distill_loss(host, Fake((8, 2)), Fake((8, 2), torch.int64), Fake((8,), torch.float32), Fake((8,), torch.float32))


# ------------------------------------------- the references' own gradients


def test_reference_gradients():
    """The formulas of the norm's and the loss's gradients against automatic
    differentiation of the forward formulas, in 64 bits (rounding: 1e-11)."""
    g = torch.Generator().manual_seed(0)
    rnd = lambda *s: torch.randn(*s, generator=g).double()  # noqa: E731
    for post, groups in ((True, 2), (False, 2), (True, 0), (False, 0)):
        v = {"parts": rnd(3, 4, 10), "residual": rnd(4, 10), "pre": rnd(10)}
        if post:
            v["post"] = rnd(10)
        if groups:
            v["gate"] = rnd(groups, 10)
        for t in v.values():
            t.requires_grad_()
        f = ref.norm_forward(v["parts"], v["residual"], v["pre"], v.get("post"), v.get("gate"), 2, 0.7, 1e-3, 1e-2)
        wo, wr = rnd(3, 4, 10), rnd(4, 10)
        ((f["out"][0] * wo.sum(0)).sum() + (f["residual"][0] * wr).sum()).backward()
        d = {k: t.detach() for k, t in v.items()}
        b = ref.norm_backward(wo, f["residual"][0].detach(), d["pre"], f["sums"][0].detach(), wr, d.get("post"), d.get("gate"), 2,
                              0.7, 1e-3, 1e-2)
        for name, t in v.items():
            want = t.grad[0] if name == "parts" else t.grad
            assert (b[name][0] - want).abs().max() < 1e-11, name
    z, t, ids, dl = rnd(5, 40).requires_grad_(), rnd(5, 6), torch.randint(-1, 40, (5, 6), generator=g), rnd(5)
    ids[1, 3] = ids[1, 2]
    ids[2] = -1
    (ref.distill_forward(z, t, ids, 1.7)["loss"][0] * dl).sum().backward()
    assert (ref.distill_backward(z.detach(), t, ids, 1.7, dl)[0] - z.grad).abs().max() < 1e-11
