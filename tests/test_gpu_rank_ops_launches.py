"""The operators' forms of several launches, which keep something in a
workspace between them: the embedding gradient's sort, sums and joining, the
distillation loss of many rows, the norms' gradient.  Captured and replayed, on
several streams at once, with guard zones around every buffer and workspace,
over tables past 2^32 bytes and more tokens than one rank may have.
"""
import ctypes

import pytest
import torch

import allreduce_reduction_amd as hc
import rankops_ref as ref
from test_gpu_rank_ops import guarded, same

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
CODE = {torch.float32: 0, torch.float16: 1, torch.bfloat16: 2}


class Back:
    """One call of each operator that has a workspace, over buffers made once:
    `tokens` tokens of 3 ranks into a table of `vocab` rows of 24, `rows` rows
    of logits and of a block's end."""

    def __init__(self, tokens, vocab, rows, seed=0):
        g = torch.Generator().manual_seed(seed)
        rnd = lambda *s, dt=BF: torch.randn(*s, generator=g).to(dt).cuda()  # noqa: E731
        P, W, K = 3, 24, 9
        self.counts = [tokens // 2, 0, tokens - tokens // 2]
        self.ids = [torch.randint(-1, vocab, (n,), generator=g).cuda() for n in self.counts]
        for t in self.ids:
            t[::3] = 5  # one id of many chunks
        self.dx = [rnd(n, W) for n in self.counts]
        self.base = ref.split_rows(rnd(vocab, W, dt=F32), P)
        self.written, self.added = [[torch.empty_like(t) for t in self.base] for _ in range(2)]
        self.logits = ref.split_rows(rnd(1000, rows), P)
        self.logits = [t.t().contiguous() for t in self.logits]
        self.t, self.t_ids = rnd(rows, K), torch.randint(-1, 1000, (rows, K), generator=g).cuda()
        self.loss, self.lse = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
        self.g = rnd(P, rows, 200)
        self.hid, self.sums = ref.split_rows(rnd(rows, 200), P), ref.split_rows(rnd(rows, 200), P)
        self.pre, self.post, self.gate = rnd(200), rnd(200), rnd(2, 200)
        self.parts, self.res = torch.empty_like(self.g), [torch.empty_like(t) for t in self.hid]
        self.dpre, self.dpost, self.dgate = [torch.empty(s, device="cuda") for s in ((200,), (200,), (2, 200))]
        self.comm = hc.Comm(P, "ring")

    def run(self):
        c = self.comm
        for a, b in zip(self.added, self.base):
            a.copy_(b)
        c.embedding_grad(self.dx, self.ids, self.written, scale=0.5)
        c.embedding_grad(self.dx, self.ids, self.added, accumulate=True)
        c.distill_loss(self.logits, self.t, self.t_ids, self.loss, self.lse, temperature=2.0)
        c.reduce_norm_grad(self.g, self.hid, self.parts, self.res, self.pre, self.dpre, sums=self.sums, post_weight=self.post,
                           post_weight_grad=self.dpost, gate=self.gate, gate_grad=self.dgate, scale=0.5)

    def outputs(self):
        return self.written + self.added + [self.loss, self.lse, self.parts, self.dpre, self.dpost, self.dgate] + self.res

    def results(self):
        return [t.clone() for t in self.outputs()]


SIZES = [(3000, 2000, 600), (3000, 20000, 600), (20000, 3000, 2000), (20000, 100000, 2000)]


@pytest.mark.parametrize("tokens,vocab,rows", SIZES)
def test_captured(tokens, vocab, rows):
    """The first call captured; two graphs and eager calls in turn."""
    backs = [Back(tokens, vocab, rows, 1), Back(tokens + 700, vocab, rows + 30, 2)]
    graphs = []
    for b in backs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            b.run()
        graphs.append(g)
    want = []
    for b in backs:
        b.run()
        torch.cuda.synchronize()
        want.append(b.results())
    eager = Back(tokens, vocab, rows, 1)
    for rep in range(4):
        for b in backs:
            for t in b.outputs():
                t.fill_(rep)
        torch.cuda.synchronize()
        graphs[0].replay()
        graphs[1].replay()
        eager.run()
        torch.cuda.synchronize()
        assert same(backs[0].results(), want[0]) and same(backs[1].results(), want[1]), rep
        assert same(eager.results(), want[0]), rep


@pytest.mark.parametrize("tokens,vocab,rows", SIZES)
def test_streams_at_once(tokens, vocab, rows):
    backs = [Back(tokens - 11 * k, vocab, rows + 2 * k, k) for k in range(4)]
    want = []
    for b in backs:
        b.run()
        torch.cuda.synchronize()
        want.append(b.results())
        for t in b.outputs():
            t.fill_(1)
    streams = [torch.cuda.Stream() for _ in backs]
    torch.cuda.synchronize()
    for _ in range(5):
        for b, q in zip(backs, streams):
            with torch.cuda.stream(q):
                b.run()
    torch.cuda.synchronize()
    for b, w in zip(backs, want):
        assert same(b.results(), w)


def workspace(need):
    """`need` bytes, 16-byte aligned, between guard zones, and their check."""
    flat = torch.full((need + 512 + 16,), 0xa5, dtype=torch.uint8, device="cuda")
    lo = 256 + -(flat.data_ptr() + 256) % 16
    return flat.data_ptr() + lo, lambda: bool((flat[:lo] == 0xa5).all()) and bool((flat[lo + need:] == 0xa5).all())


def addresses(tensors):
    return (ctypes.c_void_p * len(tensors))(*[t.data_ptr() if t.numel() else None for t in tensors])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("width", [5, 77, 1003])
@pytest.mark.parametrize("tokens,vocab", [(1025, 50), (1300, 6001), (9000, 50), (9001, 40001), (20000, 5003)])
def test_embedding_gradient_stays_inside(tokens, vocab, width, dtype):
    """Through the C ABI, whose workspace is exactly as large as it asks for;
    what it holds before plays no part."""
    g = torch.Generator().manual_seed(width + tokens)
    P, L = 3, hc.load_library()
    counts = [tokens // 3, 0, tokens - tokens // 3]
    ids = torch.randint(-1, vocab + 1, (tokens,), generator=g)
    ids[::5] = vocab - 1
    grads = torch.randn(tokens, width, generator=g).to(dtype)
    dev_ids = [guarded(t) for t in ids.split(counts)]
    dev_grads = [guarded(t) for t in grads.split(counts)]
    n, need = (ctypes.c_size_t * P)(*counts), ctypes.c_size_t()
    e = hc.Embedding(vocab, width, CODE[dtype], 8, 0.5)
    most = int(torch.bincount(ids[(ids >= 0) & (ids < vocab)]).max())
    stream = torch.cuda.current_stream().cuda_stream
    with hc.Comm(P, "ring") as c:
        assert L.hbmc_embedding_grad_workspace(c._h, e, n, ctypes.byref(need)) == 0 and need.value > 0
        for acc in (0, 1):
            for dt in dict.fromkeys((dtype, F32)):
                base = torch.randn(vocab, width, generator=g).to(dt)
                table = [guarded(t) for t in ref.split_rows(base, P)]
                ws, ws_ok = workspace(need.value)
                torch.cuda.synchronize()
                assert L.hbmc_embedding_grad(c._h, e, addresses([t for t, _ in dev_grads]), addresses([t for t, _ in dev_ids]), n,
                                             addresses([t for t, _ in table]), CODE[dt], acc, ws, need.value, stream) == 0
                torch.cuda.synchronize()
                assert ws_ok() and all(ok() for _, ok in table + dev_grads + dev_ids)
                want = ref.embed_backward(grads, ids, vocab, 0.5, base if acc else None)
                ref.check(torch.cat([t for t, _ in table]), want, most + 4, "table")


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,vocab,top", [(513, 77, 5), (600, 4999, 300), (1, 140001, 40)])
def test_loss_stays_inside(rows, vocab, top, dtype):
    g = torch.Generator().manual_seed(rows)
    P, L = 3, hc.load_library()
    z = torch.randn(rows, vocab, generator=g).to(dtype)
    t, ids = torch.randn(rows, top, generator=g).to(dtype), torch.randint(-1, vocab + 1, (rows, top), generator=g)
    logits = [guarded(z[:, lo:hi].contiguous()) for lo, hi in ref.segments(vocab, P)]
    dt, di, loss, lse = guarded(t), guarded(ids), guarded(torch.zeros(rows)), guarded(torch.zeros(rows))
    d = hc.Distill(rows, vocab, top, CODE[dtype], CODE[dtype], 8, 2.0, dt[0].data_ptr(), di[0].data_ptr())
    need = ctypes.c_size_t()
    with hc.Comm(P, "ring") as c:
        assert L.hbmc_distill_loss_workspace(c._h, d, ctypes.byref(need)) == 0 and need.value > 0
        ws, ws_ok = workspace(need.value)
        torch.cuda.synchronize()
        assert L.hbmc_distill_loss(c._h, d, addresses([x for x, _ in logits]), loss[0].data_ptr(), lse[0].data_ptr(), ws, need.value,
                                   torch.cuda.current_stream().cuda_stream) == 0
        torch.cuda.synchronize()
    assert ws_ok() and all(ok() for _, ok in logits + [dt, di, loss, lse])
    want = ref.distill_forward(z, t, ids, 2.0)
    ref.check(loss[0], want["loss"], 140, "loss")
    ref.check(lse[0], want["lse"], 100, "lse")


@pytest.mark.parametrize("rows,gate_rows,width", [(40, 0, 5), (700, 0, 1003), (700, 700, 77), (700, 3, 77), (1999, 40, 77),
                                                  (300, 7, 1003), (300, 150, 9001), (300, 2, 9001)])
def test_norm_gradient_stays_inside(rows, gate_rows, width):
    """gate_rows 0: no gate."""
    g = torch.Generator().manual_seed(rows + width)
    P, L = 3, hc.load_library()
    rnd = lambda *s: torch.randn(*s, generator=g).to(BF)  # noqa: E731
    groups = -(-rows // gate_rows) if gate_rows else 0
    grads, hid, sums, pre, post, gate = rnd(P, rows, width), rnd(rows, width), rnd(rows, width), rnd(width), rnd(width), rnd(groups, width)
    dg, dh, ds = [guarded(t) for t in grads], [guarded(t) for t in ref.split_rows(hid, P)], [guarded(t) for t in ref.split_rows(sums, P)]
    w2, w1, wg = guarded(pre), guarded(post), guarded(gate)
    parts, res = [guarded(torch.zeros_like(t)) for t in grads], [guarded(torch.zeros_like(t[0])) for t in dh]
    dpre, dpost, dgate = guarded(torch.zeros(width)), guarded(torch.zeros(width)), guarded(torch.zeros(groups, width))
    n = hc.Norm(rows, width, max(gate_rows, 1), 2, 0.5, 1e-6, 1e-6, w2[0].data_ptr(), w1[0].data_ptr(),
                wg[0].data_ptr() if groups else None)
    need = ctypes.c_size_t()
    first = lambda x: addresses([t for t, _ in x])  # noqa: E731
    with hc.Comm(P, "ring") as c:
        assert L.hbmc_reduce_norm_grad_workspace(c._h, n, ctypes.byref(need)) == 0 and need.value > 0
        ws, ws_ok = workspace(need.value)
        torch.cuda.synchronize()
        assert L.hbmc_reduce_norm_grad(c._h, n, first(dg), first(dh), first(ds), None, first(parts), first(res), dpre[0].data_ptr(),
                                       dpost[0].data_ptr(), dgate[0].data_ptr() if groups else None, ws, need.value,
                                       torch.cuda.current_stream().cuda_stream) == 0
        torch.cuda.synchronize()
    assert ws_ok() and all(ok() for _, ok in dg + dh + ds + parts + res + [w2, w1, wg, dpre, dpost, dgate])
    want = ref.norm_backward(grads, hid, pre, sums, None, post, gate if groups else None, max(gate_rows, 1), 0.5)
    for got, name in ((parts[0][0], "parts"), (torch.cat([t for t, _ in res]), "residual"), (dpre[0], "pre"), (dpost[0], "post")):
        ref.check(got, want[name], P + 180, name)
    if groups:
        ref.check(dgate[0], want["gate"], P + 180, "gate")


def test_tables_past_32_bit_offsets():
    """The sorted gradient over 4.6 GB: whole numbers, whose sums are exact."""
    rows, width, n = 140_000, 16_384, 2000
    g = torch.Generator("cuda").manual_seed(0)
    ids = rows - 1 - torch.randint(0, 900, (n,), device="cuda", generator=g)
    ids[::10] = torch.randint(0, 100, (n // 10,), device="cuda", generator=g)
    grads = torch.randint(-2, 3, (n, width), device="cuda", generator=g).to(BF)
    want = torch.zeros(rows, width, dtype=BF, device="cuda")
    for i in range(0, n, 100):  # below 2^8 a row: exact in bf16 too
        want.index_add_(0, ids[i:i + 100], grads[i:i + 100])
    table = torch.full((rows, width), 7, dtype=BF, device="cuda")
    with hc.Comm(1, "ring") as c:
        c.embedding_grad([grads], [ids], [table])
        assert torch.equal(table, want)
        c.embedding_grad([grads], [ids], [table], scale=2.0, accumulate=True)
        assert torch.equal(table, want.mul_(3))


def test_more_tokens_than_a_rank_may_have():
    """2^27 tokens, the first and last rank with the most that one may have:
    16384 tiles in the sort, sums of whole numbers (below 2^24) that are exact."""
    most, vocab = 2 ** 26 - 1, 3001
    g = torch.Generator("cuda").manual_seed(0)
    counts = [most, 1000, most]
    ids = [torch.randint(-1, vocab, (n,), device="cuda", dtype=torch.int32, generator=g) for n in counts]
    grads = [torch.randint(-4, 5, (n, 1), device="cuda", generator=g).to(BF) for n in counts]
    want = torch.zeros(vocab + 1, 1, dtype=torch.float64, device="cuda")
    for i, x in zip(ids, grads):
        for a in range(0, i.numel(), 1 << 24):
            want.index_add_(0, i[a:a + (1 << 24)].long() + 1, x[a:a + (1 << 24)].double())
    table = [torch.full((hi - lo, 1), 7.0, device="cuda") for lo, hi in ref.segments(vocab, 3)]
    with hc.Comm(3, "ring") as c:
        c.embedding_grad(grads, ids, table)
        assert torch.equal(torch.cat(table).double(), want[1:])
        c.embedding_grad(grads, ids, table, accumulate=True)
        assert torch.equal(torch.cat(table).double(), 2 * want[1:])
