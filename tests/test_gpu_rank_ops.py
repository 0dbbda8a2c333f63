"""The operators over the ranks as a program uses them: a whole training step
through all of them, captured and replayed, on other streams, several calls at
once, rows past 32-bit offsets.
"""
import pytest
import torch

import allreduce_reduction_amd as hc
import rankops_ref as ref

pytestmark = pytest.mark.gpu

P, T, H, V, K = 4, 24, 192, 1000, 12
BF = torch.bfloat16


class Step:
    """A small model of P ranks: embedding, a block whose rank r multiplies by
    its own slice of two matrices, the norms at its end, logits over the rank's
    vocabulary columns (the embedding's rows), the distillation loss; then the
    whole way back.  Every buffer is made once, so the step can be captured."""

    def __init__(self, seed=0):
        g = torch.Generator().manual_seed(seed)
        rnd = lambda *s, by=1.0: (by * torch.randn(*s, generator=g)).to(BF).cuda()  # noqa: E731
        new = lambda *s, dtype=BF: torch.empty(*s, dtype=dtype, device="cuda")  # noqa: E731
        self.table = ref.split_rows(rnd(V, H, by=0.2), P)
        self.w = [rnd(H, H, by=H ** -0.5) for _ in range(P)]
        self.pre, self.post, self.gate = 1 + rnd(H, by=0.1), 1 + rnd(H, by=0.1), rnd(2, H)
        self.ids = [torch.randint(0, V, (T,), generator=g).cuda()] * P
        self.t = rnd(T, K, by=2.0)
        self.t_ids = torch.randint(0, V, (T, K), generator=g).cuda()
        self.dl = torch.full((T,), 1.0 / T, device="cuda")
        self.x, self.parts, self.y = new(P, T, H), [new(T, H) for _ in range(P)], [new(T, H) for _ in range(P)]
        self.segs = ref.segments(T, P)
        self.res = [new(hi - lo, H) for lo, hi in self.segs]
        self.hid, self.sums, self.dres = [[torch.empty_like(t) for t in self.res] for _ in range(3)]
        self.logits = [new(T, t.shape[0]) for t in self.table]
        self.loss, self.lse = new(T, dtype=torch.float32), new(T, dtype=torch.float32)
        self.dy, self.dx = [new(T, H) for _ in range(P)], [new(T, H) for _ in range(P)]
        f32 = dict(dtype=torch.float32)
        self.dpre, self.dpost, self.dgate = new(H, **f32), new(H, **f32), new(2, H, **f32)
        self.dtable = [new(*t.shape, **f32) for t in self.table]
        self.dres_in = [torch.zeros_like(t) for t in self.res]
        self.comm = hc.Comm(P, "rhd")

    def run(self):
        c = self.comm
        c.embedding(self.table, self.ids, self.x, scale=H ** 0.5)
        for r in range(P):
            torch.mm(self.x[r], self.w[r], out=self.parts[r])
            lo, hi = self.segs[r]
            self.res[r].copy_(self.x[r, lo:hi])
        kw = dict(post_weight=self.post, gate=self.gate, scale=0.5)
        c.reduce_norm(self.parts, self.res, self.y, self.pre, residual_out=self.hid, sums=self.sums, **kw)
        for r in range(P):
            torch.mm(self.y[r], self.table[r].t(), out=self.logits[r])
        c.distill_loss(self.logits, self.t, self.t_ids, self.loss, self.lse, temperature=2.0)
        c.distill_loss_grad(self.logits, self.t, self.t_ids, self.lse, self.dl, self.logits, temperature=2.0)
        for r in range(P):
            torch.mm(self.logits[r], self.table[r], out=self.dy[r])
            self.dtable[r].copy_(torch.mm(self.logits[r].t().contiguous(), self.y[r]))
        c.reduce_norm_grad(self.dy, self.hid, self.dx, self.dres, self.pre, self.dpre, sums=self.sums,
                           residual_grad_in=self.dres_in, post_weight_grad=self.dpost, gate_grad=self.dgate, **kw)
        for r in range(P):
            torch.mm(self.dx[r], self.w[r].t().contiguous(), out=self.dy[r])
            lo, hi = self.segs[r]
            self.dy[r][lo:hi].add_(self.dres[r])
        c.embedding_grad(self.dy, self.ids, self.dtable, scale=H ** 0.5, accumulate=True)

    def results(self):
        return [t.clone() for t in [self.loss, self.lse, self.dpre, self.dpost, self.dgate] + self.dtable + self.dx + self.hid]

    def reference(self):
        """The step's loss and gradients by automatic differentiation in 64 bits."""
        table = torch.cat(self.table).double().cpu().requires_grad_()
        w = [t.double().cpu().requires_grad_() for t in self.w]
        pre, post, gate = [t.double().cpu().requires_grad_() for t in (self.pre, self.post, self.gate)]
        ids = self.ids[0].cpu()
        x = table[ids] * H ** 0.5
        s = sum(x @ m for m in w)
        n = s / (s.pow(2).mean(1, keepdim=True) + 1e-6).sqrt() * post * gate[torch.arange(T) // (T // 2)]
        h = x + 0.5 * n
        y = h / (h.pow(2).mean(1, keepdim=True) + 1e-6).sqrt() * pre
        loss = ref.distill_forward(y @ table.t(), self.t.cpu(), self.t_ids.cpu(), 2.0)["loss"][0]
        loss.mean().backward()
        return loss.detach(), pre.grad, post.grad, gate.grad, table.grad


def same(a, b):
    return all(torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for x, y in zip(a, b))


def test_a_whole_step():
    """Against 64 bits.  Between the operators the step rounds to bf16 some
    eight times (rows of x, products, residual, y, logits, their gradients, the
    way back), each by 2^-8 relative to a row's size and independent: in the
    2-norm 8 * 2^-8 = 3.1% is the worst case; the gradients pass twice that
    many."""
    s = Step()
    s.run()
    loss, pre, post, gate, table = s.reference()
    for got, want, bound in ((s.loss, loss, 8), (s.dpre, pre, 16), (s.dpost, post, 16), (s.dgate, gate, 16),
                             (torch.cat(s.dtable), table, 16)):
        off = (got.double().cpu() - want).norm() / want.norm()
        assert off <= bound * 2.0 ** -8, (tuple(want.shape), off)


def test_captured_step():
    s = Step(1)
    s.run()
    torch.cuda.synchronize()
    want = s.results()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        s.run()
    for rep in range(4):
        for t in s.dtable + s.dx + s.hid + [s.loss, s.lse, s.dpre]:
            t.fill_(rep)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert same(s.results(), want), rep


def test_first_calls_captured():
    """Nothing is cached, so the first call of a shape may be captured; two
    graphs and eager calls, replayed in turn, do not disturb each other."""
    steps = [Step(2), Step(3)]
    for s in steps:  # the products' own first-call work happens outside
        s.run()
    torch.cuda.synchronize()
    want = [s.results() for s in steps]
    graphs = []
    for s in steps:
        s.comm = hc.Comm(P, "ring")
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            s.run()
        graphs.append(g)
    for _ in range(3):
        for s in steps:
            for t in s.dtable + s.dx:
                t.fill_(3)
        graphs[0].replay()
        graphs[1].replay()
        eager = Step(2)
        eager.run()
        torch.cuda.synchronize()
        assert same(steps[0].results(), want[0]) and same(steps[1].results(), want[1]) and same(eager.results(), want[0])


def test_streams_at_once():
    """Calls on several streams at the same time, by torch's current stream."""
    steps = [Step(k) for k in range(4)]
    want = []
    for s in steps:
        s.run()
        torch.cuda.synchronize()
        want.append(s.results())
        for t in s.dtable + s.dx:
            t.fill_(1)
    streams = [torch.cuda.Stream() for _ in steps]
    torch.cuda.synchronize()
    for _ in range(5):
        for s, q in zip(steps, streams):
            with torch.cuda.stream(q):
                s.run()
    torch.cuda.synchronize()
    for s, w in zip(steps, want):
        assert same(s.results(), w)


def test_named_stream():
    """A stream given by name, as a torch stream and as a raw handle."""
    g = torch.Generator().manual_seed(0)
    n, h, v = 3000, 256, 5000
    ids, grads = torch.randint(0, v, (n,), generator=g).cuda(), torch.randn(n, h, generator=g).cuda()
    with hc.Comm(1, "ring") as c:
        want = torch.empty(v, h, device="cuda")
        c.embedding_grad([grads], [ids], [want])
        q = torch.cuda.Stream()
        q.wait_stream(torch.cuda.current_stream())
        outs = [torch.zeros(v, h, device="cuda") for _ in range(6)]
        torch.cuda.synchronize()
        for k, out in enumerate(outs):
            stream = (q, q.cuda_stream, torch.cuda.default_stream())[k % 3]
            c.embedding_grad([grads], [ids], [out], stream=stream)
            torch.empty(1 << 20, device="cuda").fill_(k)  # reuses what the current stream's allocator has free
        torch.cuda.synchronize()
        for out in outs:
            assert torch.equal(out, want)
        with torch.cuda.stream(q):
            out = torch.zeros(v, h, device="cuda")
            c.embedding_grad([grads], [ids], [out], stream=0)
            torch.cuda.synchronize()
        assert torch.equal(out, want)


def test_rows_past_32_bit_offsets():
    """Matrices of more than 2^32 bytes: the last rows are those of a small
    call on the same rows."""
    rows, width = 140_000, 16_384  # 4.6 GB in bf16
    with hc.Comm(1, "ring") as c:
        x = torch.randn(rows, width, dtype=BF, device="cuda")
        w = torch.ones(width, dtype=BF, device="cuda")
        out, res = torch.empty_like(x), torch.empty_like(x)
        c.reduce_norm([x], [x], [out], w, residual_out=[res], post_weight=w)
        few, few_res = torch.empty(50, width, dtype=BF, device="cuda"), torch.empty(50, width, dtype=BF, device="cuda")
        c.reduce_norm([x[-50:]], [x[-50:]], [few], w, residual_out=[few_res], post_weight=w)
        assert torch.equal(out[-50:], few) and torch.equal(res[-50:], few_res)
        ids = torch.arange(rows - 1, rows - 301, -1, device="cuda")
        got = torch.empty(300, width, dtype=BF, device="cuda")
        c.embedding([x], [ids], [got])
        assert torch.equal(got, x[ids])
        c.embedding_grad([got], [ids], [out])
        assert torch.equal(out[-300:], x[-300:]) and not out[:-300].any()
        t, ids = torch.ones(rows, 1, dtype=BF, device="cuda"), torch.full((rows, 1), 7, device="cuda")
        loss, lse = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
        c.distill_loss([x], t, ids, loss, lse)
        c.distill_loss_grad([x], t, ids, lse, torch.ones(rows, device="cuda"), [res])
        l2, e2 = torch.empty(50, device="cuda"), torch.empty(50, device="cuda")
        c.distill_loss([x[-50:]], t[-50:], ids[-50:], l2, e2)
        c.distill_loss_grad([x[-50:]], t[-50:], ids[-50:], e2, torch.ones(50, device="cuda"), [few])
        assert torch.equal(loss[-50:], l2) and torch.equal(lse[-50:], e2) and torch.equal(res[-50:], few)


def guarded(t, pad=40):
    """A copy of t on the GPU, one element past alignment, between guard zones;
    the copy and the check that the zones are as they were."""
    flat = torch.full((t.numel() + 2 * pad + 1,), 7, dtype=t.dtype, device="cuda")
    view = flat[pad + 1:pad + 1 + t.numel()].view(t.shape)
    view.copy_(t)
    return view, lambda: bool((flat[:pad + 1] == 7).all()) and bool((flat[pad + 1 + t.numel():] == 7).all())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("width", [5, 77, 1003, 2055, 9001])
def test_nothing_outside_is_written(dtype, width):
    g = torch.Generator().manual_seed(width)
    ranks, rows, vocab = 3, 7, 50
    checks = []

    def buf(*shape, dt=dtype):
        v, ok = guarded(torch.randn(*shape, generator=g).to(dt))
        checks.append(ok)
        return v

    segs = [hi - lo for lo, hi in ref.segments(rows, ranks)]
    cols = [hi - lo for lo, hi in ref.segments(width, ranks)]
    vocs = [hi - lo for lo, hi in ref.segments(vocab, ranks)]
    f32 = dict(dt=torch.float32)
    full = lambda: [buf(rows, width) for _ in range(ranks)]  # noqa: E731
    part = lambda: [buf(n, width) for n in segs]  # noqa: E731
    with hc.Comm(ranks, "ring") as c:
        w, w1 = buf(width), buf(width)
        for gate, gate_grad in ((buf(1, width), buf(1, width, **f32)), (buf(7, width), buf(7, width, **f32))):
            c.reduce_norm(full(), part(), full(), w, residual_out=part(), sums=part(), post_weight=w1, gate=gate)
            c.reduce_norm_grad(full(), part(), full(), part(), w, buf(width, **f32), sums=part(), residual_grad_in=part(),
                               post_weight=w1, post_weight_grad=buf(width, **f32), gate=gate, gate_grad=gate_grad)
        tokens = [4, 0, 9]
        ids = [torch.randint(-1, vocab + 1, (n,), generator=g).cuda() for n in tokens]
        c.embedding([buf(n, width) for n in vocs], ids, [buf(n, width) for n in tokens])
        for acc in (False, True):
            for dt in (dtype, torch.float32):
                c.embedding_grad([buf(n, width) for n in tokens], ids, [buf(n, width, dt=dt) for n in vocs], accumulate=acc)
        teacher, t_ids = buf(rows, 9), torch.randint(-1, width, (rows, 9), generator=g).cuda()
        logits, loss, lse = [buf(rows, n) for n in cols], buf(rows, **f32), buf(rows, **f32)
        c.distill_loss(logits, teacher, t_ids, loss, lse)
        c.distill_loss_grad(logits, teacher, t_ids, lse, buf(rows, **f32), [buf(rows, n) for n in cols])
    torch.cuda.synchronize()
    assert all(ok() for ok in checks)


@pytest.mark.parametrize("rows,gate_rows,width", [(10, 4, 48), (1999, 3, 48), (700, 300, 1000), (5, 1000, 64), (531, 2, 16384)])
def test_uneven_gate_groups(rows, gate_rows, width):
    """The C ABI takes a last group of fewer rows."""
    import ctypes
    g = torch.Generator().manual_seed(rows)
    rnd = lambda *s: torch.randn(*s, generator=g).to(BF)  # noqa: E731
    groups = -(-rows // gate_rows)
    ranks, L = 2, hc.load_library()
    grads, hid, sums = rnd(ranks, rows, width), rnd(rows, width), rnd(rows, width)
    pre, post, gate = rnd(width), rnd(width), rnd(groups, width)
    d = [t.cuda() for t in (grads, hid, sums, pre, post, gate)]
    new = lambda *s, dt=torch.float32: torch.empty(*s, dtype=dt, device="cuda")  # noqa: E731
    parts, res, y = new(ranks, rows, width, dt=BF), new(rows, width, dt=BF), new(ranks, rows, width, dt=BF)
    dpre, dpost, dgate = new(width), new(width), new(groups, width)
    n = hc.Norm(rows, width, gate_rows, 2, 0.5, 1e-6, 1e-6, d[3].data_ptr(), d[4].data_ptr(), d[5].data_ptr())
    whole = lambda t: (ctypes.c_void_p * ranks)(*[t[r].data_ptr() for r in range(ranks)])  # noqa: E731
    each = -(-rows // ranks)
    seg = lambda t: (ctypes.c_void_p * ranks)(*[t.data_ptr() + r * each * width * 2 for r in range(ranks)])  # noqa: E731
    need = ctypes.c_size_t()
    with hc.Comm(ranks, "ring") as c:
        torch.cuda.synchronize()
        stream = torch.cuda.current_stream().cuda_stream
        assert L.hbmc_reduce_norm(c._h, n, whole(d[0]), seg(d[1]), seg(res), whole(y), None, stream) == 0
        f = ref.norm_forward(grads, hid, pre, post, gate, gate_rows, 0.5)
        ref.check(y[1], f["out"], ranks + 80, "out")
        ref.check(res, f["residual"], ranks + 80, "residual")
        assert L.hbmc_reduce_norm_grad_workspace(c._h, n, ctypes.byref(need)) == 0
        ws = new(need.value, dt=torch.uint8)
        assert L.hbmc_reduce_norm_grad(c._h, n, whole(d[0]), seg(d[1]), seg(d[2]), None, whole(parts), seg(res), dpre.data_ptr(),
                                       dpost.data_ptr(), dgate.data_ptr(), ws.data_ptr(), need.value, stream) == 0
        b = ref.norm_backward(grads, hid, pre, sums, None, post, gate, gate_rows, 0.5)
    for got, name in ((parts[0], "parts"), (parts[1], "parts"), (res, "residual"), (dpre, "pre"), (dpost, "post"), (dgate, "gate")):
        ref.check(got, b[name], ranks + 180, name)


@pytest.mark.parametrize("n", [100, 9000])
def test_the_largest_vocabulary(n):
    """2^30 ids (four digits to sort) of one or two columns; each id's sum in
    the order of its tokens: below 2^-8 for the roundings to bf16 of results."""
    vocab = 2 ** 30
    ids = torch.randint(0, vocab, (n,), device="cuda", generator=torch.Generator("cuda").manual_seed(n))
    ids[1::2] = vocab - 1 - ids[1::2] % 1000  # many at the far end
    ids[0], ids[n // 2] = vocab - 1, 0
    grads = torch.randint(-4, 5, (n, 1), device="cuda").to(BF)  # exact sums
    table = torch.zeros(vocab, 1, dtype=BF, device="cuda")
    with hc.Comm(1, "ring") as c:
        c.embedding_grad([grads], [ids], [table], accumulate=True)
        want = torch.zeros(vocab, 1, dtype=torch.float32, device="cuda").index_add_(0, ids, grads.float())
        assert bool((table.float() - want).abs().le(2.0 ** -8 * want.abs()).all())
        table.fill_(3)
        c.embedding_grad([grads], [ids], [table])
        assert bool((table.float() - want).abs().le(2.0 ** -8 * want.abs()).all())
        got = torch.empty(n, 1, dtype=BF, device="cuda")
        c.embedding([table], [ids], [got])
        assert torch.equal(got, table[ids])


def test_operators_of_every_algorithm():
    """The algorithm of the communicator plays no part."""
    x = torch.randn(4, 6, 80, generator=torch.Generator().manual_seed(0)).to(BF).cuda()
    outs = []
    for algo, kw in (("ring", {}), ("rhd", {}), ("flat", {}), ("tree", {}), ("auto", {}), ("auto_rules", {}),
                     ("pipeline", dict(servers=2, ranks_per_server=2)), ("hier", dict(servers=2, ranks_per_server=2))):
        with hc.Comm(4, algo, **kw) as c:
            res = [torch.zeros(hi - lo, 80, dtype=BF, device="cuda") for lo, hi in ref.segments(6, 4)]
            out = torch.empty_like(x)
            c.reduce_norm(x, res, out, torch.ones(80, dtype=BF, device="cuda"))
            outs.append(out)
    assert all(torch.equal(o, outs[0]) for o in outs)
