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
