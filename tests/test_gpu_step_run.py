"""The operators of a step together, as they are used: a decoding step of a model
spread over the ranks, and a training step's gradients through their collective
to their clipping."""
import math

import pytest
import torch

import allreduce_reduction_amd as hc
import rankops_ref as ref
import stepops_ref as step
from test_gpu_rank_ops import same

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


class Decode:
    """Tokens' rows -> codes -> a layer whose inner width is dealt out, as partial
    sums -> the norms at its end -> codes -> the logits, their channels dealt out ->
    penalties, biases and a mask, in place."""

    def __init__(self, rows, width, vocab, P, seed=0):
        g = torch.Generator().manual_seed(seed)
        self.P, self.rows, self.width, self.vocab = P, rows, width, vocab
        self.table = torch.randn(vocab, width, generator=g).to(BF)
        self.ids = torch.randint(0, vocab, (rows,), generator=g)
        self.w1, self.s1 = step.codes(torch.randn(width, width, generator=g) / math.sqrt(width))
        self.w2, self.s2 = step.codes(torch.randn(vocab, width, generator=g) / math.sqrt(width))
        self.pre, self.post = torch.rand(width, generator=g).to(BF) + 0.5, torch.rand(width, generator=g).to(BF) + 0.5
        on = torch.rand(rows, vocab, generator=g) < 0.3
        self.lists = dict(tokens=torch.randint(-1, vocab, (rows, 50), generator=g), prompt_lengths=torch.full((rows,), 20),
                          lengths=torch.full((rows,), 45), repetition=torch.full((rows,), 1.2), frequency=torch.full((rows,), 0.1),
                          presence=torch.full((rows,), 0.2), bias_ids=torch.randint(0, vocab, (rows, 4), generator=g),
                          bias=torch.randn(rows, 4, generator=g), mask=step.bits(on))
        cols = lambda x: [x[:, lo:hi].contiguous().cuda() for lo, hi in ref.segments(x.shape[1], P)]  # noqa: E731
        rows_of = lambda x: [t.cuda() for t in ref.split_rows(x, P)]  # noqa: E731
        e = lambda *s, dt=BF: torch.empty(*s, dtype=dt, device="cuda")  # noqa: E731
        self.d_table, self.d_ids, self.x = rows_of(self.table), self.ids.cuda(), e(rows, width)
        self.d_w1, self.d_s1 = cols(self.w1), self.s1.cuda()
        self.d_w2, self.d_s2 = rows_of(self.w2), rows_of(self.s2)
        self.d_pre, self.d_post = self.pre.cuda(), self.post.cuda()
        self.d_lists = {k: v.cuda() for k, v in self.lists.items()}
        self.xs = [e(rows, hi - lo) for lo, hi in ref.segments(width, P)]
        self.q = [e(*t.shape, dt=torch.int8) for t in self.xs]
        self.scale, self.scale2 = e(rows, dt=F32), e(rows, dt=F32)
        self.parts, self.y = e(P, rows, width), e(P, rows, width)
        self.residual = [e(hi - lo, width) for lo, hi in ref.segments(rows, P)]
        self.q2 = e(rows, width, dt=torch.int8)
        self.logits = [e(rows, hi - lo) for lo, hi in ref.segments(vocab, P)]
        self.raw = [torch.empty_like(t) for t in self.logits]
        self.sum = e(P, rows, width)
        self.comm, self.one = hc.Comm(P, "ring"), hc.Comm(1, "ring")

    def run(self):
        c = self.comm
        c.embedding(self.d_table, [self.d_ids] + [self.d_ids[:0]] * (self.P - 1), [self.x] + [self.x[:0]] * (self.P - 1))
        for r, (lo, hi) in enumerate(ref.segments(self.width, self.P)):
            self.xs[r].copy_(self.x[:, lo:hi])
        for r, (lo, hi) in enumerate(ref.segments(self.rows, self.P)):
            self.residual[r].copy_(self.x[lo:hi])
        c.quantize_rows(self.xs, self.q, self.scale)
        c.product(self.q, self.scale, self.d_w1, self.d_s1, list(self.parts))
        c.reduce_product(self.q, self.scale, self.d_w1, self.d_s1, list(self.sum))
        c.reduce_norm(self.parts, self.residual, self.y, self.d_pre, post_weight=self.d_post)
        self.one.quantize_rows([self.y[0]], [self.q2], self.scale2)
        c.product([self.q2] * self.P, self.scale2, self.d_w2, self.d_s2, self.logits)
        for a, b in zip(self.raw, self.logits):
            a.copy_(b)
        c.adjust_logits(self.logits, **self.d_lists)

    def outputs(self):
        return [self.x, self.scale, self.parts, self.sum, self.y, self.q2, self.scale2] + self.q + self.residual + self.raw + self.logits

    def check(self):
        """Each operator against its formula on what the one before it left."""
        rows, P = self.rows, self.P
        x = self.x.cpu()
        assert torch.equal(x, self.table[self.ids])
        q, scale = step.codes(x)
        assert torch.equal(torch.cat([t.cpu() for t in self.q], 1), q) and torch.equal(self.scale.cpu(), scale)
        for r, (lo, hi) in enumerate(ref.segments(self.width, P)):
            ref.check(self.parts[r], step.product(q[:, lo:hi], scale, self.w1[:, lo:hi], self.s1), 3, "parts")
        for s in self.sum:
            ref.check(s, step.product(q, scale, self.w1, self.s1), 3, "sum")
        want = ref.norm_forward(self.parts.cpu(), x, self.pre, self.post)
        y = self.y[0].cpu()
        ref.check(self.y[0], want["out"], P + 120, "y")
        ref.check(torch.cat([t.cpu() for t in self.residual]), want["residual"], P + 120, "residual")
        q2, scale2 = step.codes(y)
        assert torch.equal(self.q2.cpu(), q2) and torch.equal(self.scale2.cpu(), scale2)
        raw = torch.cat([t.cpu() for t in self.raw], 1)
        ref.check(raw, step.product(q2, scale2, self.w2, self.s2), 3, "raw")
        z, mag = step.adjust(raw, **self.lists)
        got = torch.cat([t.cpu() for t in self.logits], 1)
        finite = torch.isfinite(z)
        assert bool((got == -torch.inf)[~finite].all())
        ref.check(got[finite], (z[finite], mag[finite]), 10, "logits")


@pytest.mark.parametrize("rows,width,vocab,P", [(1, 512, 1000, 8), (7, 240, 1003, 3), (40, 1024, 4096, 4), (150, 512, 2000, 2)])
def test_decoding_step(rows, width, vocab, P):
    s = Decode(rows, width, vocab, P)
    s.run()
    torch.cuda.synchronize()
    s.check()


def test_decoding_steps_captured():
    """Two steps' graphs and an eager one in turn."""
    steps = [Decode(3, 512, 1000, 4, 1), Decode(33, 256, 2001, 4, 2), Decode(3, 512, 1000, 4, 3)]
    want = []
    for s in steps:
        s.run()
        torch.cuda.synchronize()
        want.append([t.clone() for t in s.outputs()])
    graphs = []
    for s in steps[:2]:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            s.run()
        graphs.append(g)
    for rep in range(3):
        for s in steps:
            for t in s.outputs():
                t.fill_(rep)
        torch.cuda.synchronize()
        for g in graphs:
            g.replay()
        steps[2].run()
        torch.cuda.synchronize()
        assert all(same(s.outputs(), w) for s, w in zip(steps, want)), rep


@pytest.mark.parametrize("P,algo", [(8, "ring"), (4, "rhd"), (3, "ring")])
def test_gradients_from_an_allreduce_to_their_clipping(P, algo):
    """Two matrices' gradients of each rank's own tokens, made by torch, summed by an
    AllReduce in one bucket, made a mean and clipped."""
    g = torch.Generator().manual_seed(P)
    w = [torch.randn(64, 33, generator=g), torch.randn(7, 64, generator=g)]
    flats, lists, want = [], [], None
    for r in range(P):
        ws = [x.clone().requires_grad_() for x in w]
        x = torch.randn(50, 33, generator=g)
        (torch.tanh(x @ ws[0].t()) @ ws[1].t()).square().sum().backward()
        grads = [t.grad for t in ws]
        flat = torch.cat([t.flatten() for t in grads]).cuda()
        flats.append(flat)
        lists.append([flat[:64 * 33].view(64, 33), flat[64 * 33:].view(7, 64)])
        want = [t.double() for t in grads] if want is None else [a + t.double() for a, t in zip(want, grads)]
    size = step.norm(want, 2.0, 1.0 / P)
    out = torch.empty(1, device="cuda")
    with hc.Comm(P, algo) as c, c.gradients(same=lists) as grads:
        c.allreduce(flats, "fp32", "sum")
        grads.clip(0.3 * float(size), out, scale=1.0 / P)
    torch.cuda.synchronize()
    # the AllReduce's P - 1 roundings to 32 bits move each sum by P * 2^-24 of its terms' sizes; their own rounding by autograd is P more
    assert abs(float(out) - float(size)) <= 4 * P * 2.0 ** -24 * float(size)
    by = step.factor(size, 0.3 * float(size), 1.0 / P)
    for mine in lists:
        for t, v in zip(mine, want):
            scale = float(v.abs().max())
            assert float((t.cpu().double() - v * by).abs().max()) <= 16 * P * 2.0 ** -24 * scale * by
    assert same(lists[0], lists[-1])


def test_dealt_out_gradients_clipped_where_they_lie():
    """A reduce-scatter leaves rank r its segment of every bucket: views of it, clipped in place."""
    P, n = 4, 4003
    g = torch.Generator().manual_seed(5)
    host = [torch.randint(-8, 9, (n,), generator=g).float() for _ in range(P)]  # sums are exact
    bufs = [t.cuda() for t in host]
    total = torch.stack(host).sum(0)
    out = torch.empty(1, device="cuda")
    dealt = [[bufs[r][lo:hi]] for r, (lo, hi) in enumerate(ref.segments(n, P))]
    with hc.Comm(P, "ring") as c, c.gradients(dealt=dealt) as grads:
        c.reduce_scatter(bufs, "fp32", "sum")
        grads.clip(1.0, out, norm_type=1.0)
    size = step.norm([total], 1.0)
    assert float(out) == float(size)
    by = step.factor(size, 1.0)
    got = torch.cat([d[0].cpu() for d in dealt])
    ref.check(got, (total.double() * by, total.double().abs() * by), 2, "gradient")


def test_training_steps_with_one_handle_of_gradients():
    """A handle made after the first backward pass, whose gradients the next steps
    fill again: zero_grad(set_to_none=False) leaves them where they are."""
    g = torch.Generator().manual_seed(3)
    shapes, steps = [(64, 33), (7, 64)], 3
    params = [torch.randn(*s, generator=g).cuda().requires_grad_() for s in shapes]
    twin = [p.detach().clone().requires_grad_() for p in params]
    optimizer, plain = torch.optim.SGD(params, lr=0.1), torch.optim.SGD(twin, lr=0.1)
    out, grads = torch.empty(1, device="cuda"), None
    with hc.Comm(1, "ring") as c:
        for _ in range(steps):
            x = torch.randn(50, 33, generator=g).cuda()
            for p, opt in ((params, optimizer), (twin, plain)):
                opt.zero_grad(set_to_none=False)
                (torch.tanh(x @ p[0].t()) @ p[1].t()).square().sum().backward()
            before = [t.grad.cpu() for t in twin]
            if grads is None:
                grads = c.gradients(dealt=[[p.grad for p in params]])
            grads.clip(1.0, out)
            size = step.norm(before, 2.0)
            by = step.factor(size, 1.0)
            assert by < 1.0
            # both sides' gradients are the same products of the same values
            assert abs(float(out) - float(size)) <= 1.01 * 2.0 ** -24 * float(size)
            for p, b, t in zip(params, before, twin):
                ref.check(p.grad, (b.double() * by, b.double().abs() * by), 2, "gradient")
                t.grad.copy_(p.grad)
            optimizer.step()
            plain.step()
            assert same([p.detach() for p in params], [t.detach() for t in twin])
        grads.close()
