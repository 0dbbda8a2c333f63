"""The row operators over the ranks in 64 bits, written from their formulas,
and the bounds that their kernels' 32-bit arithmetic and one final rounding
stay within.

Each function returns {name: (value, magnitude)}.  The magnitude is the same
formula with every term replaced by its absolute value, so that a chain of n
roundings to 32 bits moves the value by at most about n * 2^-24 * magnitude.
"""
import torch

HALF = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}


def segments(n, P):
    """[lo, hi) of each rank's rows or columns (the ceiling split)."""
    each = -(-n // P)
    return [(min(n, r * each), min(n, (r + 1) * each)) for r in range(P)]


def split_rows(whole, P):
    return [whole[lo:hi].clone() for lo, hi in segments(whole.shape[0], P)]


def check(got, ref, steps, name):
    """|got - value| within half a step of got's type relative to the value,
    and `steps` roundings to 32 bits of the magnitude (plus half a step of
    the type's smallest numbers, for results below its normal range)."""
    value, mag = ref
    info = torch.finfo(got.dtype)
    tol = HALF[got.dtype] * value.abs() + steps * 2.0 ** -24 * mag + info.smallest_normal * info.eps / 2
    off = (got.double().cpu() - value).abs()
    assert got.shape == value.shape, (name, got.shape, value.shape)
    assert not bool(torch.isnan(got).any()), name
    worst = (off / tol.clamp_min(1e-300)).max().item() if off.numel() else 0.0
    assert worst <= 1.0, f"{name}: {worst:.3f} of the bound"


def _rows(gate, gate_rows, T):
    return gate[torch.arange(T) // gate_rows]


def norm_forward(parts, residual, pre, post=None, gate=None, gate_rows=1, scale=1.0, eps=1e-6, post_eps=None):
    post_eps = eps if post_eps is None else post_eps
    P, T, H = parts.shape
    x, xa = parts.double().sum(0), parts.double().abs().sum(0)
    sums = (x, xa)
    n, na = x, xa
    if post is not None:
        r1 = 1 / (x.pow(2).mean(1, keepdim=True) + post_eps).sqrt()
        # cancellation between the ranks moves r1 by as much relative to it
        k = (xa.pow(2).mean(1, keepdim=True) * r1 ** 2).sqrt().clamp_min(1)
        n, na = x * r1 * post.double(), (xa + x.abs() * k) * r1 * post.double().abs()
    if gate is not None:
        g = _rows(gate.double(), gate_rows, T)
        n, na = n * g, na * g.abs()
    h, ha = residual.double() + scale * n, residual.double().abs() + abs(scale) * na
    r2 = 1 / (h.pow(2).mean(1, keepdim=True) + eps).sqrt()
    k = (ha.pow(2).mean(1, keepdim=True) * r2 ** 2).sqrt().clamp_min(1)
    y, ya = h * r2 * pre.double(), (ha + h.abs() * k) * r2 * pre.double().abs()
    return {"sums": sums, "residual": (h, ha), "out": (y, ya)}


def norm_backward(out_grads, hidden, pre, sums=None, residual_in=None, post=None, gate=None, gate_rows=1, scale=1.0,
                  eps=1e-6, post_eps=None):
    post_eps = eps if post_eps is None else post_eps
    P, T, H = out_grads.shape
    g, ga = out_grads.double().sum(0), out_grads.double().abs().sum(0)
    h, w = hidden.double(), pre.double()
    r2 = 1 / (h.pow(2).mean(1, keepdim=True) + eps).sqrt()
    a, aa = g * w, ga * w.abs()
    dh = r2 * a - h * r2 ** 3 * (a * h).mean(1, keepdim=True)
    dha = r2 * aa + h.abs() * r2 ** 3 * (aa * h.abs()).mean(1, keepdim=True)
    if residual_in is not None:
        dh, dha = dh + residual_in.double(), dha + residual_in.double().abs()
    res = {"residual": (dh, dha), "pre": ((g * h * r2).sum(0), (ga * h.abs() * r2).sum(0))}
    d, da = scale * dh, abs(scale) * dha
    if post is not None or gate is not None:
        x = sums.double()
        r1 = 1 / (x.pow(2).mean(1, keepdim=True) + post_eps).sqrt() if post is not None else torch.ones(T, 1).double()
        w1 = post.double() if post is not None else torch.ones(H).double()
    if gate is not None:
        G = gate.shape[0]
        at = torch.arange(T) // gate_rows
        zero = torch.zeros(G, H).double()
        res["gate"] = (zero.index_add(0, at, d * x * r1 * w1), zero.index_add(0, at, da * (x * r1 * w1).abs()))
        rows = _rows(gate.double(), gate_rows, T)
        d, da = d * rows, da * rows.abs()
    if post is not None:
        res["post"] = ((d * x * r1).sum(0), (da * (x * r1).abs()).sum(0))
        d, da = d * w1, da * w1.abs()
        d, da = (r1 * d - x * r1 ** 3 * (d * x).mean(1, keepdim=True),
                 r1 * da + x.abs() * r1 ** 3 * (da * x.abs()).mean(1, keepdim=True))
    res["parts"] = (d, da)
    return res


def embed_forward(table, ids, scale):
    inside = (ids >= 0) & (ids < table.shape[0])
    rows = table.double()[torch.where(inside, ids.long(), 0)] * inside[:, None] * scale
    return rows, rows.abs()


def embed_backward(grads, ids, vocab, scale, base=None):
    """grads [N, H], ids [N] of all ranks in order."""
    inside = (ids >= 0) & (ids < vocab)
    kept, at = grads.double()[inside], ids.long()[inside]
    out = torch.zeros(vocab, grads.shape[1]).double()
    value, mag = out.index_add(0, at, kept) * scale, out.index_add(0, at, kept.abs()) * abs(scale)
    return (value, mag) if base is None else (value + base.double(), mag + base.double().abs())


def teacher(t, ids, vocab, tau):
    """q and log q, and whether a row has an entry that counts."""
    t = torch.where((ids >= 0) & (ids < vocab), t.double() / tau, -torch.inf)
    some = (t > -torch.inf).any(1)
    t = torch.where(some[:, None], t, 0.0)
    log_q = torch.log_softmax(t, 1)
    return log_q.exp() * some[:, None], log_q, some


def distill_forward(logits, t, ids, tau):
    z = logits.double() / tau
    lse = torch.logsumexp(z, 1)
    q, log_q, some = teacher(t, ids, z.shape[1], tau)
    at = ids.long().clamp(0, z.shape[1] - 1)
    log_p = z.gather(1, at) - lse[:, None]
    terms = torch.where(q > 0, q * (log_q - log_p), 0.0)
    top = torch.where(torch.isfinite(t), t.double().abs(), 0).max(1).values / tau
    big = torch.where(torch.isfinite(z), z.abs(), 0).max(1).values
    mag = torch.where(q > 0, q * (log_q.abs() + log_p.abs() + big[:, None] + top[:, None] + lse.abs()[:, None]), 0.0)
    return {"loss": (tau * tau * terms.sum(1), tau * tau * mag.sum(1)), "lse": (lse, lse.abs() + big)}


def distill_backward(logits, t, ids, tau, loss_grad, lse=None):
    z = logits.double() / tau
    lse = torch.logsumexp(z, 1) if lse is None else lse.double()
    q, _, some = teacher(t, ids, z.shape[1], tau)
    on = some & (loss_grad != 0)
    p = torch.where(torch.isneginf(lse)[:, None], 0.0, (z - lse[:, None]).exp())
    by = (loss_grad.double() * tau)[:, None]
    at = ids.long().clamp(0, z.shape[1] - 1)
    d = p.scatter_add(1, at, -q) * by
    # z / tau and lse are each rounded to 32 bits before their difference is raised
    x = torch.where(torch.isfinite(z), z.abs(), 0) + torch.where(torch.isfinite(lse), lse.abs(), 0)[:, None]
    top = torch.where(torch.isfinite(t), t.double().abs(), 0).max(1, keepdim=True).values / tau
    mag = (p * (1 + x) + torch.zeros_like(p).scatter_add(1, at, q * (1 + top))) * by.abs()
    keep = on[:, None]
    return torch.where(keep, d, 0.0), torch.where(keep, mag, 0.0)
