"""The operators of a training and a decoding step over the ranks in 64 bits,
written from their formulas: clipping of gradients, what is done to logits
before a token is chosen, products of 8-bit codes.  As in rankops_ref, a value
comes with its magnitude: a chain of n roundings to 32 bits moves it by at most
about n * 2^-24 * magnitude.
"""
import torch


def norm(tensors, norm_type, scale=1.0):
    """Each tensor once, on the CPU, in 64 bits."""
    flat = torch.cat([t.double().flatten().abs() for t in tensors] + [torch.zeros(1, dtype=torch.float64)])
    by = {1.0: lambda: flat.sum(), 2.0: lambda: flat.square().sum().sqrt(), float("inf"): lambda: flat.max()}[norm_type]()
    return abs(scale) * by


def factor(size, max_norm, scale=1.0, eps=1e-6):
    most = size + eps
    return scale * (1.0 if max_norm >= most else float(max_norm / most))


def adjust(logits, tokens=None, prompt_lengths=None, lengths=None, repetition=None, frequency=None, presence=None,
           bias_ids=None, bias=None, mask=None):
    """[rows, vocab] of every rank together, in 64 bits; its magnitude."""
    z = logits.double().clone()
    mag = z.abs()
    rows, vocab = z.shape
    for r in range(rows):
        if tokens is not None:
            end = tokens.shape[1] if lengths is None else min(max(int(lengths[r]), 0), tokens.shape[1])
            start = 0 if prompt_lengths is None else min(max(int(prompt_lengths[r]), 0), end)
            line = tokens[r, :end].long()
            seen, said = [x[(x >= 0) & (x < vocab)] for x in (line, line[start:])]
            at = seen.unique()
            if repetition is not None:
                by = float(repetition[r])
                z[r, at] = torch.where(z[r, at] > 0, z[r, at] / by, z[r, at] * by)
                mag[r, at] *= max(abs(by), abs(1 / by) if by else 0)
            at, count = said.unique(return_counts=True)
            if frequency is not None:
                z[r, at] -= float(frequency[r]) * count
                mag[r, at] += abs(float(frequency[r])) * count
            if presence is not None:
                z[r, at] -= float(presence[r])
                mag[r, at] += abs(float(presence[r]))
        if bias_ids is not None:
            at = bias_ids[r].long()
            on = (at >= 0) & (at < vocab)
            z[r].index_add_(0, at[on], bias[r][on].double())
            mag[r].index_add_(0, at[on], bias[r][on].double().abs())
    if mask is not None:
        z[~allowed(mask, vocab)] = -torch.inf
    return z, mag


def allowed(mask, vocab):
    v = torch.arange(vocab)
    return (mask[:, v // 32].long() >> (v % 32)) & 1 != 0


def bits(on):
    """The mask [rows, ceil(vocab / 32)] of the allowed columns [rows, vocab]."""
    rows, vocab = on.shape
    padded = torch.zeros(rows, -(-vocab // 32) * 32, dtype=torch.int64)
    padded[:, :vocab] = on
    words = (padded.view(rows, -1, 32) << torch.arange(32)).sum(2)
    return torch.where(words >= 2 ** 31, words - 2 ** 32, words).to(torch.int32)


def codes(x):
    """The codes and scales of rows, in the 32-bit steps that define them."""
    x = x.float()
    most = x.abs().amax(1) if x.shape[1] else torch.zeros(x.shape[0])
    by = torch.div(torch.ones_like(most), most) * torch.tensor(127.0)
    good = torch.isfinite(by) & torch.isfinite(most) & (most > 0)
    q = torch.where(good[:, None], torch.round(x * by[:, None]).clamp(-127, 127), 0.0).to(torch.int8)
    scale = torch.where(good, torch.div(most, torch.full_like(most, 127.0)), 0.0)
    return q, torch.where(torch.isfinite(x).all(1), scale, torch.nan)


def product(q, x_scale, w, w_scale):
    y = (q.double() @ w.double().t()) * x_scale.double()[:, None] * w_scale.double()
    return y, y.abs()
