"""Operators of a training and a decoding step over the ranks, as they are measured: the global norm of the gradients
that an AllReduce or a reduce-scatter leaves, and their clipping; a layer's product in 8-bit whole numbers, with a scale
for each token and channel, whose inner width or whose channels are dealt out to the ranks; and the penalties, biases and
grammar masks of logits whose columns are dealt out to the ranks.
"""
import math
import random

import torch

own = False

_TYPES = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16}
_SIZE = {"fp32": 4, "fp16": 2, "bf16": 2}
_EPS = 1e-6
_SIGMA = 0.02
_comms = {}


def _comm(ranks):
    """The communicator that a program keeps for its ranks."""
    if ranks not in _comms:
        import allreduce_reduction_amd as hc
        _comms[ranks] = hc.Comm(ranks, "ring")
    return _comms[ranks]


def listed():
    return [
        # the adapters' gradients of a fine-tuned model after their AllReduce: a few small tensors, launches alone
        {"name": "clip_few", "op": "clip", "ranks": 8, "layout": "same", "elements": 40013, "tensors": 13, "dtype": "bf16",
         "norm": "2"},
        # a data-parallel step: every rank holds the summed gradients of the model, the sum made a mean on the way
        {"name": "clip_same", "op": "clip", "ranks": 8, "layout": "same", "elements": 48000000, "tensors": 290,
         "dtype": "bf16", "norm": "2"},
        # a step whose gradients a reduce-scatter dealt out: each rank holds and clips its own share in 32 bits
        {"name": "clip_dealt", "op": "clip", "ranks": 8, "layout": "dealt", "elements": 268435456, "tensors": 96,
         "dtype": "fp32", "norm": "2"},
        # five ranks, half of the tensors in 32 bits, odd lengths, clipped by their largest value
        {"name": "clip_odd", "op": "clip", "ranks": 5, "layout": "dealt", "elements": 30000001, "tensors": 173,
         "dtype": "mixed", "norm": "inf"},
        # a decode step of one sequence of a few hundred tokens
        {"name": "logits_token", "op": "logits", "ranks": 8, "rows": 1, "vocab": 131072, "dtype": "bf16", "history": 700,
         "bias": 12, "mask": True, "in_place": True, "wide_ids": True},
        # a decode step of a full batch, in place
        {"name": "logits_batch", "op": "logits", "ranks": 8, "rows": 256, "vocab": 131072, "dtype": "bf16", "history": 2048,
         "bias": 32, "mask": True, "in_place": True, "wide_ids": True},
        # an odd vocabulary over six ranks, no grammar, the model's own logits kept
        {"name": "logits_odd", "op": "logits", "ranks": 6, "rows": 33, "vocab": 50001, "dtype": "fp16", "history": 301,
         "bias": 5, "mask": False, "in_place": False, "wide_ids": False},
        # many sequences of a long history, the model's own logits kept in 32 bits
        {"name": "logits_long", "op": "logits", "ranks": 4, "rows": 128, "vocab": 200064, "dtype": "fp32", "history": 16384,
         "bias": 0, "mask": True, "in_place": False, "wide_ids": False},
        # a decode step of three sequences through a layer whose inner width is dealt out, its sum on every rank
        {"name": "w8_token", "op": "w8", "form": "reduce", "ranks": 8, "rows": 3, "inner": 8192, "channels": 4096,
         "dtype": "bf16"},
        # odd sizes, the channels dealt out to five ranks
        {"name": "w8_odd", "op": "w8", "form": "own", "ranks": 5, "rows": 77, "inner": 1001, "channels": 5003,
         "dtype": "fp16"},
        # the logits of 64 sequences, the vocabulary dealt out
        {"name": "w8_logits", "op": "w8", "form": "own", "ranks": 8, "rows": 64, "inner": 4096, "channels": 131072,
         "dtype": "bf16"},
        # the prompts of a batch through a layer whose inner width is dealt out, each rank left with its own tokens' rows
        {"name": "w8_batch", "op": "w8", "form": "scatter", "ranks": 8, "rows": 4096, "inner": 8192, "channels": 4096,
         "dtype": "bf16"},
    ]


def _spread(rng, lo, hi):
    """A whole number of [lo, hi], even over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    most = {k: max(work(c)[k] for c in listed()) for k in ("bytes", "flops")}
    op = rng.choice(("clip", "clip", "clip", "logits", "logits", "logits", "w8", "w8", "w8"))
    case = {"op": op, "ranks": rng.choice((1, 2, 3, 4, 5, 7, 8, 8, 12, 16)), "dtype": rng.choice(("bf16", "bf16", "fp16", "fp32"))}
    if op == "clip":
        case.update(layout=rng.choice(("same", "dealt")), elements=_spread(rng, 1000, 1 << 28), tensors=_spread(rng, 1, 400),
                    norm=rng.choice(("2", "2", "2", "1", "inf")))
        if rng.random() < 0.3:
            case["dtype"] = "mixed"
        axes = ("elements",)
    elif op == "logits":
        case.update(rows=_spread(rng, 1, 512), vocab=_spread(rng, 500, 262144), history=rng.choice((0, 1, 1, 1)) * _spread(rng, 1, 16384),
                    bias=rng.choice((0, 1, 1)) * _spread(rng, 1, 300), mask=rng.random() < 0.6, in_place=rng.random() < 0.5,
                    wide_ids=rng.random() < 0.5)
        case["mask"] = case["mask"] or not (case["history"] or case["bias"])
        axes = ("rows", "vocab")
    else:
        even = rng.random() < 0.5
        case.update(form=rng.choice(("reduce", "scatter", "own")), rows=_spread(rng, 1, 4096),
                    inner=256 * rng.randint(1, 56) if even else _spread(rng, 16, 14336),
                    channels=256 * rng.randint(1, 56) if even else _spread(rng, 16, 65536))
        axes = ("rows", "channels", "inner")
    while any(work(case)[k] > most[k] for k in most):
        axis = max(axes, key=lambda a: case[a])
        case[axis] = max(1, case[axis] // 2)
    return case


def _deal(n, ranks):
    """Rows or columns of n on each rank (the ceiling split)."""
    each = -(-n // ranks)
    return [max(0, min(each, n - r * each)) for r in range(ranks)]


def _lengths(case):
    """The tensors' lengths: matrices and vectors, the largest some thousand times the smallest."""
    rng = random.Random(case["elements"] * 1009 + case["tensors"])
    w = [math.exp(rng.uniform(0.0, 8.0)) for _ in range(case["tensors"])]
    return [max(1, int(case["elements"] * x / sum(w))) for x in w]


def _typed(case):
    """(type, lengths of the tensors that have it), the tensors' whole list dealt to the types in turn."""
    n = _lengths(case)
    if case["dtype"] != "mixed":
        return [(case["dtype"], n)]
    return [(t, n[i::2]) for i, t in enumerate(("bf16", "fp32")) if n[i::2]]


def work(case):
    ranks = case["ranks"]
    if case["op"] == "clip":
        held = sum(sum(n) * _SIZE[t] for t, n in _typed(case))
        copies = ranks if case["layout"] == "same" else 1
        return {"bytes": held * (1 + copies), "flops": sum(_lengths(case)) * (2 + copies)}
    if case["op"] == "logits":
        rows, v, size = case["rows"], case["vocab"], _SIZE[case["dtype"]]
        ids = 8 if case["wide_ids"] else 4
        lists = rows * ((case["history"] * ids + 16 + 12 if case["history"] else 0) + case["bias"] * (ids + 4))
        # in place: the masked columns are written (two in five, see prepare), and the named ones read and written
        named = rows * min(v, case["history"] + case["bias"])
        moved = (2 * rows * v // 5 * size if case["mask"] else 0) + 2 * named * size if case["in_place"] else 2 * rows * v * size
        return {"bytes": moved + lists + (rows * v // 8 if case["mask"] else 0), "flops": 4 * named + rows * v}
    t, k, n, size = case["rows"], case["inner"], case["channels"], _SIZE[case["dtype"]]
    out = t * n * size * (ranks if case["form"] == "reduce" else 1)
    # the activations in, their codes out and in again, the weights, the scales, the result
    return {"bytes": t * k * (size + 2) + n * k + 8 * t + 4 * n + out, "flops": 2 * t * n * k}


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    ranks = case["ranks"]

    def normal(*shape, by=1.0, mean=0.0):
        return torch.randn(*shape, generator=g, device=dev, dtype=torch.float32).mul_(by).add_(mean)

    def uniform(*shape, lo=0.0, hi=1.0):
        return torch.rand(*shape, generator=g, device=dev, dtype=torch.float32).mul_(hi - lo).add_(lo)

    s = dict(case)
    if case["op"] == "clip":
        s["scale"] = 1.0 / ranks if ranks > 1 else 0.5
        s["flat"], s["lists"], total = [], [[] for _ in range(ranks)], 0
        for name, lengths in _typed(case):
            n = sum(lengths)
            total += n
            flat = torch.empty(ranks if case["layout"] == "same" else 1, n, device=dev, dtype=_TYPES[name])
            for a in range(0, n, 1 << 26):
                flat[:, a:a + (1 << 26)] = normal(min(1 << 26, n - a), by=_SIGMA)
            s["flat"].append(flat)
            if case["layout"] == "same":
                for r in range(ranks):
                    s["lists"][r] += flat[r].split(lengths)
            else:
                for i, x in enumerate(flat[0].split(lengths)):
                    s["lists"][i % ranks].append(x)
        s["norm_out"] = torch.empty(1, device=dev, dtype=torch.float32)
        typical = {"2": math.sqrt(total), "1": 0.8 * total, "inf": 4.0}[case["norm"]]
        s["max_norm"] = 0.4 * _SIGMA * s["scale"] * typical
        return s
    if case["op"] == "logits":
        rows, v, dt = case["rows"], case["vocab"], _TYPES[case["dtype"]]
        whole = torch.empty(rows, v, device=dev, dtype=dt)
        for a in range(0, rows, 64):
            whole[a:a + 64] = normal(min(64, rows - a), v, by=3.0)
        s["logits"] = [x.contiguous() for x in whole.split(_deal(v, ranks), 1)]
        s["out"] = s["logits"] if case["in_place"] else [torch.empty_like(x) for x in s["logits"]]
        id_type = torch.int64 if case["wide_ids"] else torch.int32
        length = case["history"]
        s["tokens"] = s["prompt_lengths"] = s["lengths"] = None
        s["repetition"] = s["frequency"] = s["presence"] = None
        if length:
            # few tokens of the vocabulary are frequent: ids even over their logarithm; sequences of unequal lengths, padded
            u = torch.rand(rows, length, generator=g, device=dev, dtype=torch.float64)
            ids = torch.exp(u * math.log(v + 1)).long().sub_(1).clamp_(0, v - 1)
            ids = (ids * 7919 + 13) % v
            s["lengths"] = (uniform(rows, lo=0.5, hi=1.0) * length).ceil().int().clamp_(0, length)
            s["prompt_lengths"] = (uniform(rows, lo=0.2, hi=0.9) * s["lengths"]).int()
            ids[torch.arange(length, device=dev) >= s["lengths"][:, None]] = -1
            s["tokens"] = ids.to(id_type)
            s["repetition"] = uniform(rows, lo=1.0, hi=1.4)
            s["frequency"] = uniform(rows, lo=0.0, hi=0.5)
            s["presence"] = uniform(rows, lo=-0.2, hi=0.5)
        s["bias_ids"] = s["bias_values"] = None
        if case["bias"]:
            start = torch.randint(0, v, (rows, 1), generator=g, device=dev)
            ids = (start + 104729 * torch.arange(case["bias"], device=dev)) % v
            ids = torch.where(torch.rand(rows, case["bias"], generator=g, device=dev) < 0.1, -1, ids)
            s["bias_ids"], s["bias_values"] = ids.to(id_type), normal(rows, case["bias"], by=4.0)
        s["bits"] = None
        if case["mask"]:
            # a third of the rows free of any grammar, a third inside strings (most columns allowed), a third at a name or
            # a bracket (hardly any)
            words = -(-v // 32)
            kind = torch.arange(rows, device=dev) + seed
            bits = torch.randint(-2 ** 31, 2 ** 31, (rows, words), generator=g, device=dev, dtype=torch.int64)
            more = torch.randint(-2 ** 31, 2 ** 31, (rows, words), generator=g, device=dev, dtype=torch.int64)
            few = bits & more & (torch.rand(rows, words, generator=g, device=dev) < 0.05)
            bits = torch.where((kind % 3 == 0)[:, None], -1, torch.where((kind % 3 == 1)[:, None], bits | more, few))
            s["bits"] = bits.to(torch.int32)
        return s
    t, k, n, dt = case["rows"], case["inner"], case["channels"], _TYPES[case["dtype"]]
    columns = case["form"] == "own"
    x = normal(t, k) * torch.where(torch.rand(k, generator=g, device=dev) < 0.01, 12.0, 1.0)
    x[t - t // 17:] = 0  # the padding of a batch
    s["x"] = [x.to(dt)] if columns else [p.contiguous() for p in x.to(dt).split(_deal(k, ranks), 1)]
    s["q"] = [torch.empty(p.shape, device=dev, dtype=torch.int8) for p in s["x"]]
    s["x_scale"] = torch.empty(t, device=dev, dtype=torch.float32)
    each = [(c, k) for c in _deal(n, ranks)] if columns else [(n, c) for c in _deal(k, ranks)]
    s["w"] = [torch.randint(-127, 128, shape, generator=g, device=dev, dtype=torch.int8) for shape in each]
    scale = uniform(n, lo=0.5, hi=1.5) / (74.0 * math.sqrt(k))
    s["w_scale"] = list(scale.split(_deal(n, ranks))) if columns else scale
    if columns:
        s["out"] = [torch.empty(t, c, device=dev, dtype=dt) for c in _deal(n, ranks)]
    elif case["form"] == "reduce":
        s["out"] = list(torch.empty(ranks, t, n, device=dev, dtype=dt))
    else:
        s["out"] = [torch.empty(c, n, device=dev, dtype=dt) for c in _deal(t, ranks)]
    return s


# ------------------------------------------------------------ the plain forms


def _clip(s):
    held = [x[:1].float() for x in s["flat"]]
    if s["norm"] == "2":
        n = torch.sqrt(sum(x.square().sum(dtype=torch.float64) for x in held))
    elif s["norm"] == "1":
        n = sum(x.abs().sum(dtype=torch.float64) for x in held)
    else:
        n = torch.stack([x.abs().max() for x in held]).max().double()
    n = s["scale"] * n
    s["norm_out"].copy_(n)
    factor = (s["scale"] * torch.clamp(s["max_norm"] / (n + _EPS), max=1.0)).float()
    s["flat"] = [x.copy_(x.float() * factor) for x in s["flat"]]


def _logits(s):
    z = torch.cat(s["logits"], 1).float()
    v = s["vocab"]
    if s["tokens"] is not None:
        at = torch.arange(s["history"], device=z.device)
        real = (s["tokens"] >= 0) & (s["tokens"] < v) & (at < s["lengths"][:, None])
        ids = torch.where(real, s["tokens"], 0).long()
        said = real & (at >= s["prompt_lengths"][:, None])
        seen = torch.zeros(z.shape, dtype=torch.int32, device=z.device).scatter_add_(1, ids, real.int())
        count = torch.zeros(z.shape, dtype=torch.int32, device=z.device).scatter_add_(1, ids, said.int())
        by = s["repetition"][:, None]
        z = torch.where(seen > 0, torch.where(z > 0, z / by, z * by), z)
        z = torch.where(count > 0, z - s["frequency"][:, None] * count - s["presence"][:, None], z)
    if s["bias_ids"] is not None:
        real = (s["bias_ids"] >= 0) & (s["bias_ids"] < v)
        z = z.scatter_add(1, torch.where(real, s["bias_ids"], 0).long(), torch.where(real, s["bias_values"], 0.0))
    if s["bits"] is not None:
        column = torch.arange(v, device=z.device)
        allowed = (s["bits"][:, column >> 5] >> (column & 31)) & 1
        z = torch.where(allowed != 0, z, -math.inf)
    torch._foreach_copy_(s["out"], list(z.split([x.shape[1] for x in s["out"]], 1)))


def _w8(s):
    x = torch.cat(s["x"], 1).float()
    most = x.abs().amax(1, keepdim=True)
    q = torch.where(most > 0, torch.round(x * (127.0 / most)).clamp(-127, 127), 0.0)
    s["x_scale"].copy_(most[:, 0] / 127.0)
    torch._foreach_copy_(s["q"], list(q.split([p.shape[1] for p in s["q"]], 1)))
    columns = s["form"] == "own"
    w = torch.cat(s["w"], 0 if columns else 1).float()
    y = (q @ w.t()) * s["x_scale"][:, None] * (torch.cat(s["w_scale"]) if columns else s["w_scale"])
    parts = y.split([p.shape[1] for p in s["out"]], 1) if columns else y.split([p.shape[0] for p in s["out"]]) if s["form"] == "scatter" else [y] * s["ranks"]
    torch._foreach_copy_(s["out"], list(parts))


def run(s):
    op = s["op"]
    if own:
        comm = _comm(s["ranks"])
        if op == "clip":
            if "gradients" not in s:  # what a program keeps for its gradients' buffers
                s["gradients"] = comm.gradients(**{s["layout"]: s["lists"]})
            s["gradients"].clip(s["max_norm"], s["norm_out"], norm_type=float(s["norm"]), scale=s["scale"], eps=_EPS)
        elif op == "logits":
            comm.adjust_logits(s["logits"], s["out"], tokens=s["tokens"], prompt_lengths=s["prompt_lengths"], lengths=s["lengths"],
                               repetition=s["repetition"], frequency=s["frequency"], presence=s["presence"],
                               bias_ids=s["bias_ids"], bias=s["bias_values"], mask=s["bits"])
        elif s["form"] == "own":
            _comm(1).quantize_rows(s["x"], s["q"], s["x_scale"])
            comm.product(s["q"] * s["ranks"], s["x_scale"], s["w"], s["w_scale"], s["out"])
        else:
            comm.quantize_rows(s["x"], s["q"], s["x_scale"])
            comm.reduce_product(s["q"], s["x_scale"], s["w"], s["w_scale"], s["out"], scatter=s["form"] == "scatter")
    else:
        {"clip": _clip, "logits": _logits, "w8": _w8}[op](s)
    if op == "clip":
        return {"norm": s["norm_out"], "grads": s["flat"]}
    if op == "logits":
        return {"logits": s["out"]}
    return {"out": s["out"], "codes": s["q"], "scale": s["x_scale"]}


# ------------------------------------------------- the definitions in 64 bits


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "clip":
        size = 0.0
        for flat in s["flat"]:
            for part in flat[0].split(1 << 26):
                x = part.double().abs()
                size = max(size, float(x.max())) if case["norm"] == "inf" else size + float(x.sum() if case["norm"] == "1" else (x * x).sum())
        size = s["scale"] * (math.sqrt(size) if case["norm"] == "2" else size)
        norm = torch.full((1,), size, dtype=torch.float64)
        by = s["scale"] * min(1.0, s["max_norm"] / (size + _EPS))
        return {"norm": norm, "grads": [(x[:1].double() * by).expand(x.shape) for x in s["flat"]]}
    if op == "logits":
        found = []
        edges = [0]
        for x in s["logits"]:
            edges.append(edges[-1] + x.shape[1])
        for row in range(case["rows"]):
            z = torch.cat([x[row] for x in s["logits"]]).double()
            if case["history"]:
                end, start = int(s["lengths"][row]), int(s["prompt_lengths"][row])
                line = s["tokens"][row].long()
                every, said = line[:end], line[start:end]
                names = every[(every >= 0) & (every < case["vocab"])].unique()
                by = float(s["repetition"][row])
                z[names] = torch.where(z[names] > 0, z[names] / by, z[names] * by)
                names, count = said[(said >= 0) & (said < case["vocab"])].unique(return_counts=True)
                z[names] -= float(s["frequency"][row]) * count + float(s["presence"][row])
            if case["bias"]:
                names = s["bias_ids"][row].long()
                known = (names >= 0) & (names < case["vocab"])
                z.index_add_(0, names[known], s["bias_values"][row][known].double())
            if case["mask"]:
                on = (s["bits"][row][:, None] >> torch.arange(32, device="cuda")).reshape(-1)[:case["vocab"]] & 1
                z[on == 0] = -math.inf
            found.append(z)
        whole = torch.stack(found)
        return {"logits": [whole[:, a:b].contiguous() for a, b in zip(edges, edges[1:])]}
    # the codes are defined by their 32-bit arithmetic, all that follows from them is taken in 64 bits
    x = torch.cat(s["x"], 1).float()
    most = x.abs().max(1).values
    codes = torch.round(x * (127.0 / torch.where(most > 0, most, 1.0))[:, None])
    scale = most.double() / 127.0
    w_scale = (torch.cat(s["w_scale"]) if case["form"] == "own" else s["w_scale"]).double()
    w = torch.cat(s["w"], 0 if case["form"] == "own" else 1)
    y = torch.cat([codes.double() @ part.double().t() for part in w.split(8192)], 1) * scale[:, None] * w_scale
    if case["form"] == "own":
        out = [p.contiguous() for p in y.split([p.shape[1] for p in s["out"]], 1)]
    else:
        out = list(y.split([p.shape[0] for p in s["out"]])) if case["form"] == "scatter" else [y] * case["ranks"]
    return {"out": out, "codes": [None] * len(s["q"]), "scale": scale}
