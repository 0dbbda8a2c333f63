"""The operators where a model's own work meets a collective, as they are measured: the norms at a block's end over
the ranks' partial sums, the embedding whose rows are dealt out to the ranks, and the distillation loss over logits whose
columns are dealt out to the ranks, each with its gradient.

Every case holds the P logical ranks' buffers in one allocation, rank after rank, so that the plain forms need no loop
over the ranks; the framework's operators take the ranks' own buffers (views of it).
"""
import math

import torch

own = False

_TYPES = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16}
_EPS = 1e-6
_comms = {}


def _comm(ranks):
    """The communicator that a program keeps for its ranks."""
    if ranks not in _comms:
        import allreduce_reduction_amd as hc
        _comms[ranks] = hc.Comm(ranks, "ring")
    return _comms[ranks]


def listed():
    return [
        # one token of one sequence at the end of a block of 8 ranks: a decode step's latency
        {"name": "norm_token", "op": "norm", "ranks": 8, "rows": 1, "width": 4096, "dtype": "bf16", "post": True,
         "gates": 1, "save": False},
        # a training step's forward pass: 4096 tokens, the sums kept for the backward pass
        {"name": "norm_batch", "op": "norm", "ranks": 8, "rows": 4096, "width": 4096, "dtype": "bf16", "post": True,
         "gates": 1, "save": True},
        # odd rows and width, a gate row for each of nine sequences of 37 tokens
        {"name": "norm_grad_odd", "op": "norm_grad", "ranks": 5, "rows": 333, "width": 1001, "dtype": "fp16",
         "post": True, "gates": 9},
        # the training step's backward pass
        {"name": "norm_grad_batch", "op": "norm_grad", "ranks": 8, "rows": 4096, "width": 4096, "dtype": "bf16",
         "post": True, "gates": 1},
        # a decode step of three sequences a rank
        {"name": "embed_token", "op": "embed", "ranks": 8, "tokens": 3, "vocab": 32768, "width": 2048, "dtype": "bf16",
         "wide_ids": True, "uneven": False},
        # the prompts of a batch: 4096 tokens a rank
        {"name": "embed_batch", "op": "embed", "ranks": 8, "tokens": 4096, "vocab": 131072, "width": 4096,
         "dtype": "bf16", "wide_ids": True, "uneven": False},
        # few tokens, unequal over five ranks, a whole gradient written in the activations' type
        {"name": "embed_grad_odd", "op": "embed_grad", "ranks": 5, "tokens": 701, "vocab": 50001, "width": 1000,
         "dtype": "fp16", "grad": "fp16", "accumulate": False, "wide_ids": False, "uneven": True},
        # a micro-batch added to the 32-bit gradient of a training step
        {"name": "embed_grad_batch", "op": "embed_grad", "ranks": 8, "tokens": 4096, "vocab": 65536, "width": 4096,
         "dtype": "bf16", "grad": "fp32", "accumulate": True, "wide_ids": True, "uneven": False},
        # a few rows in 32 bits
        {"name": "distill_rows", "op": "distill", "ranks": 4, "rows": 7, "vocab": 50001, "top": 20, "dtype": "fp32",
         "temperature": 1.0, "wide_ids": True},
        # a training step's loss over 2048 tokens
        {"name": "distill_batch", "op": "distill", "ranks": 8, "rows": 2048, "vocab": 131072, "top": 64,
         "dtype": "bf16", "temperature": 2.0, "wide_ids": True},
        # an odd vocabulary over six ranks, the last one shorter
        {"name": "distill_grad_odd", "op": "distill_grad", "ranks": 6, "rows": 100, "vocab": 32003, "top": 33,
         "dtype": "fp16", "temperature": 1.5, "wide_ids": False},
        # the training step's gradient of the logits
        {"name": "distill_grad_batch", "op": "distill_grad", "ranks": 8, "rows": 2048, "vocab": 131072, "top": 64,
         "dtype": "bf16", "temperature": 2.0, "wide_ids": True},
    ]


def _spread(rng, lo, hi):
    """A whole number of [lo, hi], even over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    most = max(work(c)["bytes"] for c in listed())
    op = rng.choice(("norm", "norm_grad", "embed", "embed_grad", "distill", "distill_grad"))
    case = {"op": op, "ranks": rng.choice((1, 2, 3, 4, 5, 7, 8, 8, 12, 16)), "dtype": rng.choice(("bf16", "bf16", "fp16", "fp32"))}
    if op.startswith("norm"):
        case.update(rows=_spread(rng, 1, 8192), width=_spread(rng, 64, 16384) if rng.random() < 0.5 else 256 * rng.randint(1, 64),
                    post=rng.random() < 0.7)
        rows = case["rows"]
        case["gates"] = rng.choice([0, 1, 1] + [d for d in (2, 3, 4, 8, rows) if rows % d == 0])
        if op == "norm":
            case["save"] = rng.random() < 0.5
        axis = "rows"
    elif op.startswith("embed"):
        case.update(tokens=_spread(rng, 1, 8192), vocab=_spread(rng, 500, 131072),
                    width=_spread(rng, 64, 8192) if rng.random() < 0.5 else 256 * rng.randint(1, 32),
                    wide_ids=rng.random() < 0.5, uneven=rng.random() < 0.5)
        if op == "embed_grad":
            case.update(grad=rng.choice(("fp32", case["dtype"])), accumulate=rng.random() < 0.5)
        axis = "tokens"
    else:
        case.update(rows=_spread(rng, 1, 4096), vocab=_spread(rng, 1000, 262144), top=_spread(rng, 1, 256),
                    temperature=rng.choice((1.0, 1.5, 2.0, 4.0)), wide_ids=rng.random() < 0.5)
        axis = "rows"
    while work(case)["bytes"] > most and case[axis] > 1:
        case[axis] = max(1, case[axis] // 2)
        if op.startswith("norm") and case["gates"] > 1:
            case["gates"] = 1
    while work(case)["bytes"] > most:
        case["vocab"] = case["vocab"] // 2
    return case


def _tokens(case):
    """Tokens of each rank: equal, or fewer from rank to rank with some ranks left without any."""
    n, ranks = case["tokens"], case["ranks"]
    return [n] * ranks if not case["uneven"] else [max(0, n - (r * r * n) // (ranks + 3)) for r in range(ranks)]


def _columns(case):
    """Columns of the vocabulary on each rank (the ceiling split)."""
    n, ranks = case["vocab"], case["ranks"]
    each = -(-n // ranks)
    return [max(0, min(each, n - r * each)) for r in range(ranks)]


def work(case):
    size = 4 if case["dtype"] == "fp32" else 2
    ranks = case["ranks"]
    if case["op"] == "norm":
        block = case["rows"] * case["width"]
        held = 2 + (1 if case["save"] else 0)
        return {"bytes": (2 * ranks + held) * block * size + (1 + case["post"] + case["gates"]) * case["width"] * size,
                "flops": (ranks + 11) * block}
    if case["op"] == "norm_grad":
        block = case["rows"] * case["width"]
        kept = 1 if case["post"] or case["gates"] else 0
        return {"bytes": (2 * ranks + 3 + kept) * block * size + (1 + case["post"] + case["gates"]) * case["width"] * (size + 4),
                "flops": (ranks + 25) * block}
    if case["op"].startswith("embed"):
        total, width = sum(_tokens(case)), case["width"]
        ids = total * (8 if case["wide_ids"] else 4)
        # distinct ids of ids drawn evenly over the logarithm of their rank
        v = case["vocab"]
        seen = sum(1.0 - (1.0 - 0.97 * math.log1p(1.0 / x) / math.log(v + 1)) ** total * 1.0 for x in range(1, min(v, 64) + 1))
        if v > 64:
            edges = [64 * (v / 64) ** (k / 64) for k in range(65)]
            seen += sum((b - a) * (1.0 - (1.0 - 0.97 / (0.5 * (a + b)) / math.log(v + 1)) ** total) for a, b in zip(edges, edges[1:]))
        if case["op"] == "embed":
            return {"bytes": (min(total, seen) + total) * width * size + ids, "flops": total * width}
        out = 4 if case["grad"] == "fp32" else 2
        written = 2 * min(total, seen) if case["accumulate"] else v
        return {"bytes": total * width * size + written * width * out + ids, "flops": 2 * total * width}
    block = case["rows"] * case["vocab"]
    top = case["rows"] * case["top"] * (4 + (8 if case["wide_ids"] else 4))
    if case["op"] == "distill":
        return {"bytes": block * size + top + 8 * case["rows"], "flops": 4 * block}
    return {"bytes": 2 * block * size + top + 8 * case["rows"], "flops": 4 * block}


def _rows_of(whole, ranks):
    """The ranks' row segments of a matrix (the ceiling split), as views."""
    n = whole.shape[0]
    each = -(-n // ranks)
    return [whole[min(n, r * each):min(n, (r + 1) * each)] for r in range(ranks)]


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    dt = _TYPES[case["dtype"]]
    ranks = case["ranks"]

    def normal(*shape, by=1.0, mean=0.0):
        return torch.randn(*shape, generator=g, device=dev, dtype=torch.float32).mul_(by).add_(mean)

    s = dict(case)
    if case["op"].startswith("norm"):
        t, h = case["rows"], case["width"]
        s["scale"] = 0.5
        s["pre"] = normal(h, by=0.1, mean=1.0).to(dt)
        s["post_w"] = normal(h, by=0.1, mean=1.0).to(dt) if case["post"] else None
        s["gate"] = normal(case["gates"], h, by=0.3, mean=0.7).to(dt) if case["gates"] else None
        stack = torch.empty(ranks, t, h, device=dev, dtype=dt)
        for r in range(ranks):
            stack[r] = normal(t, h, by=1.0 / math.sqrt(ranks) if case["op"] == "norm" else 0.1)
        s["parts" if case["op"] == "norm" else "out_grads"] = stack
        s["out" if case["op"] == "norm" else "part_grads"] = torch.empty_like(stack)
        if case["op"] == "norm":
            s["residual"] = normal(t, h, by=2.0).to(dt)
            s["residual_out"] = torch.empty_like(s["residual"])
            s["sums"] = torch.empty_like(s["residual"]) if case["save"] else None
            names = ("residual", "residual_out", "sums")
        else:
            s["hidden"] = normal(t, h, by=2.0).to(dt)
            s["sums"] = normal(t, h).to(dt) if case["post"] or case["gates"] else None
            s["residual_grad"] = normal(t, h, by=0.1).to(dt)
            s["residual_grad_out"] = torch.empty_like(s["hidden"])
            s["pre_grad"] = torch.empty(h, device=dev, dtype=torch.float32)
            s["post_grad"] = torch.empty(h, device=dev, dtype=torch.float32) if case["post"] else None
            s["gate_grad"] = torch.empty(case["gates"], h, device=dev, dtype=torch.float32) if case["gates"] else None
            names = ("hidden", "sums", "residual_grad", "residual_grad_out")
        for n in names:
            s[n + "_ranks"] = None if s[n] is None else _rows_of(s[n], ranks)
        return s
    if case["op"].startswith("embed"):
        counts, v, h = _tokens(case), case["vocab"], case["width"]
        total = sum(counts)
        # few tokens of the vocabulary are frequent: ids even over their logarithm; 3 of 100 are padding
        u = torch.rand(total, generator=g, device=dev, dtype=torch.float64)
        ids = torch.exp(u * math.log(v + 1)).long().sub_(1).clamp_(0, v - 1)
        ids = torch.where(torch.rand(total, generator=g, device=dev) < 0.03, -1, ids)
        s["ids"] = ids if case["wide_ids"] else ids.int()
        s["ids_ranks"] = list(s["ids"].split(counts))
        s["scale"] = math.sqrt(h)
        whole = torch.empty(v, h, device=dev, dtype=dt if case["op"] == "embed" else _TYPES[case["grad"]])
        if case["op"] == "embed":
            for a in range(0, v, 8192):
                whole[a:a + 8192] = normal(min(8192, v - a), h, by=0.02)
            s["table"], s["table_ranks"] = whole, _rows_of(whole, ranks)
            s["out"] = torch.empty(total, h, device=dev, dtype=dt)
            s["out_ranks"] = list(s["out"].split(counts))
        else:
            whole.zero_()
            s["grads"], s["grads_ranks"] = whole, _rows_of(whole, ranks)
            s["out_grads"] = normal(total, h, by=0.1).to(dt)
            s["out_grads_ranks"] = list(s["out_grads"].split(counts))
        return s
    n, v, k = case["rows"], case["vocab"], case["top"]
    start = torch.randint(0, v, (n, 1), generator=g, device=dev)
    ids = (start + 7919 * torch.arange(k, device=dev)) % v
    logits = torch.empty(n, v, device=dev, dtype=dt)
    for a in range(0, n, 256):
        z = normal(min(256, n - a), v, by=2.0)
        z.scatter_add_(1, ids[a:a + 256], normal(z.shape[0], k, by=1.0, mean=5.0))
        logits[a:a + 256] = z
    s["logits"] = [x.contiguous() for x in logits.split(_columns(case), 1)]
    teacher = normal(n, k, by=2.0, mean=8.0)
    s["teacher"] = teacher.sort(dim=1, descending=True).values.to(dt)
    rows = torch.arange(n, device=dev)[:, None]
    ids = torch.where((rows % 37 == 36) | (torch.arange(k, device=dev) >= k - rows % 3), -1, ids) if k > 3 else ids
    s["ids"] = ids.contiguous() if case["wide_ids"] else ids.int().contiguous()
    if case["op"] == "distill":
        s["loss"] = torch.empty(n, device=dev, dtype=torch.float32)
        s["lse"] = torch.empty(n, device=dev, dtype=torch.float32)
    else:
        s["lse"] = torch.cat([torch.logsumexp(logits[a:a + 256].double() / case["temperature"], 1) for a in range(0, n, 256)]).float()
        s["loss_grad"] = normal(n, by=0.1, mean=1.0)
        s["grads"] = [torch.empty_like(x) for x in s["logits"]]
    return s


# ------------------------------------------------------------ the plain forms


def _norm(s):
    x = s["parts"].float().sum(0)
    n = x
    if s["post_w"] is not None:
        n = x * torch.rsqrt((x * x).mean(1, keepdim=True) + _EPS) * s["post_w"].float()
    if s["gate"] is not None:
        n = n.view(s["gates"], -1, s["width"]).mul(s["gate"].float()[:, None]).view_as(x)
    h = s["residual"].float() + s["scale"] * n
    y = h * torch.rsqrt((h * h).mean(1, keepdim=True) + _EPS) * s["pre"].float()
    s["residual_out"].copy_(h)
    if s["sums"] is not None:
        s["sums"].copy_(x)
    s["out"].copy_(y)


def _norm_grad(s):
    g = s["out_grads"].float().sum(0)
    h = s["hidden"].float()
    a = g * s["pre"].float()
    r = torch.rsqrt((h * h).mean(1, keepdim=True) + _EPS)
    dh = r * a - h * (r * r * r * (a * h).mean(1, keepdim=True)) + s["residual_grad"].float()
    s["residual_grad_out"].copy_(dh)
    s["pre_grad"].copy_((g * h * r).sum(0))
    dn = s["scale"] * dh
    if s["sums"] is not None:
        x = s["sums"].float()
        q = torch.rsqrt((x * x).mean(1, keepdim=True) + _EPS) if s["post_w"] is not None else torch.ones_like(x[:, :1])
        w = s["post_w"].float() if s["post_w"] is not None else torch.ones_like(x[0])
    if s["gate"] is not None:
        s["gate_grad"].copy_((dn * (x * q * w)).view(s["gates"], -1, s["width"]).sum(1))
        dn = dn.view(s["gates"], -1, s["width"]).mul(s["gate"].float()[:, None]).view_as(h)
    if s["post_w"] is not None:
        s["post_grad"].copy_((dn * x * q).sum(0))
        b = dn * w
        dn = q * b - x * (q * q * q * (b * x).mean(1, keepdim=True))
    s["part_grads"].copy_(dn)


def _embed(s):
    inside = (s["ids"] >= 0) & (s["ids"] < s["vocab"])
    rows = s["table"][torch.where(inside, s["ids"], 0)].float()
    s["out"].copy_(rows * (inside * s["scale"])[:, None].float())


def _embed_grad(s):
    inside = (s["ids"] >= 0) & (s["ids"] < s["vocab"])
    rows = s["out_grads"].float() * (inside * s["scale"])[:, None].float()
    at = torch.where(inside, s["ids"], 0)
    if s["accumulate"] and s["grads"].dtype == torch.float32:
        s["grads"].index_add_(0, at, rows)
    else:
        total = torch.zeros(s["grads"].shape, device=rows.device, dtype=torch.float32).index_add_(0, at, rows)
        s["grads"].copy_(s["grads"].float() + total if s["accumulate"] else total)


def _teacher(s, t, valid):
    """The teacher's distribution over its valid entries and its logarithm (zeros where there is none)."""
    t = torch.where(valid, t, -math.inf)
    m = t.max(1, keepdim=True).values
    e = torch.where(valid, torch.exp(t - torch.where(torch.isfinite(m), m, 0)), 0)
    total = e.sum(1, keepdim=True)
    some = total > 0
    q = e / torch.where(some, total, 1)
    log_q = torch.where(q > 0, t - torch.where(some, m, 0) - torch.log(torch.where(some, total, 1)), 0)
    return q, log_q


def _distill(s):
    tau = s["temperature"]
    z = torch.cat(s["logits"], 1).float() / tau
    m = z.max(1, keepdim=True).values
    lse = (m + torch.log(torch.exp(z - m).sum(1, keepdim=True)))
    valid = (s["ids"] >= 0) & (s["ids"] < s["vocab"])
    q, log_q = _teacher(s, s["teacher"].float() / tau, valid)
    at = torch.where(valid, s["ids"], 0).long()
    log_p = z.gather(1, at) - lse
    s["loss"].copy_((tau * tau) * torch.where(q > 0, q * (log_q - log_p), 0).sum(1))
    s["lse"].copy_(lse[:, 0])


def _distill_grad(s):
    tau = s["temperature"]
    z = torch.cat(s["logits"], 1).float() / tau
    valid = (s["ids"] >= 0) & (s["ids"] < s["vocab"])
    q, _ = _teacher(s, s["teacher"].float() / tau, valid)
    d = torch.exp(z - s["lse"][:, None]) * (q.sum(1, keepdim=True) > 0)
    d.scatter_add_(1, torch.where(valid, s["ids"], 0).long(), -q)
    d = d * (s["loss_grad"] * tau)[:, None]
    torch._foreach_copy_(s["grads"], list(d.split([x.shape[1] for x in s["grads"]], 1)))


def run(s):
    op = s["op"]
    if own:
        comm = _comm(s["ranks"])
        if op == "norm":
            comm.reduce_norm(s["parts"], s["residual_ranks"], s["out"], s["pre"], residual_out=s["residual_out_ranks"],
                             sums=s["sums_ranks"], post_weight=s["post_w"], gate=s["gate"], scale=s["scale"], eps=_EPS)
        elif op == "norm_grad":
            comm.reduce_norm_grad(s["out_grads"], s["hidden_ranks"], s["part_grads"], s["residual_grad_out_ranks"], s["pre"],
                                  s["pre_grad"], sums=s["sums_ranks"], residual_grad_in=s["residual_grad_ranks"],
                                  post_weight=s["post_w"], post_weight_grad=s["post_grad"], gate=s["gate"],
                                  gate_grad=s["gate_grad"], scale=s["scale"], eps=_EPS)
        elif op == "embed":
            comm.embedding(s["table_ranks"], s["ids_ranks"], s["out_ranks"], scale=s["scale"])
        elif op == "embed_grad":
            comm.embedding_grad(s["out_grads_ranks"], s["ids_ranks"], s["grads_ranks"], scale=s["scale"],
                                accumulate=s["accumulate"])
        elif op == "distill":
            comm.distill_loss(s["logits"], s["teacher"], s["ids"], s["loss"], s["lse"], temperature=s["temperature"])
        else:
            comm.distill_loss_grad(s["logits"], s["teacher"], s["ids"], s["lse"], s["loss_grad"], s["grads"],
                                   temperature=s["temperature"])
    else:
        {"norm": _norm, "norm_grad": _norm_grad, "embed": _embed, "embed_grad": _embed_grad, "distill": _distill,
         "distill_grad": _distill_grad}[op](s)
    if op == "norm":
        return {"out": s["out"], "residual": s["residual_out"], "sums": s["sums"]}
    if op == "norm_grad":
        return {"parts": s["part_grads"], "residual": s["residual_grad_out"], "pre": s["pre_grad"], "post": s["post_grad"],
                "gate": s["gate_grad"]}
    if op == "embed":
        return {"out": s["out"]}
    if op == "embed_grad":
        return {"table": s["grads"]}
    if op == "distill":
        return {"loss": s["loss"], "lse": s["lse"]}
    return {"logits": s["grads"]}


# ------------------------------------------------- the definitions in 64 bits


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("norm", "norm_grad"):
        t, width, ranks = case["rows"], case["width"], case["ranks"]
        group = torch.arange(t, device="cuda") * max(1, case["gates"]) // t
        w2 = s["pre"].double()
        w1 = s["post_w"].double() if case["post"] else None
        gate = s["gate"].double() if case["gates"] else None
        stack = s["parts"] if op == "norm" else s["out_grads"]
        total = torch.zeros(t, width, device="cuda", dtype=torch.float64)
        for r in range(ranks):
            total += stack[r].double()
    if op == "norm":
        inner = total / (total.pow(2).sum(1) / width + _EPS).sqrt()[:, None] * w1 if case["post"] else total
        h = s["residual"].double() + s["scale"] * (inner * gate[group] if case["gates"] else inner)
        y = h / (h.pow(2).sum(1) / width + _EPS).sqrt()[:, None] * w2
        return {"out": y.expand(ranks, t, width), "residual": h, "sums": total if case["save"] else None}
    if op == "norm_grad":
        h = s["hidden"].double()
        rms = (h.pow(2).sum(1) / width + _EPS).sqrt()[:, None]
        unit = h / rms
        u = total * w2
        dh = (u - unit * ((u * unit).sum(1) / width)[:, None]) / rms + s["residual_grad"].double()
        found = {"residual": dh, "pre": (total * unit).sum(0), "post": None, "gate": None}
        back = s["scale"] * dh
        if case["post"] or case["gates"]:
            x = s["sums"].double()
            size = (x.pow(2).sum(1) / width + _EPS).sqrt()[:, None] if case["post"] else 1.0
            direction = x / size
        if case["gates"]:
            inner = direction * w1 if case["post"] else direction
            found["gate"] = torch.zeros(case["gates"], width, device="cuda", dtype=torch.float64).index_add_(0, group, back * inner)
            back = back * gate[group]
        if case["post"]:
            found["post"] = (back * direction).sum(0)
            u = back * w1
            back = (u - direction * ((u * direction).sum(1) / width)[:, None]) / size
        found["parts"] = back.expand(ranks, t, width)
        return found
    if op == "embed":
        got = torch.zeros(s["ids"].shape[0], case["width"], device="cuda", dtype=torch.float64)
        known = ((s["ids"] >= 0) & (s["ids"] < case["vocab"])).nonzero()[:, 0]
        got[known] = s["table"][s["ids"][known].long()].double() * s["scale"]
        return {"out": got}
    if op == "embed_grad":
        got = s["grads"].double() if case["accumulate"] else torch.zeros(case["vocab"], case["width"], device="cuda", dtype=torch.float64)
        known = ((s["ids"] >= 0) & (s["ids"] < case["vocab"])).nonzero()[:, 0]
        got.index_add_(0, s["ids"][known].long(), s["out_grads"][known].double() * s["scale"])
        return {"table": got}
    tau, rows = case["temperature"], case["rows"]
    loss, lse, grads = [], [], []
    for a in range(0, rows, 128):
        z = torch.cat([x[a:a + 128] for x in s["logits"]], 1).double() / tau
        norm = torch.logsumexp(z, 1, keepdim=True)
        ids = s["ids"][a:a + 128].long()
        t = s["teacher"][a:a + 128].double() / tau
        t[(ids < 0) | (ids >= case["vocab"])] = -math.inf
        some = torch.isfinite(t).any(1)
        t[~some] = 0.0
        log_q = torch.log_softmax(t, 1)
        q = log_q.exp() * some[:, None]
        safe = ids.clamp(0, case["vocab"] - 1)
        if op == "distill":
            terms = q * (log_q - (z.gather(1, safe) - norm))
            loss.append(tau * tau * torch.nan_to_num(terms, nan=0.0).sum(1))
            lse.append(norm[:, 0])
        else:
            p = (z - norm).exp() * some[:, None]
            p.scatter_add_(1, safe, -q)
            grads.append(p * (tau * s["loss_grad"][a:a + 128].double())[:, None])
    if op == "distill":
        return {"loss": torch.cat(loss), "lse": torch.cat(lse)}
    return {"logits": [x.contiguous() for x in torch.cat(grads).split(_columns(case), 1)]}
