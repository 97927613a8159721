"""Operators around the optimizer step: what is measured, and their plain forms.

* ``clip``: the global L2 norm of a list of gradients, and clipping by it in place.
* ``norm``: the norm alone.
* ``step``: the norm, then a multi-tensor AdamW step whose gradients are taken clipped.
* ``lookup``: rows of an embedding table by token, scaled.
* ``embed``: the table's gradient from the rows' gradients, by sorted tokens.
* ``qk``: each attention head's largest logit, and the QK-Clip of the query and key weights by it.

``run`` computes them with elementary torch operations in 32 bits (64 for long
sums) where ``own`` is false, and with this package's kernels where it is true.
"""
from __future__ import annotations

import math

import numpy as np
import torch

own = False

DT = {"bf16": torch.bfloat16, "fp32": torch.float32}
BYTES = {"bf16": 2, "fp32": 4}
ALIGN = 64  # elements: the tensors of a list sit at such offsets of one buffer, as the sharded step lays them out
MAX_NORM = 1.0
HP = {"lr": 0.02, "beta1": 0.9, "beta2": 0.95, "eps": 1e-8, "weight_decay": 0.01, "step": 100}
TAU = 100.0
HOT = 4  # every HOT-th head's logits are large enough to be clipped


# ------------------------------------------------------------------ cases

def listed():
    return [
        # the gains and scalars of the depth-20 set: 81 tensors of 1 to 1280 values, where latency is all
        {"name": "clip gains d20", "op": "clip", "tensors": "gains d20", "dtype": "fp32"},
        # every gradient of the depth-20 set
        {"name": "clip d20", "op": "clip", "tensors": "d20", "dtype": "bf16"},
        # every gradient of the 7B set, only measured (the step applies the factor)
        {"name": "norm 7b", "op": "norm", "tensors": "7b", "dtype": "bf16"},
        # the RMSNorm gains of the 7B set on AdamW, clipped
        {"name": "step gains 7b", "op": "step", "tensors": "gains 7b", "dtype": "fp32"},
        # embedding, unembedding and gains of the 7B set on AdamW, clipped
        {"name": "step adamw 7b", "op": "step", "tensors": "adamw 7b", "dtype": "bf16"},
        # one token each of 16 sequences that are being continued, table of the depth-20 set
        {"name": "lookup 16", "op": "lookup", "tokens": 16, "rows": 65536, "dim": 1280, "table": "fp32", "out": "bf16",
         "scale": 1.0},
        # a training batch of the 7B set: 4 sequences of 2048
        {"name": "lookup 8192", "op": "lookup", "tokens": 8192, "rows": 32000, "dim": 4096, "table": "fp32",
         "out": "bf16", "scale": 64.0},
        # a short odd batch whose gradient is added to what an earlier micro-batch left
        {"name": "embed 301 added", "op": "embed", "tokens": 301, "rows": 5003, "dim": 514, "rowgrad": "fp32",
         "grad": "fp32", "scale": 1.0, "add": True},
        # the training batch's gradient of the 7B table
        {"name": "embed 8192", "op": "embed", "tokens": 8192, "rows": 32000, "dim": 4096, "rowgrad": "bf16",
         "grad": "bf16", "scale": 64.0, "add": False},
        # a large batch of the depth-20 set: 64 sequences of 2048, frequent tokens thousands of times
        {"name": "embed 131072", "op": "embed", "tokens": 131072, "rows": 65536, "dim": 1280, "rowgrad": "bf16",
         "grad": "bf16", "scale": 1.0, "add": False},
        # one sequence of the 7B set: 32 heads of 128
        {"name": "qk 4096x32", "op": "qk", "seqs": 1, "length": 4096, "heads": 32, "kv_heads": 32, "dim": 128,
         "causal": True, "packed": False, "absolute": False, "width": 4096},
        # ragged sequences packed end to end, depth-20 widths, shared key heads
        {"name": "qk packed 12x1000 gqa", "op": "qk", "seqs": 12, "length": 1000, "heads": 10, "kv_heads": 2,
         "dim": 128, "causal": True, "packed": True, "absolute": True, "width": 1280},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["clip", "clip", "norm", "step", "lookup", "embed", "embed", "qk", "qk"])
    if op in ("clip", "norm", "step"):
        total = _log(rng, 2000, 500_000_000 if op != "step" else 150_000_000)
        return {"op": op, "tensors": "drawn", "count": min(_log(rng, 1, 600), total), "total": total,
                "order": rng.randrange(1 << 20), "dtype": rng.choice(["bf16", "fp32"])}
    if op == "qk":
        dim = rng.choice([64, 72, 96, 128, 128, 160, 192, 256])
        kv = rng.choice([1, 2, 3, 4, 8])
        heads = kv * rng.choice([1, 1, 2, 4])
        length = _log(rng, 1, 4096)
        most = max(1, min(16, int((4096.0 * 4096 * 32 / (heads * length * length)) ** 0.5), 16384 // length))
        return {"op": op, "seqs": rng.randint(1, most), "length": length, "heads": heads, "kv_heads": kv, "dim": dim,
                "causal": rng.random() < 0.7, "packed": rng.random() < 0.5, "absolute": rng.random() < 0.5,
                "width": 8 * rng.randint(8, 300)}
    rows = _log(rng, 7, 70000)
    dim = rng.choice([_log(rng, 1, 5000), 8 * _log(rng, 1, 640)])
    case = {"op": op, "tokens": min(_log(rng, 1, 131072), 170_000_000 // dim), "rows": rows, "dim": dim,
            "scale": rng.choice([1.0, 1.0, round(math.sqrt(dim), 3)])}
    if op == "lookup":
        return case | {"table": rng.choice(["fp32", "bf16"]), "out": rng.choice(["fp32", "bf16"])}
    return case | {"rowgrad": rng.choice(["bf16", "fp32"]), "grad": rng.choice(["bf16", "fp32"]),
                   "add": rng.random() < 0.3}


def _gains(layers, dim, scalars):
    return [n for _ in range(layers) for n in [dim, dim] + [1] * scalars] + [dim]


def _sizes(case):
    """Elements of each tensor of the case's list."""
    kind = case["tensors"]
    if kind == "gains d20":
        return _gains(20, 1280, 2)
    if kind == "gains 7b":
        return _gains(32, 4096, 0)
    if kind == "adamw 7b":
        return [32000 * 4096] + _gains(32, 4096, 0) + [32000 * 4096]
    if kind == "d20":
        return [65536 * 1280] + 20 * (4 * [1280 * 1280] + 2 * [1280 * 5120]) + _gains(20, 1280, 2) + [65536 * 1280]
    if kind == "7b":
        return [32000 * 4096] + 32 * (4 * [4096 * 4096] + 3 * [4096 * 11008]) + _gains(32, 4096, 0) + [32000 * 4096]
    r = np.random.default_rng(case["order"])
    part = r.pareto(0.7, case["count"]) + 1e-3
    part = np.maximum(1, (part * (case["total"] / part.sum())).astype(np.int64))
    return [int(n) for n in part]


def _lengths(case):
    """Lengths of packed sequences: odd, one of them full, and one empty where there are enough."""
    r = np.random.default_rng([case["seqs"], case["length"], case["dim"]])
    n = r.integers(1, case["length"] + 1, case["seqs"])
    n[0] = case["length"]
    if case["seqs"] > 2:
        n[case["seqs"] // 2] = 0
    return [int(x) for x in n]


def _tokens(case):
    return sum(_lengths(case)) if case["packed"] else case["seqs"] * case["length"]


# ------------------------------------------------------------------ inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 2654435761 % (1 << 62) + 17)
    return g


def _randn(g, shape, dtype, std):
    return torch.randn(shape, generator=g, device="cuda", dtype=dtype).mul_(std)


def _views(flat, sizes):
    at, out = 0, []
    for n in sizes:
        out.append(flat[at:at + n])
        at += -(-n // ALIGN) * ALIGN
    return out


def _zipf(g, n, rows):
    """Token ids with the frequencies of text: id of rank r with probability about 1/r, ranks in random order."""
    u = torch.rand(n, generator=g, device="cuda", dtype=torch.float64)
    rank = torch.exp(u * math.log(rows + 1.0)).long().sub_(1).clamp_(0, rows - 1)
    return torch.randperm(rows, generator=g, device="cuda")[rank]


def prepare(case, seed):
    g, op = _gen(seed), case["op"]
    if op in ("clip", "norm", "step"):
        sizes, dt = _sizes(case), DT[case["dtype"]]
        flat = torch.zeros(sum(-(-n // ALIGN) * ALIGN for n in sizes), dtype=dt, device="cuda")
        views = _views(flat, sizes)
        for v in views:
            v.copy_(_randn(g, v.shape, dt, 1e-3))
        s = {"op": op, "flat": flat, "grads": views, "turn": 0}
        if op == "step":
            for name, std in (("P", 0.02), ("M", 1e-4), ("V", 1e-4)):
                x = torch.zeros(flat.shape, dtype=torch.float32, device="cuda")
                s[name], s[name + "s"] = x, _views(x, sizes)
                for v in s[name + "s"]:
                    v.copy_(_randn(g, v.shape, torch.float32, std))
            s["V"].square_()
        if own:  # the handle a training loop keeps for its gradients, and the hyperparameters of its step
            import adamw_hybrid_optimizer_muon_b200 as ma
            s["clip"] = ma.GradClip(views)
            s["hp"] = ma.adamw_hparams(**HP)
        return s
    if op == "lookup":
        ids = _zipf(g, case["tokens"], case["rows"])
        return {"op": op, "ids": ids, "scale": case["scale"], "dtype": DT[case["out"]],
                "table": _randn(g, (case["rows"], case["dim"]), DT[case["table"]], 0.02)}
    if op == "embed":
        grad = torch.zeros((case["rows"], case["dim"]), dtype=DT[case["grad"]], device="cuda")
        if case["add"]:
            grad = _randn(g, grad.shape, grad.dtype, 1e-3)
        return {"op": op, "ids": _zipf(g, case["tokens"], case["rows"]), "scale": case["scale"], "add": case["add"],
                "dy": _randn(g, (case["tokens"], case["dim"]), DT[case["rowgrad"]], 1e-3), "grad": grad}
    h, kv, d, n = case["heads"], case["kv_heads"], case["dim"], _tokens(case)
    gain = torch.rand(h, generator=g, device="cuda") * 2 + 1
    gain[::HOT] = 40.0
    shape = (n,) if case["packed"] else (case["seqs"], case["length"])
    q = (_randn(g, shape + (h, d), torch.float32, 1.0) * gain[:, None]).bfloat16()
    k = _randn(g, shape + (kv, d), torch.bfloat16, 1.0)
    s = {"op": op, "q": q, "k": k, "causal": case["causal"], "absolute": case["absolute"], "scale": d ** -0.5,
         "length": case["length"], "offsets": None, "wq": _randn(g, (h * d, case["width"]), torch.float32, 0.02),
         "wk": _randn(g, (kv * d, case["width"]), torch.float32, 0.02)}
    if case["packed"]:
        s["offsets"] = torch.tensor(np.concatenate([[0], np.cumsum(_lengths(case))]), dtype=torch.int32, device="cuda")
    return s


# ------------------------------------------------------------------ the operators

def _bounds(s):
    """(largest norm, factor before it) of this pass. Clipping in place changes the gradients, so passes in turn clip
    to one and to two: the summed gradients of four micro-batches come back over either each time."""
    s["turn"] ^= 1
    return (MAX_NORM if s["turn"] else 2 * MAX_NORM), 4.0


def _norm(flat):
    x = flat.float()
    return torch.sqrt((x * x).sum(dtype=torch.float64)).float()


def _plain_clip(s):
    max_norm, scale = _bounds(s)
    norm = scale * _norm(s["flat"])
    factor = scale * torch.clamp(max_norm / norm, max=1.0)
    s["flat"].copy_(s["flat"].float() * factor)
    return [s["flat"], norm]


def _plain_step(s):
    norm = _norm(s["flat"])
    grad = s["flat"].float() * torch.clamp(MAX_NORM / norm, max=1.0)
    p, m, v, h = s["P"], s["M"], s["V"], HP
    m.copy_(h["beta1"] * m + (1 - h["beta1"]) * grad)
    v.copy_(h["beta2"] * v + (1 - h["beta2"]) * (grad * grad))
    b1, b2 = 1 - h["beta1"] ** h["step"], 1 - h["beta2"] ** h["step"]
    p.copy_(p * (1 - h["lr"] * h["weight_decay"]) - h["lr"] * (m / b1) / (torch.sqrt(v / b2) + h["eps"]))
    return [p, m, v, norm]


def _plain_embed(s):
    total = torch.zeros(s["grad"].shape, dtype=torch.float32, device="cuda")
    total.index_add_(0, s["ids"], s["dy"].float())
    total *= s["scale"]
    s["grad"].copy_(s["grad"].float() + total if s["add"] else total)
    return s["grad"]


def _visible(s, n):
    """n x n truth values: whether the query of a row sees the key of a column."""
    at = torch.arange(n, device="cuda")
    see = at[:, None] >= at[None, :] if s["causal"] else torch.ones((n, n), dtype=torch.bool, device="cuda")
    if s["offsets"] is not None:
        seq = torch.bucketize(at, s["offsets"][1:], right=True)
        see = see & (seq[:, None] == seq[None, :])
    return see


def _plain_qk(s):
    q, k = s["q"].float(), s["k"].float()
    if s["offsets"] is not None:
        q, k = q[None], k[None]
    group = q.shape[2] // k.shape[2]
    k = k.repeat_interleave(group, dim=2)
    logits = torch.matmul(q.permute(0, 2, 1, 3), k.permute(0, 2, 3, 1)) * s["scale"]
    if s["absolute"]:
        logits = logits.abs()
    top = logits.masked_fill(~_visible(s, q.shape[1]), -math.inf).amax(dim=(0, 2, 3))
    gamma = torch.clamp(TAU / top.clamp(min=1e-30), max=1.0)  # per query head
    fk = gamma.view(-1, group).amin(dim=1).sqrt()              # per key head
    fq = gamma / fk.repeat_interleave(group)
    wq, wk = s["wq"], s["wk"]
    wq.copy_((wq.view(fq.numel(), -1) * fq[:, None]).view(wq.shape))
    wk.copy_((wk.view(fk.numel(), -1) * fk[:, None]).view(wk.shape))
    return [top, wq, wk]


def _own(s):
    import adamw_hybrid_optimizer_muon_b200 as ma
    op = s["op"]
    if op == "clip":
        max_norm, scale = _bounds(s)
        return [s["flat"], s["clip"].clip(max_norm, scale=scale)]
    if op == "norm":
        return s["clip"].norm()
    if op == "step":
        norm = s["clip"].norm(max_norm=MAX_NORM)
        ma.adamw_step_fused(s["Ps"], s["grads"], s["Ms"], s["Vs"], s["hp"], clip=s["clip"].buffer)
        return [s["P"], s["M"], s["V"], norm]
    if op == "lookup":
        return ma.embedding_lookup(s["ids"], s["table"], scale=s["scale"], dtype=s["dtype"])
    if op == "embed":
        return ma.embedding_grad(s["ids"], s["dy"], s["grad"], scale=s["scale"], accumulate=s["add"])
    top = ma.qk_max_logit(s["q"], s["k"], scale=s["scale"], causal=s["causal"], offsets=s["offsets"],
                          max_len=s["length"], absolute=s["absolute"])
    ma.qk_clip(s["wq"], s["wk"], top, tau=TAU, kv_heads=s["k"].shape[-2])
    return [top, s["wq"], s["wk"]]


def run(s):
    if own:
        return _own(s)
    op = s["op"]
    if op == "clip":
        return _plain_clip(s)
    if op == "norm":
        return _norm(s["flat"])
    if op == "step":
        return _plain_step(s)
    if op == "lookup":
        return (s["table"][s["ids"]].float() * s["scale"]).to(s["dtype"])
    return _plain_embed(s) if op == "embed" else _plain_qk(s)


# ------------------------------------------------------------------ work

def work(case):
    op = case["op"]
    if op in ("clip", "norm", "step"):
        n, b = sum(_sizes(case)), BYTES[case["dtype"]]
        # clip: read, written back; step: gradients read, parameters and two moments read and written
        return {"bytes": n * {"clip": 2 * b, "norm": b, "step": b + 24}[op],
                "flops": n * {"clip": 3, "norm": 2, "step": 17}[op]}
    if op == "lookup":
        # as many rows read as distinct tokens can be; Zipf draws repeat some
        n, d = case["tokens"], case["dim"]
        return {"bytes": d * (_distinct(n, case["rows"]) * BYTES[case["table"]] + n * BYTES[case["out"]]) + 8 * n,
                "flops": n * d}
    if op == "embed":
        n, d, b = case["tokens"], case["dim"], BYTES[case["grad"]]
        touched = _distinct(n, case["rows"])
        rows = 2 * touched if case["add"] else case["rows"]
        return {"bytes": d * (n * BYTES[case["rowgrad"]] + rows * b) + 8 * n, "flops": 2 * n * d}
    h, kv, d, n = case["heads"], case["kv_heads"], case["dim"], _tokens(case)
    lens = _lengths(case) if case["packed"] else [case["length"]] * case["seqs"]
    pairs = sum(t * (t + 1) // 2 if case["causal"] else t * t for t in lens)
    hot = -(-h // HOT)
    hot_kv = len({i // (h // kv) for i in range(0, h, HOT)})
    return {"bytes": 2 * n * d * (h + kv) + 8 * d * case["width"] * (hot + hot_kv), "flops": 2 * pairs * d * h}


def _distinct(n, rows):
    """Expected number of distinct ids among n draws of _zipf."""
    r = np.arange(1, rows + 1, dtype=np.float64)
    p = np.log1p(1.0 / r) / math.log(rows + 1.0)
    return float(np.sum(-np.expm1(n * np.log1p(-np.minimum(p, 1 - 1e-12)))))


# ------------------------------------------------------------------ in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("clip", "norm", "step"):
        squares = [g.double().pow(2).sum() for g in s["grads"]]
        norm = torch.stack(squares).sum().sqrt()
        if op == "norm":
            return norm
        if op == "clip":
            max_norm, scale = _bounds(s)
            factor = max_norm / norm if float(scale * norm) > max_norm else torch.full_like(norm, scale)
            return [s["flat"].double() * factor, norm * scale]
        h = {k: (float(np.float32(v)) if k != "step" else v) for k, v in HP.items()}
        g = s["flat"].double() * min(1.0, MAX_NORM / float(norm))
        m = s["M"].double().mul_(h["beta1"]).add_(g, alpha=1 - h["beta1"])
        v = s["V"].double().mul_(h["beta2"]).add_(g.square_(), alpha=1 - h["beta2"])
        root = (v / (1 - h["beta2"] ** h["step"])).sqrt_().add_(h["eps"])
        p = s["P"].double().mul_(1 - h["lr"] * h["weight_decay"])
        p.sub_((m / root).mul_(h["lr"] / (1 - h["beta1"] ** h["step"])))
        return [p, m, v, norm]
    if op == "lookup":
        return s["table"].double().index_select(0, s["ids"]) * float(np.float32(case["scale"]))
    if op == "embed":
        # sums over runs of equal tokens, as differences of running sums along the sorted tokens
        order = torch.argsort(s["ids"], stable=True)
        ends = torch.bincount(s["ids"], minlength=case["rows"]).cumsum(0)
        out = torch.empty(s["grad"].shape, dtype=torch.float64, device="cuda")
        for c in range(0, case["dim"], 256):
            run_sum = s["dy"][:, c:c + 256].double()[order].cumsum(0)
            run_sum = torch.cat([torch.zeros_like(run_sum[:1]), run_sum])[ends]
            out[:, c:c + 256] = torch.diff(run_sum, dim=0, prepend=torch.zeros_like(run_sum[:1]))
        out *= float(np.float32(case["scale"]))
        return out + s["grad"].double() if case["add"] else out
    h, kv, t = case["heads"], case["kv_heads"], case["length"]
    ends = np.cumsum(_lengths(case)).tolist() if case["packed"] else [t * (i + 1) for i in range(case["seqs"])]
    q, k = s["q"].view(-1, h, case["dim"]), s["k"].view(-1, kv, case["dim"])
    top = np.full(h, -math.inf)
    for lo, hi in zip([0] + ends[:-1], ends):
        for j in range(h if hi > lo else 0):
            x = q[lo:hi, j].double() @ k[lo:hi, j // (h // kv)].double().T * case["dim"] ** -0.5
            x = x.abs() if case["absolute"] else x
            if case["causal"]:
                x = torch.where(torch.ones_like(x, dtype=torch.bool).tril(), x, -math.inf)
            top[j] = max(top[j], float(x.max()))
    gamma = np.array([TAU / x if x > TAU else 1.0 for x in top])
    fk = gamma.reshape(kv, -1).min(axis=1) ** 0.5
    fq = gamma / np.repeat(fk, h // kv)
    rows = lambda w, f: w.double() * torch.from_numpy(np.repeat(f, case["dim"])).cuda()[:, None]  # noqa: E731
    return [torch.from_numpy(top), rows(s["wq"], fq), rows(s["wk"], fk)]
