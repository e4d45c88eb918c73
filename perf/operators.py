"""Workloads of the 8-bit floating point products and the mixture-of-experts operators.

Each case names one operator and its sizes.  ``run`` computes it in elementary
torch operations (``own`` false) or through the package's entry points (``own``
true); ``exact`` computes it in 64 bits from its definition.

Definitions.  A block is 128 consecutive columns; kb = ceil(k / 128) blocks a
row, the columns past k are zero.  E4M3 is the finite-only 8-bit type of largest
value 448.

* quant: v = x, or silu(gate) * up of rows [gate | up]; a = max |v| over a
  token's block; scale = max(a / 448, 2^-126), 1 for a block of zeros;
  codes = E4M3(clamp(v / scale, -448, 448)).  codes [m, 128 kb], scale [kb, m].
* gemm: y[t, r] = sum_b sx[b, t] * sw[r / 128, b] * (codes of t, block b) . (codes of r, block b).
* grouped: the same with the matrix of the expert whose range [off[e], off[e + 1])
  holds the output row p, and token row_ids[p].
* route: the k largest logits of a token (lowest index first on ties; -inf is
  never chosen), their softmax weights over the chosen or over all experts, and the
  chosen (token, expert) pairs sorted by expert, then token.
* combine: out[t] = sum_j weights[t, j] * y[slots[t, j]].
"""
import math

import torch

own = False

DEV = "cuda"
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZE = {"f32": 4, "bf16": 2, "f16": 2}
F8 = torch.float8_e4m3fn
TINY, HUGE = 2.0 ** -126, torch.finfo(torch.float32).max


# ------------------------------------------------------------------ the cases

def listed():
    return [
        # one token's hidden state before its products: a launch and little else
        dict(name="quant_1x4096", op="quant", m=1, k=4096, swiglu=False, dtype="bf16", gap=0),
        # a prefill's gate and up rows on their way into the down projection
        dict(name="quant_swiglu_2048x14336", op="quant", m=2048, k=14336, swiglu=True, dtype="bf16", gap=0),
        # decode of one token: the weights are read once
        dict(name="gemm_1x4096x4096", op="gemm", m=1, n=4096, k=4096, ytype="bf16"),
        # a small model's up projection with odd sizes and fp32 results
        dict(name="gemm_77x1092x312", op="gemm", m=77, n=1092, k=312, ytype="f32"),
        # prefill of a long prompt: bound by the matrix cores
        dict(name="gemm_4096x14336x4096", op="gemm", m=4096, n=14336, k=4096, ytype="bf16"),
        # decode of one token through the 8 experts it is sent to
        dict(name="grouped_1of64_2048x2048", op="grouped", tokens=1, experts=64, top=8, n=2048, k=2048, gather=True, skew=0.5, ytype="bf16"),
        # few tokens, odd sizes, some experts without any
        dict(name="grouped_37of12_1092x312", op="grouped", tokens=37, experts=12, top=3, n=1092, k=312, gather=False, skew=1.5, ytype="f32"),
        # prefill: 32768 rows over 64 experts, some with several times others' share
        dict(name="grouped_4096of64_4096x2048", op="grouped", tokens=4096, experts=64, top=8, n=4096, k=2048, gather=True, skew=0.5, ytype="bf16"),
        # the router's step of a small decode batch
        dict(name="route_4of64", op="route", tokens=4, experts=64, top=8, renorm=True, masked=0.0, dtype="f32"),
        # the router over a long prefill, some experts masked
        dict(name="route_16384of256", op="route", tokens=16384, experts=256, top=8, renorm=True, masked=0.02, dtype="bf16"),
        # one token's eight expert rows back into one
        dict(name="combine_1x8x2048", op="combine", tokens=1, top=8, d=2048, masked=0.0, dtype="bf16"),
        # a prefill's rows back into tokens
        dict(name="combine_8192x8x4096", op="combine", tokens=8192, top=8, d=4096, masked=0.01, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _size(rng, lo, hi):
    """A size over the logarithm of the range: a multiple of 64 two times in three, any number otherwise."""
    v = _log(rng, lo, hi)
    return max(lo, v // 64 * 64) if rng.random() < 0.67 and v >= 64 else v


def draw(rng):
    most = {c["op"]: c for c in listed()}            # the last listed of an operator is its largest
    most["gemm"], most["grouped"] = listed()[4], listed()[7]
    op = rng.choice(["quant", "gemm", "gemm", "grouped", "grouped", "route", "combine"])
    while True:
        if op == "quant":
            c = dict(op=op, m=_log(rng, 1, 8192), k=_size(rng, 64, 14336), swiglu=rng.random() < 0.5,
                     dtype=rng.choice(["bf16", "bf16", "f16", "f32"]), gap=rng.choice([0, 0, 64, 1]))
        elif op == "gemm":
            c = dict(op=op, m=_log(rng, 1, 8192), n=_size(rng, 64, 14336), k=_size(rng, 64, 14336),
                     ytype=rng.choice(["bf16", "bf16", "f16", "f32"]))
        elif op == "grouped":
            experts = _log(rng, 4, 128)
            c = dict(op=op, tokens=_log(rng, 1, 8192), experts=experts, top=rng.randint(1, min(8, experts)),
                     n=_size(rng, 64, 4096), k=_size(rng, 64, 4096), gather=rng.random() < 0.6,
                     skew=rng.choice([0.0, 0.5, 1.0]), ytype=rng.choice(["bf16", "bf16", "f16", "f32"]))
        elif op == "route":
            experts = _log(rng, 4, 256)
            c = dict(op=op, tokens=_log(rng, 1, 16384), experts=experts, top=rng.randint(1, min(8, experts)),
                     renorm=rng.random() < 0.5, masked=rng.choice([0.0, 0.02, 0.3]),
                     dtype=rng.choice(["f32", "bf16", "f16"]))
        else:
            c = dict(op=op, tokens=_log(rng, 1, 8192), top=rng.randint(1, 8), d=_size(rng, 64, 8192),
                     masked=rng.choice([0.0, 0.01]), dtype=rng.choice(["bf16", "f16", "f32"]))
        w, top = work(c), work(most[op])
        if w["bytes"] <= top["bytes"] and w["flops"] <= top["flops"]:
            return c


def _blocks(k):
    return (k + 127) // 128


def work(case):
    c = case
    if c["op"] == "quant":
        reads = c["m"] * c["k"] * SIZE[c["dtype"]] * (2 if c["swiglu"] else 1)
        return {"bytes": reads + c["m"] * _blocks(c["k"]) * 132, "flops": c["m"] * c["k"] * (6 if c["swiglu"] else 3)}
    if c["op"] == "gemm":
        kp = 128 * _blocks(c["k"])
        return {"bytes": (c["n"] + c["m"]) * kp + c["m"] * c["n"] * SIZE[c["ytype"]], "flops": 2 * c["m"] * c["n"] * c["k"]}
    if c["op"] == "grouped":
        kp, rows = 128 * _blocks(c["k"]), c["tokens"] * c["top"]
        read = (min(rows, c["experts"]) * c["n"] + (c["tokens"] if c["gather"] else rows)) * kp
        return {"bytes": read + rows * c["n"] * SIZE[c["ytype"]], "flops": 2 * rows * c["n"] * c["k"]}
    if c["op"] == "route":
        pairs = c["tokens"] * c["top"]
        return {"bytes": c["tokens"] * c["experts"] * SIZE[c["dtype"]] + 16 * pairs, "flops": 4 * c["tokens"] * c["experts"]}
    pairs = c["tokens"] * c["top"]
    return {"bytes": (pairs + c["tokens"]) * c["d"] * SIZE[c["dtype"]] + 8 * pairs, "flops": 2 * pairs * c["d"]}


# ------------------------------------------------------------------ the inputs

def _activations(g, m, k, dtype):
    """Hidden states: normal, a few columns many times larger, tokens of unlike size."""
    x = torch.randn((m, k), device=DEV, generator=g)
    col = torch.rand((k,), device=DEV, generator=g)
    x *= torch.where(col < 0.01, 20.0, 1.0)
    x *= torch.exp(0.5 * torch.randn((m, 1), device=DEV, generator=g))
    return x.to(dtype)


def _codes(g, m, k):
    """Quantized activations in the operators' layout: codes [m, 128 kb], scale [kb, m]."""
    kb = _blocks(k)
    x = torch.zeros((m, 128 * kb), device=DEV)
    x[:, :k] = _activations(g, m, k, torch.float32)
    x = x.view(m, kb, 128)
    s = (x.abs().amax(-1) / 448.0).clamp(min=TINY)
    q = (x / s[..., None]).clamp(-448.0, 448.0).to(F8)
    return q.view(m, 128 * kb), s.t().contiguous()


def _weights(g, experts, n, k):
    """Quantized weights: codes [experts, n, 128 kb], scale [experts, ceil(n / 128), kb]."""
    kb, nb = _blocks(k), (n + 127) // 128
    codes = torch.empty((experts, n, 128 * kb), dtype=F8, device=DEV)
    scale = torch.empty((experts, nb, kb), device=DEV)
    for e in range(experts):
        w = torch.zeros((128 * nb, 128 * kb), device=DEV)
        w[:n, :k] = 0.02 * torch.randn((n, k), device=DEV, generator=g)
        w = w.view(nb, 128, kb, 128)
        s = (w.abs().amax((1, 3)) / 448.0).clamp(min=TINY)
        codes[e] = (w / s[:, None, :, None]).clamp(-448.0, 448.0).to(F8).view(128 * nb, 128 * kb)[:n]
        scale[e] = s
    return codes, scale


def _sorted_pairs(ids, experts):
    """ids [tokens, top] (-1: none) -> offsets, row_ids, slots of the stable order by expert."""
    top = ids.shape[1]
    key = torch.where(ids >= 0, ids, experts).reshape(-1)
    by, order = torch.sort(key, stable=True)
    offsets = torch.searchsorted(by, torch.arange(experts + 1, device=ids.device))
    place = torch.empty_like(order)
    place[order] = torch.arange(order.numel(), device=ids.device)
    slots = torch.where(key < experts, place, -1).view(ids.shape)
    row_ids = torch.where(by < experts, order // top, -1)
    return offsets.to(torch.int32), row_ids.to(torch.int32), slots.to(torch.int32)


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    s = {"case": c}
    if c["op"] == "quant":
        width = c["k"] * (2 if c["swiglu"] else 1)
        x = _activations(g, c["m"], width + c["gap"], TYPES[c["dtype"]])
        s["x"] = x[:, :width]                                  # with a gap: part of a wider buffer's rows
    elif c["op"] == "gemm":
        s["q"], s["qs"] = _codes(g, c["m"], c["k"])
        w, ws = _weights(g, 1, c["n"], c["k"])
        s["w"], s["ws"] = w[0], ws[0]
    elif c["op"] == "grouped":
        love = -c["skew"] * torch.log(1.0 + torch.arange(c["experts"], device=DEV))
        love = love[torch.randperm(c["experts"], device=DEV, generator=g)]
        gate = torch.randn((c["tokens"], c["experts"]), device=DEV, generator=g) + love
        ids = torch.sort(gate, dim=1, descending=True).indices[:, :c["top"]]
        s["offsets"], s["row_ids"], _ = _sorted_pairs(ids, c["experts"])
        s["most"] = int((s["offsets"][1:] - s["offsets"][:-1]).max())
        s["q"], s["qs"] = _codes(g, c["tokens"] if c["gather"] else c["tokens"] * c["top"], c["k"])
        s["w"], s["ws"] = _weights(g, c["experts"], c["n"], c["k"])
    elif c["op"] == "route":
        x = 1.5 * torch.randn((c["tokens"], c["experts"]), device=DEV, generator=g)
        if c["masked"]:
            hide = torch.rand(x.shape, device=DEV, generator=g) < c["masked"]
            hide |= torch.rand((c["tokens"], 1), device=DEV, generator=g) < 0.001     # tokens with no expert left
            x = x.masked_fill(hide, -math.inf)
        s["logits"] = x.to(TYPES[c["dtype"]])
    else:
        pairs = c["tokens"] * c["top"]
        s["y"] = torch.randn((pairs, c["d"]), device=DEV, generator=g).to(TYPES[c["dtype"]])
        slots = torch.randperm(pairs, device=DEV, generator=g).view(c["tokens"], c["top"]).to(torch.int32)
        w = torch.softmax(torch.randn(slots.shape, device=DEV, generator=g), 1)
        gone = torch.rand(slots.shape, device=DEV, generator=g) < c["masked"]
        s["slots"], s["weights"] = slots.masked_fill(gone, -1), w.masked_fill(gone, 0.0)
    return s


# ------------------------------------------------------------------ the package's operators

def _own(s):
    from bit_quantized_matmul_amd import binding as B
    c = s["case"]
    if c["op"] == "quant":
        q, scale = B.fp8_quant(s["x"], swiglu=c["swiglu"])
        return {"codes": q, "scale": scale}
    if c["op"] == "gemm":
        return {"y": B.fp8_gemm(s["w"], s["ws"], c["k"], s["q"], s["qs"], dtype=TYPES[c["ytype"]])}
    if c["op"] == "grouped":
        return {"y": B.fp8_gemm_grouped(s["w"], s["ws"], c["k"], s["q"], s["qs"], s["offsets"],
                                        row_ids=s["row_ids"] if c["gather"] else None, dtype=TYPES[c["ytype"]])}
    if c["op"] == "route":
        r = B.moe_route(s["logits"], c["top"], renorm=c["renorm"])
        return {"ids": r.ids, "weights": r.weights, "offsets": r.offsets, "row_ids": r.row_ids, "slots": r.slots}
    return {"out": B.moe_combine(s["y"], s["slots"], s["weights"])}


# ------------------------------------------------------------------ the plain forms

def _plain_quant(c, x):
    x = x.to(torch.float32)
    m, k, kb = c["m"], c["k"], _blocks(c["k"])
    if c["swiglu"]:
        gate, up = x[:, :k], x[:, k:]
        x = gate / (1.0 + torch.exp(-gate)) * up
    v = torch.nn.functional.pad(x, (0, 128 * kb - k)).view(m, kb, 128)
    a = v.abs().amax(-1)
    s = torch.where(a > 0, (a / 448.0).clamp(min=TINY), 1.0)
    s = torch.where(torch.isfinite(a), s, math.nan)
    q = (v / s[..., None]).clamp(-448.0, 448.0).to(F8)
    return {"codes": q.view(m, 128 * kb), "scale": s.t().contiguous()}


def _values(q, scale):
    """Activations as fp32 values: [m, 128 kb]."""
    m, kp = q.shape
    return (q.to(torch.float32).view(m, kp // 128, 128) * scale.t()[..., None]).view(m, kp)


def _matrix(w, scale):
    """Weights [..., n, 128 kb] as fp32 values."""
    rows = scale.repeat_interleave(128, -2)[..., :w.shape[-2], :]
    return (w.to(torch.float32).unflatten(-1, (-1, 128)) * rows[..., None]).flatten(-2)


def _plain_grouped(c, s):
    """Every expert's rows as one padded batch, rows that no expert has left out afterwards."""
    rows = s["row_ids"].numel()
    place = torch.arange(rows, device=DEV)
    expert = torch.searchsorted(s["offsets"][1:].to(torch.int64), place, right=True)
    at = place - s["offsets"].to(torch.int64)[expert]
    x = _values(s["q"], s["qs"])
    x = x[s["row_ids"].to(torch.int64)] if c["gather"] else x
    if rows < c["experts"]:                                   # few rows: the matrices of their experts
        y = torch.bmm(_matrix(s["w"][expert], s["ws"][expert]), x[:, :, None])[..., 0]
    else:
        batch = torch.zeros((c["experts"], s["most"], x.shape[1]), device=DEV)
        batch[expert, at] = x
        y = torch.bmm(batch, _matrix(s["w"], s["ws"]).transpose(1, 2))[expert, at]
    return {"y": y.to(TYPES[c["ytype"]])}


def _plain_route(c, logits):
    x = logits.to(torch.float32)
    x = torch.where(torch.isnan(x), -math.inf, x).clamp(max=HUGE)
    by, order = torch.sort(x, dim=1, descending=True, stable=True)
    some = by[:, :c["top"]] > -math.inf
    first = torch.where(some[:, :1], by[:, :1], 0.0)
    e = torch.exp(by - first)
    total = e[:, :c["top"]].sum(1, keepdim=True) if c["renorm"] else e.sum(1, keepdim=True)
    w = torch.where(some, e[:, :c["top"]] / total, 0.0)
    ids = torch.where(some, order[:, :c["top"]], -1)
    offsets, row_ids, slots = _sorted_pairs(ids, c["experts"])
    return {"ids": ids.to(torch.int32), "weights": w, "offsets": offsets, "row_ids": row_ids, "slots": slots}


def _plain_combine(c, s):
    rows = s["y"][s["slots"].clamp(min=0).to(torch.int64)].to(torch.float32)
    part = torch.where(s["slots"][..., None] >= 0, rows * s["weights"][..., None], 0.0)
    return {"out": part.sum(1).to(TYPES[c["dtype"]])}


def run(state):
    if own:
        return _own(state)
    c = state["case"]
    if c["op"] == "quant":
        return _plain_quant(c, state["x"])
    if c["op"] == "gemm":
        y = _values(state["q"], state["qs"]) @ _matrix(state["w"], state["ws"]).t()
        return {"y": y.to(TYPES[c["ytype"]])}
    if c["op"] == "grouped":
        return _plain_grouped(c, state)
    if c["op"] == "route":
        return _plain_route(c, state["logits"])
    return _plain_combine(c, state)


# ------------------------------------------------------------------ 64 bits

def exact(case, seed):
    c, s = case, prepare(case, seed)
    f64 = torch.float64
    if c["op"] == "quant":
        k, kb = c["k"], _blocks(c["k"])
        x = s["x"].to(f64)
        if c["swiglu"]:
            x = x[:, :k] * x[:, k:] * torch.sigmoid(x[:, :k])
        codes = torch.zeros((c["m"], 128 * kb), dtype=f64, device=DEV)
        scale = torch.ones((kb, c["m"]), dtype=f64, device=DEV)
        for b in range(kb):
            v = x[:, 128 * b:min(k, 128 * b + 128)]
            a = v.abs().max(1).values
            scale[b] = torch.where(a > 0, torch.maximum(a / 448.0, torch.full_like(a, TINY)), torch.ones_like(a))
            r = v / scale[b][:, None]
            # the nearest E4M3 value: steps of 2^(e - 3), 2^-9 below 2^-6; ties to even
            step = torch.exp2(torch.floor(torch.log2(r.abs().clamp(min=2.0 ** -6))) - 3.0)
            codes[:, 128 * b:128 * b + v.shape[1]] = (torch.round(r / step) * step).clamp(-448.0, 448.0)
        return {"codes": codes, "scale": scale}
    if c["op"] in ("gemm", "grouped"):
        grouped = c["op"] == "grouped"
        w, ws = (s["w"], s["ws"]) if grouped else (s["w"][None], s["ws"][None])
        offsets = s["offsets"].tolist() if grouped else [0, c["m"]]
        tokens = s["row_ids"].long() if grouped and c["gather"] else torch.arange(offsets[-1], device=DEV)
        column = torch.arange(s["q"].shape[1], device=DEV) // 128
        block_row = torch.arange(c["n"], device=DEV) // 128
        y = torch.empty((offsets[-1], c["n"]), dtype=f64, device=DEV)
        for e in range(w.shape[0]):
            lo, hi = offsets[e], offsets[e + 1]
            if lo == hi:
                continue
            matrix = w[e].to(f64) * ws[e].to(f64)[block_row][:, column]
            t = tokens[lo:hi]
            y[lo:hi] = (s["q"][t].to(f64) * s["qs"].to(f64)[column][:, t].t()) @ matrix.t()
        return {"y": y}
    if c["op"] == "route":
        x = s["logits"].to(f64)
        x = torch.where(torch.isnan(x), -math.inf, x).clamp(max=HUGE)
        p = torch.softmax(x, 1).nan_to_num(0.0)
        w = torch.zeros((c["tokens"], c["top"]), dtype=f64, device=DEV)
        left = x.clone()
        for j in range(c["top"]):
            best = left.max(1, keepdim=True).values
            at = (left == best).to(torch.int8).argmax(1, keepdim=True)      # the lowest index of the largest
            w[:, j] = torch.where(best > -math.inf, p.gather(1, at), 0.0)[:, 0]
            left.scatter_(1, at, -math.inf)
        if c["renorm"]:
            w = torch.where(w > 0, w / w.sum(1, keepdim=True), 0.0)
        return {"ids": None, "weights": w, "offsets": None, "row_ids": None, "slots": None}
    out = torch.zeros((c["tokens"], c["d"]), dtype=f64, device=DEV)
    for j in range(c["top"]):
        at = s["slots"][:, j].long()
        term = s["y"][at.clamp(min=0)].to(f64) * s["weights"][:, j, None].to(f64)
        out += torch.where(at[:, None] >= 0, term, 0.0)
    return {"out": out}
