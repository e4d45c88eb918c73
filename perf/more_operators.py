"""Workloads of rotary positions, the 8-bit paged cache with its attention, and the expert layer of few tokens.

Each case names one operator and its sizes.  ``run`` computes it in elementary
torch operations (``own`` false) or through the package's entry points (``own``
true); ``exact`` computes it in 64 bits from its definition.

Definitions.  E4M3 is the finite-only 8-bit type of largest value 448.

* rope: the first r of a head's d columns are r / 2 pairs, columns (i, i + r / 2) or, interleaved,
  (2 i, 2 i + 1); at position p pair i is turned by the angle p f_i and scaled by ms:
  y1 = ms (x1 cos - x2 sin), y2 = ms (x1 sin + x2 cos).  The other columns are copied.
  Backward turns by -p f_i.
* append: a sequence's tokens lie in pages of 64, the page of position p is pages[s, p / 64].
  A page's keys of one head are codes [64, dp] with one scale, its values codes [dp, 64] with another; dp
  is d rounded up to 32, 64, 96, 128, 192 or 256.  The new tokens of sequence s are the rows
  offsets[s] .. offsets[s + 1] - 1 and take its last positions below lens[s]; keys are turned as
  by rope.  scale = the smallest power of two, 2^-126 at least, with |new values| <= 448 scale, but no
  smaller than the page's scale where the page held tokens before; codes = E4M3(value / scale), and
  where the scale has grown the page's earlier codes become E4M3(code * earlier scale / scale).
* attend: o[t, h] = sum_j p_j v_j, p = softmax over j of scale * (q[t, h] . k_j), over the positions j of the
  cache with t's position - window < j <= t's position (no lower bound with window 0).
* moe: each token's `top` largest logits (lowest index first on ties), w their softmax;
  out[t] = sum_j w[t, j] W2[e_j] (silu(G[e_j] x_t) * (U[e_j] x_t)), W13 = [G | U] and W2 in E4M3 with a
  scale for each 128 x 128 block.
"""
import math
import random

import torch

own = False

DEV = "cuda"
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZE = {"f32": 4, "bf16": 2, "f16": 2}
F8 = torch.float8_e4m3fn
TINY = 2.0 ** -126
PAGE = 64
THETA = 10000.0


# ------------------------------------------------------------------ the cases

def listed():
    return [
        # one token's queries between their product and the attention: a launch and little else
        dict(name="rope_1x32x128", op="rope", tokens=1, heads=32, dim=128, rotary=128, interleaved=False, kind="none", backward=False, most=4096, gap=8, dtype="bf16"),
        # a long prompt's queries, cut out of the projections' rows, half of each head turned, scaled for a long context
        dict(name="rope_16384x32x128", op="rope", tokens=16384, heads=32, dim=128, rotary=64, interleaved=False, kind="linear", backward=False, most=131072, gap=16, dtype="bf16"),
        # one decoded token's keys and values
        dict(name="append_1of4096", op="append", seqs=1, new=1, most=4096, ragged=False, kv=8, dim=128, rotary=128, interleaved=False, dtype="bf16"),
        # a decode batch, sequences of unlike length
        dict(name="append_64of2048", op="append", seqs=64, new=1, most=2048, ragged=True, kv=8, dim=128, rotary=128, interleaved=False, dtype="bf16"),
        # prompts and their continuations, starting and ending within pages
        dict(name="append_8x4096of8192", op="append", seqs=8, new=4096, most=8192, ragged=True, kv=8, dim=128, rotary=128, interleaved=False, dtype="bf16"),
        # a small model's heads of 26 columns in fp32, a few tokens a sequence, a window of 1024
        dict(name="attend_9x7of1500_26", op="attend", seqs=9, new=7, most=1500, ragged=True, heads=12, kv=4, dim=26, window=1024, dtype="f32"),
        # one token of one long sequence: few rows, a long cache
        dict(name="attend_1of131072", op="attend", seqs=1, new=1, most=131072, ragged=False, heads=32, kv=8, dim=128, window=0, dtype="bf16"),
        # a decode batch: the cache is read once
        dict(name="attend_64of8192", op="attend", seqs=64, new=1, most=8192, ragged=True, heads=32, kv=8, dim=128, window=0, dtype="bf16"),
        # pieces of prompts against all that came before: bound by arithmetic
        dict(name="attend_4x2048of8192", op="attend", seqs=4, new=2048, most=8192, ragged=False, heads=32, kv=8, dim=128, window=0, dtype="bf16"),
        # one token's expert layer
        dict(name="moe_1of64_2048x1024", op="moe", tokens=1, experts=64, top=8, hidden=2048, ffn=1024, dtype="bf16"),
        # odd sizes in fp32
        dict(name="moe_7of12_312x1092", op="moe", tokens=7, experts=12, top=3, hidden=312, ffn=1092, dtype="f32"),
        # a decode batch: nearly every expert has a few tokens
        dict(name="moe_32of64_2048x1024", op="moe", tokens=32, experts=64, top=8, hidden=2048, ffn=1024, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _size(rng, lo, hi):
    """A size over the logarithm of the range: a multiple of 64 two times in three, any number otherwise."""
    v = _log(rng, lo, hi)
    return max(lo, v // 64 * 64) if rng.random() < 0.67 and v >= 64 else v


def draw(rng):
    most = {}
    for c in listed():
        w = work(c)
        old = most.get(c["op"], {"bytes": 0, "flops": 0})
        most[c["op"]] = {k: max(w[k], old[k]) for k in w}
    op = rng.choice(["rope", "append", "append", "attend", "attend", "attend", "moe", "moe"])
    while True:
        dim = rng.choice([26, 64, 80, 96, 128, 128, 128, 192, 256])
        rotary = rng.choice([dim, dim, dim // 4 * 2])
        dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
        if op == "rope":
            c = dict(op=op, tokens=_log(rng, 1, 16384), heads=_log(rng, 1, 64), dim=dim, rotary=rotary, interleaved=rng.random() < 0.5,
                     kind=rng.choice(["none", "linear", "base"]), backward=rng.random() < 0.3, most=_log(rng, 64, 1 << 20),
                     gap=rng.choice([0, 1, 16]), dtype=dtype)
        elif op == "append":
            new = 1 if rng.random() < 0.5 else _log(rng, 1, 4096)
            c = dict(op=op, seqs=_log(rng, 1, 64), new=new, most=_log(rng, max(64, new), max(4096, 2 * new)), ragged=rng.random() < 0.7, kv=_log(rng, 1, 16), dim=dim,
                     rotary=rotary, interleaved=rng.random() < 0.5, dtype=dtype)
        elif op == "attend":
            kv = _log(rng, 1, 8)
            new = 1 if rng.random() < 0.5 else _log(rng, 1, 2048)
            c = dict(op=op, seqs=_log(rng, 1, 64), new=new, most=_log(rng, max(64, new), 131072), ragged=rng.random() < 0.7, heads=kv * rng.choice([1, 3, 4, 8]), kv=kv,
                     dim=dim, window=rng.choice([0, 0, 1024]), dtype=dtype)
        else:
            experts = _log(rng, 4, 128)
            c = dict(op=op, tokens=_log(rng, 1, 32), experts=experts, top=rng.randint(1, min(8, experts)), hidden=_size(rng, 64, 4096), ffn=_size(rng, 64, 4096),
                     dtype=dtype)
        w = work(c)
        if w["bytes"] <= most[op]["bytes"] and w["flops"] <= most[op]["flops"]:
            # the plain form lays every sequence out at its longest's length
            if op != "attend" or c["seqs"] * c["most"] * c["kv"] * c["dim"] <= 64 * 8192 * 8 * 128 and c["seqs"] * c["heads"] * c["new"] * c["most"] <= 4 * 32 * 2048 * 8192:
                return c


def _lens(c):
    """Each sequence's (new tokens, length with them), from the case alone."""
    r = random.Random(c["seqs"] * 7919 + c["most"] * 31 + c["new"])
    got = []
    for i in range(c["seqs"]):
        new, length = c["new"], c["most"]
        if c["ragged"]:
            new = r.randint((new + 3) // 4, new) if i % 8 != 5 else 0          # some have nothing new
            length = r.randint(new, c["most"])
        got.append((new, length))
    return got


def _keys(c):
    """(query-key pairs, positions of the cache that some query of theirs sees), of one head."""
    pairs = seen = 0
    for new, length in _lens(c):
        first = length - new                                                    # the first query's position
        w = c["window"] or length + 1
        short = max(0, min(new, w - first))                                     # queries that see fewer than w
        pairs += short * first + short * (short + 1) // 2 + (new - short) * w
        seen += min(length, w + new - 1) if new else 0
    return pairs, seen


def _blocks(k):
    return (k + 127) // 128


def work(case):
    c = case
    if c["op"] == "rope":
        n = c["tokens"] * c["heads"]
        return {"bytes": 2 * n * c["dim"] * SIZE[c["dtype"]], "flops": 3 * n * c["rotary"]}
    if c["op"] == "append":
        n = sum(new for new, _ in _lens(c)) * c["kv"] * c["dim"]
        return {"bytes": 2 * n * (SIZE[c["dtype"]] + 1), "flops": 6 * n}
    if c["op"] == "attend":
        pairs, seen = _keys(c)
        rows = sum(new for new, _ in _lens(c)) * c["heads"]
        return {"bytes": 2 * seen * c["kv"] * c["dim"] + 2 * rows * c["dim"] * SIZE[c["dtype"]], "flops": 4 * pairs * c["heads"] * c["dim"]}
    pairs = c["tokens"] * c["top"]
    chosen = c["experts"] * (1.0 - (1.0 - c["top"] / c["experts"]) ** c["tokens"])   # experts with a token, in the mean
    codes = c["hidden"] * (2 * 128 * _blocks(c["ffn"])) + c["ffn"] * 128 * _blocks(c["hidden"])
    return {"bytes": chosen * codes + 2 * c["tokens"] * c["hidden"] * SIZE[c["dtype"]], "flops": 6 * pairs * c["hidden"] * c["ffn"]}


# ------------------------------------------------------------------ the inputs

def _freqs(rotary, kind):
    """Radians a position, in 64 bits: as trained, all divided by 8, or with a base that turns the last pair 8 times slower."""
    r = max(rotary, 1)
    theta = THETA * 8.0 ** (r / max(r - 2, 1)) if kind == "base" else THETA
    f = theta ** -(torch.arange(0, rotary, 2, dtype=torch.float64, device=DEV) / r)
    return f / 8.0 if kind == "linear" else f


def _heads(g, tokens, heads, dim, dtype):
    """Projections of hidden states: normal, a few columns of a head larger, tokens of unlike size."""
    x = torch.randn((tokens, heads, dim), device=DEV, generator=g)
    x *= torch.where(torch.rand((heads, dim), device=DEV, generator=g) < 0.03, 4.0, 1.0)
    x *= torch.exp(0.3 * torch.randn((tokens, 1, 1), device=DEV, generator=g))
    return x.to(dtype)


def _padded(dim):
    return min(p for p in (32, 64, 96, 128, 192, 256) if p >= dim)


def _pow2(amax):
    """The smallest power of two, TINY at least, with amax <= 448 times it."""
    frac, e = torch.frexp(amax / 448.0)                                        # amax / 448 = frac 2^e, frac in [0.5, 1)
    return torch.ldexp(torch.ones_like(amax), torch.where(frac == 0.5, e - 1, e).clamp(min=-126)).clamp(min=TINY)


def _coded(x, scale):
    return (x / scale).clamp(-448.0, 448.0).to(F8)


def _cache(g, pages, heads, dim):
    """Keys and values of pages that are full: codes [pages, heads, 64, dp], [pages, heads, dp, 64] and scales [pages, heads]."""
    dp = _padded(dim)
    k = torch.zeros((pages, heads, PAGE, dp), dtype=F8, device=DEV)
    v = torch.zeros((pages, heads, dp, PAGE), dtype=F8, device=DEV)
    ks, vs = torch.empty((pages, heads), device=DEV), torch.empty((pages, heads), device=DEV)
    large = torch.where(torch.rand((heads, 1, dim), device=DEV, generator=g) < 0.03, 4.0, 1.0)
    for p in range(0, pages, 4096):                                            # a part at a time: the inputs are larger than the codes
        n = min(4096, pages - p)
        x = torch.randn((n, heads, PAGE, dim), device=DEV, generator=g) * large
        ks[p:p + n] = _pow2(x.abs().amax((2, 3)))
        k[p:p + n, :, :, :dim] = _coded(x, ks[p:p + n, :, None, None])
        x = torch.randn((n, heads, dim, PAGE), device=DEV, generator=g)
        vs[p:p + n] = _pow2(x.abs().amax((2, 3)))
        v[p:p + n, :, :dim] = _coded(x, vs[p:p + n, :, None, None])
    return k, v, ks, vs


def _tables(c, g, s):
    """The batch: lens, offsets, the pages of each sequence in a random order, and what a scheduler knows of them on the host."""
    lens = _lens(c)
    need = [max(1, -(-length // PAGE)) for _, length in lens]
    width, count = max(need), sum(need) + 3
    order = torch.randperm(count, device=DEV, generator=g).to(torch.int32)
    used = torch.arange(width, device=DEV)[None] < torch.tensor(need, device=DEV)[:, None]
    pages = torch.full((c["seqs"], width), -1, dtype=torch.int32, device=DEV)
    pages[used] = order[:sum(need)]
    s["pages"], s["count"] = pages, count
    s["lens"] = torch.tensor([length for _, length in lens], dtype=torch.int32, device=DEV)
    new = torch.tensor([n for n, _ in lens], device=DEV)
    s["offsets"] = torch.nn.functional.pad(torch.cumsum(new, 0), (1, 0)).to(torch.int32)
    s["tokens"], s["most_new"] = sum(n for n, _ in lens), max(n for n, _ in lens)
    s["seq"] = torch.repeat_interleave(torch.arange(c["seqs"], device=DEV), new)
    s["place"] = torch.arange(s["tokens"], device=DEV) - s["offsets"].long()[s["seq"]]
    s["positions"] = (s["lens"].long()[s["seq"]] - new[s["seq"]] + s["place"]).to(torch.int32)


def _matrices(g, experts, n, k):
    """Quantized weights: codes [experts, n, 128 kb], scale [experts, ceil(n / 128), kb]."""
    kb, nb = _blocks(k), _blocks(n)
    codes = torch.empty((experts, n, 128 * kb), dtype=F8, device=DEV)
    scale = torch.empty((experts, nb, kb), device=DEV)
    for e in range(experts):
        w = torch.zeros((128 * nb, 128 * kb), device=DEV)
        w[:n, :k] = k ** -0.5 * torch.randn((n, k), device=DEV, generator=g)
        w = w.view(nb, 128, kb, 128)
        s = (w.abs().amax((1, 3)) / 448.0).clamp(min=TINY)
        codes[e] = (w / s[:, None, :, None]).clamp(-448.0, 448.0).to(F8).view(128 * nb, 128 * kb)[:n]
        scale[e] = s
    return codes, scale


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    s = {"case": c}
    dtype = TYPES[c["dtype"]]
    if c["op"] == "rope":
        wide = _heads(g, c["tokens"], c["heads"] + c["gap"], c["dim"], dtype)
        s["x"] = wide[:, :c["heads"]]                                          # with a gap: part of the projections' rows
        s["positions"] = torch.randint(0, c["most"], (c["tokens"],), device=DEV, generator=g).to(torch.int32)
        s["freqs"] = _freqs(c["rotary"], c["kind"])
        s["mscale"] = 1.0 if c["kind"] == "none" else 0.1 * math.log(8.0) + 1.0
    elif c["op"] == "append":
        _tables(c, g, s)
        s["cache"] = _cache(g, s["count"], c["kv"], c["dim"])
        both = _heads(g, max(1, s["tokens"]), 2 * c["kv"], c["dim"], dtype)    # keys and values side by side
        s["k"], s["v"] = both[:, :c["kv"]], both[:, c["kv"]:]
        s["freqs"] = _freqs(c["rotary"], "none")
        at = s["positions"].long()
        s["slot"], s["page"] = at % PAGE, s["pages"].long()[s["seq"], at // PAGE]
        s["touched"], s["which"] = torch.unique(s["page"], return_inverse=True)
        s["held"] = torch.full((s["count"],), PAGE, device=DEV).scatter_reduce(0, s["page"], s["slot"], "amin")[s["touched"]]
    elif c["op"] == "attend":
        _tables(c, g, s)
        s["cache"] = _cache(g, s["count"], c["kv"], c["dim"])
        s["q"] = _heads(g, max(1, s["tokens"]), c["heads"], c["dim"], dtype)
    else:
        s["x"] = _heads(g, c["tokens"], 1, c["hidden"], dtype)[:, 0]
        s["logits"] = torch.randn((c["tokens"], c["experts"]), device=DEV, generator=g).to(dtype)
        s["w13"], s["s13"] = _matrices(g, c["experts"], 2 * c["ffn"], c["hidden"])
        s["w2"], s["s2"] = _matrices(g, c["experts"], c["hidden"], c["ffn"])
    return s


# ------------------------------------------------------------------ the package's operators

def _own(s):
    from bit_quantized_matmul_amd import binding as B
    c = s["case"]
    if c["op"] == "rope":
        return {"y": B.rope(s["x"], s["positions"], s["freqs"], interleaved=c["interleaved"], mscale=s["mscale"], backward=c["backward"])}
    if c["op"] == "append":
        cache = B.KvCache(*s["cache"])
        B.kv_append(cache, s["k"], s["v"], s["pages"], s["lens"], offsets=s["offsets"], positions=s["positions"], freqs=s["freqs"], interleaved=c["interleaved"])
        return dict(zip(("k", "v", "k_scale", "v_scale"), cache))
    if c["op"] == "attend":
        return {"o": B.kv_attention(s["q"], B.KvCache(*s["cache"]), s["pages"], s["lens"], offsets=s["offsets"], window=c["window"])}
    return {"out": B.moe_ffn(s["x"], s["w13"], s["s13"], s["w2"], s["s2"], s["logits"], c["top"])}


# ------------------------------------------------------------------ the plain forms

def _turned(x, positions, freqs, interleaved, mscale, backward):
    """rope of x [tokens, heads, dim] in fp32; angles in 64 bits."""
    x = x.to(torch.float32)
    r = 2 * freqs.numel()
    angle = positions.to(torch.float64)[:, None] * freqs
    cos, sin = (mscale * torch.cos(angle)).to(torch.float32)[:, None], (mscale * torch.sin(angle)).to(torch.float32)[:, None]
    sin = -sin if backward else sin
    x1, x2 = (x[..., 0:r:2], x[..., 1:r:2]) if interleaved else (x[..., :r // 2], x[..., r // 2:r])
    y1, y2 = x1 * cos - x2 * sin, x1 * sin + x2 * cos
    y = torch.stack((y1, y2), -1).flatten(-2) if interleaved else torch.cat((y1, y2), -1)
    return torch.cat((y, x[..., r:]), -1)


def _plain_append(c, s):
    k, v, ks, vs = s["cache"]
    n, dim = s["tokens"], c["dim"]
    new_k = _turned(s["k"][:n], s["positions"], s["freqs"], c["interleaved"], 1.0, False)
    new_v = s["v"][:n].to(torch.float32)
    touched, which, slot = s["touched"], s["which"], s["slot"]
    held = s["held"][:, None]
    before = torch.arange(PAGE, device=DEV) < held                              # slots of tokens that were there before
    for codes, scale, x, turn in ((k, ks, new_k, False), (v, vs, new_v, True)):
        part = codes[touched, :, :, :dim] if not turn else codes[touched, :, :dim].transpose(2, 3)
        amax = torch.zeros((touched.numel(), c["kv"]), device=DEV).scatter_reduce(0, which[:, None].expand(-1, c["kv"]), x.abs().amax(2), "amax")
        old, need = scale[touched], _pow2(amax)
        now = torch.where(held > 0, torch.maximum(old, need), need)
        page = part.to(torch.float32) * torch.where(before[:, None], (old / now)[..., None], 1.0)[..., None]
        page[which, :, slot] = x / now[which][..., None]
        page = page.clamp(-448.0, 448.0).to(F8)
        if turn:
            codes[touched, :, :dim] = page.transpose(2, 3)
        else:
            codes[touched, :, :, :dim] = page
        scale[touched] = now
    return {"k": k, "v": v, "k_scale": ks, "v_scale": vs}


def _plain_attend(c, s):
    """Every sequence at the longest's length, the others masked."""
    k, v, ks, vs = s["cache"]
    seqs, kv, dim, most = c["seqs"], c["kv"], c["dim"], s["most_new"]
    rep, at = c["heads"] // kv, s["pages"].clamp(min=0).long()
    length = at.shape[1] * PAGE
    keys = (k[at][..., :dim].to(torch.float32) * ks[at][..., None, None]).transpose(1, 2).reshape(seqs * kv, length, dim)
    values = (v[at][..., :dim, :].to(torch.float32) * vs[at][..., None, None]).permute(0, 2, 1, 4, 3).reshape(seqs * kv, length, dim)
    q = torch.zeros((seqs, most, kv, rep, dim), device=DEV)
    where = torch.full((seqs, most), -1, dtype=torch.int64, device=DEV)
    n = s["tokens"]
    q[s["seq"], s["place"]] = s["q"][:n].to(torch.float32).view(n, kv, rep, dim)
    where[s["seq"], s["place"]] = s["positions"].long()
    score = torch.bmm(q.permute(0, 2, 1, 3, 4).reshape(seqs * kv, most * rep, dim), keys.transpose(1, 2)).view(seqs, kv, most, rep, length)
    j = torch.arange(length, device=DEV)
    see = j <= where[..., None]
    if c["window"]:
        see &= j > where[..., None] - c["window"]
    score = (score * dim ** -0.5).masked_fill_(~see[:, None, :, None], -math.inf)
    top = score.amax(-1, keepdim=True)
    score -= torch.where(top > -math.inf, top, 0.0)
    p = score.exp_()
    total = p.sum(-1, keepdim=True)
    o = torch.bmm(p.view(seqs * kv, most * rep, length), values).view(seqs, kv, most, rep, dim) / torch.where(total > 0, total, 1.0)
    o = o.permute(0, 2, 1, 3, 4)[s["seq"], s["place"]].reshape(n, c["heads"], dim)
    return {"o": o.to(TYPES[c["dtype"]])}


def _matrix(w, scale):
    """Weights [..., n, 128 kb] as fp32 values."""
    rows = scale.repeat_interleave(128, -2)[..., :w.shape[-2], :]
    return (w.to(torch.float32).unflatten(-1, (-1, 128)) * rows[..., None]).flatten(-2)


def _plain_moe(c, s):
    m, hidden, ffn, top = c["tokens"], c["hidden"], c["ffn"], c["top"]
    best, ids = torch.sort(s["logits"].to(torch.float32), dim=1, descending=True, stable=True)
    e = torch.exp(best[:, :top] - best[:, :1])
    weights, ids = e / e.sum(1, keepdim=True), ids[:, :top]
    x = s["x"].to(torch.float32)
    if m * top < c["experts"]:                                # few pairs: the matrices of their experts
        at = ids.reshape(-1)
        x = x.repeat_interleave(top, 0)[:, None]
        h = torch.bmm(x, _matrix(s["w13"][at], s["s13"][at])[..., :hidden].transpose(1, 2))
        a = h[..., :ffn] / (1.0 + torch.exp(-h[..., :ffn])) * h[..., ffn:]
        y = torch.bmm(a, _matrix(s["w2"][at], s["s2"][at])[..., :ffn].transpose(1, 2)).view(m, top, hidden)
        return {"out": (y * weights[..., None]).sum(1).to(TYPES[c["dtype"]])}
    share = torch.zeros((m, c["experts"]), device=DEV).scatter(1, ids, weights)
    h = torch.matmul(x, _matrix(s["w13"], s["s13"])[..., :hidden].transpose(1, 2))                    # [experts, m, 2 ffn]
    a = h[..., :ffn] / (1.0 + torch.exp(-h[..., :ffn])) * h[..., ffn:]
    y = torch.bmm(a, _matrix(s["w2"], s["s2"])[..., :ffn].transpose(1, 2))
    return {"out": (y * share.t()[..., None]).sum(0).to(TYPES[c["dtype"]])}


def run(state):
    if own:
        return _own(state)
    c = state["case"]
    if c["op"] == "rope":
        y = _turned(state["x"], state["positions"], state["freqs"], c["interleaved"], state["mscale"], c["backward"])
        return {"y": y.to(TYPES[c["dtype"]])}
    if c["op"] == "append":
        return _plain_append(c, state)
    if c["op"] == "attend":
        return _plain_attend(c, state)
    return _plain_moe(c, state)


# ------------------------------------------------------------------ 64 bits

def _exact_rope(x, positions, freqs, interleaved, mscale, backward):
    """Each pair as a complex number times exp(i angle)."""
    f64 = torch.float64
    x, r = x.to(f64), 2 * freqs.numel()
    if r == 0:
        return x.clone()
    first = torch.arange(0, r, 2, device=DEV) if interleaved else torch.arange(r // 2, device=DEV)
    second = first + (1 if interleaved else r // 2)
    angle = positions.to(f64).outer(freqs) * (-1.0 if backward else 1.0)
    z = torch.complex(x[..., first], x[..., second]) * torch.polar(torch.full_like(angle, mscale), angle)[:, None]
    y = x.clone()
    y[..., first], y[..., second] = z.real, z.imag
    return y


def _nearest(r):
    """The nearest E4M3 value: steps of 2^(e - 3), 2^-9 below 2^-6; ties to even."""
    step = torch.exp2(torch.floor(torch.log2(r.abs().clamp(min=2.0 ** -6))) - 3.0)
    return (torch.round(r / step) * step).clamp(-448.0, 448.0)


def _exact_append(c, s):
    f64 = torch.float64
    got = [t.to(f64) for t in s["cache"]]
    new = (_exact_rope(s["k"], torch.nn.functional.pad(s["positions"], (0, s["k"].shape[0] - s["tokens"])), s["freqs"], c["interleaved"], 1.0, False), s["v"].to(f64))
    table, dim, row = s["pages"].tolist(), c["dim"], 0
    for seq, (count, length) in enumerate(_lens(c)):
        at = length - count
        while at < length:                                                      # a page at a time
            slot, page = at % PAGE, table[seq][at // PAGE]
            n = min(PAGE - slot, length - at)
            for i in (0, 1):
                x = new[i][row:row + n].transpose(0, 1)                         # [heads, n, dim]
                codes = got[i][page] if i == 0 else got[i][page].transpose(1, 2)
                scale = got[2 + i][page].clone()
                need = torch.exp2(torch.ceil(torch.log2(x.abs().amax((1, 2)) / 448.0)).clamp(min=-126.0))
                now = torch.maximum(need, scale) if slot else need
                codes[:, :slot, :dim] = _nearest(codes[:, :slot, :dim] * (scale / now)[:, None, None])
                codes[:, slot:slot + n, :dim] = _nearest(x / now[:, None, None])
                got[2 + i][page] = now
            at, row = at + n, row + n
    return dict(zip(("k", "v", "k_scale", "v_scale"), got))


def _exact_attend(c, s):
    f64 = torch.float64
    k, v, ks, vs = s["cache"]
    rep, o, row = c["heads"] // c["kv"], torch.zeros((s["tokens"], c["heads"], c["dim"]), dtype=f64, device=DEV), 0
    for seq, (count, length) in enumerate(_lens(c)):
        if count == 0:
            continue
        at = s["pages"][seq, :-(-length // PAGE)].long()
        first = length - count
        t, j = torch.arange(first, length, device=DEV)[:, None], torch.arange(length, device=DEV)[None]
        hidden = (j > t) | ((j <= t - c["window"]) if c["window"] else (j < 0))
        for h in range(c["kv"]):
            keys = (k[at, h].to(f64) * ks[at, h].to(f64)[:, None, None]).reshape(-1, k.shape[3])[:length, :c["dim"]]
            values = (v[at, h].to(f64) * vs[at, h].to(f64)[:, None, None]).transpose(1, 2).reshape(-1, k.shape[3])[:length, :c["dim"]]
            for i in range(h * rep, h * rep + rep):
                score = (s["q"][row:row + count, i].to(f64) @ keys.t() / math.sqrt(c["dim"])).masked_fill(hidden, -math.inf)
                o[row:row + count, i] = torch.softmax(score, 1) @ values
        row += count
    return {"o": o}


def _exact_moe(c, s):
    f64 = torch.float64
    out = torch.zeros((c["tokens"], c["hidden"]), dtype=f64, device=DEV)
    logits = s["logits"].to(f64)
    column = lambda n: torch.arange(n, device=DEV) // 128                       # noqa: E731
    for t in range(c["tokens"]):
        left, ids = logits[t].clone(), []
        for _ in range(c["top"]):
            ids.append(int((left == left.max()).to(torch.int8).argmax()))       # the lowest index of the largest
            left[ids[-1]] = -math.inf
        share = torch.softmax(logits[t, ids], 0)
        for e, w in zip(ids, share):
            m13 = s["w13"][e].to(f64)[:, :c["hidden"]] * s["s13"][e].to(f64)[column(2 * c["ffn"])][:, column(c["hidden"])]
            m2 = s["w2"][e].to(f64)[:, :c["ffn"]] * s["s2"][e].to(f64)[column(c["hidden"])][:, column(c["ffn"])]
            h = m13 @ s["x"][t].to(f64)
            out[t] += w * (m2 @ (h[:c["ffn"]] * torch.sigmoid(h[:c["ffn"]]) * h[c["ffn"]:]))
    return {"out": out}


def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["op"] == "rope":
        return {"y": _exact_rope(s["x"], s["positions"], s["freqs"], c["interleaved"], s["mscale"], c["backward"])}
    return {"append": _exact_append, "attend": _exact_attend, "moe": _exact_moe}[c["op"]](c, s)
