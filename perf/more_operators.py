"""Cases for the operators of a cheaper block: norms around a branch, 4-bit projections, attention over chosen blocks.

Six operators, each in a plain form (elementary torch operations in 32 bits) and, where `own` is true, through the
library's entry points:

  norm    the norm after a branch, its gate, the scaled residual and the norm before the next branch
  linear  a projection in microscaled 4-bit floating point: rows quantised as they come, weights once when loaded
  swiglu  the same for the gate/up projection with SwiGLU
  scores  a cheap score of every (query block, key block): the product of the blocks' mean rows
  select  the best-scored key blocks of every query block
  attend  attention of the query blocks over their chosen key blocks

Sizes are a function of the case alone, values of the seed.
"""
import math
import random

import torch

own = False

DEV = "cuda"
DH = 128
QB = 256          # rows of a query block
EPS = 1e-6


# ------------------------------------------------------------------- cases
def _norm(name=None, **kw):
    c = {"op": "norm", "rows": 1, "D": 5376, "rms": False, "groups": 0, "rscale": 1.0, "after": True}
    return _named(c, name, kw)


def _gemm(op, name=None, **kw):
    c = {"op": op, "rows": 1, "N": 5376, "K": 5376, "form": "nv"}
    return _named(c, name, kw)


def _blocks(op, name=None, **kw):
    c = {"op": op, "Lq": 1, "Lk": 1, "H": 42, "Hkv": 42, "kb": 64, "sel": 1, "first": 0, "last": 0, "ragged": False,
         "mix": 1}
    return _named(c, name, kw)


def _named(c, name, kw):
    c.update(kw)
    if name:
        c["name"] = name
    return c


def listed():
    return [
        # the 22 text and audio rows at the end of a packed sequence: latency
        _norm("norm_rows", rows=22, rms=True),
        # a 10 s packed sequence, two token groups with modulations of their own
        _norm("norm_packed", rows=58758, groups=2, rscale=0.75),
        # the output projection of the 22 text and audio rows: the weights' bytes count
        _gemm("linear", "linear_rows", rows=22, form="mx"),
        # the QKV projection of a 10 s sequence
        _gemm("linear", "linear_packed", rows=58758, N=16128),
        # odd sizes of a small model
        _gemm("swiglu", "swiglu_ragged", rows=1999, N=1408, K=1056, form="mx"),
        # the gate/up projection of a 5 s sequence
        _gemm("swiglu", "swiglu_packed", rows=29034, N=14336),
        # one latent frame against a 5 s sequence, grouped heads, large blocks
        _blocks("scores", "scores_frame", Lq=1896, Lk=29034, H=40, Hkv=8, kb=128),
        _blocks("scores", "scores_packed", Lq=58758, Lk=58758),
        # one latent frame: a tenth of the blocks, the text's last one among them
        _blocks("select", "select_frame", Lq=1896, Lk=29034, H=40, kb=128, sel=23, last=1),
        _blocks("select", "select_packed", Lq=58758, Lk=58758, sel=92, first=1, last=1),
        # the text rows over a tenth of a 5 s sequence, grouped heads: few items, long lists
        _blocks("attend", "attend_rows", Lq=22, Lk=29034, H=40, Hkv=8, kb=128, sel=23, ragged=True, mix=3),
        # a 10 s sequence over a tenth of its blocks
        _blocks("attend", "attend_packed", Lq=58758, Lk=58758, sel=92),
    ]


_HEADS = [(42, 42), (4, 4), (32, 8), (32, 4), (40, 8), (16, 2), (24, 1), (12, 12), (28, 4), (64, 8)]
_WIDTHS = [512, 1024, 1152, 1928, 2048, 2560, 4096, 5120, 5376, 8192]
_PACKED = 58758


def _log(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(max(lo, hi)))))))


def draw(rng):
    op = rng.choice(["norm", "linear", "swiglu", "scores", "select", "attend"])
    if op == "norm":
        D = rng.choice(_WIDTHS)
        return _norm(rows=_log(rng, 1, _PACKED * 5376 // max(D, 5376)), D=D, rms=rng.random() < 0.5,
                     groups=rng.choice([0, 0, 2, 3]), rscale=rng.choice([1.0, 0.5, 0.75]), after=rng.random() < 0.8)
    if op in ("linear", "swiglu"):
        K = 32 * _log(rng, 4, 448)
        if op == "linear":
            N = 8 * _log(rng, 8, 2016)
            top = _PACKED * 16128 * 5376 // (N * K)
        else:
            N = 128 * _log(rng, 2, 112)
            top = 29034 * 14336 * 5376 // (N * K)
        return _gemm(op, rows=_log(rng, 1, min(_PACKED, top)), N=N, K=K, form=rng.choice(["mx", "nv"]))
    H, Hkv = rng.choice(_HEADS)
    kb = rng.choice([64, 128])
    c = _blocks(op, H=H, Hkv=Hkv, kb=kb, mix=rng.randrange(1, 1 << 20))
    c["Lk"] = _log(rng, 1, _PACKED * 42 // max(42, H))
    c["Lq"] = _log(rng, 1, _PACKED * 42 // max(42, H))
    nk = -(-c["Lk"] // kb)
    if op == "select":
        c["sel"] = _log(rng, 1, nk)
        c["first"], c["last"] = rng.choice([(0, 0), (1, 0), (0, 1), (1, 2)])
        if c["first"] + c["last"] > c["sel"]:
            c["first"] = c["last"] = 0
    if op == "attend":
        c["ragged"] = rng.random() < 0.4
        pairs = _PACKED * 92 * 64 * 42          # rows x keys x heads of the largest case
        c["sel"] = _log(rng, 1, min(nk, max(1, pairs // (-(-c["Lq"] // QB) * QB * kb * H)), 256))
    return c


def _counts(case):
    """Key blocks that a head's query block is given: all of them the same number, or ragged with some none."""
    n = case["H"] * -(-case["Lq"] // QB)
    if not case["ragged"]:
        return [case["sel"]] * n
    r = random.Random(case["mix"])
    return [r.randint(0, case["sel"]) for _ in range(n)]


def work(case):
    op = case["op"]
    if op == "norm":
        n = case["rows"] * case["D"]
        return {"bytes": n * (12 if case["after"] else 10), "flops": n * 16}
    if op in ("linear", "swiglu"):
        M, N, K = case["rows"], case["N"], case["K"]
        wide = N * (2 if op == "swiglu" else 1)
        bits = 4 + (8 / 32 if case["form"] == "mx" else 8 / 16)
        return {"bytes": M * K * 2 + wide * K * bits / 8 + M * N * 2, "flops": 2 * M * wide * K}
    nq, nk = -(-case["Lq"] // QB), -(-case["Lk"] // case["kb"])
    if op == "scores":
        rows = case["Lq"] * case["H"] + case["Lk"] * case["Hkv"]
        return {"bytes": rows * DH * 2 + case["H"] * nq * nk * 4,
                "flops": rows * DH + 2 * DH * case["H"] * nq * nk}
    if op == "select":
        n = case["H"] * nq
        return {"bytes": n * (nk + case["sel"] + 1) * 4, "flops": n * nk}
    counts = _counts(case)
    per = [min(QB, case["Lq"] - (i % nq) * QB) for i in range(len(counts))]
    pairs = case["kb"] * sum(a * b for a, b in zip(per, counts))
    chosen = min(case["Lk"] * case["Hkv"], sum(counts) * case["kb"])  # key rows that are read at all, at most
    return {"bytes": case["Lq"] * case["H"] * DH * 4 + chosen * DH * 4 + sum(counts) * 4, "flops": 4 * DH * pairs}


# ------------------------------------------------------------------ inputs
def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    op = case["op"]

    def rnd(*shape, std=1.0):
        return torch.randn(*shape, generator=g, device=DEV) * std

    def bf(*shape, std=1.0):
        x = torch.randn(*shape, generator=g, device=DEV, dtype=torch.bfloat16)
        return x if std == 1.0 else x * std

    def unit(*shape):  # unit root-mean-square per head, as a normed head has
        x = bf(*shape)
        for part in x.split(max(1, (1 << 28) // max(1, x[0].numel()))):
            f = part.float()
            part.copy_(f * torch.rsqrt(f.square().mean(-1, keepdim=True)))
        return x

    s = {"case": dict(case)}
    if op == "norm":
        L, D, G = case["rows"], case["D"], case["groups"]
        s["resid"] = rnd(L, D)
        s["resid_out"] = torch.empty_like(s["resid"])
        s["delta"] = bf(L, D, std=3.0)
        s["normed"] = torch.empty_like(s["delta"])
        s["post_gain"] = 1 + rnd(D, std=0.1) if case["after"] else None
        mod = rnd(max(G, 1), 6, D, std=0.1)
        s["seg"] = (torch.arange(L, device=DEV) * max(G, 1) // L).to(torch.int32) if G else None
        s["gate"], s["shift"], s["scale"] = (mod[:, i] if G else mod[0, i] for i in (2, 3, 4))
        return s
    if op in ("linear", "swiglu"):
        M, N, K = case["rows"], case["N"], case["K"]
        # activations with a few wide channels, as a normed and modulated row has
        s["x"] = bf(M, K)
        s["x"][:, :: 97] *= 8
        s["w"] = bf(N * (2 if op == "swiglu" else 1), K, std=0.02)
        s["y"] = torch.empty(M, N, device=DEV, dtype=torch.bfloat16)
        return s
    nq, nk, H = -(-case["Lq"] // QB), -(-case["Lk"] // case["kb"]), case["H"]
    if op == "select":
        # pooled scores: coarse enough that some tie, and some blocks masked out
        x = rnd(H, nq, nk).to(torch.bfloat16).float()
        x[torch.rand(H, nq, nk, generator=g, device=DEV) < 0.02] = -math.inf
        s["scores"] = x
        s["ids"] = torch.empty(H, nq, case["sel"], dtype=torch.int32, device=DEV)
        s["count"] = torch.empty(H, nq, dtype=torch.int32, device=DEV)
        return s
    s["q"], s["k"] = unit(case["Lq"], H, DH), unit(case["Lk"], case["Hkv"], DH)
    if op == "scores":
        s["scores"] = torch.empty(H, nq, nk, device=DEV)
        return s
    s["v"] = bf(case["Lk"], case["Hkv"], DH)
    s["o"] = torch.empty_like(s["q"])
    ids = torch.empty(H * nq, case["sel"], dtype=torch.int32, device=DEV)
    for a, part in zip(range(0, H * nq, 4096), ids.split(4096)):  # distinct blocks, ascending
        part.copy_(torch.rand(part.shape[0], nk, generator=g, device=DEV).topk(case["sel"], -1).indices.sort(-1).values)
    s["count"] = torch.tensor(_counts(case), dtype=torch.int32, device=DEV).view(H, nq)
    listed_ = torch.arange(case["sel"], device=DEV) < s["count"].view(-1, 1)
    s["ids"] = torch.where(listed_, ids, -1).to(torch.int32).view(H, nq, case["sel"])
    return s


# -------------------------------------------------------------- plain forms
def _centred(x, rms):
    if not rms:
        x = x - x.mean(-1, keepdim=True)
    return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)


def _plain_norm(s):
    c = s["case"]
    pick = (lambda t: t[s["seg"].long()]) if c["groups"] else (lambda t: t)
    y = s["delta"].float()
    if c["after"]:
        y = _centred(y, c["rms"]) * s["post_gain"]
    r = c["rscale"] * s["resid"] + pick(s["gate"]) * y
    h = _centred(r, c["rms"]) * (1 + pick(s["scale"])) + pick(s["shift"])
    return {"resid": r, "normed": h.to(torch.bfloat16)}


def _e2m1(y):
    """The nearest of 0, 0.5, 1, 1.5, 2, 3, 4, 6 (ties to the even code, larger ones to 6), with y's sign."""
    a = y.abs()
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    return torch.copysign(torch.minimum((a / step).round() * step, torch.full_like(a, 6.0)), y)


def _rows4(x, form):
    """Values that x [R, K] bf16 has after quantisation, without the rows' own scales, and those [R, 1]."""
    R, K = x.shape
    if form == "mx":
        b = x.float().view(R, K // 32, 32)
        top = b.abs().amax(-1, keepdim=True)
        e = torch.floor(torch.log2(top.clamp(min=2.0 ** -125))).clamp(min=-125.0) - 2
        e = torch.where(torch.exp2(e + 2) > top.clamp(min=2.0 ** -125), e - 1, e)     # where the logarithm rounded up
        return (_e2m1(b * torch.exp2(-e)) * torch.exp2(e)).view(R, K), torch.ones(R, 1, device=DEV)
    b = x.float().view(R, K // 16, 16)
    row = b.abs().amax((-1, -2)).view(R, 1, 1)
    safe = torch.where(row > 0, row, 1.0)
    one = torch.ones_like(safe)
    sf = (b.abs().amax(-1, keepdim=True) * (448 * one / safe)).to(torch.float8_e4m3fn).float()
    inv = torch.where(sf > 0, (2688 * one / safe) / torch.where(sf > 0, sf, 1.0), 0.0)
    return (_e2m1(b * inv) * sf).view(R, K), (row / (2688 * one)).view(R, 1)


def _plain_product(s):
    c = s["case"]
    if "w_rows" not in s:  # once, when the weights are loaded
        s["w_rows"] = _rows4(s["w"], c["form"])
    (x, rx), (w, rw) = _rows4(s["x"], c["form"]), s["w_rows"]
    y = (x @ w.T).mul_(rx).mul_(rw.view(1, -1))
    if c["op"] == "linear":
        return {"y": y.to(torch.bfloat16)}
    g, u = (t.to(torch.bfloat16).float() for t in y.chunk(2, -1))   # rounded between the product and the gate
    return {"y": (g / (1 + torch.exp(-g)) * u).to(torch.bfloat16)}


def _means(x, block):
    """Means of every `block` rows of [L, heads, 128]: [heads, blocks, 128]."""
    L, heads, _ = x.shape
    n = -(-L // block)
    full = L // block
    m = torch.empty(n, heads, DH, device=DEV)
    for a in range(0, full, 256):
        b = min(full, a + 256)
        m[a:b] = x[a * block:b * block].float().view(b - a, block, heads, DH).mean(1)
    if full < n:
        m[full] = x[full * block:].float().mean(0)
    return m.transpose(0, 1)


def _plain_scores(s):
    c = s["case"]
    mq, mk = _means(s["q"], QB), _means(s["k"], c["kb"])
    mk = mk.repeat_interleave(c["H"] // c["Hkv"], 0)
    return {"scores": (mq * DH ** -0.5) @ mk.transpose(-1, -2)}


def _plain_select(s):
    c, x = s["case"], s["scores"]
    nk = x.shape[-1]
    j = torch.arange(nk, device=DEV)
    kept = ((j < c["first"]) | (j >= nk - c["last"])).expand(x.shape)
    x = torch.where(x.isnan(), -math.inf, x)
    order = x.sort(dim=-1, descending=True, stable=True).indices
    order = order.gather(-1, kept.gather(-1, order).int().sort(dim=-1, descending=True, stable=True).indices)
    order = order[..., :c["sel"]]
    some = kept.gather(-1, order) | (x.gather(-1, order) > -math.inf)
    ids = torch.where(some, order, nk).sort(-1).values
    ids = torch.where(ids < nk, ids, -1)
    if ids.shape[-1] < c["sel"]:
        ids = torch.nn.functional.pad(ids, (0, c["sel"] - ids.shape[-1]), value=-1)
    return {"ids": ids.to(torch.int32), "count": some.sum(-1).to(torch.int32)}


def _plain_attend(s):
    c = s["case"]
    Lq, Lk, H, kb = c["Lq"], c["Lk"], c["H"], c["kb"]
    nq, nk, n = -(-Lq // QB), -(-Lk // kb), c["sel"] * kb
    items = H * nq
    head = torch.arange(items, device=DEV) // nq
    first = torch.arange(items, device=DEV) % nq * QB
    ids, count = s["ids"].view(items, -1).long(), s["count"].view(items, 1)
    o = torch.zeros(Lq, H, DH, device=DEV, dtype=torch.bfloat16)
    per = max(1, (1 << 28) // (QB * n))
    slot = torch.arange(c["sel"], device=DEV)
    for a in range(0, items, per):
        h, rows = head[a:a + per, None], first[a:a + per, None] + torch.arange(min(QB, Lq), device=DEV)
        q = s["q"][rows.clamp(max=Lq - 1), h].float() * DH ** -0.5                       # [items, 256, 128]
        ok = (slot < count[a:a + per]) & (ids[a:a + per] >= 0) & (ids[a:a + per] < nk)
        at = ids[a:a + per, :, None].clamp(0, nk - 1) * kb + torch.arange(kb, device=DEV)
        ok = (ok[..., None] & (at < Lk)).flatten(1)[:, None]
        at = at.clamp(max=Lk - 1).flatten(1)
        g = h // (H // c["Hkv"])
        z = (q @ s["k"][at, g].float().transpose(-1, -2)).masked_fill_(~ok, -math.inf)
        top = z.amax(-1, keepdim=True)
        p = z.sub_(torch.where(top == -math.inf, 0.0, top)).exp_()
        total = p.sum(-1, keepdim=True)
        y = p @ s["v"][at, g].float()
        y = torch.where(total > 0, y / total, 0.0).to(torch.bfloat16)
        real = rows < Lq
        o[rows[real], h.expand_as(rows)[real]] = y[real]
    return {"o": o}


def _handles(s):
    """What a program keeps: the 4-bit weights, room for the rows' codes, scratch memory."""
    from dit_transformer_block_gb300 import h3
    c = s["case"]
    if c["op"] in ("linear", "swiglu"):
        s["w4"] = h3.fp4_rows(*s["w"].shape, format=c["form"])
        h3.quantize_fp4_rows(s["w"], s["w4"])
        s["x4"] = h3.fp4_rows(*s["x"].shape, format=c["form"])
    elif c["op"] == "scores":
        s["scratch"] = torch.empty(h3.block_scores_workspace_bytes(c["Lq"], c["Lk"], c["H"], c["Hkv"], c["kb"]),
                                   dtype=torch.uint8, device=DEV)
    s["h3"] = h3


def run(s):
    c = s["case"]
    op = c["op"]
    if not own:
        return {"norm": _plain_norm, "linear": _plain_product, "swiglu": _plain_product, "scores": _plain_scores,
                "select": _plain_select, "attend": _plain_attend}[op](s)
    if "h3" not in s:
        _handles(s)
    h3 = s["h3"]
    if op == "norm":
        h3.sandwich_norm(s["resid"], s["delta"], s["normed"], resid_out=s["resid_out"], post_norm=c["after"],
                         post_gain=s["post_gain"], gate=s["gate"], resid_scale=c["rscale"], shift=s["shift"],
                         scale=s["scale"], seg=s["seg"], rms=c["rms"], eps=EPS)
        return {"resid": s["resid_out"], "normed": s["normed"]}
    if op in ("linear", "swiglu"):
        h3.quantize_fp4_rows(s["x"], s["x4"])
        (h3.linear_fp4 if op == "linear" else h3.linear_swiglu_fp4)(s["x4"], s["w4"], s["y"])
        return {"y": s["y"]}
    if op == "scores":
        h3.block_scores(s["q"], s["k"], s["scores"], s["scratch"], k_block=c["kb"])
        return {"scores": s["scores"]}
    if op == "select":
        h3.block_select(s["scores"], s["ids"], s["count"], keep_first=c["first"], keep_last=c["last"])
        return {"ids": s["ids"], "count": s["count"]}
    h3.attention_blocks(s["q"], s["k"], s["v"], s["o"], s["ids"], s["count"], k_block=c["kb"])
    return {"o": s["o"]}


# -------------------------------------------------------------------- exact
def _f32(x):
    """64-bit values rounded to 32 bits, held in 64: a step that the definition takes in 32 bits."""
    return x.float().double()


def _nearest(y, grid):
    """The nearest value of an ascending grid whose even places are the even codes; ties go to those."""
    g = torch.tensor(grid, dtype=torch.float64, device=DEV)
    a = y.abs()
    hi = torch.searchsorted(g, a).clamp(max=len(grid) - 1)
    lo = (hi - 1).clamp(min=0)
    up, down = g[hi] - a, a - g[lo]
    near = torch.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)
    return torch.copysign(g[near], y)


_E2M1 = [0, 0.5, 1, 1.5, 2, 3, 4, 6]
_E4M3 = [m * 2.0 ** -9 for m in range(8)] + [(8 + m) * 2.0 ** (e - 10) for e in range(1, 16) for m in range(8)][:-1]


def _exact_rows(x, form):
    parts = []
    for p in x.split(2048):
        n = 32 if form == "mx" else 16
        b = p.double().view(p.shape[0], -1, n)
        top = b.abs().amax(-1, keepdim=True)
        if form == "mx":  # the largest power of two in top, over the largest in 6
            e = (torch.frexp(top).exponent.double() - 3).clamp(min=-127)
            e = torch.where(top > 0, e, -127.0)
            parts.append((_nearest(b / torch.exp2(e), _E2M1) * torch.exp2(e)).flatten(1))
            continue
        row = top.amax(1, keepdim=True)
        safe = torch.where(row > 0, row, 1.0)
        sf = _nearest(_f32(top * _f32(448 / safe)), _E4M3)
        inv = torch.where(sf > 0, _f32(_f32(2688 / safe) / torch.where(sf > 0, sf, 1.0)), 0.0)
        parts.append((_nearest(_f32(b * inv), _E2M1) * sf * _f32(row / 2688)).flatten(1))
    return torch.cat(parts)


def _norm64(x, rms):
    mean = 0 if rms else x.sum(-1, keepdim=True) / x.shape[-1]
    return (x - mean) / ((x - mean).pow(2).sum(-1, keepdim=True) / x.shape[-1] + EPS).sqrt()


def exact(case, seed):
    """The definitions in 64 bits (what a definition rounds to 32 or fewer bits on its way is rounded)."""
    if work(case)["flops"] > 1.1e13:
        return None
    s = prepare(case, seed)
    op = case["op"]
    if op == "norm":
        out = {"resid": [], "normed": []}
        for a in range(0, case["rows"], 4096):
            at = slice(a, a + 4096)
            seg = s["seg"][at].long() if case["groups"] else None
            gate, shift, scale = (t.double() if seg is None else t.double()[seg]
                                  for t in (s["gate"], s["shift"], s["scale"]))
            y = s["delta"][at].double()
            if case["after"]:
                y = _norm64(y, case["rms"]) * s["post_gain"].double()
            r = case["rscale"] * s["resid"][at].double() + gate * y
            out["resid"].append(r)
            out["normed"].append(_norm64(r, case["rms"]) * (1 + scale) + shift)
        return {k: torch.cat(v) for k, v in out.items()}
    if op in ("linear", "swiglu"):
        w = _exact_rows(s["w"], case["form"])
        out = []
        for p in s["x"].split(8192):
            y = _exact_rows(p, case["form"]) @ w.T
            if op == "swiglu":
                g, u = y.to(torch.bfloat16).double().chunk(2, -1)
                y = g * torch.sigmoid(g) * u
            out.append(y)
        return {"y": torch.cat(out)}
    Lq, Lk, H, Hkv, kb = (case[k] for k in ("Lq", "Lk", "H", "Hkv", "kb"))
    nq, nk = -(-Lq // QB), -(-Lk // kb)
    if op == "scores":
        out = torch.empty(H, nq, nk, dtype=torch.float64, device=DEV)
        for h in range(H):
            mean = [torch.stack([p.double().sum(0) / p.shape[0] for p in t.split(n)])
                    for t, n in ((s["q"][:, h], QB), (s["k"][:, h // (H // Hkv)], kb))]
            out[h] = mean[0] @ mean[1].T / math.sqrt(DH)
        return {"scores": out}
    if op == "select":
        j = torch.arange(nk, device=DEV)
        must = (j < case["first"]) | (j >= nk - case["last"])
        ids = torch.full((H * nq, case["sel"]), -1, dtype=torch.int32, device=DEV)
        count = torch.empty(H * nq, dtype=torch.int32, device=DEV)
        per = max(1, (1 << 27) // (nk * nk))
        for a in range(0, H * nq, per):
            x = s["scores"].view(H * nq, nk)[a:a + per].double()
            one, two = x[:, :, None], x[:, None, :]
            ahead = (two > one) | ((two == one) & (j[None, None, :] < j[None, :, None]))   # two comes before one
            ahead = torch.where(must[None, :] == must[:, None], ahead, must[None, :])
            mine = (ahead.sum(-1) < case["sel"]) & (must | (x > -math.inf))
            count[a:a + per] = mine.sum(-1)
            row, at = mine.nonzero(as_tuple=True)
            place = mine.long().cumsum(-1)[row, at] - 1
            ids[a + row, place] = at.to(torch.int32)
        return {"ids": ids.view(H, nq, -1), "count": count.view(H, nq)}
    o = torch.zeros(Lq, H, DH, dtype=torch.float64, device=DEV)
    count = _counts(case)
    lists = s["ids"].cpu().tolist()
    for h in range(H):
        k, v = (t[:, h // (H // Hkv)].double() for t in (s["k"], s["v"]))
        for t in range(nq):
            mine = [b for b in lists[h][t][:count[h * nq + t]]]
            if not mine:
                continue
            at = (torch.tensor(mine, device=DEV)[:, None] * kb + torch.arange(kb, device=DEV)).flatten()
            at = at[at < Lk]
            z = s["q"][t * QB:(t + 1) * QB, h].double() @ k[at].T / math.sqrt(DH)
            o[t * QB:(t + 1) * QB, h] = torch.softmax(z, -1) @ v[at]
    return {"o": o}
