"""Cases for the paged key/value cache operators of dit_transformer_block_gb300.

Three operators, each in a plain form (elementary torch operations in 32 bits) and, where `own` is true, through the
library's entry points:

  append  per-head Q/K RMSNorm + rotary embedding with the keys and values written to a paged cache on the way
  paged   attention of a ragged batch over its paged keys, single rows per sequence (decode) or chunks of rows
  prefix  the same where all sequences of the batch share a long prefix of keys

Sequence lengths are a function of the case alone (its "mix"), values a function of the seed.
"""
import math
import random

import torch

own = False

DEV = "cuda"
DH = 128


# ------------------------------------------------------------------- cases
def _case(op, name=None, **kw):
    c = {"op": op, "B": 1, "q_max": 1, "ragged_q": False, "kv_max": 1, "ragged_kv": False, "H": 42, "Hkv": 42,
         "page": 64, "causal": False, "prefix": 0, "pairing": 0, "axis": "32/48/48", "norm": True, "mix": 1}
    c.update(kw)
    if name:
        c["name"] = name
    return c


def listed():
    return [
        # one new row for each of 64 requests on the block's 42 heads: latency
        _case("append", "append_rows", B=64, kv_max=520, ragged_kv=True),
        # grouped heads, ragged chunks, split-half pairs, rotation without a norm, small pages
        _case("append", "append_ragged", B=9, q_max=301, ragged_q=True, kv_max=700, ragged_kv=True, H=32, Hkv=8,
              page=16, pairing=1, axis="128/0/0", norm=False, mix=2),
        # the whole packed 10 s sequence goes to the cache
        _case("append", "append_packed", q_max=58758, kv_max=58758, page=128),
        # the smallest call: one row of a 4-head block against 250 keys
        _case("paged", "row_small", kv_max=250, H=4, Hkv=4),
        # single rows, grouped heads, many ragged requests, small pages
        _case("paged", "rows_grouped", B=96, kv_max=8191, ragged_kv=True, H=32, Hkv=4, page=16, mix=3),
        # single rows of the block's heads against eight 10 s sequences: the largest cache
        _case("paged", "rows_long", B=8, kv_max=58758, page=128, mix=4),
        # one latent frame (24 x 79 rows) against the 10 s sequence it ends
        _case("paged", "frame_chunk", q_max=1896, kv_max=58758, page=128, mix=5),
        # ragged causal chunks, some of one row, on grouped heads
        _case("paged", "causal_ragged", B=6, q_max=901, ragged_q=True, kv_max=6007, ragged_kv=True, H=32, Hkv=8,
              page=32, causal=True, mix=6),
        # eight requests behind a short shared prompt: latency
        _case("prefix", "prefix_small", B=8, kv_max=100, ragged_kv=True, H=16, Hkv=2, prefix=4099, mix=7),
        # 64 variants of one 5 s sequence, single rows
        _case("prefix", "prefix_rows", B=64, kv_max=512, ragged_kv=True, prefix=29034, mix=8),
        # grouped heads behind a longer prefix, single rows
        _case("prefix", "prefix_grouped", B=48, kv_max=1500, ragged_kv=True, H=40, Hkv=8, prefix=58758, page=32,
              mix=9),
        # four variants, a quarter of a latent frame each, behind the 5 s sequence
        _case("prefix", "prefix_chunks", B=4, q_max=474, kv_max=1896, ragged_kv=True, prefix=29034, mix=10),
    ]


_HEADS = [(42, 42), (4, 4), (32, 8), (32, 4), (40, 8), (16, 2), (24, 1), (12, 12), (28, 4), (64, 8)]
_AXES = ["32/48/48", "128/0/0", "16/64/48"]
_KEYS = 8 * 58758 * 42          # key rows x key heads of the largest cache
_SCORES = 1896 * 58758 * 42     # query rows x keys x heads of the largest chunk


def _log(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(max(lo, hi)))))))


def draw(rng):
    H, Hkv = rng.choice(_HEADS)
    c = _case(rng.choice(["append", "paged", "paged", "prefix"]), H=H, Hkv=Hkv, page=rng.choice([16, 32, 64, 128]),
              mix=rng.randrange(1, 1 << 20), ragged_kv=rng.random() < 0.7)
    if c["op"] == "append":
        c["B"] = _log(rng, 1, 128)
        c["q_max"] = _log(rng, 1, 58758 // c["B"] * 42 // max(42, H))
        c["kv_max"] = c["q_max"] + _log(rng, 1, 600)
        c["ragged_q"] = rng.random() < 0.5
        c["pairing"] = rng.randrange(2)
        c["axis"] = rng.choice(_AXES)
        c["norm"] = rng.random() < 0.7
        return c
    chunk = rng.random() < 0.4
    if c["op"] == "prefix":
        c["prefix"] = _log(rng, 100, 58758)
        c["B"] = _log(rng, 2, 8 if chunk else 128)
        c["kv_max"] = _log(rng, 1, 2048)
    else:
        c["B"] = _log(rng, 1, 8 if chunk else 256)
        c["kv_max"] = _log(rng, 1, min(58758, _KEYS // (c["B"] * Hkv)))
    if chunk:
        keys = c["kv_max"] + c["prefix"]
        c["q_max"] = _log(rng, 2, max(2, min(1896 // (1 if c["op"] == "paged" else c["B"]),
                                             _SCORES // (c["B"] * keys * H))))
        c["kv_max"] = max(c["kv_max"], c["q_max"])
        c["ragged_q"] = rng.random() < 0.5
        c["causal"] = rng.random() < 0.5
    return c


def _lengths(case):
    """(q_len, kv_len) of every sequence; kv_len counts the call's own rows."""
    r = random.Random(case["mix"])
    q = [r.randint(1, case["q_max"]) if case["ragged_q"] else case["q_max"] for _ in range(case["B"])]
    kv = [r.randint(1, case["kv_max"]) if case["ragged_kv"] else case["kv_max"] for _ in range(case["B"])]
    return q, [max(a, b) for a, b in zip(q, kv)]


def work(case):
    q, kv = _lengths(case)
    T, H, Hkv = sum(q), case["H"], case["Hkv"]
    row = 2 * DH
    if case["op"] == "append":
        return {"bytes": T * (H + 2 * Hkv) * row * 2 + T * 12, "flops": T * (H + Hkv) * DH * 8}
    pairs = 0
    for a, n in zip(q, kv):
        pairs += a * case["prefix"] + (a * n - a * (a - 1) // 2 if case["causal"] else a * n)
    return {"bytes": (case["prefix"] + sum(kv)) * Hkv * row * 2 + T * H * row * 2, "flops": 4 * DH * H * pairs}


# ------------------------------------------------------------------ inputs
def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    q_len, kv_len = _lengths(case)
    B, T, H, Hkv, P = case["B"], sum(q_len), case["H"], case["Hkv"], case["page"]
    per = -(-max(kv_len) // P)
    n_prefix = -(-case["prefix"] // P)
    used = sum(-(-n // P) for n in kv_len)
    pages = used + n_prefix + 1
    # pages in the order in which a server's free list hands them out: none
    order = torch.randperm(pages, generator=g, device=DEV).to(torch.int32)
    table = torch.zeros(B, per, dtype=torch.int32, device=DEV)
    at = n_prefix
    for b, n in enumerate(kv_len):
        k = -(-n // P)
        table[b, :k] = order[at:at + k]
        at += k

    def unit(*shape):  # unit root-mean-square per head, as a normed head has
        x = torch.randn(*shape, generator=g, device=DEV, dtype=torch.bfloat16)
        for part in x.split(max(1, (1 << 28) // max(1, x[0].numel()))):
            f = part.float()
            part.copy_(f * torch.rsqrt(f.square().mean(-1, keepdim=True)))
        return x

    cu = torch.tensor([0] + q_len, dtype=torch.int64).cumsum(0).to(torch.int32).to(DEV)
    s = {"case": dict(case), "T": T, "per": per, "cu_q": cu,
         "kv_len": torch.tensor(kv_len, dtype=torch.int32, device=DEV), "table": table,
         "k_cache": unit(pages, Hkv, P, DH),
         "v_cache": torch.randn(pages, Hkv, P, DH, generator=g, device=DEV, dtype=torch.bfloat16)}
    if case["prefix"]:
        s["prefix_pages"] = order[:n_prefix].contiguous()
    if case["op"] == "append":
        # the merged projection's output: q, k and v of a row side by side
        qkv = torch.randn(T, (H + 2 * Hkv) * DH, generator=g, device=DEV, dtype=torch.bfloat16) * 2
        s["q"] = qkv[:, :H * DH].unflatten(1, (H, DH))
        s["k"] = qkv[:, H * DH:(H + Hkv) * DH].unflatten(1, (Hkv, DH))
        s["v"] = qkv[:, (H + Hkv) * DH:].unflatten(1, (Hkv, DH))
        s["q_out"] = torch.empty(T, H, DH, device=DEV, dtype=torch.bfloat16)
        axis = [int(x) for x in case["axis"].split("/")]
        s["axis"] = axis
        # (t, h, w) of a packed sequence: the row's key index walked over a 24 x 79 grid, or the index alone
        first = s["kv_len"] - (cu[1:] - cu[:-1])
        rows = torch.arange(T, device=DEV)
        b = torch.searchsorted(cu[1:].contiguous(), rows.to(torch.int32), right=True)
        idx = rows - cu[b].long() + first[b].long()
        if axis[1]:
            pos = torch.stack([idx // (24 * 79), idx // 79 % 24, idx % 79], 1)
        else:
            pos = torch.stack([idx, idx * 0, idx * 0], 1)
        s["pos"] = pos.to(torch.int32).contiguous()
        gains = 1 + 0.1 * torch.randn(2, DH, generator=g, device=DEV)
        s["q_gain"], s["k_gain"] = (gains[0].contiguous(), gains[1].contiguous()) if case["norm"] else (None, None)
    else:
        s["q"] = unit(T, H, DH)
        s["o"] = torch.empty_like(s["q"])
    return s


THETA, EPS = 1e4, 1e-6


# -------------------------------------------------------------- plain forms
def _turn(axis, pairing, pos):
    """cos, sin [T, 64] of every pair and the channels of its two elements; angles in 64 bits."""
    first, second, freq, which = [], [], [], []
    o = 0
    for a, d in enumerate(axis):
        j = torch.arange(d // 2, device=DEV)
        first.append(o + (j if pairing else 2 * j))
        second.append(o + (d // 2 + j if pairing else 2 * j + 1))
        freq.append(THETA ** (-2.0 * j.double() / max(d, 1)))
        which.append(torch.full((d // 2,), a, device=DEV))
        o += d
    phi = pos.double()[:, torch.cat(which)] * torch.cat(freq)
    return phi.cos(), phi.sin(), torch.cat(first), torch.cat(second)


def _norm_turn(x, gain, cs, sn, first, second):
    x = x.to(cs.dtype)
    if gain is not None:
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * gain.to(x.dtype)
    a, b = x[..., first], x[..., second]
    cs, sn = cs[:, None], sn[:, None]
    y = torch.empty_like(x)
    y[..., first] = a * cs - b * sn
    y[..., second] = a * sn + b * cs
    return y


def _plain_append(s):
    c, cu = s["case"], s["cu_q"].long()
    cs, sn, first, second = _turn(s["axis"], c["pairing"], s["pos"])
    cs, sn = cs.float(), sn.float()
    rows = torch.arange(s["T"], device=DEV)
    b = torch.searchsorted(cu[1:].contiguous(), rows, right=True)
    at = s["kv_len"].long()[b] - (cu[b + 1] - cu[b]) + rows - cu[b]
    page, off = s["table"].long()[b, at // c["page"]], at % c["page"]
    s["k_cache"][page, :, off] = _norm_turn(s["k"], s["k_gain"], cs, sn, first, second).to(torch.bfloat16)
    s["v_cache"][page, :, off] = s["v"]
    q = _norm_turn(s["q"], s["q_gain"], cs, sn, first, second).to(torch.bfloat16)
    return {"q": q, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _plain_attention(s):
    c = s["case"]
    H, Hkv, B, Q, n = c["H"], c["Hkv"], c["B"], c["q_max"], s["per"] * c["page"]
    G, cu, kv_len = H // Hkv, s["cu_q"].long(), s["kv_len"].long()
    q_len = cu[1:] - cu[:-1]
    i = torch.arange(Q, device=DEV)
    rows = (cu[:-1, None] + i).clamp(max=s["T"] - 1)                       # [B, Q]
    q = s["q"].float()[rows] * DH ** -0.5                                  # [B, Q, H, 128]
    q = q.view(B, Q, Hkv, G, DH).permute(0, 2, 1, 3, 4).reshape(B, Hkv, Q * G, DH)
    table = s["table"].long()

    def keys(cache):  # [B, Hkv, n, 128]
        return cache[table].float().permute(0, 2, 1, 3, 4).reshape(B, Hkv, n, DH)

    z = q @ keys(s["k_cache"]).transpose(-1, -2)                           # [B, Hkv, Q*G, n]
    j = torch.arange(n, device=DEV)
    limit = kv_len[:, None].expand(B, Q)
    if c["causal"]:
        limit = torch.minimum(limit, (kv_len - q_len)[:, None] + i + 1)
    limit = limit.repeat_interleave(G, 1)[:, None, :, None]
    z = z.masked_fill_(j >= limit, -math.inf)
    if c["prefix"]:
        m = s["prefix_pages"].long()

        def shared(cache):  # [Hkv, prefix, 128]
            return cache[m].float().permute(1, 0, 2, 3).reshape(Hkv, -1, DH)[:, :c["prefix"]]

        def stack(x):  # the rows of all sequences over the shared keys: [Hkv, B*Q*G, ...]
            return x.transpose(0, 1).reshape(Hkv, B * Q * G, -1)

        def unstack(x):
            return x.view(Hkv, B, Q * G, -1).transpose(0, 1)

        z = torch.cat([unstack(stack(q) @ shared(s["k_cache"]).transpose(-1, -2)), z], -1)
    top = z.amax(-1, keepdim=True)
    p = z.sub_(torch.where(top == -math.inf, 0.0, top)).exp_()
    total = p.sum(-1, keepdim=True)
    o = p[..., c["prefix"]:] @ keys(s["v_cache"])
    if c["prefix"]:
        o = o + unstack(stack(p[..., :c["prefix"]]) @ shared(s["v_cache"]))
    o = torch.where(total > 0, o / total, 0.0)
    o = o.view(B, Hkv, Q, G, DH).permute(0, 2, 1, 3, 4).reshape(B, Q, H, DH)
    r = torch.arange(s["T"], device=DEV)
    b = torch.searchsorted(cu[1:].contiguous(), r, right=True)
    return {"o": o[b, r - cu[b]].to(torch.bfloat16)}


def _handles(s):
    """What a serving program keeps of its cache, its batch and its scratch memory."""
    from dit_transformer_block_gb300 import h3
    c = s["case"]
    s["cache"] = h3.kv_cache(s["k_cache"], s["v_cache"])
    s["batch"] = h3.kv_batch(s["cu_q"], s["kv_len"], s["table"], s["T"])
    if c["op"] != "append":
        s["scratch"] = torch.empty(h3.attention_paged_workspace_bytes(s["T"], c["H"], c["prefix"]),
                                   dtype=torch.uint8, device=DEV)
    s["h3"] = h3


def run(s):
    op = s["case"]["op"]
    if not own:
        return _plain_append(s) if op == "append" else _plain_attention(s)
    if "h3" not in s:
        _handles(s)
    h3 = s["h3"]
    if op == "append":
        h3.kv_append_paged(s["q"], s["k"], s["v"], s["q_out"], s["cache"], s["batch"], s["pos"], s["axis"],
                           s["q_gain"], s["k_gain"], theta=THETA, eps=EPS, pairing=s["case"]["pairing"])
        return {"q": s["q_out"], "k_cache": s["k_cache"], "v_cache": s["v_cache"]}
    if op == "paged":
        h3.attention_paged(s["q"], s["o"], s["cache"], s["batch"], s["scratch"], causal=s["case"]["causal"])
    else:
        h3.attention_paged_prefix(s["q"], s["o"], s["cache"], s["batch"], s["prefix_pages"], s["case"]["prefix"],
                                  s["scratch"], causal=s["case"]["causal"])
    return {"o": s["o"]}


# -------------------------------------------------------------------- exact
def exact(case, seed):
    """The definitions, row by row and sequence by sequence, in 64 bits."""
    s = prepare(case, seed)
    q_len, kv_len = _lengths(case)
    P, H, Hkv = case["page"], case["H"], case["Hkv"]
    if case["op"] == "append":
        pos, T = s["pos"], s["T"]
        out = {"k_cache": s["k_cache"].double(), "v_cache": s["v_cache"].double()}

        def head(x, gain):
            x = x.double()
            if gain is not None:
                x = x / (x.pow(2).sum(-1, keepdim=True) / DH + EPS).sqrt() * gain.double()
            y, o = x.clone(), 0
            for a, d in enumerate(s["axis"]):
                for j in range(d // 2):
                    u, w = (o + j, o + d // 2 + j) if case["pairing"] else (o + 2 * j, o + 2 * j + 1)
                    turn = torch.exp(1j * (pos[:, a, None].double() * THETA ** (-2.0 * j / d)))
                    r = torch.complex(x[..., u], x[..., w]) * turn
                    y[..., u], y[..., w] = r.real, r.imag
                o += d
            return y

        out["q"] = head(s["q"], s["q_gain"])
        k, v, t = head(s["k"], s["k_gain"]), s["v"].double(), 0
        table = s["table"].cpu()
        for b in range(case["B"]):
            done = 0
            while done < q_len[b]:  # the run of rows that falls into one page
                j = kv_len[b] - q_len[b] + done
                n = min(P - j % P, q_len[b] - done)
                page = int(table[b, j // P])
                out["k_cache"][page, :, j % P:j % P + n] = k[t + done:t + done + n].transpose(0, 1)
                out["v_cache"][page, :, j % P:j % P + n] = v[t + done:t + done + n].transpose(0, 1)
                done += n
            t += q_len[b]
        return {"q": out["q"], "k_cache": out["k_cache"], "v_cache": out["v_cache"]}
    o = torch.empty(s["T"], H, DH, dtype=torch.float64, device=DEV)
    t = 0
    for b in range(case["B"]):
        mine = s["table"][b, :-(-kv_len[b] // P)].long()
        for h in range(Hkv):
            k = s["k_cache"][mine, h].reshape(-1, DH)[:kv_len[b]]
            v = s["v_cache"][mine, h].reshape(-1, DH)[:kv_len[b]]
            if case["prefix"]:
                m = s["prefix_pages"].long()
                k = torch.cat([s["k_cache"][m, h].reshape(-1, DH)[:case["prefix"]], k])
                v = torch.cat([s["v_cache"][m, h].reshape(-1, DH)[:case["prefix"]], v])
            k, v = k.double(), v.double()
            for g in range(h * (H // Hkv), (h + 1) * (H // Hkv)):
                z = s["q"][t:t + q_len[b], g].double() @ k.T / math.sqrt(DH)
                if case["causal"]:
                    last = case["prefix"] + kv_len[b] - q_len[b] + torch.arange(q_len[b], device=DEV)
                    z = z.masked_fill(torch.arange(k.shape[0], device=DEV) > last[:, None], -math.inf)
                o[t:t + q_len[b], g] = torch.softmax(z, -1) @ v
        t += q_len[b]
    return {"o": o}
