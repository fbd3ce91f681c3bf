"""Attention over so many keys that a CTA sums more than 131,072 of them: long
tables over few pages, so that a softmax over the pages' keys, each weighted with
the times that it stands in the table, is the answer in 64 bits.

Tolerances, derived before their first run (u = 2^-8): |o - ref| <= e + u (|ref| + e)
with e = (u + 2 (ln 2) dz + 2^-20 + s) sum p |v| / sum p as in test_gpu_paged.py, but
for s, which does not grow with the keys: an accumulator takes 8 products for each of
1,024 key tiles, each cut off by at most 2^-23 of it (2^-10); its sum as many
additions (2^-13); and at most 512 such runs and 160 CTAs' parts are added (2^-14).
The values have one sign, the worst case of a cut, so the mean relative error over
all outputs is tested too: within s, as the roundings of weights and outputs go both
ways (of 2,000 outputs and more: 5 standard deviations of u / sqrt(12) in the mean
are 2^-13)."""
import math

import pytest
import torch

from test_gpu_paged import DH, U, cumul, gen, i32

pytestmark = pytest.mark.gpu
dev = "cuda"
S = 2.0 ** -10 + 2.0 ** -13 + 2.0 ** -14
PAGES = 16


def run(h3lib, q_len, kv_len, Hkv, G, page=128, causal=False, prefix=0, rising=False, bad=False):
    g = gen(7)
    H, B, T, P = Hkv * G, len(kv_len), sum(q_len), page
    k = torch.randn(PAGES, Hkv, P, DH, generator=g, device=dev)
    if rising:  # the maximum rises from run to run of the keys
        k *= torch.linspace(0.05, 4, PAGES, device=dev)[:, None, None, None]
    k = k.to(torch.bfloat16)
    v = (torch.randn(PAGES, Hkv, P, DH, generator=g, device=dev).abs() + 1).to(torch.bfloat16)
    q = (0.5 * torch.randn(T, H, DH, generator=g, device=dev)).to(torch.bfloat16)

    def pages(n):
        x = torch.randint(0, PAGES, (-(-n // P),), generator=g, device=dev)
        return (x.sort().values if rising else x).to(torch.int32)

    table = torch.zeros(B, -(-max(kv_len) // P), dtype=torch.int32, device=dev)
    for b, n in enumerate(kv_len):
        table[b, :-(-n // P)] = pages(n)
    pre = pages(prefix) if prefix else None
    cu = cumul(q_len)
    ws = torch.full((h3lib.attention_paged_workspace_bytes(T, H, prefix),), 0xFF, dtype=torch.uint8,
                    device=dev)
    if bad:
        q[0, 0] = q[-1, -1] = float("nan")
    o = torch.empty_like(q)
    h3lib.attention_paged_prefix(q, o, h3lib.kv_cache(k, v), h3lib.kv_batch(i32(cu), i32(kv_len), table, T),
                                 pre, prefix, ws, causal=causal)
    h3lib.check_device_error()
    if bad:
        assert bool(torch.isnan(o[0, 0]).all()) and bool(torch.isnan(o[-1, -1]).all())
        q[0, 0] = q[-1, -1] = 0

    def times(tab, n):  # of every key of the pages, among the first n of the table
        c = torch.bincount(tab[:n // P].long(), minlength=PAGES).double()[:, None].repeat(1, P)
        if n % P:
            c[int(tab[n // P]), :n % P] += 1
        return c.view(-1)

    kd, vd = (x.transpose(0, 1).reshape(Hkv, PAGES * P, DH).double() for x in (k, v))
    ref, dz = torch.zeros(T, H, DH, dtype=torch.float64, device=dev), 0.0
    for b in range(B):
        lim = [kv_len[b] - q_len[b] + i + 1 if causal else kv_len[b] for i in range(q_len[b])]
        c = torch.stack([times(table[b], n) + (times(pre, prefix) if prefix else 0) for n in lim])
        qb = q[cu[b]:cu[b + 1]].double().view(-1, Hkv, G, DH)
        for h in range(Hkv):
            z = torch.einsum("igd,jd->gij", qb[:, h], kd[h]) * DH ** -0.5
            w = (z - z.amax(-1, keepdim=True)).exp() * c
            w /= w.sum(-1, keepdim=True)
            ref[cu[b]:cu[b + 1], h * G:(h + 1) * G] = torch.einsum("gij,jd->igd", w, vd[h])
        dz = max(dz, 2.0 ** -16 * float((qb.abs().sum(-1).amax() * kd.abs().amax())) * DH ** -0.5 * 1.4427)
    dz = min(dz, 2.0 ** -12) if not rising else dz
    if bad:
        o[0, 0], o[-1, -1] = ref[0, 0].to(torch.bfloat16), ref[-1, -1].to(torch.bfloat16)
    d = o.double() - ref
    e = (U + 2 * math.log(2) * dz + 2.0 ** -20 + S) * ref  # the values are positive
    worst, mean = float((d.abs() / (e + U * (ref + e))).max()), float((d / ref).mean())
    print(f"q {q_len[:3]} kv {kv_len[:3]} heads {H}/{Hkv} prefix {prefix}: worst {worst:.3g} of the "
          f"bound, mean {mean:+.2e}")
    assert worst <= 1.0 and abs(mean) <= S + 2.0 ** -13


M = 1 << 20


@pytest.mark.parametrize("G", [1, 4, 16])
def test_one_row(h3lib, G):
    # 160 key heads on fewer CTAs: whole items, ends and beginnings of split ones
    run(h3lib, [1], [4 * M], 160, G)


def test_the_longest_table(h3lib):
    run(h3lib, [1], [64 * M], 160, 16)


@pytest.mark.parametrize("G,page", [(1, 128), (12, 64)])
def test_few_heads_over_several_ctas_each(h3lib, G, page):
    # every CTA has one part of more than 131,072 keys of a split item
    run(h3lib, [1], [16 * M + 1000], 38, G, page)


@pytest.mark.parametrize("keys", [131071, 131072, 131073, 131072 + 128, 262144, 262145, 400077])
def test_about_the_length_of_a_run(h3lib, keys):
    # many items of one CTA, one after the other
    run(h3lib, [1, 1, 1, 1], [keys, keys - 1, 130, keys], 160, 2)
    run(h3lib, [3, 40], [keys, keys + 5], 160, 3)


@pytest.mark.parametrize("causal", [False, True])
def test_chunks(h3lib, causal):
    # two query tiles; the second one of four rows
    run(h3lib, [33], [1 * M + 77], 160, 4, causal=causal)
    run(h3lib, [3], [300000], 80, 100, causal=causal)
    run(h3lib, [200, 1], [500000, 270000], 40, 2, causal=causal)


@pytest.mark.parametrize("G", [1, 16])
def test_behind_a_prefix(h3lib, G):
    run(h3lib, [1, 1], [1000, 5], 160, G, prefix=2 * M + 3)
    run(h3lib, [2, 30], [300000, 140000], 160, G, prefix=270000, causal=True)


@pytest.mark.parametrize("G", [1, 16])
def test_a_rising_maximum(h3lib, G):
    run(h3lib, [1, 1], [600000, 150000], 160, G, rising=True)
    run(h3lib, [1, 40], [9, 270000], 160, G, rising=True, prefix=400000)


@pytest.mark.parametrize("G", [1, 16])
def test_a_query_of_nan(h3lib, G):
    run(h3lib, [1, 2], [300000, 400000], 160, G, bad=True)
