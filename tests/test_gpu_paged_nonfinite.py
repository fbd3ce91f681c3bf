"""Query rows that are not finite over the paged cache. A softmax over scores
that are NaN, or all infinite, has no value, so such a row gives NaN whatever
kernel takes it and however its keys are split; zeros are for rows without keys
alone. The other rows and heads of the call keep their values, against 64 bits,
within the bound of test_gpu_paged.py."""
import math

import pytest
import torch

import test_gpu_paged as paged

pytestmark = pytest.mark.gpu
dev = "cuda"
CH = 5  # the channel of a query that is infinite

# q_len, kv_len, H, Hkv, page, causal, prefix, keys that a table has room for at least
FORMS = {
    "rows": ([1, 1, 1], [200, 0, 77], 4, 2, 16, False, 0, 0),
    "rows, a cluster each": ([1], [4000], 3, 1, 64, False, 0, 0),
    "rows of a chunk, some without keys": ([300, 5], [40, 7], 4, 2, 16, True, 0, 0),
    "rows, many heads": ([1, 2], [700, 300], 40, 2, 32, False, 0, 0),
    "rows behind a prefix": ([1, 1, 2, 1], [50, 0, 30, 1], 6, 2, 16, True, 300, 0),
    "tiles of a few rows": ([1, 2, 1], [300, 40, 0], 4, 2, 64, False, 0, 12000),
    "tiles of a few rows, split": ([1, 3], [11000, 900], 4, 2, 64, True, 0, 12000),
    "tiles of a few rows, many parts": ([3], [27000], 24, 1, 64, False, 0, 0),
    "tiles": ([40, 1, 30], [400, 200, 10], 6, 2, 32, True, 0, 12000),
    "tiles, split": ([40, 1], [9000, 200], 6, 2, 32, False, 0, 12000),
    "two query tiles, split": ([300, 140], [3500, 100], 6, 3, 64, True, 0, 12000),
    "a prefix, whole": ([1, 4, 30], [70, 0, 200], 6, 2, 16, True, 300, 12000),
    "a prefix, split": ([1, 4, 90], [70, 0, 1200], 6, 2, 16, True, 5000, 12000),
    "a prefix, many parts": ([1, 1], [40, 0], 6, 2, 64, False, 20000, 12000),
    "a prefix, own keys by rows": ([1] * 170, [(i * 37) % 230 for i in range(170)], 4, 2, 16, False,
                                   1500, 0),
}


def seen_keys(q_len, kv_len, causal, prefix):
    """Keys that every row sees."""
    out = []
    for n, kv in zip(q_len, kv_len):
        out += [prefix + (min(max(kv - n + i + 1, 0), kv) if causal else kv) for i in range(n)]
    return torch.tensor(out, device=dev)


@pytest.mark.parametrize("kind", ["nan", "inf", "-inf"])
@pytest.mark.parametrize("form", FORMS)
def test_a_query_that_is_not_finite(h3lib, monkeypatch, form, kind):
    q_len, kv, H, Hkv, page, causal, prefix, least = FORMS[form]
    monkeypatch.setattr(paged, "LEAST_KEYS", least)
    P = paged.Paged(kv, Hkv, page, 3, prefix)
    P.k[..., CH] = P.k[..., CH].abs() + 0.5  # an infinite query has scores of one sign
    cu = paged.cumul(q_len)
    g = paged.gen(103)
    ok = paged.rnd(g, cu[-1], H, paged.DH)
    bad = torch.rand(cu[-1], H, generator=g, device=dev) < 0.3
    bad[0, 0] = bad[-1, -1] = True
    q = ok.clone()
    if kind == "nan":
        q[bad] = float("nan")
    else:
        q[bad] = 0
        q[..., CH][bad] = float(kind)
    o = paged.attend(h3lib, q, P, cu, causal)
    seen = (seen_keys(q_len, kv, causal, prefix) > 0)[:, None]
    assert bool(torch.isnan(o[bad & seen]).all()), "a row that is not finite has another value"
    assert bool((o[bad & ~seen] == 0).all()), "a row without keys"
    ref = paged.ref_attention(ok, P, cu, causal, paged.DH ** -0.5)[0]
    o = torch.where(bad[..., None], ref.to(torch.bfloat16), o)
    paged.check_attention(o, ok, P, cu, causal, paged.DH ** -0.5, f"{form}, {kind}")


@pytest.mark.parametrize("least", [0, 12000])
@pytest.mark.parametrize("kv,q_len,H", [(600, 1, 2), (4000, 3, 2), (4000, 40, 4), (11000, 1, 6)])
def test_a_run_of_keys_whose_scores_are_minus_infinity(h3lib, monkeypatch, kv, q_len, H, least):
    # every score of the first half overflows to -inf: weights of 0, whole parts of
    # them, and the rest as if those keys were not there
    monkeypatch.setattr(paged, "LEAST_KEYS", least)
    P = paged.Paged([kv], 2, 64, 4)
    k, v = (x.to(torch.bfloat16) for x in P.keys(0))
    k[:kv // 2, :, CH], k[kv // 2:, :, CH] = -2.0 ** 70, 0
    P.put(P.table[0], k, v)
    q = paged.rnd(paged.gen(104), q_len, H, paged.DH)
    q[..., CH] = 2.0 ** 70
    o = paged.attend(h3lib, q, P, [0, q_len]).double()
    scale, G = paged.DH ** -0.5, H // 2
    k, v = (x[kv // 2:].double() for x in (k, v))
    qh = q.double().view(q_len, 2, G, paged.DH).clone()
    qh[..., CH] = 0
    p = torch.softmax(torch.einsum("ihgd,jhd->hgij", qh, k) * scale, -1)
    ref, a1 = (torch.einsum("hgij,jhd->ihgd", p, x).reshape(o.shape) for x in (v, v.abs()))
    dz = 2.0 ** -16 * float(torch.einsum("ihgd,jhd->hgij", qh.abs(), k.abs()).amax()) * scale * 1.4427
    e = (paged.U + 2 * math.log(2) * dz + 2.0 ** -20 + 2 * kv * 2.0 ** -23) * a1
    assert bool(((o - ref).abs() <= e + paged.U * (ref.abs() + e)).all())
