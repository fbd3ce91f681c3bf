"""Block-sparse attention: scores of pooled blocks, their selection, and attention over the listed
blocks, against 64-bit forms.

Scores: within (n + 4) 2^-24 + 2^-20 of scale * sum over channels of mean |q| * mean |k|, where n counts
the roundings that a value goes through: at most 40 additions in each mean and 128 in the product; 2^-20
for the means' two TF32 parts (each mean 2^-23 off, the product of the smaller parts, 2^-24, left out) and
for the tensor cores' sums, which are cut off and not rounded (48 of them, 2^-23 each, are below 128 2^-24).
Selection: equal.
Attention, with A the sum of weight times |v|: 2^-8 |o| for the output's own rounding (half a
bf16 step), 2^-8 A for the weights', 2^-10 A for the sums in FP32 and 2^-11 A for the scores (their
FP32 sums of 128 products are off by at most 8 2^-23 sum |q k|, here below 300)."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
dev = "cuda"
SENT = -7.25
QB = 256


def gen(seed):
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    return g


def heads(L, H, g, std=1.0):
    return (torch.randn(L, H, 128, generator=g, device=dev) * std).to(torch.bfloat16)


# ------------------------------------------------------------------- scores
def ref_scores(q, k, kb, scale):
    def means(x, n):
        return torch.stack([p.mean(0) for p in x.split(n)], 1)   # [heads, blocks, 128]
    G = q.shape[1] // k.shape[1]
    q, k = q.double(), k.double()
    s = means(q, QB) @ means(k, kb).repeat_interleave(G, 0).transpose(1, 2) * scale
    m = means(q.abs(), QB) @ means(k.abs(), kb).repeat_interleave(G, 0).transpose(1, 2) * abs(scale)
    return s, m


@pytest.mark.parametrize("kb", [64, 128])
@pytest.mark.parametrize("Lq,Lk,H,Hkv", [(1, 1, 1, 1), (5, 70, 3, 1), (256, 128, 4, 4), (257, 129, 6, 2),
                                         (700, 5000, 5, 5), (1896, 3001, 40, 8), (17000, 900, 2, 1),
                                         (4096, 8200, 3, 1), (4097, 16500, 4, 2), (33000, 300, 2, 2)])
def test_scores(h3lib, Lq, Lk, H, Hkv, kb):
    g = gen(Lq + Lk)
    q, k = heads(Lq, H, g), heads(Lk, Hkv, g) + 0.25
    nq, nk = -(-Lq // QB), -(-Lk // kb)
    out = torch.full((H * nq * nk + 64,), SENT, device=dev)
    scores = out[:H * nq * nk].view(H, nq, nk)
    ws = torch.empty(h3lib.block_scores_workspace_bytes(Lq, Lk, H, Hkv, kb), dtype=torch.uint8, device=dev)
    h3lib.block_scores(q, k, scores, ws, k_block=kb, scale=0.3)
    h3lib.check_device_error()
    ref, mag = ref_scores(q, k, kb, 0.3)
    assert ((scores.double() - ref).abs() <= ((208 + 4) * 2.0 ** -24 + 2.0 ** -20) * mag).all()
    assert (out[H * nq * nk:] == SENT).all()


def test_scores_of_strided_rows_and_a_bad_row(h3lib):
    g = gen(3)
    qkv = heads(600, 12, g)
    q, k = qkv[:, :6], qkv[:, 6:9]
    ws = torch.empty(h3lib.block_scores_workspace_bytes(600, 600, 6, 3, 64), dtype=torch.uint8, device=dev)
    a, b = (torch.empty(6, 3, 10, device=dev) for _ in range(2))
    h3lib.block_scores(q, k, a, ws)
    h3lib.block_scores(q.contiguous(), k.contiguous(), b, ws)
    h3lib.check_device_error()
    assert torch.equal(a, b)
    k[130, 1, 5] = float("nan")    # one block of one key head
    h3lib.block_scores(q, k, b, ws)
    h3lib.check_device_error()
    bad = torch.zeros(6, 3, 10, dtype=torch.bool, device=dev)
    bad[2:4, :, 2] = True
    assert torch.equal(b.isnan(), bad) and torch.equal(b[~bad], a[~bad])


# ---------------------------------------------------------------- selection
def ref_select(s, most, first, last):
    rows, nk = s.shape
    ids = np.full((rows, most), -1, np.int32)
    counts = np.zeros(rows, np.int32)
    for r in range(rows):
        kept = [b for b in range(nk) if b < first or b >= nk - last]
        rest = [b for b in range(nk) if not (b < first or b >= nk - last) and s[r, b] > -np.inf]
        rest.sort(key=lambda b: (-s[r, b], b))
        mine = sorted((kept + rest)[:most])
        ids[r, :len(mine)], counts[r] = mine, len(mine)
    return ids, counts


def check_select(h3lib, s, most, first=0, last=0):
    rows, nk = s.shape
    ids = torch.full((rows * most + 16,), 77, dtype=torch.int32, device=dev)
    counts = torch.full((rows + 16,), 77, dtype=torch.int32, device=dev)
    h3lib.block_select(s.to(dev), ids[:rows * most].view(rows, most), counts[:rows], first, last)
    h3lib.check_device_error()
    want, n = ref_select(s.numpy(), most, first, last)
    assert np.array_equal(counts[:rows].cpu().numpy(), n)
    assert np.array_equal(ids[:rows * most].view(rows, most).cpu().numpy(), want)
    assert (ids[rows * most:] == 77).all() and (counts[rows:] == 77).all()


@pytest.mark.parametrize("nk", [1, 2, 31, 128, 129, 460, 919, 2048, 2049, 4097, 20000])
def test_select(h3lib, nk):
    g = torch.Generator()
    g.manual_seed(nk)
    rows = 12 if nk < 5000 else 4
    for most in sorted({1, 2, max(1, nk // 10), max(1, nk // 2), nk, nk + 3}):
        s = torch.randn(rows, nk, generator=g)
        check_select(h3lib, s, most)
        check_select(h3lib, (s * 4).round() / 4, most)         # many equal scores
        if most > 3:
            check_select(h3lib, s, most, 1, 2)
            check_select(h3lib, (s * 2).round() / 2, most, 2, 0)


def test_select_odd_scores(h3lib):
    inf, nan = float("inf"), float("nan")
    g = torch.Generator()
    g.manual_seed(1)
    s = torch.randn(14, 300, generator=g)
    s[0] = -inf                          # nothing to select
    s[1] = nan
    s[2, ::2] = -inf
    s[3, 5:290] = nan
    s[4] = 0.0
    s[4, ::3] = -0.0                     # equal to +0
    s[5, [7, 200, 299]] = inf
    s[6] = -3.0e38
    s[7] = torch.arange(300) * 1e-45     # subnormal
    s[8] = -torch.arange(300) * 1e-45
    s[9] = 1.0
    s[9, 150] = 1.0 + 2.0 ** -23
    s[10] = torch.arange(300) % 2 * 2.0 - 1
    s[11, :] = -3.4028234663852886e38
    s[12, 3:] = -inf
    for most, first, last in ((1, 0, 0), (40, 0, 0), (40, 2, 3), (150, 0, 1), (300, 0, 0), (301, 300, 1),
                              (5, 5, 0), (299, 1, 1)):
        check_select(h3lib, s, most, first, last)


# ---------------------------------------------------------------- attention
def ref_attention(q, k, v, ids, counts, kb, scale):
    """(o, A): the output and the weighted sum of |v|, [Lq, H, 128] in 64 bits."""
    Lq, H, _ = q.shape
    Lk, Hkv, _ = k.shape
    nk = -(-Lk // kb)
    o = torch.zeros(Lq, H, 128, dtype=torch.float64, device=dev)
    mag = torch.zeros_like(o)
    lists, n = ids.cpu().tolist(), counts.cpu().tolist()
    for h in range(H):
        kk, vv = k[:, h // (H // Hkv)].double(), v[:, h // (H // Hkv)].double()
        for t in range(-(-Lq // QB)):
            mine = [b for b in lists[h][t][:max(0, n[h][t])] if 0 <= b < nk]
            at = [j for b in mine for j in range(b * kb, min(Lk, b * kb + kb))]
            if not at:
                continue
            at = torch.tensor(at, device=dev)
            p = torch.softmax(q[t * QB:(t + 1) * QB, h].double() @ kk[at].T * scale, -1)
            o[t * QB:(t + 1) * QB, h] = p @ vv[at]
            mag[t * QB:(t + 1) * QB, h] = p @ vv[at].abs()
    return o, mag


def lists(H, nq, nk, most, g, ragged=True):
    ids = torch.rand(H, nq, nk, generator=g, device=dev).argsort(-1)[..., :most].sort(-1).values
    if ids.shape[-1] < most:
        ids = torch.nn.functional.pad(ids, (0, most - ids.shape[-1]), value=-1)
    n = torch.full((H, nq), min(most, nk), device=dev)
    if ragged:
        n = torch.randint(0, min(most, nk) + 1, (H, nq), generator=g, device=dev)
    return ids.to(torch.int32).contiguous(), n.to(torch.int32)


def check_attention(h3lib, q, k, v, ids, counts, kb, scale=None, o=None):
    if o is None:
        o = torch.full((q.shape[0], q.shape[1], 128), SENT, dtype=torch.bfloat16, device=dev)
    h3lib.attention_blocks(q, k, v, o, ids, counts, k_block=kb, scale=scale)
    h3lib.check_device_error()
    ref, mag = ref_attention(q, k, v, ids, counts, kb, 128 ** -0.5 if scale is None else scale)
    err = (o.double() - ref).abs()
    bound = 2.0 ** -8 * ref.abs() + (2.0 ** -8 + 2.0 ** -10 + 2.0 ** -11) * mag
    assert (err <= bound).all(), float((err / (bound + 1e-300)).max())
    return o


@pytest.mark.parametrize("kb", [64, 128])
@pytest.mark.parametrize("Lq,Lk,H,Hkv,most", [
    (1, 1, 1, 1, 1), (1, 300, 2, 1, 3), (22, 2000, 4, 4, 9), (22, 9000, 8, 2, 64), (128, 640, 3, 3, 4),
    (129, 700, 3, 1, 7), (256, 256, 2, 2, 2), (257, 1000, 4, 2, 5), (600, 600, 5, 5, 10),
    (1500, 3333, 12, 4, 20), (3000, 1024, 24, 8, 6), (1, 20000, 1, 1, 300), (700, 8000, 1, 1, 60)])
def test_attention(h3lib, Lq, Lk, H, Hkv, most, kb):
    g = gen(Lq + Lk)
    q, k, v = heads(Lq, H, g), heads(Lk, Hkv, g), heads(Lk, Hkv, g)
    nq, nk = -(-Lq // QB), -(-Lk // kb)
    for ragged in (False, True):
        ids, n = lists(H, nq, nk, most, g, ragged)
        check_attention(h3lib, q, k, v, ids, n, kb)


@pytest.mark.parametrize("kb", [64, 128])
@pytest.mark.parametrize("Lq,Lk,H,Hkv,most", [
    (768, 900, 51, 17, 7), (2000, 1500, 20, 4, 9), (1793, 2500, 20, 20, 24), (256, 3000, 160, 32, 41),
    (200, 700, 155, 5, 5), (256, 64, 153, 1, 1), (2048, 5000, 19, 19, 70)])
def test_attention_of_many_items(h3lib, Lq, Lk, H, Hkv, most, kb):
    # two (query block, head)s to a pair of CTAs: an odd number of them, lists of unequal length, some
    # of them empty, the second half of a block's rows missing
    g = gen(Lq + Lk + H)
    q, k, v = heads(Lq, H, g), heads(Lk, Hkv, g), heads(Lk, Hkv, g)
    nq, nk = -(-Lq // QB), -(-Lk // kb)
    assert nq * H >= 152
    for ragged in (False, True):
        ids, n = lists(H, nq, nk, most, g, ragged)
        if ragged:
            n.view(-1)[::7] = 0
            n.view(-1)[1::14] = 0
            n.view(-1)[-1] = 1 << 30
            ids.view(-1, most)[3::5, 0] = nk
            ids.view(-1, most)[4::9] = -1
            ids.view(-1, most)[5::9] = nk - 1
        buf = torch.full((Lq + 2, H, 128), SENT, dtype=torch.bfloat16, device=dev)
        check_attention(h3lib, q, k, v, ids, n.clamp(max=most) if not ragged else n, kb, o=buf[1:-1])
        assert (buf[0] == SENT).all() and (buf[-1] == SENT).all()


def test_many_items_hold_anything_where_they_do_not_look(h3lib):
    g = gen(77)
    Lq, Lk, H, kb = 1000, 1030, 40, 64
    q, k, v = heads(Lq, H, g), heads(Lk, H, g), heads(Lk, H, g)
    ids, n = lists(H, 4, 17, 6, g, True)
    ids %= 10                                   # blocks 10 and on are in no list
    want = check_attention(h3lib, q, k, v, ids, n, kb)
    k2, v2 = k.clone(), v.clone()
    k2[640:], v2[640:] = float("nan"), float("inf")
    o = torch.empty_like(want)
    h3lib.attention_blocks(q, k2, v2, o, ids, n, k_block=kb)
    h3lib.check_device_error()
    assert torch.equal(o, want)
    k2[5] = float("nan")                         # a key of block 0: NaN where it is listed
    h3lib.attention_blocks(q, k2, v2, o, ids, n, k_block=kb)
    h3lib.check_device_error()
    for h in range(H):
        for t in range(4):
            bad = 0 in ids[h, t, :int(n[h, t])].tolist()
            rows = o[t * QB:(t + 1) * QB, h]
            assert torch.isnan(rows).all() if bad else torch.equal(rows, want[t * QB:(t + 1) * QB, h])


@pytest.mark.parametrize("kb", [64, 128])
def test_lists_of_any_content(h3lib, kb):
    g = gen(5)
    for Lq, Lk, most in ((300, 1000, 12), (22, 4000, 40)):
        q, k, v = heads(Lq, 4, g), heads(Lk, 4, g), heads(Lk, 4, g)
        nq, nk = -(-Lq // QB), -(-Lk // kb)
        ids, n = lists(4, nq, nk, most, g, False)
        ids[0, 0, :5] = torch.tensor([-1, nk, 1 << 30, -(1 << 31), nk + 7], device=dev)
        ids[1] = ids[1].flip(-1)                      # any order
        ids[2, 0, :] = nk - 1                         # the short last block, many times over
        ids[3, 0] = -1                                # nothing but ids outside
        o = check_attention(h3lib, q, k, v, ids, n, kb)
        assert (o[:QB, 3] == 0).all()
        n[0, 0], n[1, 0], n[2, 0] = -7, 1 << 30, 0    # counts are taken as 0 .. most
        n[3, 0] = 1
        o = check_attention(h3lib, q, k, v, ids, n.clamp(max=1 << 20), kb)
        assert (o[:QB, 0] == 0).all() and (o[:QB, 2] == 0).all()


def test_unlisted_and_masked_keys_may_hold_anything(h3lib):
    g = gen(6)
    Lq, Lk, kb = 300, 1000, 64
    q, k, v = heads(Lq, 2, g), heads(Lk, 2, g), heads(Lk, 2, g)
    ids = torch.tensor([1, 4, 15], dtype=torch.int32, device=dev).expand(2, 2, 3).contiguous()
    n = torch.full((2, 2), 3, dtype=torch.int32, device=dev)
    want = check_attention(h3lib, q, k, v, ids, n, kb)
    big_k, big_v = (torch.full((1400, 2, 128), float("nan"), dtype=torch.bfloat16, device=dev) for _ in range(2))
    for b in (1, 4, 15):
        at = slice(b * kb, min(Lk, b * kb + kb))
        big_k[at], big_v[at] = k[at], v[at]
    o = torch.empty_like(want)
    h3lib.attention_blocks(q, big_k[:Lk], big_v[:Lk], o, ids, n, k_block=kb)
    h3lib.check_device_error()
    assert torch.equal(o, want)


@pytest.mark.parametrize("Lq,most", [(300, 4), (20, 16)])
def test_rows_without_a_value(h3lib, Lq, most):
    g = gen(7)
    Lk, kb = 1024, 64
    q, k, v = heads(Lq, 1, g), heads(Lk, 1, g), heads(Lk, 1, g)
    ids, n = lists(1, -(-Lq // QB), 16, most, g, False)
    inf = float("inf")
    q[3, 0, 0] = float("nan")
    q[5] = 0
    q[5, 0, 1] = inf               # scores of +-inf by the sign of a key's channel 1
    q[7] = 0
    q[7, 0, 2] = inf
    k[:, 0, 2] = -k[:, 0, 2].abs() - 0.5   # all -inf for row 7
    o = torch.empty_like(q)
    h3lib.attention_blocks(q, k, v, o, ids, n, k_block=kb)
    h3lib.check_device_error()
    bad = torch.zeros(Lq, dtype=torch.bool, device=dev)
    bad[[3, 5, 7]] = True
    assert torch.equal(o[:, 0].isnan().all(1), bad) and torch.equal(o[:, 0].isnan().any(1), bad)


def test_large_scores_and_far_blocks(h3lib):
    # the running maximum rises by far more than the rescaling threshold, and falls
    g = gen(8)
    q, k, v = heads(260, 2, g, 3.0), heads(2048, 2, g, 1.0), heads(2048, 2, g)
    k *= torch.linspace(0.1, 3.0, 2048, device=dev).view(-1, 1, 1).to(torch.bfloat16)
    ids, n = lists(2, 2, 32, 20, g, False)
    check_attention(h3lib, q, k, v, ids, n, 64, scale=0.2)
    check_attention(h3lib, q, k, v, ids.flip(-1).contiguous(), n, 64, scale=0.2)


def test_the_longest_lists(h3lib):
    # 2^17 keys in one accumulator, of values of one sign: the tensor cores' sums come out low, by
    # little over 2^-11; the weights are all 1 and their sum exact
    g = gen(13)
    Lk = 1 << 17
    q = torch.zeros(200, 2, 128, dtype=torch.bfloat16, device=dev)
    k, v = heads(Lk, 1, g), torch.full((Lk, 1, 128), 1.0, dtype=torch.bfloat16, device=dev)
    v[:, :, 64:] += torch.rand(Lk, 1, 64, generator=g, device=dev).to(torch.bfloat16)
    for kb in (64, 128):
        most = Lk // kb
        ids = torch.arange(most, dtype=torch.int32, device=dev).expand(2, 1, most).contiguous()
        n = torch.full((2, 1), most, dtype=torch.int32, device=dev)
        o = torch.empty_like(q)
        h3lib.attention_blocks(q, k, v, o, ids, n, k_block=kb)
        h3lib.check_device_error()
        ref = v.double().mean(0)
        assert ((o.double() - ref).abs() <= (2.0 ** -8 + 2.0 ** -10) * ref).all()


def test_strided_rows_of_one_buffer(h3lib):
    g = gen(9)
    qkv = heads(700, 12, g)
    q, k, v = qkv[:, :6], qkv[:, 6:9], qkv[:, 9:]
    ids, n = lists(6, 3, 11, 5, g)
    wide = torch.full((700, 10, 128), SENT, dtype=torch.bfloat16, device=dev)
    check_attention(h3lib, q, k, v, ids, n, 64, o=wide[:, 2:8])
    assert (wide[:, :2] == SENT).all() and (wide[:, 8:] == SENT).all()


def test_all_blocks_are_dense_attention(h3lib):
    g = gen(10)
    L, H = 1100, 3
    q, k, v = heads(L, H, g), heads(L, H, g), heads(L, H, g)
    ids = torch.arange(18, dtype=torch.int32, device=dev).expand(H, 5, 18).contiguous()
    n = torch.full((H, 5), 18, dtype=torch.int32, device=dev)
    o = check_attention(h3lib, q, k, v, ids, n, 64)
    dense = torch.empty_like(o)
    h3lib.attention_varlen(q, k, v, dense)
    h3lib.check_device_error()
    assert ((o.float() - dense.float()).abs() <= 2 * 2.0 ** -8 * (dense.float().abs() + 0.5)).all()


def test_no_keys_at_all_and_bounds(h3lib):
    g = gen(11)
    q = heads(300, 2, g)
    k = torch.empty(0, 2, 128, dtype=torch.bfloat16, device=dev)
    ids, n = torch.zeros(2, 2, 3, dtype=torch.int32, device=dev), torch.ones(2, 2, dtype=torch.int32, device=dev)
    wide = torch.full((302, 4, 128), SENT, dtype=torch.bfloat16, device=dev)
    h3lib.attention_blocks(q, k, k, wide[1:301, 1:3], ids, n)
    h3lib.check_device_error()
    assert (wide[1:301, 1:3] == 0).all()
    wide[1:301, 1:3] = SENT
    assert (wide == SENT).all()
    k = heads(130, 2, g)
    for rows in (1, 127, 128, 200, 256, 299):   # rows beyond are left alone
        wide.fill_(SENT)
        nq = -(-rows // QB)
        h3lib.attention_blocks(q[:rows], k, k, wide[1:rows + 1, 1:3], ids[:, :nq].contiguous(),
                               n[:, :nq].contiguous())
        h3lib.check_device_error()
        assert (wide[1:rows + 1, 1:3] != SENT).any(-1).all()
        wide[1:rows + 1, 1:3] = SENT
        assert (wide == SENT).all()


def test_full_size(h3lib):
    g = gen(12)
    L, H, kb, most = 58758, 42, 64, 92
    q, k, v = heads(L, H, g), heads(L, H, g), heads(L, H, g)
    nq, nk = 230, 919
    ids = torch.empty(H, nq, most, dtype=torch.int32, device=dev)
    for h in range(H):
        ids[h] = torch.rand(nq, nk, generator=g, device=dev).topk(most, -1).indices.sort(-1).values
    n = torch.full((H, nq), most, dtype=torch.int32, device=dev)
    o = torch.empty_like(q)
    h3lib.attention_blocks(q, k, v, o, ids, n, k_block=kb)
    h3lib.check_device_error()
    for h, t in ((0, 0), (41, 229), (17, 100), (3, 228), (30, 7)):
        rows = slice(t * QB, min(L, t * QB + QB))
        ref, mag = ref_attention(q[rows, h:h + 1], k[:, h:h + 1], v[:, h:h + 1], ids[h:h + 1, t:t + 1],
                                 n[h:h + 1, t:t + 1], kb, 128 ** -0.5)
        err = (o[rows, h:h + 1].double() - ref).abs()
        assert (err <= 2.0 ** -8 * ref.abs() + (2.0 ** -8 + 2.0 ** -10 + 2.0 ** -11) * mag).all(), (h, t)


def test_choose_and_attend_in_a_graph(h3lib):
    """Scores, selection and attention as one captured run, on two inputs in turn, equal to the calls
    made one by one; the blocks chosen are those of the scores that came out."""
    Lq = Lk = 3000
    H, Hkv, kb, most = 8, 4, 64, 9
    ins = []
    for seed in (1, 2):
        g = gen(seed)
        ins.append([heads(Lq, H, g), heads(Lk, Hkv, g), heads(Lk, Hkv, g)])
    nq, nk = -(-Lq // QB), -(-Lk // kb)

    def buffers():
        return (torch.empty(H, nq, nk, device=dev),
                torch.empty(h3lib.block_scores_workspace_bytes(Lq, Lk, H, Hkv, kb), dtype=torch.uint8, device=dev),
                torch.empty(H, nq, most, dtype=torch.int32, device=dev),
                torch.empty(H, nq, dtype=torch.int32, device=dev),
                torch.empty(Lq, H, 128, dtype=torch.bfloat16, device=dev))

    def run(q, k, v, b):
        h3lib.block_scores(q, k, b[0], b[1], k_block=kb)
        h3lib.block_select(b[0], b[2], b[3], keep_first=1, keep_last=1)
        h3lib.attention_blocks(q, k, v, b[4], b[2], b[3], k_block=kb)

    want = []
    for q, k, v in ins:
        b = buffers()
        run(q, k, v, b)
        h3lib.check_device_error()
        s, m = ref_scores(q, k, kb, 128 ** -0.5)
        assert ((b[0].double() - s).abs() <= 212 * 2.0 ** -24 * m).all()
        ids, counts = ref_select(b[0].view(-1, nk).cpu().numpy(), most, 1, 1)
        assert np.array_equal(b[2].view(-1, most).cpu().numpy(), ids)
        ref, mag = ref_attention(q, k, v, b[2], b[3], kb, 128 ** -0.5)
        assert ((b[4].double() - ref).abs() <= 2.0 ** -8 * ref.abs() + 0.0054 * mag).all()
        want.append(b)
    live = [t.clone() for t in ins[0]]
    b = buffers()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run(*live, b)
    for i in (1, 0, 1):
        for a, t in zip(live, ins[i]):
            a.copy_(t)
        graph.replay()
        torch.cuda.synchronize()
        for x, y in zip((b[0], b[2], b[3], b[4]), (want[i][j] for j in (0, 2, 3, 4))):
            assert torch.equal(x, y)
