"""The paged key/value cache calls against plain 64-bit implementations:
appending rows (with Q/K RMSNorm and RoPE) and attention over the cache, with
and without a shared prefix, over lengths from none to several tiles, ragged
batches, page and head layouts, strides, masked rows, garbage in every place
that no row may see, streams and captured graphs.

Tolerances, derived before their first run. u = 2^-8 is a bf16 rounding.
Append: y = a cos - b sin in FP32 from exact bf16 inputs. The norm (a sum of
128 squares in a tree, rsqrt, two products) and the rotation take under 32
FP32 roundings, the angle one rounding of a half turn (pi 2^-24) and sincospif
a few ulp: |dy| <= 2^-18 (|a| + |b|), then one bf16 rounding.
Attention, per element: |o - ref| <= e + u (|ref| + e),
  e = (u + 2 (ln 2) dz + 2^-20 + 2 L 2^-23) sum p |v| / sum p
(u: the weights rounded to bf16; dz = 2^-16 max|q.k|_1 scale log2 e: a score is
an FP32 sum of 128 products; 2^-20: exp2; the sums over L keys, each addition
within 2^-23). In the mean, over inputs of random sign: the two bf16 roundings
are independent and uniform within half a step, so the relative L2 error is at
most u sqrt(2 / 3), and the other terms do not add to u: rel-L2 <= u."""
import math
import random

import pytest
import torch

pytestmark = pytest.mark.gpu
dev = "cuda"
U = 2.0 ** -8
DH = 128
SENT = -7.25
LEAST_KEYS = 0  # that a page table has room for: the choice of kernel goes by it


def gen(seed):
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    return g


def rnd(g, *shape, std=1.0):
    return (torch.randn(*shape, generator=g, device=dev) * std).to(torch.bfloat16)


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=dev)


class Paged:
    """A pool whose unused places hold NaN and infinities, and the pages of
    sequences of the given lengths in a shuffled order."""

    def __init__(self, kv_len, Hkv, page, seed=0, prefix=0, spare=2, fill=True, k_std=1.0):
        g = gen(seed)
        self.page, self.Hkv, self.kv = page, Hkv, list(kv_len)
        need = [max(1, -(-n // page)) for n in kv_len]
        npre = -(-prefix // page)
        self.pages = sum(need) + npre + spare
        self.k = torch.full((self.pages, Hkv, page, DH), float("nan"), device=dev).to(torch.bfloat16)
        self.v = torch.full((self.pages, Hkv, page, DH), float("inf"), device=dev).to(torch.bfloat16)
        self.v[..., ::2] = float("nan")
        order = torch.randperm(self.pages, generator=g, device=dev).to(torch.int32)
        self.table = torch.full((len(kv_len), max(need + [1, -(-LEAST_KEYS // page)])), -1,
                                dtype=torch.int32, device=dev)
        at = npre
        for b, n in enumerate(need):
            self.table[b, :n] = order[at:at + n]
            at += n
        self.prefix, self.prefix_pages = prefix, order[:npre].contiguous()
        if fill:
            for b, n in enumerate(kv_len):
                self.put(self.table[b], rnd(g, n, Hkv, DH, std=k_std), rnd(g, n, Hkv, DH))
            if prefix:
                self.put(self.prefix_pages, rnd(g, prefix, Hkv, DH, std=k_std),
                         rnd(g, prefix, Hkv, DH))

    def rows(self, pages, n):
        j = torch.arange(n, device=dev)
        return pages.long()[j // self.page], j % self.page

    def put(self, pages, k, v):
        p, o = self.rows(pages, k.shape[0])
        self.k[p, :, o] = k
        self.v[p, :, o] = v

    def keys(self, b):
        """k, v [n, Hkv, 128] in 64 bits: the prefix, then sequence b's own."""
        out = []
        for c in (self.k, self.v):
            parts = []
            for pages, n in ((self.prefix_pages, self.prefix), (self.table[b], self.kv[b])):
                p, o = self.rows(pages, n)
                parts.append(c[p, :, o].double())
            out.append(torch.cat(parts))
        return out

    def batch(self, h3, cu, T):
        return h3.kv_batch(i32(cu), i32(self.kv), self.table, T)


def ref_attention(q, P, cu, causal, scale):
    """(o, sum p |v| / sum p, max |q| . |k|) per row and head in 64 bits."""
    o = torch.zeros(q.shape, dtype=torch.float64, device=dev)
    a1 = torch.zeros_like(o)
    zmax = 0.0
    for b in range(len(cu) - 1):
        n = cu[b + 1] - cu[b]
        if n == 0:
            continue
        k, v = P.keys(b)
        G = q.shape[1] // P.Hkv
        qb = q[cu[b]:cu[b + 1]].double().view(n, P.Hkv, G, DH)
        z = torch.einsum("ihgd,jhd->hgij", qb, k) * scale
        if k.shape[0]:
            zmax = max(zmax, float(torch.einsum("ihgd,jhd->hgij", qb.abs(), k.abs()).amax()))
        if causal:
            j = torch.arange(k.shape[0], device=dev) - P.prefix
            i = torch.arange(n, device=dev)
            # the prefix's keys (j < 0) are seen by every row
            z = z.masked_fill((j[None, :] > (P.kv[b] - n + i)[:, None]) & (j >= 0), -math.inf)
        if k.shape[0] == 0:
            continue
        top = z.amax(-1, keepdim=True)
        p = (z - torch.where(top == -math.inf, 0.0, top)).exp()
        w = p.sum(-1, keepdim=True)
        p = torch.where(w > 0, p / w, 0.0)
        o[cu[b]:cu[b + 1]] = torch.einsum("hgij,jhd->ihgd", p, v).reshape(n, -1, DH)
        a1[cu[b]:cu[b + 1]] = torch.einsum("hgij,jhd->ihgd", p, v.abs()).reshape(n, -1, DH)
    return o, a1, zmax


def check_attention(o, q, P, cu, causal, scale, what=""):
    ref, a1, zmax = ref_attention(q, P, cu, causal, scale)
    rows = slice(cu[0], cu[-1])
    x, ref, a1 = o[rows].double(), ref[rows], a1[rows]
    L = P.prefix + max(P.kv + [0])
    dz = 2.0 ** -16 * zmax * scale * 1.4427
    e = (U + 2 * math.log(2) * dz + 2.0 ** -20 + 2 * L * 2.0 ** -23) * a1
    assert bool(torch.isfinite(x).all()), f"{what}: non-finite output"
    worst = float(((x - ref).abs() / (e + U * (ref.abs() + e) + 1e-30)).max()) if x.numel() else 0.0
    n = float(ref.norm())
    rel = float((x - ref).norm()) / n if n else float((x - ref).norm())
    print(f"{what}: worst {worst:.3g} of the bound, rel-L2 {rel:.3g}")
    assert worst <= 1.0 and rel <= U, f"{what}: worst {worst:.3g} of the bound, rel-L2 {rel:.3g}"


def attend(h3lib, q, P, cu, causal=False, scale=None, o=None, ws=None, stream=None, T=None):
    T = q.shape[0] if T is None else T
    o = torch.full(q.shape, SENT, dtype=torch.bfloat16, device=dev) if o is None else o
    need = h3lib.attention_paged_workspace_bytes(T, q.shape[1], P.prefix)
    if ws is None:
        ws = torch.full((need,), 0xFF, dtype=torch.uint8, device=dev)  # NaN floats
    c, b = h3lib.kv_cache(P.k, P.v), P.batch(h3lib, cu, T)
    if P.prefix:
        h3lib.attention_paged_prefix(q, o, c, b, P.prefix_pages, P.prefix, ws, scale, causal,
                                     stream=stream)
    else:
        h3lib.attention_paged(q, o, c, b, ws, scale, causal, stream=stream)
    h3lib.check_device_error(stream)
    return o


def cumul(lens, first=0):
    out = [first]
    for n in lens:
        out.append(out[-1] + n)
    return out


def run_attention(h3lib, q_len, kv_len, H, Hkv, page, causal=False, prefix=0, seed=1, first=0,
                  behind=0, std=1.0):
    P = Paged(kv_len, Hkv, page, seed, prefix)
    cu = cumul(q_len, first)
    T = cu[-1] + behind
    q = torch.full((T, H, DH), float("nan"), dtype=torch.bfloat16, device=dev)
    q[cu[0]:cu[-1]] = rnd(gen(seed + 100), cu[-1] - cu[0], H, DH, std=std)
    o = attend(h3lib, q, P, cu, causal)
    check_attention(o, q, P, cu, causal, DH ** -0.5,
                    f"q {q_len[:5]} kv {kv_len[:5]} H {H}/{Hkv} page {page} prefix {prefix}")
    assert bool((o[:cu[0]] == SENT).all()) and bool((o[cu[-1]:] == SENT).all()), "other rows written"


# ------------------------------------------------------------- attention
@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("kv", [1, 15, 16, 17, 127, 128, 129, 250, 1000])
def test_single_row(h3lib, kv, page):
    run_attention(h3lib, [1], [kv], 4, 4, page)


@pytest.mark.parametrize("H,Hkv", [(1, 1), (4, 4), (3, 1), (14, 2), (24, 3), (40, 8), (128, 1),
                                   (42, 42), (100, 1), (254, 2)])
def test_head_groups(h3lib, H, Hkv):
    run_attention(h3lib, [1, 1, 1], [300, 77, 513], H, Hkv, 64)
    run_attention(h3lib, [5, 1, 37], [300, 77, 513], H, Hkv, 32, causal=True)


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("q,kv", [
    ([127], [127]), ([128], [128]), ([129], [129]), ([255], [400]), ([256], [256]), ([257], [257]),
    ([600], [1000]), ([513, 1, 2], [513, 900, 130]), ([1, 300, 1, 300], [2000, 300, 5, 700]),
])
def test_chunks(h3lib, q, kv, causal):
    run_attention(h3lib, q, kv, 3, 3, 64, causal)
    run_attention(h3lib, q, kv, 6, 2, 16, causal, seed=2)


def test_ragged_decode_batch(h3lib):
    lens = [1 + (i * 977) % 1500 for i in range(150)]
    run_attention(h3lib, [1] * 150, lens, 8, 2, 16)
    run_attention(h3lib, [1] * 150, lens, 5, 5, 128)


def test_many_sequences_of_one_key(h3lib):
    run_attention(h3lib, [1] * 700, [1] * 700, 2, 2, 16)


def test_no_wait_runs_out_at_the_end_of_a_call(h3lib):
    # many key tiles per SM: a wait for copies that have long landed would show
    # as its 2 s limit
    P = Paged([20000, 7000, 12345], 8, 16, k_std=1.0)
    q = rnd(gen(40), 3, 8, DH)
    attend(h3lib, q, P, [0, 1, 2, 3])
    e = [torch.cuda.Event(enable_timing=True) for _ in range(2)]
    e[0].record()
    attend(h3lib, q, P, [0, 1, 2, 3])
    e[1].record()
    torch.cuda.synchronize()
    assert e[0].elapsed_time(e[1]) < 500


def test_empty_sequences_and_masked_rows(h3lib):
    # sequences without rows, without keys, with more rows than keys (causal:
    # the first rows see nothing and give zeros)
    run_attention(h3lib, [0, 3, 0, 1, 0], [50, 0, 0, 60, 0], 4, 2, 16)
    run_attention(h3lib, [0, 0], [5, 9], 4, 2, 16)
    for page in (16, 128):
        run_attention(h3lib, [300, 5, 4], [40, 0, 200], 4, 2, page, causal=True)
        run_attention(h3lib, [300, 5, 4], [40, 0, 200], 4, 2, page, causal=True, prefix=130)
    P = Paged([0], 2, 16)
    o = attend(h3lib, rnd(gen(1), 3, 4, DH), P, [0, 3])
    assert bool((o == 0).all())


def test_rows_before_and_behind_are_left_alone(h3lib):
    run_attention(h3lib, [3, 140, 1], [30, 140, 700], 6, 2, 64, first=5, behind=9)
    run_attention(h3lib, [3, 140, 1], [30, 140, 700], 6, 2, 64, first=5, behind=9, prefix=200,
                  causal=True)


@pytest.mark.parametrize("prefix", [1, 16, 127, 128, 129, 1000, 5000])
def test_prefix_single_rows(h3lib, prefix):
    run_attention(h3lib, [1] * 20, [(i * 37) % 300 for i in range(20)], 4, 4, 64, prefix=prefix)
    run_attention(h3lib, [1] * 50, [(i * 7) % 100 for i in range(50)], 16, 2, 16, prefix=prefix)


@pytest.mark.parametrize("causal", [False, True])
def test_prefix_chunks(h3lib, causal):
    run_attention(h3lib, [70, 1, 0, 200, 33], [170, 1, 0, 200, 400], 6, 3, 32, causal, prefix=777)
    run_attention(h3lib, [300, 300], [300, 300], 2, 1, 128, causal, prefix=300)


@pytest.mark.parametrize("G", [1, 4, 32])
def test_second_query_tile_of_few_rows(h3lib, G):
    # a piece of two query tiles whose second one has one token, between pieces
    # of one tile and of two full ones
    t = 128 // G
    run_attention(h3lib, [t + 1, 2 * t, 1, t + 2, 3 * t + 1, t], [700, 700, 300, 1500, 4000, 129],
                  2 * G, 2, 32, causal=True)
    run_attention(h3lib, [t + 1, 1, 2 * t + 1], [700, 3, 1500], 2 * G, 2, 16, prefix=400)


@pytest.mark.parametrize("prefix", [0, 300, 13000])
def test_a_table_without_pages(h3lib, prefix):
    # no sequence has a place for a key: nothing, or the prefix alone
    P = Paged([0, 0], 2, 16, prefix=prefix)
    P.table = torch.zeros(2, 0, dtype=torch.int32, device=dev)
    q = rnd(gen(34), 5, 6, DH)
    o = attend(h3lib, q, P, [0, 2, 5], causal=True)
    check_attention(o, q, P, [0, 2, 5], True, DH ** -0.5)
    assert prefix or bool((o == 0).all())


def test_a_page_in_several_places(h3lib):
    # the same page twice in a sequence, in two sequences and in the prefix
    P = Paged([200, 150, 64], 2, 32, prefix=96)
    P.table[0, 3] = P.table[0, 1]
    P.table[1, 0] = P.table[0, 1]
    P.prefix_pages[2] = P.table[0, 0]
    P.prefix_pages[1] = P.prefix_pages[0]
    q = rnd(gen(31), 8, 6, DH)
    check_attention(attend(h3lib, q, P, [0, 3, 7, 8]), q, P, [0, 3, 7, 8], False, DH ** -0.5)


def test_many_sequences(h3lib):
    # more than 32 ends per step of the search for a row's sequence, empty ones
    # among them
    B = 2100
    q_len = [0 if i % 3 == 1 else 1 + (i % 97 == 0) * 2 for i in range(B)]
    kv = [(i * 7) % 50 + q_len[i] for i in range(B)]
    run_attention(h3lib, q_len, kv, 2, 1, 16, causal=True, prefix=40)
    run_attention(h3lib, q_len, kv, 2, 1, 16, first=2, behind=3, prefix=40)


def test_nothing_but_the_rows_is_written(h3lib):
    # the columns beside o's rows, the memory behind the workspace and the pool
    for prefix in (0, 300):
        P = Paged([900, 40, 2000], 2, 16, prefix=prefix)
        k, v = P.k.clone(), P.v.clone()
        H, cu = 6, [0, 1, 30, 200]
        q = rnd(gen(32), 200, H, DH)
        wide = torch.full((200, H * DH + 24), SENT, dtype=torch.bfloat16, device=dev)
        o = wide[:, 8:8 + H * DH].unflatten(1, (H, DH))
        need = h3lib.attention_paged_workspace_bytes(200, H, prefix)
        ws = torch.full((need + 4096,), 0x5A, dtype=torch.uint8, device=dev)
        h3lib_o = attend(h3lib, q, P, cu, causal=True, o=o, ws=ws[:need])
        check_attention(h3lib_o, q, P, cu, True, DH ** -0.5)
        assert bool((wide[:, :8] == SENT).all()) and bool((wide[:, 8 + H * DH:] == SENT).all())
        assert bool((ws[need:] == 0x5A).all())
        for now, then in ((P.k, k), (P.v, v)):
            assert torch.equal(now.view(torch.int16), then.view(torch.int16))


@pytest.mark.parametrize("H,Hkv", [(1, 1), (3, 1), (8, 4), (21, 3), (8, 1), (9, 1), (20, 2), (128, 1)])
@pytest.mark.parametrize("kv", [255, 257, 511, 513, 1023, 1100, 2048, 2100, 4096, 9000, 10240, 11000])
def test_single_rows_of_growing_tables(h3lib, H, Hkv, kv):
    # lengths about those where a row's keys go to more CTAs or to the other kernel
    run_attention(h3lib, [1], [kv], H, Hkv, 16 if kv % 2 else 64)
    run_attention(h3lib, [1, 1, 0, 1], [kv, 1, 5, kv // 3], H, Hkv, 32, prefix=70 if kv < 2000 else 0)


@pytest.mark.parametrize("B", [10, 14, 15, 16, 22, 23, 27, 28, 33, 35, 45, 46, 75, 77, 151, 153, 305, 700])
def test_single_rows_of_growing_batches(h3lib, B):
    run_attention(h3lib, [1] * B, [(i * 131) % 1100 for i in range(B)], 2, 1, 64)
    run_attention(h3lib, [1] * B, [(i * 131) % 300 for i in range(B)], 18, 2, 16)
    run_attention(h3lib, [1] * B, [(i * 131) % 90 for i in range(B)], 1, 1, 16, prefix=130, causal=True)


def test_short_chunks(h3lib):
    # a few rows of a sequence, each taken by itself
    run_attention(h3lib, [4, 1, 7], [900, 40, 7], 6, 2, 32, causal=True)
    run_attention(h3lib, [4, 1, 7], [900, 40, 7], 10, 1, 16, prefix=33)
    run_attention(h3lib, [30], [20], 4, 4, 16, causal=True, first=2, behind=3)


@pytest.mark.parametrize("seed", range(48))
def test_drawn_batches(h3lib, seed):
    r = random.Random(seed)
    log = lambda lo, hi: round(math.exp(r.uniform(math.log(lo), math.log(hi))))  # noqa: E731
    G, Hkv = r.choice([1, 1, 2, 3, 5, 8, 12, 17, 40]), r.choice([1, 2, 3, 7])
    B, prefix = log(1, 60), r.choice([0, 0, 0, log(1, 3000)])
    q_len = [r.choice([0, 1, 1, 1, log(1, max(2, 700 // B))]) for _ in range(B)]
    kv = [0 if r.random() < 0.1 else log(1, r.choice([100, 1000, max(2, 40000 // B)])) for _ in q_len]
    if r.random() < 0.4:
        q_len = [min(n, 1) for n in q_len]
    if not sum(q_len):
        q_len[0] = 1
    run_attention(h3lib, q_len, kv, G * Hkv, Hkv, r.choice([16, 32, 64, 128]), r.random() < 0.4, prefix,
                  seed, first=r.choice([0, 3]), behind=r.choice([0, 5]))


def test_large_scores(h3lib):
    # sharply peaked softmax: the running maximum moves by more than one
    # rescale threshold many times
    run_attention(h3lib, [9, 1], [1500, 600], 4, 2, 64, std=12.0)
    run_attention(h3lib, [9, 1], [1500, 600], 4, 2, 64, std=12.0, prefix=1000)


def test_equal_keys_give_the_mean_of_the_values(h3lib):
    P = Paged([200], 1, 32)
    P.put(P.table[0], rnd(gen(2), 1, 1, DH).expand(200, 1, DH), rnd(gen(3), 200, 1, DH))
    q = rnd(gen(4), 1, 1, DH)
    o = attend(h3lib, q, P, [0, 1])
    mean = P.keys(0)[1].mean(0)
    a1 = P.keys(0)[1].abs().mean(0)
    assert bool(((o[0].double() - mean).abs() <= U * mean.abs() + 2 * U * a1).all())


def test_strided_rows(h3lib):
    # q as the first columns of a merged projection, o inside a wider buffer
    P = Paged([333, 60], 2, 64)
    cu, H = [0, 40, 41], 6
    wide = rnd(gen(5), 41, (H + 4) * DH)
    q = wide[:, :H * DH].unflatten(1, (H, DH))
    buf = torch.full((41, 9 * DH), SENT, dtype=torch.bfloat16, device=dev)
    o = buf[:, DH:7 * DH].unflatten(1, (H, DH))
    attend(h3lib, q, P, cu, True, o=o)
    check_attention(o, q, P, cu, True, DH ** -0.5, "strided")
    assert bool((buf[:, :DH] == SENT).all()) and bool((buf[:, 7 * DH:] == SENT).all())


def test_scale(h3lib):
    P = Paged([500], 2, 64)
    q = rnd(gen(6), 7, 2, DH)
    o = attend(h3lib, q, P, [0, 7], scale=0.02)
    check_attention(o, q, P, [0, 7], False, 0.02, "scale")


@pytest.mark.parametrize("prefix", [0, 300])
def test_repeats_are_bit_identical(h3lib, prefix):
    P = Paged([3000, 5, 700], 3, 64, prefix=prefix)
    q = rnd(gen(7), 12, 6, DH)
    outs = [attend(h3lib, q, P, [0, 1, 3, 12], causal=True) for _ in range(3)]
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])


def test_lengths_and_pages_out_of_range_are_bounded(h3lib):
    # lengths past the table are taken as the table's; pages outside the pool
    # read as zero keys and values
    P = Paged([128, 128], 2, 64, spare=1)
    q = rnd(gen(8), 2, 4, DH)
    want = attend(h3lib, q, P, [0, 1, 2])
    c = h3lib.kv_cache(P.k, P.v)
    ws = torch.empty(h3lib.attention_paged_workspace_bytes(2, 4), dtype=torch.uint8, device=dev)
    o = torch.empty_like(q)
    h3lib.attention_paged(q, o, c, h3lib.kv_batch(i32([0, 1, 2]), i32([2 ** 31 - 1, 128]),
                                                  P.table, 2), ws)
    h3lib.check_device_error()
    assert torch.equal(o, want)
    h3lib.attention_paged(q, o, c, h3lib.kv_batch(i32([0, 1, 2]), i32([-5, 128]), P.table, 2), ws)
    h3lib.check_device_error()
    assert bool((o[0] == 0).all()) and torch.equal(o[1], want[1])
    for bad in (-1, P.pages, 2 ** 31 - 1, -2 ** 31):
        table = P.table.clone()
        table[0, 1] = bad
        h3lib.attention_paged(q, o, c, h3lib.kv_batch(i32([0, 1, 2]), i32([128, 128]), table, 2),
                              ws)
        h3lib.check_device_error()
        Z = Paged([128], 2, 64)
        k, v = (x.to(torch.bfloat16).clone() for x in P.keys(0))
        k[64:], v[64:] = 0, 0
        Z.put(Z.table[0], k, v)
        check_attention(o[:1], q[:1], Z, [0, 1], False, DH ** -0.5, f"page {bad}")
        assert torch.equal(o[1], want[1])


def test_row_ranges_out_of_order_stay_inside(h3lib):
    # cu_q that runs backwards or past T: no row outside T is touched
    P = Paged([40, 40, 40], 2, 16)
    g = gen(9)
    buf = torch.full((4 + 8 + 4, 4, DH), SENT, dtype=torch.bfloat16, device=dev)
    q = rnd(g, 8, 4, DH)
    for cu in ([0, 6, 3, 100], [-5, 4, 4, 8], [8, 8, 8, 2 ** 31 - 1], [5, 2, 9, 1]):
        attend(h3lib, q, P, cu, o=buf[4:12])
        assert bool((buf[:4] == SENT).all()) and bool((buf[12:] == SENT).all())


def test_offsets_past_32_bits(h3lib):
    # a pool of 2^33 bytes per tensor whose last pages are the ones in use
    Hkv, page = 8, 128
    pages = 2 ** 33 // (Hkv * page * DH * 2)
    P = Paged([300], Hkv, page)
    k = torch.empty(pages, Hkv, page, DH, dtype=torch.bfloat16, device=dev)
    v = torch.empty_like(k)
    n = P.table.shape[1]
    k[-n:], v[-n:] = P.k[P.table[0].long()], P.v[P.table[0].long()]
    table = torch.arange(pages - n, pages, dtype=torch.int32, device=dev)[None]
    q = rnd(gen(10), 2, 16, DH)
    P.k, P.v, P.table = k, v, table
    o = attend(h3lib, q, P, [0, 2])
    check_attention(o, q, P, [0, 2], False, DH ** -0.5, "past 32 bits")
    kk, vv = rnd(gen(11), 2, Hkv, DH), rnd(gen(12), 2, Hkv, DH)
    b = h3lib.kv_batch(i32([0, 2]), i32([300]), table, 2)
    h3lib.kv_append_paged(None, kk, vv, None, h3lib.kv_cache(k, v), b,
                          torch.zeros(2, 3, dtype=torch.int32, device=dev), (128, 0, 0))
    h3lib.check_device_error()
    p, off = P.rows(table[0], 300)
    assert torch.equal(v[p, :, off][298:], vv) and torch.equal(k[p, :, off][298:], kk)


def test_another_stream_and_two_at_once(h3lib):
    P = Paged([2000, 900], 4, 64, prefix=640)
    q = rnd(gen(13), 2, 8, DH)
    want = attend(h3lib, q, P, [0, 1, 2])
    torch.cuda.synchronize()
    s = [torch.cuda.Stream(), torch.cuda.Stream()]
    outs = [torch.empty_like(q) for _ in range(8)]
    need = h3lib.attention_paged_workspace_bytes(2, 8, P.prefix)
    ws = [torch.empty(need, dtype=torch.uint8, device=dev) for _ in s]
    c, b = h3lib.kv_cache(P.k, P.v), P.batch(h3lib, [0, 1, 2], 2)
    torch.cuda.synchronize()
    for i, o in enumerate(outs):
        h3lib.attention_paged_prefix(q, o, c, b, P.prefix_pages, P.prefix, ws[i % 2],
                                     stream=s[i % 2])
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs)


def test_captured_calls_follow_the_device_arrays(h3lib):
    # append + attention captured once; replayed for growing lengths
    Hkv, H, page, n = 2, 4, 16, 40
    P = Paged([n], Hkv, page)
    k0, v0 = (x.to(torch.bfloat16) for x in P.keys(0))
    P.k.fill_(float("nan"))
    P.v.fill_(float("nan"))
    c = h3lib.kv_cache(P.k, P.v)
    kv_len = i32([1])
    b = h3lib.kv_batch(i32([0, 1]), kv_len, P.table, 1)
    q, k, v = (torch.zeros(1, h, DH, dtype=torch.bfloat16, device=dev) for h in (H, Hkv, Hkv))
    q_out, o = torch.empty_like(q), torch.empty_like(q)
    pos = torch.zeros(1, 3, dtype=torch.int32, device=dev)
    ws = torch.empty(h3lib.attention_paged_workspace_bytes(1, H), dtype=torch.uint8, device=dev)

    def step():
        h3lib.kv_append_paged(q, k, v, q_out, c, b, pos, (128, 0, 0))
        h3lib.attention_paged(q_out, o, c, b, ws)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    qs = rnd(gen(14), n, H, DH)
    R = Paged([n], Hkv, page)
    for j in range(n):
        q.copy_(qs[j:j + 1])
        k.copy_(k0[j:j + 1])
        v.copy_(v0[j:j + 1])
        kv_len.fill_(j + 1)
        graph.replay()
        h3lib.check_device_error()
        R.k, R.v, R.table, R.kv = P.k, P.v, P.table, [j + 1]
        check_attention(o, qs[j:j + 1], R, [0, 1], False, DH ** -0.5, f"replay {j}")
    assert torch.equal(P.keys(0)[0].to(torch.bfloat16), k0)


# ---------------------------------------------------------------- append
def ref_norm_turn(x, gain, pos, axis, pairing, theta=1e4, eps=1e-6):
    """(y, |a| + |b| of every element's pair) in 64 bits."""
    x = x.double()
    if gain is not None:
        x = x / (x.pow(2).mean(-1, keepdim=True) + eps).sqrt() * gain.double()
    y, mag = torch.empty_like(x), torch.empty_like(x)
    o = 0
    for a, d in enumerate(axis):
        for j in range(d // 2):
            u, w = (o + j, o + d // 2 + j) if pairing else (o + 2 * j, o + 2 * j + 1)
            phi = pos[:, a].double() * theta ** (-2.0 * j / d)
            c, s = phi.cos()[:, None], phi.sin()[:, None]
            y[..., u] = x[..., u] * c - x[..., w] * s
            y[..., w] = x[..., u] * s + x[..., w] * c
            mag[..., u] = mag[..., w] = x[..., u].abs() + x[..., w].abs()
        o += d
    return y, mag


def close_turned(x, ref, what):
    y, mag = ref
    e = 2.0 ** -18 * mag
    worst = float(((x.double() - y).abs() / (e + U * (y.abs() + e) + 1e-30)).max()) if x.numel() else 0
    assert worst <= 1.0, f"{what}: {worst:.3g} of the bound"


def run_append(h3lib, q_len, kv_len, H, Hkv, page, axis=(32, 48, 48), pairing=0, norm=True,
               merged=True, first=0, behind=0, seed=3, in_place=False, only_cache=False):
    P = Paged(kv_len, Hkv, page, seed)
    g = gen(seed + 50)
    cu = cumul(q_len, first)
    T = cu[-1] + behind
    if merged:
        qkv = rnd(g, T, (H + 2 * Hkv) * DH, std=2.0)
        q = qkv[:, :H * DH].unflatten(1, (H, DH))
        k = qkv[:, H * DH:(H + Hkv) * DH].unflatten(1, (Hkv, DH))
        v = qkv[:, (H + Hkv) * DH:].unflatten(1, (Hkv, DH))
    else:
        q, k, v = (rnd(g, T, h, DH, std=2.0) for h in (H, Hkv, Hkv))
    q0 = q.clone()
    q_out = q if in_place else torch.full((T, H, DH), SENT, dtype=torch.bfloat16, device=dev)
    pos = torch.randint(0, 60000, (T, 3), generator=g, device=dev, dtype=torch.int32)
    gains = [1 + 0.1 * torch.randn(DH, generator=g, device=dev) for _ in range(2)] if norm \
        else [None, None]
    k_before, v_before = P.k.clone(), P.v.clone()
    h3lib.kv_append_paged(None if only_cache else q, k, v, None if only_cache else q_out,
                          h3lib.kv_cache(P.k, P.v), P.batch(h3lib, cu, T), pos, axis,
                          None if only_cache else gains[0], gains[1], pairing=pairing)
    h3lib.check_device_error()
    want_k, want_v = k_before.clone(), v_before.clone()
    rows = slice(cu[0], cu[-1])
    ky, kmag = ref_norm_turn(k, gains[1], pos, axis, pairing)
    for b in range(len(q_len)):
        for i in range(q_len[b]):
            j = kv_len[b] - q_len[b] + i
            if not 0 <= j < P.table.shape[1] * page:
                continue
            p = int(P.table[b, j // page])
            if not 0 <= p < P.pages:
                continue
            t = cu[b] + i
            close_turned(P.k[p, :, j % page], (ky[t], kmag[t]), f"k of sequence {b}, key {j}")
            want_k[p, :, j % page] = P.k[p, :, j % page]
            want_v[p, :, j % page] = v[t]
    bits = lambda x: x.view(torch.int16)  # noqa: E731
    assert torch.equal(bits(P.k), bits(want_k)), "another place of the key cache was written"
    assert torch.equal(bits(P.v), bits(want_v)), "values differ"
    if not only_cache:
        close_turned(q_out[rows], [x[rows] for x in ref_norm_turn(q0, gains[0], pos, axis, pairing)],
                     "q_out")
        left = q0 if in_place else torch.full_like(q0, SENT)
        assert torch.equal(q_out[:cu[0]], left[:cu[0]]) and torch.equal(q_out[cu[-1]:], left[cu[-1]:])


@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("pairing,axis", [(0, (32, 48, 48)), (1, (32, 48, 48)), (1, (128, 0, 0)),
                                          (0, (126, 2, 0)), (1, (0, 96, 32))])
def test_append(h3lib, page, pairing, axis):
    run_append(h3lib, [1, 1, 1], [1, 130, 64], 4, 4, page, axis, pairing)
    run_append(h3lib, [20, 0, 1, 70], [20, 9, 200, 128], 6, 2, page, axis, pairing, norm=False)


@pytest.mark.parametrize("H,Hkv", [(1, 1), (3, 1), (7, 7), (42, 42), (32, 8), (40, 5), (5, 1)])
def test_append_head_layouts(h3lib, H, Hkv):
    run_append(h3lib, [1, 33], [5, 60], H, Hkv, 16, merged=False)
    run_append(h3lib, [1, 33], [5, 60], H, Hkv, 16, merged=False, in_place=True, pairing=1)
    run_append(h3lib, [1, 33], [5, 60], H, Hkv, 16, only_cache=True)


def test_append_rows_without_a_place(h3lib):
    # rows before the first key, rows outside every sequence
    run_append(h3lib, [10, 4], [3, 4], 4, 2, 16)
    run_append(h3lib, [10, 4], [12, 40], 4, 2, 16, first=3, behind=5)
    run_append(h3lib, [2], [0], 4, 2, 16)


def test_append_many_rows(h3lib):
    run_append(h3lib, [1] * 300, [1 + i % 90 for i in range(300)], 2, 1, 32)
    run_append(h3lib, [700], [900], 3, 1, 64, pairing=1)


def test_append_pages_out_of_range_write_nothing(h3lib):
    g = gen(20)
    k = torch.full((4, 2, 16, DH), SENT, dtype=torch.bfloat16, device=dev)
    v = torch.full_like(k, SENT)
    rows = rnd(g, 6, 2, DH)
    pos = torch.zeros(6, 3, dtype=torch.int32, device=dev)
    table = i32([[-1, 4], [2 ** 31 - 1, -2 ** 31], [0, 1]])
    # sequence 0: pages -1 and 4; sequence 1: the largest and smallest integers;
    # sequence 2: beyond its two pages, at a length no table holds
    for kv in ([17, 17, 34], [17, 17, 2 ** 31 - 1], [17, 17, -2 ** 31]):
        b = h3lib.kv_batch(i32([0, 2, 4, 6]), i32(kv), table, 6)
        h3lib.kv_append_paged(None, rows, rows, None, h3lib.kv_cache(k, v), b, pos, (128, 0, 0))
        h3lib.check_device_error()
        assert bool((k == SENT).all()) and bool((v == SENT).all())
    for cu in ([0, 7, 3, 100], [-3, 2, 2, 2], [6, 6, 6, 2 ** 31 - 1]):
        b = h3lib.kv_batch(i32(cu), i32([40, 40, 40]), table, 6)
        h3lib.kv_append_paged(None, rows, rows, None, h3lib.kv_cache(k, v), b, pos, (128, 0, 0))
        h3lib.check_device_error()
    assert bool((k == SENT).all())


def test_append_equals_the_in_place_kernel(h3lib):
    # the same arithmetic as h3_qk_norm_rope, so the same bits
    g = gen(21)
    T, H = 150, 6
    q, k, v = (rnd(g, T, H, DH) for _ in range(3))
    pos = torch.randint(0, 60000, (T, 3), generator=g, device=dev, dtype=torch.int32)
    gq, gk = (1 + 0.1 * torch.randn(DH, generator=g, device=dev) for _ in range(2))
    for pairing in (0, 1):
        P = Paged([T], H, 64, fill=False)
        q_out = torch.empty_like(q)
        h3lib.kv_append_paged(q, k, v, q_out, h3lib.kv_cache(P.k, P.v), P.batch(h3lib, [0, T], T),
                              pos, (32, 48, 48), gq, gk, pairing=pairing)
        q2, k2 = q.clone(), k.clone()
        h3lib.qk_norm_rope(q2, k2, gq, gk, pos, (32, 48, 48), pairing=pairing)
        h3lib.check_device_error()
        assert torch.equal(q_out, q2)
        assert torch.equal(P.keys(0)[0], k2.double()) and torch.equal(P.keys(0)[1], v.double())


# --------------------------------------------------- together, as in serving
def test_frames_through_the_cache_match_dense_attention(h3lib):
    """A packed sequence sent through the cache in ragged chunks: the last
    chunk's rows see every key, so they equal the dense attention of the whole
    sequence (h3_qk_norm_rope + h3_attention_varlen) within both calls'
    tolerances against 64 bits."""
    g = gen(30)
    H, S = 6, 700
    q, k, v = (rnd(g, S, H, DH) for _ in range(3))
    pos = torch.randint(0, 100, (S, 3), generator=g, device=dev, dtype=torch.int32)
    gq, gk = (1 + 0.1 * torch.randn(DH, generator=g, device=dev) for _ in range(2))
    P = Paged([S], H, 32, fill=False)
    c = h3lib.kv_cache(P.k, P.v)
    o, q_all = torch.empty_like(q), torch.empty_like(q)
    done = 0
    for n in (1, 255, 44, 1, 399):
        sl = slice(done, done + n)
        done += n
        b = h3lib.kv_batch(i32([0, n]), i32([done]), P.table, n)
        ws = torch.empty(h3lib.attention_paged_workspace_bytes(n, H), dtype=torch.uint8, device=dev)
        h3lib.kv_append_paged(q[sl], k[sl], v[sl], q_all[sl], c, b, pos[sl].contiguous(),
                              (32, 48, 48), gq, gk)
        h3lib.attention_paged(q_all[sl], o[sl], c, b, ws)
    h3lib.check_device_error()
    q2, k2 = q.clone(), k.clone()
    h3lib.qk_norm_rope(q2, k2, gq, gk, pos, (32, 48, 48))
    dense = torch.empty_like(q)
    h3lib.attention_varlen(q2, k2, v, dense)
    h3lib.check_device_error()
    last = slice(S - 399, S)
    rel = float((o[last].double() - dense[last].double()).norm() / dense[last].double().norm())
    assert rel <= 2 * U, rel
    check_attention(o[last], q_all[last], P, [0, 399], False, DH ** -0.5, "last chunk")


def test_variants_behind_one_prefix_equal_separate_sequences(h3lib):
    """Variants of one clip: the prefix is written once, every variant appends
    its own rows and reads prefix + own; each equals a sequence of its own that
    holds a copy of the prefix."""
    g = gen(31)
    H, Hkv, page, prefix, n = 8, 2, 64, 320, 5
    B = 6
    S = Paged([n] * B, Hkv, page, prefix=prefix)
    c = h3lib.kv_cache(S.k, S.v)
    q, k, v = rnd(g, B * n, H, DH), rnd(g, B * n, Hkv, DH), rnd(g, B * n, Hkv, DH)
    pos = torch.arange(B * n, device=dev, dtype=torch.int32)[:, None].repeat(1, 3) % n + prefix
    cu = cumul([n] * B)
    b = S.batch(h3lib, cu, B * n)
    q_out = torch.empty_like(q)
    h3lib.kv_append_paged(q, k, v, q_out, c, b, pos.contiguous(), (32, 48, 48))
    for causal in (False, True):
        o = attend(h3lib, q_out, S, cu, causal)
        check_attention(o, q_out, S, cu, causal, DH ** -0.5, "shared")
        own = Paged([prefix + n] * B, Hkv, page)
        for i in range(B):
            kk, vv = (x.to(torch.bfloat16) for x in S.keys(i))
            own.put(own.table[i], kk, vv)
        alone = attend(h3lib, q_out, own, cu, causal)
        rel = float((o.double() - alone.double()).norm() / alone.double().norm())
        assert rel <= 2 * U, rel


@pytest.mark.parametrize("prefix", [0, 260])
def test_two_captured_calls_in_turn(h3lib, prefix):
    # two graphs of one padded size with a workspace of their own, replayed in
    # turn on two streams while the batch shrinks and grows
    P = Paged([300, 40, 600], 2, 32, prefix=prefix)
    T, H = 160, 6
    c = h3lib.kv_cache(P.k, P.v)
    cu, kv = torch.zeros(4, dtype=torch.int32, device=dev), i32(P.kv)
    b = h3lib.kv_batch(cu, kv, P.table, T)
    q = rnd(gen(33), T, H, DH)
    need = h3lib.attention_paged_workspace_bytes(T, H, prefix)
    ws = [torch.full((need,), 0xFF, dtype=torch.uint8, device=dev) for _ in range(2)]
    o = [torch.empty_like(q) for _ in range(2)]
    streams, graphs = [torch.cuda.Stream() for _ in range(2)], []
    torch.cuda.synchronize()
    for i in range(2):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[i], stream=streams[i]):
            h3lib.attention_paged_prefix(q, o[i], c, b, P.prefix_pages if prefix else None, prefix,
                                         ws[i], causal=i == 1)
    for ends in ([0, 1, 1, 2], [0, 100, 140, 160], [0, 0, 0, 0], [0, 40, 70, 71], [3, 3, 30, 150]):
        cu.copy_(i32(ends))
        for x in o:
            x.fill_(SENT)
        torch.cuda.synchronize()
        for _ in range(3):
            for i in range(2):
                with torch.cuda.stream(streams[i]):
                    graphs[i].replay()
        torch.cuda.synchronize()
        h3lib.check_device_error()
        for i in range(2):
            if ends[-1] > ends[0]:
                check_attention(o[i], q, P, ends, i == 1, DH ** -0.5, f"ends {ends} causal {i}")
            assert bool((o[i][:ends[0]] == SENT).all()) and bool((o[i][ends[-1]:] == SENT).all())


def test_calls_one_after_another_share_a_workspace(h3lib):
    # rows of many sequences behind a prefix (two kernels and a join), a chunk, and a
    # long row, in turn on one stream with one workspace, directly and captured
    B = 170
    calls, want = [], []
    need = 0
    for q_len, kv, prefix, seed in (([1] * B, [(i * 37) % 230 for i in range(B)], 1500, 1),
                                    ([200], [1500], 0, 2), ([1], [15000], 0, 3),
                                    ([1] * B, [(i * 53) % 120 + 1 for i in range(B)], 900, 4)):
        P, cu = Paged(kv, 2, 16, seed, prefix), cumul(q_len)
        q = rnd(gen(seed), cu[-1], 4, DH)
        need = max(need, h3lib.attention_paged_workspace_bytes(cu[-1], 4, prefix))
        calls.append((q, torch.empty_like(q), h3lib.kv_cache(P.k, P.v), P.batch(h3lib, cu, cu[-1]),
                      P.prefix_pages if prefix else None, prefix))
        want.append(attend(h3lib, q, P, cu))
        check_attention(want[-1], q, P, cu, False, DH ** -0.5, f"call {seed}")
    ws = torch.empty(need, dtype=torch.uint8, device=dev)

    def run():
        for _ in range(4):
            for q, o, c, b, pages, n in calls:
                h3lib.attention_paged_prefix(q, o, c, b, pages, n, ws)

    run()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        run()
    for go in (run, graph.replay, run):
        for c in calls:
            c[1].fill_(SENT)
        go()
        torch.cuda.synchronize()
        h3lib.check_device_error()
        assert all(torch.equal(c[1], w) for c, w in zip(calls, want))


def test_append_many_sequences(h3lib):
    B = 2100
    q_len = [0 if i % 3 == 1 else 1 for i in range(B)]
    run_append(h3lib, q_len, [(i * 7) % 50 + q_len[i] for i in range(B)], 1, 1, 16, first=1, behind=2)
