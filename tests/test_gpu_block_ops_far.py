"""Norms around a branch, 4-bit rows and products, scores, selection and attention over chosen blocks where offsets
pass 2^31 elements: the last rows give, bit for bit, what they give as a tensor of their own."""
import pytest
import torch

pytestmark = pytest.mark.gpu
dev = "cuda"


@pytest.fixture(autouse=True)
def room():
    yield
    torch.cuda.empty_cache()


def gen(seed):
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    return g


def tail(x, n):
    return x[-n:].clone()


def test_norm(h3lib):
    S, D = 420000, 5376
    assert S * D > 1 << 31
    g = gen(1)
    r = torch.zeros(S, D, device=dev)
    r[-300:] = torch.randn(300, D, generator=g, device=dev)
    r[-7] *= 1e25                                  # and a row that is worked out apart
    d = torch.zeros(S, D, device=dev, dtype=torch.bfloat16)
    d[-300:] = torch.randn(300, D, generator=g, device=dev).to(torch.bfloat16)
    h = torch.empty_like(d)
    seg = torch.zeros(S, dtype=torch.int32, device=dev)
    seg[-100:] = 1
    mod = torch.randn(2, 3, D, generator=g, device=dev)
    few = [tail(x, 300) for x in (r, d, h)]
    h3lib.sandwich_norm(few[0], few[1], few[2], gate=mod[:, 0], shift=mod[:, 1], scale=mod[:, 2], seg=tail(seg, 300))
    h3lib.sandwich_norm(r, d, h, gate=mod[:, 0], shift=mod[:, 1], scale=mod[:, 2], seg=seg)
    h3lib.check_device_error()
    assert torch.equal(r[-300:], few[0]) and torch.equal(h[-300:], few[2])


@pytest.mark.parametrize("fmt", ["mx", "nv"])
def test_rows_and_product(h3lib, fmt):
    R, K, n = 140032, 16384, 256                  # n: whole tiles of scales, so that the last rows' are a tensor's
    assert R * K > 1 << 31 and R % 128 == 0
    x = torch.zeros(R, K, device=dev, dtype=torch.bfloat16)
    x[-n:] = torch.randn(n, K, generator=gen(2), device=dev).to(torch.bfloat16)
    q, few = h3lib.fp4_rows(R, K, fmt), h3lib.fp4_rows(n, K, fmt)
    h3lib.quantize_fp4_rows(x, q)
    h3lib.quantize_fp4_rows(tail(x, n), few)
    h3lib.check_device_error()
    assert torch.equal(q.codes[-n:], few.codes) and torch.equal(q.scales[-few.scales.numel():], few.scales)
    if fmt == "nv":
        assert torch.equal(q.row_scale[-n:], few.row_scale)
    del x
    w = h3lib.fp4_rows(16128, K, fmt)
    h3lib.quantize_fp4_rows(torch.randn(16128, K, generator=gen(3), device=dev).to(torch.bfloat16), w)
    y, z = (torch.empty(m, 16128, device=dev, dtype=torch.bfloat16) for m in (R, n))
    assert y.numel() > 1 << 31
    h3lib.linear_fp4(q, w, y)
    h3lib.linear_fp4(few, w, z)
    h3lib.check_device_error()
    assert torch.equal(y[-n:], z) and (y[:4096] == 0).all()
    s, t = (torch.empty(m, 8064, device=dev, dtype=torch.bfloat16) for m in (R, n))
    h3lib.linear_swiglu_fp4(q, w, s)
    h3lib.linear_swiglu_fp4(few, w, t)
    h3lib.check_device_error()
    assert torch.equal(s[-n:], t)


@pytest.mark.parametrize("kb", [64, 128])
def test_chosen_blocks(h3lib, kb):
    L, H, most = 410112, 42, 3
    assert L * H * 128 > 1 << 31 and L % 256 == 0
    g = gen(4)
    q, k, v = (torch.zeros(L, H, 128, device=dev, dtype=torch.bfloat16) for _ in range(3))
    for x in (q, k, v):
        x[-512:] = torch.randn(512, H, 128, generator=g, device=dev).to(torch.bfloat16)
    nq, nk = L // 256, -(-L // kb)
    at = 512 // kb                                     # the last blocks, of which all lists are
    ids = torch.randint(nk - at, nk, (H, nq, most), generator=g, device=dev).int()
    n = torch.full((H, nq), most, dtype=torch.int32, device=dev)
    o = torch.empty_like(q)
    h3lib.attention_blocks(q, k, v, o, ids, n, k_block=kb)
    h3lib.check_device_error()
    few = [tail(x, 512) for x in (q, k, v)]
    want = torch.empty_like(few[0])
    # (the same number of blocks, some of them empty, takes the kernel that many items take)
    more = torch.cat([torch.full((H, 30, most), -1, device=dev, dtype=torch.int32), ids[:, -2:] - (nk - at)], 1)
    counts = torch.full((H, 32), most, dtype=torch.int32, device=dev)
    padded = torch.cat([torch.zeros(30 * 256, H, 128, device=dev, dtype=torch.bfloat16), few[0]])
    out = torch.empty_like(padded)
    h3lib.attention_blocks(padded, few[1], few[2], out, more.contiguous(), counts, k_block=kb)
    h3lib.check_device_error()
    want = out[-512:]
    assert torch.equal(o[-512:], want) and torch.isfinite(want.float()).all()
    scores = torch.empty(1, nq, nk, device=dev)
    last = torch.empty(1, 30 + 2, at, device=dev)
    ws = torch.empty(h3lib.block_scores_workspace_bytes(L, L, 1, 1, kb), device=dev, dtype=torch.uint8)
    h3lib.block_scores(q[:, 41:], k[:, 41:], scores, ws, k_block=kb)
    h3lib.block_scores(padded[:, 41:], few[1][:, 41:], last, ws, k_block=kb)
    h3lib.check_device_error()
    assert torch.equal(scores[:, -2:, -at:], last[:, -2:]) and (scores[:, :-2] == 0).all()


@pytest.mark.parametrize("rows,nk,most", [(2300000, 900, 4), (430000, 1100, 900)])
def test_selection(h3lib, rows, nk, most):
    assert rows * max(nk, most) < 1 << 31          # (the call's own bound; bytes pass 2^32)
    s = torch.zeros(rows, nk, device=dev)
    s[-500:] = torch.randn(500, nk, generator=gen(5), device=dev)
    ids, n = torch.empty(rows, most, device=dev, dtype=torch.int32), torch.empty(rows, device=dev, dtype=torch.int32)
    h3lib.block_select(s, ids, n, keep_last=1)
    want, m = torch.empty_like(ids[:500]), torch.empty_like(n[:500])
    h3lib.block_select(tail(s, 500), want, m, keep_last=1)
    h3lib.check_device_error()
    assert torch.equal(ids[-500:], want) and torch.equal(n[-500:], m) and (n == most).all()
    first = torch.arange(most - 1, device=dev, dtype=torch.int32)
    assert (ids[:-500, :-1] == first).all() and (ids[:-500, -1] == nk - 1).all()
