"""Block scores of means that are infinite or NaN: what the definition says of them, whichever kernel a call takes
(at most eight query blocks by the CUDA cores, more on the tensor cores), and every other score as it was."""
import pytest
import torch

from test_gpu_blocks import QB, gen, heads

pytestmark = pytest.mark.gpu
dev = "cuda"
INF, NAN = float("inf"), float("nan")


def scores(h3lib, q, k, kb, scale):
    H, nq, nk = q.shape[1], -(-q.shape[0] // QB), -(-k.shape[0] // kb)
    out = torch.full((H * nq * nk + 64,), -7.25, device=dev)
    ws = torch.empty(h3lib.block_scores_workspace_bytes(q.shape[0], k.shape[0], H, k.shape[1], kb), dtype=torch.uint8,
                     device=dev)
    h3lib.block_scores(q, k, out[:-64].view(H, nq, nk), ws, k_block=kb, scale=scale)
    h3lib.check_device_error()
    assert (out[-64:] == -7.25).all()
    return out[:-64].view(H, nq, nk)


def definition(q, k, kb, scale):
    mean = lambda x, n: torch.stack([p.double().mean(0) for p in x.split(n)], 1)     # [heads, blocks, 128]
    q, k = mean(q, QB), mean(k, kb).repeat_interleave(q.shape[1] // k.shape[1], 0)
    return (q[:, :, None] * k[:, None]).sum(-1) * scale


@pytest.mark.parametrize("kb", [64, 128])
@pytest.mark.parametrize("Lq,Lk,H,Hkv", [(2048, 700, 4, 2), (2049, 700, 4, 2), (2600, 9000, 3, 1), (33100, 330, 2, 2),
                                         (34000, 17000, 1, 1)])
def test_infinite_and_nan_means(h3lib, Lq, Lk, H, Hkv, kb):
    g = gen(Lq + Lk)
    # means of at least a sixteenth in magnitude, of both signs: no product of one with infinity is in doubt
    def side(L, n):
        x = heads(L, n, g, 0.25)
        sign = torch.randint(0, 2, (1, n, 128), generator=g, device=dev) * 2 - 1
        return (x.float() + sign).to(torch.bfloat16)
    q, k = side(Lq, H), side(Lk, Hkv)
    clean = scores(h3lib, q, k, kb, -0.3)
    q[3, 0, 7] = INF                       # one channel of one block of a head
    q[QB * 2 + 5, 0, 99] = -INF
    q[QB * 3 + 1, H - 1, 3] = NAN
    q[Lq - 1, H - 1, 64] = INF             # the last, short block
    q[QB * 4, 0, 11], q[QB * 4 + 1, 0, 11] = INF, -INF    # a mean of inf - inf
    q[QB * 5, 0, 20], q[QB * 5, 0, 21] = INF, INF         # two channels: inf + inf or inf - inf by the key's signs
    k[kb + 2, Hkv - 1, 3] = -INF
    k[Lk - 1, 0, 120] = INF
    k[Lk // 2, 0, 0] = NAN
    got = scores(h3lib, q, k, kb, -0.3)
    want = definition(q, k, kb, -0.3)
    same = torch.isfinite(want)
    assert torch.equal(got.isnan(), want.isnan())
    assert torch.equal(got.isposinf(), want.isposinf()) and torch.equal(got.isneginf(), want.isneginf())
    assert want.isposinf().any() and want.isneginf().any() and want.isnan().any()
    assert torch.equal(got[same], clean[same])


def test_the_same_blocks_are_chosen_with_more_query_rows(h3lib):
    # a block whose score is +inf is selected, one of NaN or -inf is not, with 2,048 query rows as with 2,049
    g = gen(5)
    q, k = heads(2049, 2, g) + 0.5, heads(1000, 2, g) + 0.5
    k[70, :, 9] = INF
    k[200, :, 9] = -INF
    k[400, :, 9] = NAN
    picked = []
    for L in (2048, 2049):
        s = scores(h3lib, q[:L], k, 64, 1.0)
        nq = s.shape[1]
        ids = torch.empty(2, nq, 1, dtype=torch.int32, device=dev)
        n = torch.empty(2, nq, dtype=torch.int32, device=dev)
        h3lib.block_select(s, ids, n)
        h3lib.check_device_error()
        picked.append(ids[:, :8])
    assert (picked[0] == 1).all() and torch.equal(picked[0], picked[1])


@pytest.mark.parametrize("Lq", [2000, 2600])
def test_sums_beyond_fp32(h3lib, Lq):
    # finite means whose products, or their sum, FP32 cannot hold
    q = torch.full((Lq, 1, 128), 2.0 ** 100, dtype=torch.bfloat16, device=dev)
    k = torch.full((256, 1, 128), 2.0 ** 20, dtype=torch.bfloat16, device=dev)
    k[64:128] = -(2.0 ** 50)
    k[128:192] = 0
    s = scores(h3lib, q, k, 64, 1.0)
    assert (s[:, :, 0] == 2.0 ** 127).all() and s[:, :, 1].isneginf().all() and (s[:, :, 2] == 0).all()


def test_nothing_but_nan(h3lib):
    q = torch.full((20000, 3, 128), NAN, dtype=torch.bfloat16, device=dev)
    k = torch.full((20000, 3, 128), INF, dtype=torch.bfloat16, device=dev)
    assert scores(h3lib, q, k, 64, 1.0).isnan().all()
    q[:, 1] = -1.0
    s = scores(h3lib, q, k, 64, 1.0)
    assert s[1].isneginf().all() and s[::2].isnan().all()
