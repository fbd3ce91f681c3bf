"""Appends of so many rows that a CTA takes two of them: odd numbers of rows, rows
outside every sequence and without a place beside others, several rounds of heads,
both pairings, in place and of keys alone, against the 64-bit form and within the
bound of test_gpu_paged.py. And a block put together from the public calls with its
keys and values in a cache, against the oracle."""
import pytest
import torch

import test_gpu_paged as paged
from dit_transformer_block_gb300 import inputs as I
from test_gpu_block import check_block
from test_gpu_paged import DH, SENT, cumul, gen, i32, ref_norm_turn, rnd

pytestmark = pytest.mark.gpu
dev = "cuda"


def least_rows():
    """Two rows per CTA from 16 CTAs of them per SM on."""
    return 32 * torch.cuda.get_device_properties(0).multi_processor_count


def bits(x):
    return x.view(torch.int16)


def run(h3lib, q_len, kv_len, H, Hkv, page=64, axis=(32, 48, 48), pairing=0, norm=True, first=0,
        behind=0, in_place=False, only_cache=False):
    P = paged.Paged(kv_len, Hkv, page, 3, fill=False)
    g, cu = gen(53), cumul(q_len, first)
    T = cu[-1] + behind
    assert T >= least_rows()
    heads = (0 if only_cache else H) + 2 * Hkv
    if in_place:
        q, k, v = (rnd(g, T, h, DH, std=2.0) for h in (H, Hkv, Hkv))
    else:
        qkv = rnd(g, T, heads * DH, std=2.0).unflatten(1, (heads, DH))
        q, k, v = qkv[:, :heads - 2 * Hkv], qkv[:, heads - 2 * Hkv:heads - Hkv], qkv[:, heads - Hkv:]
    q0 = q.clone()
    q_out = q if in_place else torch.full_like(q0, SENT)
    pos = torch.randint(0, 60000, (T, 3), generator=g, device=dev, dtype=torch.int32)
    gq, gk = (1 + 0.1 * torch.randn(DH, generator=g, device=dev) for _ in range(2)) if norm \
        else (None, None)
    want_k, want_v = P.k.clone(), P.v.clone()
    h3lib.kv_append_paged(None if only_cache else q, k, v, None if only_cache else q_out,
                          h3lib.kv_cache(P.k, P.v), P.batch(h3lib, cu, T), pos, axis,
                          None if only_cache else gq, gk, pairing=pairing)
    h3lib.check_device_error()

    def close(x, ref, what):
        y, mag = ref
        e = 2.0 ** -18 * mag
        worst = float(((x.double() - y).abs() / (e + paged.U * (y.abs() + e) + 1e-30)).max())
        assert worst <= 1.0, f"{what}: {worst:.3g} of the bound"

    # the place of every row: key index kv_len - q_len + i of its sequence
    t = torch.arange(cu[0], cu[-1], device=dev)
    b = torch.searchsorted(i32(cu[1:]), t.to(torch.int32), right=True)
    start, n, kv = (i32(x).long()[b] for x in (cu[:-1], q_len, kv_len))
    j = kv - n + t - start
    t, b, j = (x[j >= 0] for x in (t, b, j))
    at = P.table.long()[b, j // page], slice(None), j % page
    close(P.k[at], [x[t] for x in ref_norm_turn(k, gk, pos, axis, pairing)], "keys")
    want_k[at], want_v[at] = P.k[at], v[t]
    assert torch.equal(bits(P.k), bits(want_k)), "another place of the key cache was written"
    assert torch.equal(bits(P.v), bits(want_v)), "values differ"
    if not only_cache:
        rows = slice(cu[0], cu[-1])
        close(q_out[rows], [x[rows] for x in ref_norm_turn(q0, gq, pos, axis, pairing)], "q_out")
        left = q0 if in_place else torch.full_like(q0, SENT)
        for other in (slice(0, cu[0]), slice(cu[-1], T)):
            assert torch.equal(q_out[other], left[other]), "other rows written"


@pytest.mark.parametrize("pairing,axis", [(0, (32, 48, 48)), (1, (32, 48, 48)), (1, (128, 0, 0))])
@pytest.mark.parametrize("H,Hkv", [(1, 1), (5, 1), (4, 4), (32, 8), (42, 42)])
def test_one_long_sequence(h3lib, H, Hkv, pairing, axis):
    n = least_rows() + 1  # the last CTA has one row
    run(h3lib, [n], [n + 9], H, Hkv, 128, axis, pairing)


@pytest.mark.parametrize("pairing", [0, 1])
def test_rows_of_many_sequences(h3lib, pairing):
    # rows outside every sequence at both ends, so that a CTA's two rows are of
    # different kinds; sequences of no rows, and of more rows than keys
    n = least_rows() // 2
    q_len = [1] * n + [0, 7, 3] + [n]
    kv = [1 + i % 40 for i in range(n)] + [5, 4, 0] + [n + 77]
    run(h3lib, q_len, kv, 6, 2, 16, pairing=pairing, first=1, behind=2)
    run(h3lib, q_len, kv, 6, 2, 32, pairing=pairing, first=3, behind=4, norm=False)


@pytest.mark.parametrize("pairing", [0, 1])
def test_in_place_and_keys_alone(h3lib, pairing):
    n = least_rows()
    run(h3lib, [n - 40, 53], [n, 60], 40, 5, 64, pairing=pairing, in_place=True)
    run(h3lib, [n - 40, 53], [n, 60], 0, 3, 64, pairing=pairing, only_cache=True)
    run(h3lib, [n - 40, 53], [n, 60], 0, 20, 64, pairing=pairing, only_cache=True, norm=False)


@pytest.mark.parametrize("pairing", ["interleaved", "half"])
def test_a_block_over_the_cache(h3lib, pairing):
    """Projection, append in two calls, attention over the cache, output projection
    and SwiGLU, from the public calls: the block of the packed sequence."""
    shape = I.BlockShape(S=384, L=321, D=768, H=6, Dh=DH, F=2048, axis_dims=(32, 48, 48),
                         pos_kind="3d", grid=(2, 10, 16), n_tail=22)
    L, D, H = shape.L, shape.D, shape.H
    inp = {k: v.to(dev) for k, v in I.block_inputs(shape, seed=6).items()}
    resid, mod = inp["resid"].clone(), inp["mod"]
    empty = lambda *s: torch.empty(*s, dtype=torch.bfloat16, device=dev)  # noqa: E731
    h, qkv, q, o = empty(shape.S, D), empty(shape.S, 3 * D), empty(L, H, DH), empty(shape.S, D)
    P = paged.Paged([L], H, 32, fill=False)
    cache = h3lib.kv_cache(P.k, P.v)
    h3lib.mod_norm_residual(resid, shift=mod[0], scale=mod[1], normed=h, L=L, eps=shape.eps_ln)
    h3lib.linear(h, inp["w_qkv"], qkv, L=L)
    x = qkv.unflatten(1, (3, H, DH))
    done = 0
    for n in (200, L - 200):  # what is kept of an earlier call, then the rest
        sl = slice(done, done + n)
        done += n
        b = h3lib.kv_batch(i32([0, n]), i32([done]), P.table, n)
        h3lib.kv_append_paged(x[sl, 0], x[sl, 1], x[sl, 2], q[sl], cache, b, inp["pos"][sl].contiguous(),
                              shape.axis_dims, inp["q_gain"], inp["k_gain"], theta=shape.theta,
                              eps=shape.eps_qk, pairing=int(pairing == "half"))
    b = h3lib.kv_batch(i32([0, L]), i32([L]), P.table, L)
    ws = torch.empty(h3lib.attention_paged_workspace_bytes(L, H), dtype=torch.uint8, device=dev)
    h3lib.attention_paged(q, o[:L].unflatten(1, (H, DH)), cache, b, ws)
    h3lib.linear_residual(o, inp["w_o"], resid, mod[2], L=L)
    h3lib.mod_norm_residual(resid, shift=mod[3], scale=mod[4], normed=h, L=L, eps=shape.eps_ln)
    act = empty(shape.S, shape.F)
    h3lib.linear_swiglu(h, inp["w_gu"], act, L=L)
    h3lib.linear_residual(act, inp["w_down"], resid, mod[5], L=L)
    h3lib.check_device_error()
    check_block(resid[:L], shape, inp, what="block over the cache", rope_pairing=pairing)
    assert torch.equal(resid[L:], inp["resid"][L:]), "pad rows written"
