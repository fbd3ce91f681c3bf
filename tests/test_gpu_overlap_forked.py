"""Launches that overlap the one before them, on streams that wait for one another: a run that forks to a second stream
and joins it, made call by call and captured into a graph, gives the bits of the calls one after another."""
import pytest
import torch

from test_gpu_blocks import QB, gen, heads

pytestmark = pytest.mark.gpu
dev = "cuda"


@pytest.mark.parametrize("Lq,Lk", [(22, 9000), (2600, 2600)])
@pytest.mark.parametrize("fmt", ["mx", "nv"])
def test_fork_and_join(h3lib, fmt, Lq, Lk):
    H, Hkv, kb, most = 4, 2, 64, 12
    D, nq, nk = H * 128, -(-Lq // QB), -(-Lk // kb)
    g = gen(Lq)
    q, k, v = heads(Lq, H, g), heads(Lk, Hkv, g), heads(Lk, Hkv, g)
    resid = torch.randn(Lq, D, generator=g, device=dev)
    w = [h3lib.fp4_rows(n, D, fmt) for n in (D, D, 2 * D)]
    for x in w:
        h3lib.quantize_fp4_rows((torch.randn(*x.shape, generator=g, device=dev) * 0.05).to(torch.bfloat16), x)
    e = lambda *s, dtype=torch.bfloat16: torch.empty(*s, dtype=dtype, device=dev)
    ws = e(h3lib.block_scores_workspace_bytes(Lq, Lk, H, Hkv, kb), dtype=torch.uint8)
    scores, ids, n = e(H, nq, nk, dtype=torch.float32), e(H, nq, most, dtype=torch.int32), e(H, nq, dtype=torch.int32)
    o, h, y, z, s, r = e(Lq, H, 128), e(Lq, D), e(Lq, D), e(Lq, D), e(Lq, D), e(Lq, D, dtype=torch.float32)
    a4, h4, y4 = (h3lib.fp4_rows(Lq, D, fmt) for _ in range(3))

    def left():      # the attention over chosen blocks and its projection
        h3lib.block_scores(q, k, scores, ws, k_block=kb)
        h3lib.block_select(scores, ids, n, keep_first=1)
        h3lib.attention_blocks(q, k, v, o, ids, n, k_block=kb)
        h3lib.quantize_fp4_rows(o.view(Lq, D), a4)
        h3lib.linear_fp4(a4, w[0], y)

    def right():     # a branch of its own on the normed residual
        h3lib.sandwich_norm(resid, normed=h, rms=True)
        h3lib.quantize_fp4_rows(h, h4)
        h3lib.linear_fp4(h4, w[1], z)

    def join():      # both of them
        h3lib.sandwich_norm(resid, y, h, resid_out=r)
        h3lib.sandwich_norm(r, z, h, resid_out=r, post_norm=False)
        h3lib.quantize_fp4_rows(h, y4)
        h3lib.linear_swiglu_fp4(y4, w[2], s)

    outs = (scores, ids, n, o, y, z, r, s)
    for f in (left, right, join):
        f()
        torch.cuda.synchronize()
    h3lib.check_device_error()
    want = [t.clone() for t in outs]
    side = torch.cuda.Stream()

    def forked():
        main = torch.cuda.current_stream()
        side.wait_stream(main)
        with torch.cuda.stream(side):
            right()
        left()
        main.wait_stream(side)
        join()

    def clear():
        for t in outs:
            t.zero_()

    for _ in range(10):
        clear()
        forked()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want))
    clear()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        forked()
        forked()
    for _ in range(5):
        clear()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want))
    h3lib.check_device_error()
