"""Few tiles and few items, which clusters share, captured into graphs: replayed on other inputs and lists, two graphs
over one workspace one after the other, and each equal to the calls made one by one."""
import pytest
import torch

from test_gpu_blocks import QB, gen, heads

pytestmark = pytest.mark.gpu
dev = "cuda"


@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("Lq,Lk,most", [(22, 20000, 40), (200, 6000, 24), (1, 9000, 30)])
def test_tail_rows(h3lib, fmt, Lq, Lk, most):
    H, Hkv, kb, N = 8, 2, 64, 5376
    K = H * 128
    nq, nk = -(-Lq // QB), -(-Lk // kb)

    class Run:
        def __init__(self, seed, ws, w):
            g = gen(seed)
            self.q, self.k, self.v = heads(Lq, H, g), heads(Lk, Hkv, g), heads(Lk, Hkv, g)
            self.s, self.ws, self.w = torch.empty(H, nq, nk, device=dev), ws, w
            self.ids = torch.empty(H, nq, most, device=dev, dtype=torch.int32)
            self.n = torch.empty(H, nq, device=dev, dtype=torch.int32)
            self.o, self.y = torch.empty_like(self.q), torch.empty(Lq, N, device=dev, dtype=torch.bfloat16)
            self.x4, self.z = h3lib.fp4_rows(Lq, K, fmt), torch.empty(Lq, 8, device=dev, dtype=torch.bfloat16)
            self.t4 = h3lib.fp4_rows(Lq, N, fmt)

        def go(self):
            h3lib.block_scores(self.q, self.k, self.s, self.ws, k_block=kb)
            h3lib.block_select(self.s, self.ids, self.n, keep_last=1)
            h3lib.attention_blocks(self.q, self.k, self.v, self.o, self.ids, self.n, k_block=kb)
            h3lib.quantize_fp4_rows(self.o.view(Lq, K), self.x4)
            h3lib.linear_fp4(self.x4, self.w[0], self.y)
            h3lib.quantize_fp4_rows(self.y, self.t4)
            h3lib.linear_fp4(self.t4, self.w[1], self.z)

        def outs(self):
            return [t.clone() for t in (self.s, self.ids, self.n, self.o, self.y, self.z)]

    ws = torch.empty(h3lib.block_scores_workspace_bytes(Lq, Lk, H, Hkv, kb), device=dev, dtype=torch.uint8)
    w = [h3lib.fp4_rows(N, K, fmt), h3lib.fp4_rows(8, N, fmt)]
    for x in w:
        h3lib.quantize_fp4_rows((torch.randn(*x.shape, generator=gen(7), device=dev) * 0.05).to(torch.bfloat16), x)
    runs = [Run(1, ws, w), Run(2, ws, w)]
    want = []
    for r in runs:
        r.go()
        torch.cuda.synchronize()
        want.append(r.outs())
    h3lib.check_device_error()
    assert all(torch.isfinite(t.float()).all() for o in want for t in o)
    graphs = []
    for r in runs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            r.go()
        graphs.append(g)
    for r in runs:
        for t in (r.s, r.o, r.y, r.z, r.ids, r.n):
            t.zero_()
    for i in (0, 1, 1, 0):
        graphs[i].replay()
    torch.cuda.synchronize()
    for r, o in zip(runs, want):
        assert all(torch.equal(a, b) for a, b in zip(r.outs(), o))
    for t, u in zip((runs[0].q, runs[0].k, runs[0].v), (runs[1].q, runs[1].k, runs[1].v)):
        t.copy_(u)
    graphs[0].replay()
    torch.cuda.synchronize()
    h3lib.check_device_error()
    assert all(torch.equal(a, b) for a, b in zip(runs[0].outs(), want[1]))
