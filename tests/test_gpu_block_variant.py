"""A block of the cheaper kind, run as a program would run it: norms around both branches, 4-bit
projections, attention over chosen key blocks. Every step is held to its 64-bit form on what the step
before it left, and the whole run, captured into a graph, repeats its results on other inputs."""
import numpy as np
import pytest
import torch

from test_gpu_blocks import ref_attention, ref_scores, ref_select
from test_gpu_fp4 import check_linear, check_swiglu, reference, unpack
from test_gpu_sandwich_norm import check as check_norm

pytestmark = pytest.mark.gpu
dev = "cuda"
L, D, H, F, KB, MOST = 900, 512, 4, 1408, 64, 6
NQ, NK = 4, 15


class Block:
    def __init__(self, h3, fmt, seed):
        g = torch.Generator(device=dev)
        g.manual_seed(seed)
        rnd = lambda *s, std=1.0: torch.randn(*s, generator=g, device=dev) * std
        bf = lambda *s, std=1.0: rnd(*s, std=std).to(torch.bfloat16)
        empty = lambda *s, dtype=torch.bfloat16: torch.empty(*s, dtype=dtype, device=dev)
        self.h3, self.fmt = h3, fmt
        self.r, self.mod = rnd(L, D), rnd(6, D, std=0.2)
        self.gains = [1 + rnd(D, std=0.1) for _ in range(4)]
        self.qk_gain, self.pos = 1 + rnd(2, 128, std=0.1), torch.arange(L, device=dev, dtype=torch.int32)
        self.pos = torch.stack([self.pos // 64, self.pos // 8 % 8, self.pos % 8], 1).contiguous()
        w = dict(qkv=bf(3 * D, D, std=0.05), o=bf(D, D, std=0.05), gu=bf(2 * F, D, std=0.05), down=bf(D, F, std=0.03))
        self.w = {k: h3.fp4_rows(*x.shape, format=fmt) for k, x in w.items()}
        for k, x in w.items():
            h3.quantize_fp4_rows(x, self.w[k])
        self.x4, self.f4 = h3.fp4_rows(L, D, fmt), h3.fp4_rows(L, F, fmt)
        self.a4, self.h24 = h3.fp4_rows(L, D, fmt), h3.fp4_rows(L, D, fmt)
        self.h1, self.h2, self.o, self.down = (empty(L, D) for _ in range(4))
        self.r1, self.r2 = (empty(L, D, dtype=torch.float32) for _ in range(2))
        self.qkv, self.q, self.k = empty(L, 3, H, 128), empty(L, H, 128), empty(L, H, 128)
        self.scores, self.ids = empty(H, NQ, NK, dtype=torch.float32), empty(H, NQ, MOST, dtype=torch.int32)
        self.counts, self.a, self.s = empty(H, NQ, dtype=torch.int32), empty(L, H, 128), empty(L, F)
        self.ws = empty(h3.block_scores_workspace_bytes(L, L, H, H, KB), dtype=torch.uint8)

    def run(self):
        h3, m = self.h3, self.mod
        h3.sandwich_norm(self.r, normed=self.h1, pre_gain=self.gains[0], shift=m[0], scale=m[1], rms=True)
        h3.quantize_fp4_rows(self.h1, self.x4)
        h3.linear_fp4(self.x4, self.w["qkv"], self.qkv.view(L, 3 * D))
        self.q.copy_(self.qkv[:, 0])
        self.k.copy_(self.qkv[:, 1])
        h3.qk_norm_rope(self.q, self.k, self.qk_gain[0], self.qk_gain[1], self.pos, (32, 48, 48))
        h3.block_scores(self.q, self.k, self.scores, self.ws, k_block=KB)
        h3.block_select(self.scores, self.ids, self.counts, keep_first=1, keep_last=1)
        h3.attention_blocks(self.q, self.k, self.qkv[:, 2], self.a, self.ids, self.counts, k_block=KB)
        h3.quantize_fp4_rows(self.a.view(L, D), self.a4)
        h3.linear_fp4(self.a4, self.w["o"], self.o)
        h3.sandwich_norm(self.r, self.o, self.h2, resid_out=self.r1, post_gain=self.gains[1], gate=m[2],
                         pre_gain=self.gains[2], shift=m[3], scale=m[4], rms=True)
        h3.quantize_fp4_rows(self.h2, self.h24)
        h3.linear_swiglu_fp4(self.h24, self.w["gu"], self.s)
        h3.quantize_fp4_rows(self.s, self.f4)
        h3.linear_fp4(self.f4, self.w["down"], self.down)
        h3.sandwich_norm(self.r1, self.down, resid_out=self.r2, post_gain=self.gains[3], gate=m[5], rms=True)

    def check(self):
        m, rows = self.mod, np.arange(L)
        norm = dict(resid=self.r, delta=None, post_norm=False, resid_scale=1.0, rms=True, eps=1e-6, seg=None,
                    pre_gain=self.gains[0], shift=m[0], scale=m[1])
        check_norm(None, self.h1, norm, L, "h1")
        for x, q in ((self.h1, self.x4), (self.a.view(L, D), self.a4), (self.h2, self.h24), (self.s, self.f4)):
            code, byte, row = reference(x.double().cpu().numpy(), self.fmt)
            got = unpack(q)
            assert np.array_equal(got[0], code) and np.array_equal(got[1], byte)
            assert row is None or np.array_equal(q.row_scale.double().cpu().numpy(), row)
        check_linear(self.qkv.view(L, 3 * D), self.x4, self.w["qkv"], rows, "qkv")
        s, mag = ref_scores(self.q, self.k, KB, 128 ** -0.5)
        assert ((self.scores.double() - s).abs() <= (212 * 2.0 ** -24 + 2.0 ** -20) * mag).all()
        ids, counts = ref_select(self.scores.view(-1, NK).cpu().numpy(), MOST, 1, 1)
        assert np.array_equal(self.ids.view(-1, MOST).cpu().numpy(), ids)
        assert np.array_equal(self.counts.view(-1).cpu().numpy(), counts)
        a, mag = ref_attention(self.q, self.k, self.qkv[:, 2], self.ids, self.counts, KB, 128 ** -0.5)
        assert ((self.a.double() - a).abs() <= 2.0 ** -8 * a.abs() + (2.0 ** -8 + 2.0 ** -10 + 2.0 ** -11) * mag).all()
        check_linear(self.o, self.a4, self.w["o"], rows, "o")
        check_norm(self.r1, self.h2, norm | dict(delta=self.o, post_norm=True, post_gain=self.gains[1], gate=m[2],
                                                 pre_gain=self.gains[2], shift=m[3], scale=m[4]), L, "r1")
        gu = torch.empty(L, 2 * F, dtype=torch.bfloat16, device=dev)
        self.h3.linear_fp4(self.h24, self.w["gu"], gu)
        check_linear(gu, self.h24, self.w["gu"], rows, "gate and up")
        check_swiglu(self.s, gu)
        check_linear(self.down, self.f4, self.w["down"], rows, "down")
        check_norm(self.r2, None, dict(norm, resid=self.r1, delta=self.down, post_norm=True, post_gain=self.gains[3],
                                       gate=m[5], pre_gain=None, shift=None, scale=None), L, "r2")


@pytest.mark.parametrize("fmt", ["mx", "nv"])
def test_block_and_its_graph(h3lib, fmt):
    b = Block(h3lib, fmt, 1)
    b.run()
    h3lib.check_device_error()
    b.check()
    first, r = b.r2.clone(), b.r.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        b.run()
    b.r.copy_(r.flip(0))
    graph.replay()
    torch.cuda.synchronize()
    h3lib.check_device_error()
    b.check()
    assert not torch.equal(b.r2, first)
    b.r.copy_(r)
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(b.r2, first)
    # and back to back without a graph, each launch overlapping the one before it
    for _ in range(20):
        b.run()
    torch.cuda.synchronize()
    h3lib.check_device_error()
    assert torch.equal(b.r2, first)
