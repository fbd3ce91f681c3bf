"""Launches that overlap the end of the kernel before them: a chain of calls, among them ones of the paged
cache and of torch, gives the bits that it gives with a wait after every call, and calls of several
streams at once, with outputs and workspaces of their own, give those of one call after another."""
import pytest
import torch

pytestmark = pytest.mark.gpu
dev = "cuda"


def gen(seed):
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    return g


def rnd(g, *s, std=1.0):
    return (torch.randn(*s, generator=g, device=dev) * std).to(torch.bfloat16)


def empty(*s, dtype=torch.bfloat16):
    return torch.empty(*s, dtype=dtype, device=dev)


@pytest.mark.parametrize("T,keys,prefix", [(8, 700, 0), (200, 3000, 0), (8, 130, 2000), (1, 65, 0)])
@pytest.mark.parametrize("fmt", ["mx", "nv"])
def test_decoding_chain(h3lib, fmt, T, keys, prefix):
    H, D, B, page = 4, 512, (T if T <= 8 else 1), 64
    g = gen(T + keys)
    per = -(-keys // page)
    npre = -(-prefix // page)
    k, v = (rnd(g, B * per + npre, H, page, 128) for _ in range(2))
    cache = h3lib.kv_cache(k, v)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=dev)
    rows = T // B
    batch = h3lib.kv_batch(i32([i * rows for i in range(B + 1)]), i32([keys] * B),
                           torch.arange(B * per, dtype=torch.int32, device=dev).view(B, per), T)
    pages = torch.arange(B * per, B * per + npre, dtype=torch.int32, device=dev)
    ws = empty(h3lib.attention_paged_workspace_bytes(T, H, prefix), dtype=torch.uint8)
    w = [h3lib.fp4_rows(D, D, format=fmt) for _ in range(2)]
    for x in w:
        h3lib.quantize_fp4_rows(rnd(g, D, D, std=0.06), x)
    start, gain = rnd(g, T, H, 128), 1 + torch.randn(D, generator=g, device=dev) * 0.1
    resid = torch.randn(T, D, generator=g, device=dev)

    def chain(after):
        q, o, y, h, r = start.clone(), empty(T, H, 128), empty(T, D), empty(T, D), resid.clone()
        x4 = h3lib.fp4_rows(T, D, format=fmt)
        out = []
        torch.cuda.synchronize()
        for i in range(6):
            if prefix:
                h3lib.attention_paged_prefix(q, o, cache, batch, pages, prefix, ws)
            else:
                h3lib.attention_paged(q, o, cache, batch, ws)
            after()
            h3lib.quantize_fp4_rows(o.view(T, D), x4)
            after()
            h3lib.linear_fp4(x4, w[0], y)
            after()
            h3lib.sandwich_norm(r, y, h, post_gain=gain, pre_gain=gain, rms=i % 2 == 1)
            after()
            h3lib.quantize_fp4_rows(h, x4)
            after()
            h3lib.linear_fp4(x4, w[1], q.view(T, D))
            after()
            q.mul_(4.0)   # a kernel that knows nothing of the others
            after()
            out.append((q.clone(), r.clone()))
        torch.cuda.synchronize()
        h3lib.check_device_error()
        return out

    want = chain(torch.cuda.synchronize)
    for _ in range(10):
        for a, b in zip(chain(lambda: None), want):
            assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_streams_at_once(h3lib):
    H, Hkv, kb = 8, 4, 64

    def work(seed, Lq, Lk, most, N, K, fmt):
        g = gen(seed)
        q, kk, vv = rnd(g, Lq, H, 128), rnd(g, Lk, Hkv, 128), rnd(g, Lk, Hkv, 128)
        x, w = rnd(g, Lq, K), h3lib.fp4_rows(N, K, format=fmt)
        h3lib.quantize_fp4_rows(rnd(g, N, K, std=0.03), w)
        nq, nk = -(-Lq // h3lib.QUERY_BLOCK), -(-Lk // kb)
        s, o, y = empty(H, nq, nk, dtype=torch.float32), empty(Lq, H, 128), empty(Lq, N)
        ids, counts = empty(H, nq, most, dtype=torch.int32), empty(H, nq, dtype=torch.int32)
        ws = empty(h3lib.block_scores_workspace_bytes(Lq, Lk, H, Hkv, kb), dtype=torch.uint8)
        x4 = h3lib.fp4_rows(Lq, K, format=fmt)
        h, r = empty(Lq, K), torch.randn(Lq, K, generator=g, device=dev)

        def run():
            h3lib.block_scores(q, kk, s, ws, k_block=kb)
            h3lib.block_select(s, ids, counts, keep_last=1)
            h3lib.attention_blocks(q, kk, vv, o, ids, counts, k_block=kb)
            h3lib.sandwich_norm(r, normed=h, rms=True)
            h3lib.quantize_fp4_rows(h, x4)
            h3lib.linear_fp4(x4, w, y)
            return o, y, s, ids, counts
        return run

    # few items and tiles (clusters that share them), and many
    runs = [work(1, 22, 20000, 40, 5376, 5376, "nv"), work(2, 3000, 3000, 9, 2048, 1056, "mx"),
            work(3, 200, 9000, 24, 2560, 4096, "mx")]
    want = []
    for f in runs:
        want.append([t.clone() for t in f()])
        torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in runs]
    for _ in range(10):
        got = []
        for f, st in zip(runs, streams):
            with torch.cuda.stream(st):
                for _ in range(4):
                    outs = f()
                got.append(outs)
        torch.cuda.synchronize()
        h3lib.check_device_error()
        for a, b in zip(got, want):
            assert all(torch.equal(x, y) for x, y in zip(a, b))
