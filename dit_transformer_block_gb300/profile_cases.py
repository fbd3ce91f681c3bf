"""Small, fixed cases for ncu captures of the library's kernels.

    python -m dit_transformer_block_gb300.profile_cases [attention] [gemm] [elementwise] [fp8] [sage] [paged]
                                                        [norms] [fp4] [blocks]

Each selected kernel runs twice on inputs larger than L2 (129 MB) but a few
hundred MB in total, so that an `ncu --set full -k <kernel> -s 1 -c 1`
capture of the second launch ends within a minute or two:
  attention   S = L = 16384, 42 heads x 128 (q, k, v, o: 704 MB)
  gemm        M = 8192, N = 16128, K = 5376 (the QKV projection shape; 520 MB),
              plain and with Q/K RMSNorm + RoPE in the epilogue (after its RoPE
              table), then the down projection shape M = 8192, N = 5376,
              K = 14336 with the residual update in the epilogue (565 MB)
  elementwise qk_norm_rope on 16384 x 42 x 128 (interleaved, then split-half
              pairs), SwiGLU on 16384 x 2 x 14336,
              modulation/LN/residual on 16384 x 5376
  fp8         FP8 GEMM (QKV shape, M = 8192), per-row FP8 quantisation of
              8192 x 5376, SAGE quantisation and FP8 attention at S = L = 16384
  sage        SAGE quantisation alone (K mean, V absmax, Q/K tile and V codes)
              at S = L = 16384, 42 heads
  paged       the paged cache: 16384 rows appended (42 heads, interleaved pairs),
              1896 rows against 16384 keys (42 heads), 64 rows of 4096 keys (40
              heads on 8), and 512 rows of 256 keys (32 heads on 8)
  norms       norms around a gated branch, 16384 x 5376
  fp4         4-bit rows: quantisation of 16384 x 5376 (both formats), the QKV
              projection shape with M = 8192 (both), SwiGLU M = 4096, F = 14336,
              16 rows of the QKV shape (63 tiles, a pair of CTAs each), and 22 rows of
              the output projection (21 tiles, three pairs each)
  blocks      16384 rows of 42 heads: scores of key blocks of 64, selection of 56
              per query block, attention over them; and selection of 92 of 919
              blocks in 9660 rows
"""
from __future__ import annotations

import sys

import torch

from dit_transformer_block_gb300 import build, h3


def main(argv):
    which = set(argv) or {"attention", "gemm", "elementwise", "fp8", "sage", "paged", "norms", "fp4", "blocks"}
    build.build()
    h3.lib()
    dev = "cuda"
    g = torch.Generator(device=dev)
    g.manual_seed(0)
    rnd = lambda *s, std=1.0: (torch.randn(*s, generator=g, device=dev) * std).to(torch.bfloat16)
    runs = []
    if "attention" in which:
        S = 16384
        q, k, v = rnd(S, 42, 128), rnd(S, 42, 128), rnd(S, 42, 128)
        o = torch.empty_like(q)
        runs.append(lambda: h3.attention_varlen(q, k, v, o, S))
    if "gemm" in which:
        M, N, K = 8192, 16128, 5376
        x, w = rnd(M, K), rnd(N, K, std=0.02)
        y = torch.empty(M, N, device=dev, dtype=torch.bfloat16)
        runs.append(lambda: h3.linear(x, w, y, M))
        from dit_transformer_block_gb300 import inputs as I
        pos = I.positions_3d(M, M, grid=(31, 24, 79), n_tail=22).to(dev)
        tab = torch.empty(M, 64, 2, device=dev)
        gains = torch.ones(128, device=dev)
        runs.append(lambda: h3.rope_table(pos, (32, 48, 48), tab, M))
        runs.append(lambda: h3.linear_qk_norm_rope(x, w, y, gains, gains, tab, (32, 48, 48), M))
        xd, wd = rnd(M, 14336), rnd(5376, 14336, std=0.02)
        rd = torch.randn(M, 5376, generator=g, device=dev)
        gate = torch.randn(5376, generator=g, device=dev) * 0.1
        runs.append(lambda: h3.linear_residual(xd, wd, rd, gate, M))
    if "elementwise" in which:
        S = 16384
        qq, kk = rnd(S, 42, 128), rnd(S, 42, 128)
        ones = torch.ones(128, device=dev)
        pos = torch.zeros(S, 3, dtype=torch.int32, device=dev)
        gu = rnd(S, 2 * 14336)
        u = torch.empty(S, 14336, device=dev, dtype=torch.bfloat16)
        r = torch.randn(S, 5376, generator=g, device=dev)
        d = rnd(S, 5376)
        hh = torch.empty(S, 5376, device=dev, dtype=torch.bfloat16)
        mod = torch.randn(6, 5376, generator=g, device=dev) * 0.1
        runs.append(lambda: h3.qk_norm_rope(qq, kk, ones, ones, pos, (32, 48, 48), S))
        runs.append(lambda: h3.qk_norm_rope(qq, kk, ones, ones, pos, (32, 48, 48), S, pairing=1))
        runs.append(lambda: h3.swiglu(gu, u, S))
        runs.append(lambda: h3.mod_norm_residual(r, d, mod[2], mod[3], mod[4], hh, S))
    if "fp8" in which:
        M, N, K = 8192, 16128, 5376
        x8, w8 = rnd(M, K), rnd(N, K, std=0.02)
        qx = torch.empty(M, K, dtype=torch.uint8, device=dev)
        sx = torch.empty(M, device=dev)
        qw = torch.empty(N, K, dtype=torch.uint8, device=dev)
        sw = torch.empty(N, device=dev)
        h3.quantize_fp8_rows(w8, qw, sw)
        y8 = torch.empty(M, N, device=dev, dtype=torch.bfloat16)
        runs.append(lambda: h3.quantize_fp8_rows(x8, qx, sx))
        runs.append(lambda: h3.linear_fp8(qx, sx, qw, sw, y8, M))
        S = 16384
        qa, ka, va = rnd(S, 42, 128), rnd(S, 42, 128), rnd(S, 42, 128)
        oa = torch.empty_like(qa)
        ops = h3.sage_quantize(qa, ka, va, S)
        runs.append(lambda: h3.attention_fp8(ops, oa, S))
    if "sage" in which:
        S = 16384
        qs, ks, vs = rnd(S, 42, 128), rnd(S, 42, 128), rnd(S, 42, 128)
        runs.append(lambda: h3.sage_quantize(qs, ks, vs, S))
    if "paged" in which:
        i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=dev)

        def pool(B, keys, Hkv, page=64):
            n = keys // page
            c = h3.kv_cache(rnd(B * n, Hkv, page, 128), rnd(B * n, Hkv, page, 128))
            order = torch.randperm(B * n, generator=g, device=dev).to(torch.int32).view(B, n)
            return c, order

        def attend(B, rows, keys, H, Hkv):
            c, table = pool(B, keys, Hkv)
            T = B * rows
            b = h3.kv_batch(i32([i * rows for i in range(B + 1)]), i32([keys] * B), table, T)
            q, o = rnd(T, H, 128), torch.empty(T, H, 128, device=dev, dtype=torch.bfloat16)
            ws = torch.empty(h3.attention_paged_workspace_bytes(T, H), device=dev, dtype=torch.uint8)
            runs.append(lambda: h3.attention_paged(q, o, c, b, ws))

        T = 16384
        ca, table = pool(1, T, 42)
        ba = h3.kv_batch(i32([0, T]), i32([T]), table, T)
        qkv = rnd(T, 3, 42, 128)
        qp, ones3 = torch.empty(T, 42, 128, device=dev, dtype=torch.bfloat16), torch.ones(128, device=dev)
        pos3 = torch.zeros(T, 3, dtype=torch.int32, device=dev)
        runs.append(lambda: h3.kv_append_paged(qkv[:, 0], qkv[:, 1], qkv[:, 2], qp, ca, ba, pos3,
                                               (32, 48, 48), ones3, ones3))
        attend(1, 1896, 16384, 42, 42)
        attend(64, 1, 4096, 40, 8)
        attend(512, 1, 256, 32, 8)
    if "norms" in which:
        S, D = 16384, 5376
        rn, dn = torch.randn(S, D, generator=g, device=dev), rnd(S, D)
        on, hn = torch.empty_like(rn), torch.empty_like(dn)
        vecs = torch.randn(5, D, generator=g, device=dev) * 0.1
        runs.append(lambda: h3.sandwich_norm(rn, dn, hn, resid_out=on, post_gain=vecs[0], gate=vecs[1],
                                             pre_gain=vecs[2], shift=vecs[3], scale=vecs[4], rms=True))
    if "fp4" in which:
        def rows(R, K, form, std=1.0):
            x, q = rnd(R, K, std=std), h3.fp4_rows(R, K, format=form)
            h3.quantize_fp4_rows(x, q)
            return x, q

        def product(M, N, K, form, swiglu=False):
            xq, wq = rows(M, K, form)[1], rows(2 * N if swiglu else N, K, form, 0.02)[1]
            yq = torch.empty(M, N, device=dev, dtype=torch.bfloat16)
            fn = h3.linear_swiglu_fp4 if swiglu else h3.linear_fp4
            runs.append(lambda: fn(xq, wq, yq))

        def quantise(R, K, form):
            xq, qq4 = rows(R, K, form)
            runs.append(lambda: h3.quantize_fp4_rows(xq, qq4))

        for form in ("mx", "nv"):
            quantise(16384, 5376, form)
        for form in ("mx", "nv"):
            product(8192, 16128, 5376, form)
        product(4096, 14336, 5376, "mx", swiglu=True)
        product(16, 16128, 5376, "nv")
        product(22, 5376, 5376, "mx")
    if "blocks" in which:
        S, H, most = 16384, 42, 56
        qb, kb, vb = rnd(S, H, 128), rnd(S, H, 128), rnd(S, H, 128)
        ob = torch.empty_like(qb)
        nq, nk = S // h3.QUERY_BLOCK, S // 64
        sc = torch.empty(H, nq, nk, device=dev)
        ids = torch.empty(H, nq, most, dtype=torch.int32, device=dev)
        counts = torch.empty(H, nq, dtype=torch.int32, device=dev)
        wsb = torch.empty(h3.block_scores_workspace_bytes(S, S, H, H, 64), device=dev, dtype=torch.uint8)
        runs.append(lambda: h3.block_scores(qb, kb, sc, wsb, k_block=64))
        runs.append(lambda: h3.block_select(sc, ids, counts, keep_first=1, keep_last=1))
        runs.append(lambda: h3.attention_blocks(qb, kb, vb, ob, ids, counts, k_block=64))
        many = torch.randn(9660, 919, generator=g, device=dev)
        many_ids = torch.empty(9660, 92, dtype=torch.int32, device=dev)
        many_counts = torch.empty(9660, dtype=torch.int32, device=dev)
        runs.append(lambda: h3.block_select(many, many_ids, many_counts, keep_first=1, keep_last=1))
    torch.cuda.synchronize()
    for _ in range(2):
        for fn in runs:
            fn()
    torch.cuda.synchronize()
    h3.check_device_error()
    print("ok")


if __name__ == "__main__":
    main(sys.argv[1:])
