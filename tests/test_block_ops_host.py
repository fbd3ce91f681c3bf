"""Refusals of the norms around a branch, the 4-bit rows and products and the block-sparse
attention, on the host: each call returns its status and message and launches nothing."""
import ctypes

import pytest
import torch

from dit_transformer_block_gb300 import build as B
from dit_transformer_block_gb300 import h3

P, Q, R_, S_ = (ctypes.c_void_p(4096 * i) for i in (1, 2, 3, 4))  # never dereferenced
PM = ctypes.c_void_p(4096 + 4)
NULL = None
F = ctypes.c_float


@pytest.fixture(scope="module")
def lib():
    B.build()
    return h3.lib()


def norm(lib, **kw):
    a = dict(resid=P, delta=Q, resid_out=P, normed=R_, post_norm=1, post_gain=S_, gate=S_, resid_scale=F(1.0),
             pre_gain=NULL, shift=S_, scale=S_, seg=NULL, num_seg=1, seg_stride=0, rms=0, S=10, L=0, D=512,
             eps=F(1e-6), stream=NULL)
    assert set(kw) <= set(a)
    return lib.h3_sandwich_norm(*(a | kw).values())


@pytest.mark.parametrize("status,text,kw", [
    (0, "", {}),
    (0, "", dict(delta=NULL, post_norm=0, post_gain=NULL, gate=NULL, resid_out=NULL)),
    (0, "", dict(normed=NULL, shift=NULL, scale=NULL)),
    (1, "L=11", dict(L=11)),
    (1, "negative", dict(S=-1)),
    (1, "resid is NULL", dict(resid=NULL)),
    (1, "nothing to do", dict(resid_out=NULL, normed=NULL)),
    (1, "resid_out is NULL", dict(resid_out=NULL)),
    (1, "resid_out is NULL", dict(resid_out=NULL, delta=NULL, post_norm=0, post_gain=NULL, gate=NULL,
                                  resid_scale=F(0.5))),
    (1, "nothing to do", dict(normed=NULL, delta=NULL, post_norm=0, post_gain=NULL, gate=NULL, shift=NULL,
                              scale=NULL)),
    (1, "without delta", dict(delta=NULL)),
    (1, "without post_norm", dict(post_norm=0)),
    (1, "without normed", dict(normed=NULL)),
    (2, "multiple of 8", dict(D=500)),
    (2, "multiple of 8", dict(D=0)),
    (2, "8192", dict(D=8200)),
    (1, "eps", dict(eps=F(-1.0))),
    (1, "finite", dict(resid_scale=F(float("nan")))),
    (3, "aligned", dict(delta=PM)),
    (3, "aligned", dict(scale=PM)),
    (1, "num_seg", dict(seg=Q, num_seg=0, seg_stride=512)),
    (1, "seg_stride", dict(seg=Q, num_seg=2, seg_stride=508)),
    (1, "seg_stride", dict(seg=Q, num_seg=2, seg_stride=514)),
    (3, "seg", dict(seg=ctypes.c_void_p(4097), num_seg=2, seg_stride=512)),
    (1, "overlaps", dict(normed=Q)),
    (1, "delta", dict(resid_out=Q)),
])
def test_sandwich_norm(lib, status, text, kw):
    assert norm(lib, **kw) == status, h3.last_error()
    assert text in h3.last_error()


def test_fp4_scale_bytes(lib):
    # tiles of 128 rows x 4 scales
    assert h3.fp4_scale_bytes(1, 32, "mx") == 512 and h3.fp4_scale_bytes(1, 32, "nv") == 512
    assert h3.fp4_scale_bytes(129, 160, "mx") == 2 * 2 * 512
    assert h3.fp4_scale_bytes(129, 160, "nv") == 2 * 3 * 512
    assert h3.fp4_scale_bytes(16128, 5376, "nv") == 16128 * 5376 // 16
    assert h3.fp4_scale_bytes(0, 64, "nv") == 512
    for a in ((-1, 64, 1), (4, 48, 1), (4, 0, 0), (4, 64, 2)):
        assert lib.h3_fp4_scale_bytes(*a) == 0 and h3.last_error()


def test_quantize_fp4_rows(lib):
    f = lib.h3_quantize_fp4_rows
    assert f(P, 64, Q, R_, S_, 0, 64, 1, NULL) == 0
    for status, text, a in (
            (2, "multiple of 32", (P, 48, Q, R_, S_, 4, 48, 1)), (2, "16384", (P, 16416, Q, R_, S_, 4, 16416, 1)),
            (1, "format", (P, 64, Q, R_, S_, 4, 64, 3)), (1, "R=-2", (P, 64, Q, R_, S_, -2, 64, 1)),
            (1, "row_scale", (P, 64, Q, R_, NULL, 4, 64, 1)), (1, "row_scale", (P, 64, Q, R_, S_, 4, 64, 0)),
            (1, "NULL", (NULL, 64, Q, R_, S_, 4, 64, 1)), (1, "NULL", (P, 64, Q, NULL, S_, 4, 64, 1)),
            (1, "stride", (P, 56, Q, R_, S_, 4, 64, 1)), (3, "aligned", (P, 68, Q, R_, S_, 4, 64, 1)),
            (3, "aligned", (PM, 64, Q, R_, S_, 4, 64, 1)), (3, "128", (P, 64, Q, ctypes.c_void_p(4096 + 64), S_, 4, 64, 1)),
            (1, "overlap", (P, 64, P, R_, S_, 4, 64, 1))):
        assert f(*a, NULL) == status, (a, h3.last_error())
        assert text in h3.last_error()


@pytest.mark.parametrize("name,N,odd", [("h3_linear_fp4", 40, 44), ("h3_linear_swiglu_fp4", 128, 64)])
def test_fp4_products(lib, name, N, odd):
    f = getattr(lib, name)
    X, W = (P, P, P), (Q, Q, Q)
    assert f(*X, *W, R_, 8, 0, N, 64, 1, NULL) == 0
    assert f(P, P, NULL, Q, Q, NULL, R_, 8, 0, N, 64, 0, NULL) == 0
    for status, text, a in (
            (1, "L=9", (*X, *W, R_, 8, 9, N, 64, 1)), (2, "multiple of", (*X, *W, R_, 8, 8, odd, 64, 1)),
            (2, "multiple of 32", (*X, *W, R_, 8, 8, N, 80, 1)), (1, "format", (*X, *W, R_, 8, 8, N, 64, -1)),
            (1, "NULL", (NULL, P, P, *W, R_, 8, 8, N, 64, 1)), (1, "NULL", (*X, Q, NULL, Q, R_, 8, 8, N, 64, 1)),
            (1, "row scales", (P, P, NULL, *W, R_, 8, 8, N, 64, 1)), (1, "row scales", (*X, *W, R_, 8, 8, N, 64, 0)),
            (3, "aligned", (PM, P, P, *W, R_, 8, 8, N, 64, 1)), (3, "aligned", (*X, Q, Q, PM, R_, 8, 8, N, 64, 1)),
            (1, "overlaps", (*X, *W, P, 8, 8, N, 64, 1)), (2, "16384", (*X, *W, R_, 8, 8, N, 16416, 1)), (2, "2^30", (*X, *W, R_, (1 << 30) + 1, (1 << 30) + 1, N, 64, 1))):
        assert f(*a, NULL) == status, (a, h3.last_error())
        assert text in h3.last_error()


def test_block_scores_and_workspace(lib):
    n = lib.h3_block_scores_workspace_bytes
    assert n(257, 129, 4, 2, 64) == (2 * 4 + 3 * 2) * 512 and n(0, 0, 4, 2, 64) > 0
    assert n(4097, 129, 4, 2, 64) == (17 * 4 + 3 * 2) * 1024   # means in two parts
    for a in ((-1, 5, 4, 2, 64), (5, 5, 4, 3, 64), (5, 5, 0, 1, 64), (5, 5, 4, 2, 32), (5, (1 << 26) + 1, 4, 2, 64)):
        assert n(*a) == 0 and h3.last_error()
    f = lib.h3_block_scores
    ok = dict(q=P, ld_q=512, k=Q, ld_k=256, scores=R_, Lq=300, Lk=200, H=4, Hkv=2, Dh=128, kb=64, scale=F(0.1), ws=S_,
              n=1 << 20, stream=NULL)
    assert f(*(ok | dict(Lq=0)).values()) == 0 and f(*(ok | dict(Lk=0)).values()) == 0
    for status, text, kw in (
            (1, "multiple", dict(Hkv=3)), (2, "k_block", dict(kb=100)), (2, "head_dim", dict(Dh=64)),
            (1, "negative", dict(Lk=-1)), (1, "q is NULL", dict(q=NULL)), (3, "aligned", dict(ld_q=516)),
            (1, "row stride", dict(ld_k=248)), (1, "scores", dict(scores=NULL)), (4, "workspace", dict(n=100)),
            (4, "workspace", dict(ws=NULL)), (3, "256", dict(ws=ctypes.c_void_p(4096 + 128))),
            (2, "2^31", dict(Lq=1 << 26, Lk=1 << 26)), (1, "finite", dict(scale=F(float("inf"))))):
        assert f(*(ok | kw).values()) == status, (kw, h3.last_error())
        assert text in h3.last_error()


def test_block_select(lib):
    f = lib.h3_block_select
    assert f(P, Q, R_, 0, 10, 4, 0, 0, NULL) == 0 and f(P, Q, R_, 5, 0, 4, 0, 0, NULL) == 0
    for status, text, a in (
            (1, "rows", (P, Q, R_, -1, 10, 4, 0, 0)), (1, "max_blocks", (P, Q, R_, 5, 10, 0, 0, 0)),
            (2, "2^20", (P, Q, R_, 5, (1 << 20) + 1, 4, 0, 0)), (1, "keep_first", (P, Q, R_, 5, 10, 4, 3, 2)),
            (1, "keep_first", (P, Q, R_, 5, 10, 4, -1, 0)), (1, "NULL", (P, NULL, R_, 5, 10, 4, 0, 0)),
            (2, "2^31", (P, Q, R_, 1 << 20, 10, 1 << 12, 0, 0)), (2, "2^31", (P, Q, R_, 1 << 20, 1 << 12, 4, 0, 0)),
            (1, "keep_first", (P, Q, R_, 5, 10, 4, 2147483647, 2147483647)),
            (3, "aligned", (ctypes.c_void_p(4097), Q, R_, 5, 10, 4, 0, 0))):
        assert f(*a, NULL) == status, (a, h3.last_error())
        assert text in h3.last_error()


def test_attention_blocks(lib):
    f = lib.h3_attention_blocks
    V, O, I = (ctypes.c_void_p(4096 * i) for i in (5, 6, 7))
    ok = dict(q=P, ld_q=512, k=Q, ld_k=256, v=V, ld_v=256, o=O, ld_o=512, ids=I, counts=I, most=4, Lq=300, Lk=200, H=4,
              Hkv=2, Dh=128, kb=64, scale=F(0.1), stream=NULL)
    assert f(*(ok | dict(Lq=0)).values()) == 0
    for status, text, kw in (
            (1, "multiple", dict(Hkv=3)), (2, "k_block", dict(kb=16)), (2, "head_dim", dict(Dh=256)),
            (2, "2^20", dict(Lq=(1 << 28) + 1)),
            (1, "negative", dict(Lq=-1)), (1, "max_blocks", dict(most=0)), (1, "scale", dict(scale=F(0.0))),
            (1, "scale", dict(scale=F(float("nan")))), (1, "o is q", dict(o=P)), (1, "o is k", dict(o=Q)),
            (1, "v is NULL", dict(v=NULL)), (3, "aligned", dict(ld_v=260)), (1, "row stride", dict(ld_o=504)),
            (1, "ids", dict(ids=NULL)), (3, "4-byte", dict(counts=ctypes.c_void_p(4097))),
            (2, "65535", dict(H=65536, Hkv=1)), (2, "2^31", dict(Lq=1 << 28, most=1 << 12)),
            (2, "2^17", dict(most=2049)), (2, "2^17", dict(most=1025, kb=128))):
        assert f(*(ok | kw).values()) == status, (kw, h3.last_error())
        assert text in h3.last_error()


def test_binding_refuses_before_the_library(lib):
    bf, i32 = torch.bfloat16, torch.int32
    t = lambda *s, dtype=torch.float32: torch.zeros(*s, dtype=dtype)
    with pytest.raises((ValueError, TypeError)):
        h3.sandwich_norm(t(4, 64, dtype=bf))
    with pytest.raises(ValueError, match="format"):
        h3.fp4_rows(4, 64, format="int4", device="cpu")
    with pytest.raises(h3.H3Error, match="multiple of 32"):
        h3.fp4_rows(4, 48, device="cpu")
    for k_block in (0, 32, 256):
        with pytest.raises(ValueError, match="k_block"):
            h3._block_shape(10, 10, 1, k_block)
    with pytest.raises(ValueError, match="wanted"):
        h3.block_select(t(2, 3, 9), t(2, 3, 4, dtype=i32), t(2, 4, dtype=i32))
    # tensors that are not on the current CUDA device
    for call in (lambda: h3.sandwich_norm(t(4, 64)),
                 lambda: h3.block_select(t(2, 9), t(2, 4, dtype=i32), t(2, dtype=i32)),
                 lambda: h3.block_scores(t(4, 1, 128, dtype=bf), t(4, 1, 128, dtype=bf), t(1, 1, 1), t(8)),
                 lambda: h3.quantize_fp4_rows(t(4, 64, dtype=bf), h3.fp4_rows(4, 64, device="meta"))):
        with pytest.raises(ValueError, match="CUDA device"):
            call()
