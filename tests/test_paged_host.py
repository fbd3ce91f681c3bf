"""Host-side checks of the paged key/value cache calls: every refusal with its
status before any launch, empty calls, workspace sizes, and the binding's own
checks of shapes, types and devices. No GPU."""
import ctypes

import pytest
import torch

from dit_transformer_block_gb300 import build as B
from dit_transformer_block_gb300 import h3

NULL = None
A = 4096              # 16- and 256-byte aligned fake device address (never dereferenced)
P = ctypes.c_void_p(A)
PM = ctypes.c_void_p(A + 2)
INVALID, UNSUPPORTED, MISALIGNED, WORKSPACE = 1, 2, 3, 4


@pytest.fixture(scope="module")
def lib():
    B.build()
    return h3.lib()


def cache(**kw):
    d = dict(k=A, v=A, num_pages=10, page_size=64, Hkv=4, Dh=128)
    d.update(kw)
    return h3.KvCache(*d.values())


def batch(**kw):
    d = dict(T=6, B=2, max_pages=3, cu_q=A, kv_len=A, page_table=A)
    d.update(kw)
    return h3.KvBatch(*d.values())


def attend(lib, c=None, b=None, **kw):
    d = dict(q=P, ld_q=8 * 128, o=P, ld_o=8 * 128, H=8, scale=0.1, causal=0, prefix=P,
             prefix_len=100, ws=P, bytes=None)
    d.update(kw)
    c, b = c or cache(), b or batch()
    if d["bytes"] is None:
        d["bytes"] = lib.h3_attention_paged_workspace_bytes(max(b.T, 0), 8, 100)
    return lib.h3_attention_paged_prefix(
        d["q"], d["ld_q"], d["o"], d["ld_o"], d["H"], ctypes.c_float(d["scale"]), d["causal"],
        ctypes.addressof(c), ctypes.addressof(b), d["prefix"], d["prefix_len"], d["ws"],
        d["bytes"], NULL)


def append(lib, c=None, b=None, axis=(32, 48, 48), **kw):
    d = dict(q=P, ld_q=8 * 128, k=P, ld_k=4 * 128, v=P, ld_v=4 * 128, q_out=ctypes.c_void_p(A * 2),
             H=8, qg=P, kg=P, pos=P, pairing=0, theta=1e4, eps=1e-6)
    d.update(kw)
    c, b = c or cache(), b or batch()
    ax = ctypes.cast((ctypes.c_int * 3)(*axis), ctypes.c_void_p) if axis is not None else None
    return lib.h3_kv_append_paged(
        d["q"], d["ld_q"], d["k"], d["ld_k"], d["v"], d["ld_v"], d["q_out"], d["H"], d["qg"],
        d["kg"], d["pos"], ax, d["pairing"], ctypes.c_float(d["theta"]), ctypes.c_float(d["eps"]),
        ctypes.addressof(c), ctypes.addressof(b), NULL)


CACHE_AND_BATCH = [
    (dict(k=None), {}, INVALID), (dict(v=None), {}, INVALID),
    (dict(k=A + 2), {}, MISALIGNED), (dict(Dh=64), {}, UNSUPPORTED),
    (dict(page_size=48), {}, UNSUPPORTED), (dict(page_size=8), {}, UNSUPPORTED),
    (dict(page_size=256), {}, UNSUPPORTED), (dict(page_size=0), {}, UNSUPPORTED),
    (dict(num_pages=0), {}, INVALID), (dict(Hkv=0), {}, INVALID), (dict(Hkv=-1), {}, INVALID),
    # 2^23 pages x 4 heads x 64 keys = 2^31 rows
    (dict(num_pages=1 << 23), {}, UNSUPPORTED),
    ({}, dict(T=-1), INVALID), ({}, dict(B=-1), INVALID), ({}, dict(max_pages=-1), INVALID),
    ({}, dict(max_pages=(1 << 24) + 1), UNSUPPORTED), ({}, dict(B=65537), UNSUPPORTED),
    ({}, dict(cu_q=None), INVALID), ({}, dict(kv_len=None), INVALID),
    ({}, dict(page_table=None), INVALID), ({}, dict(cu_q=A + 2), MISALIGNED),
]


@pytest.mark.parametrize("c,b,want", CACHE_AND_BATCH)
def test_cache_and_batch_refusals(lib, c, b, want):
    assert attend(lib, cache(**c), batch(**b)) == want, h3.last_error()
    assert append(lib, cache(**c), batch(**b)) == want, h3.last_error()
    assert h3.last_error()


@pytest.mark.parametrize("kw,want", [
    (dict(q=NULL), INVALID), (dict(o=NULL), INVALID), (dict(q=PM), MISALIGNED),
    (dict(o=PM), MISALIGNED), (dict(ld_q=8 * 128 + 4), MISALIGNED),
    (dict(ld_o=8 * 128 - 8), INVALID), (dict(ld_q=1 << 31), UNSUPPORTED),
    (dict(H=6), INVALID), (dict(H=0), INVALID), (dict(H=-4), INVALID),
    (dict(scale=0.0), INVALID), (dict(scale=-1.0), INVALID), (dict(scale=float("nan")), INVALID),
    (dict(prefix_len=-1), INVALID), (dict(prefix_len=(1 << 30) + 1, bytes=1 << 50), UNSUPPORTED), (dict(prefix=NULL), INVALID), (dict(prefix=PM), MISALIGNED),
    (dict(ws=NULL), WORKSPACE), (dict(ws=ctypes.c_void_p(A + 16)), MISALIGNED),
])
def test_attention_refusals(lib, kw, want):
    assert attend(lib, **kw) == want, h3.last_error()


def test_attention_workspace_and_group_limits(lib):
    need = lib.h3_attention_paged_workspace_bytes(6, 8, 100)
    assert attend(lib, bytes=need - 1) == WORKSPACE
    assert attend(lib, b=batch(T=(1 << 26) + 1), bytes=1 << 50) == UNSUPPORTED  # T * H > 2^29
    # 129 query heads on one key head
    assert attend(lib, cache(Hkv=1), ld_q=129 * 128, ld_o=129 * 128, H=129,
                  bytes=1 << 40) == UNSUPPORTED
    assert lib.h3_attention_paged_workspace_bytes(-1, 8, 0) == 0 and h3.last_error()
    assert lib.h3_attention_paged_workspace_bytes(4, 0, 0) == 0
    assert lib.h3_attention_paged_workspace_bytes(4, 8, -1) == 0
    with pytest.raises(h3.H3Error):
        h3.attention_paged_workspace_bytes(4, 0)
    # sizes grow with the rows and never shrink with a prefix
    sizes = [h3.attention_paged_workspace_bytes(t, 42, 0) for t in (0, 1, 64, 1896, 58758)]
    assert sizes == sorted(sizes) and sizes[0] > 0
    assert h3.attention_paged_workspace_bytes(64, 42, 1) >= sizes[2]


@pytest.mark.parametrize("kw,want", [
    (dict(q=NULL), INVALID), (dict(q_out=NULL), INVALID), (dict(k=NULL), INVALID),
    (dict(v=NULL), INVALID), (dict(pos=NULL), INVALID), (dict(axis=None), INVALID),
    (dict(axis=(32, 48, 46)), INVALID), (dict(axis=(33, 47, 48)), INVALID),
    (dict(axis=(40, 40, 48), pairing=1), UNSUPPORTED), (dict(pairing=2), INVALID),
    (dict(theta=0.5), INVALID), (dict(theta=float("nan")), INVALID), (dict(eps=-1.0), INVALID),
    (dict(qg=NULL), INVALID), (dict(kg=NULL), INVALID), (dict(qg=PM), MISALIGNED),
    (dict(k=PM), MISALIGNED), (dict(v=PM), MISALIGNED), (dict(q_out=PM), MISALIGNED),
    (dict(ld_k=4 * 128 + 2), MISALIGNED), (dict(ld_v=3 * 128), INVALID), (dict(H=0), INVALID),
    (dict(q=NULL, q_out=NULL), INVALID),  # H query heads without q
    (dict(q_out=P, ld_q=9 * 128), INVALID),  # in place on strided rows
])
def test_append_refusals(lib, kw, want):
    assert append(lib, **kw) == want, h3.last_error()


def test_empty_calls_do_nothing(lib):
    for kw in (dict(T=0), dict(B=0), dict(T=0, cu_q=None, kv_len=None, page_table=None)):
        assert attend(lib, b=batch(**kw)) == 0 and h3.last_error() == ""
        assert append(lib, b=batch(**kw)) == 0 and h3.last_error() == ""
    assert append(lib, b=batch(T=0), q=NULL, q_out=NULL, H=0, qg=NULL) == 0


def test_binding_checks_before_the_library():
    f = torch.zeros(2, 4, 64, 128, dtype=torch.bfloat16)
    with pytest.raises(TypeError):
        h3.kv_cache(f.float(), f.float())
    with pytest.raises(ValueError, match="current CUDA device"):
        h3.kv_cache(f, f)  # host memory
    with pytest.raises(ValueError, match="contiguous"):
        h3.kv_cache(f.transpose(1, 2), f.transpose(1, 2))
    i = torch.zeros(3, dtype=torch.int32)
    with pytest.raises(TypeError):
        h3.kv_batch(i.long(), i, i, 4)
    with pytest.raises(ValueError, match="current CUDA device"):
        h3.kv_batch(i, i, i, 4)
    c, b = cache(), batch()
    x = torch.zeros(6, 8, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="current CUDA device"):
        h3.attention_paged(x, x, c, b, torch.zeros(16, dtype=torch.uint8))
    with pytest.raises(ValueError, match="heads, 128"):
        h3.attention_paged(x[:5], x, c, b, torch.zeros(16, dtype=torch.uint8))
    with pytest.raises(ValueError, match="contiguous"):
        h3.attention_paged(x.transpose(0, 1)[:6].expand(6, 6, 128), x, c, b,
                           torch.zeros(16, dtype=torch.uint8))
    with pytest.raises(TypeError):
        h3.kv_append_paged(x.float(), x[:, :4], x[:, :4], x, c, b,
                           torch.zeros(6, 3, dtype=torch.int32), (128, 0, 0))


def test_attention_in_place_is_refused(lib):
    assert attend(lib, q=P, o=P) == INVALID and "o is q" in h3.last_error()


@pytest.mark.parametrize("page", [16, 128])
def test_longest_table_and_prefix(lib, page):
    c, most = cache(page_size=page), (1 << 26) // page
    assert attend(lib, c, batch(max_pages=most + 1)) == UNSUPPORTED
    assert append(lib, c, batch(max_pages=most + 1)) == UNSUPPORTED
    assert attend(lib, c, prefix_len=(1 << 26) + 1, bytes=1 << 50) == UNSUPPORTED
    # at the limit the next check is the first to refuse
    assert attend(lib, c, batch(max_pages=most), q=NULL) == INVALID
    assert attend(lib, c, prefix_len=1 << 26, bytes=1 << 50, prefix=NULL) == INVALID


def test_cache_and_batch_of_another_device_are_refused(monkeypatch):
    x = torch.zeros(6, 8, 128, dtype=torch.bfloat16)
    for at in ("cache", "batch"):
        c, b = cache(), batch()
        (c if at == "cache" else b).device = 1
        monkeypatch.setattr(h3, "_device", lambda: 0)
        with pytest.raises(ValueError, match=f"the {at} must be on the current CUDA device"):
            h3.attention_paged(x, x, c, b, torch.zeros(16, dtype=torch.uint8))
        with pytest.raises(ValueError, match=f"the {at} must be on the current CUDA device"):
            h3.kv_append_paged(None, x[:, :4], x[:, :4], None, c, b,
                               torch.zeros(6, 3, dtype=torch.int32), (128, 0, 0))


def test_append_of_keys_alone_needs_their_gain(lib):
    # a gain for the queries that the call does not have, none for its keys
    kw = dict(q=NULL, q_out=NULL, H=0)
    assert append(lib, kg=NULL, **kw) == INVALID and "k_gain" in h3.last_error()
