"""Room for 4-bit rows, made on the host."""
import pytest
import torch

from dit_transformer_block_gb300 import build, h3


@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("R,K", [(1, 32), (130, 96), (128, 256)])
def test_scales_begin_as_zeros(monkeypatch, fmt, R, K):
    # a product reads scales past the last block of a row of 32, 96, ... values, which nothing has to
    # write: with what memory holds by chance (here 0xff everywhere, a NaN in both formats) it gave NaN
    build.build()
    monkeypatch.setattr(h3, "Fp4Rows", lambda codes, scales, row_scale, format: scales)   # (it takes CUDA tensors only)
    was = torch.are_deterministic_algorithms_enabled()
    torch.use_deterministic_algorithms(True)      # fills what torch.empty returns with ones
    try:
        assert torch.utils.deterministic.fill_uninitialized_memory
        assert (torch.empty(64, dtype=torch.uint8) == 255).all()
        scales = h3.fp4_rows(R, K, format=fmt, device="cpu")
    finally:
        torch.use_deterministic_algorithms(was)
    assert (scales == 0).all() and scales.numel() == h3.fp4_scale_bytes(R, K, fmt)


@pytest.mark.parametrize("format", ["int4", "", None, 1])
def test_a_format_that_is_none_is_refused(format):
    build.build()
    for call in (lambda: h3.fp4_scale_bytes(4, 64, format), lambda: h3.fp4_rows(4, 64, format=format, device="cpu"),
                 lambda: h3.Fp4Rows(torch.empty(4, 32, dtype=torch.uint8), torch.empty(512, dtype=torch.uint8), None, format)):
        with pytest.raises(ValueError, match="format must be one of"):
            call()
