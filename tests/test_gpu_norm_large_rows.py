"""Norms around a branch of rows whose squares, or sums, FP32 cannot hold: the formula of the row all the same,
within the bound of the other rows (derived where it stands)."""
import pytest
import torch

from test_gpu_sandwich_norm import call, check, draw

pytestmark = pytest.mark.gpu
dev = "cuda"


@pytest.mark.parametrize("rms", [False, True])
@pytest.mark.parametrize("D", [8, 256, 504, 1024, 1280, 1928, 2560, 3080, 4096, 5120, 5376, 8192])
def test_rows_of_large_magnitude(h3lib, D, rms):
    a = draw(40, D, D, groups=2) | dict(rms=rms)
    top = 2.0 ** 118 if D > 8 else 2.0 ** 122
    for i, big in enumerate((2.0 ** 50, 2.0 ** 60, 1e18, 1e19, 2.0 ** 64, 1e20, 1e25, 1e30, 2.0 ** 110, top)):
        a["resid"][2 * i] *= big              # rows that are large all over, with an ordinary branch
        a["delta"][20 + i] *= big             # an ordinary residual and a large branch: its norm is ordinary
        a["resid"][30 + i, 1] = big           # one large value in an ordinary row
    if D > 8:
        a["resid"][1] = a["resid"][1] * 2.0 ** 100 + 2.0 ** 121   # far from zero: the sum itself overflows
        a["delta"][3] = 2.0 ** 120                                # a constant row: its norm is near 0
        a["delta"][5, ::2] = -3.0e38
        a["delta"][5, 1::2] = 1.0e38
    out = torch.empty(40, D, device=dev)
    normed = torch.empty(40, D, device=dev, dtype=torch.bfloat16)
    call(h3lib, a, out, normed)
    assert torch.isfinite(out).all() and torch.isfinite(normed.float()).all()
    check(out, normed, a, 40, f"{D} wide")


@pytest.mark.parametrize("rms", [False, True])
def test_a_constant_row_is_its_shift(h3lib, rms):
    # powers of two: the mean is exact, and what LayerNorm has left is 0; a root mean square gives 1
    for D, big in ((512, 2.0 ** 120), (512, 2.0 ** 126), (5376, 2.0 ** 100), (8192, 2.0 ** 124), (8192, 1.0)):
        x = torch.full((3, D), big, device=dev)
        h = torch.empty(3, D, device=dev, dtype=torch.bfloat16)
        h3lib.sandwich_norm(x, normed=h, rms=rms)
        h3lib.check_device_error()
        if rms:
            assert ((h.float() - 1).abs() <= 2.0 ** -8).all(), (D, big)
        elif D & (D - 1) == 0:
            assert (h == 0).all(), (D, big)


def test_rows_that_are_not_finite_show_as_before(h3lib):
    for rms in (False, True):
        a = draw(6, 1024, 3) | dict(rms=rms)
        a["resid"][1, 5] = float("inf")
        a["resid"][2] *= 1e30
        a["resid"][2, 700] = float("nan")
        a["delta"][4, 9] = -float("inf")
        out, normed = torch.empty(6, 1024, device=dev), torch.empty(6, 1024, device=dev, dtype=torch.bfloat16)
        call(h3lib, a, out, normed)
        bad = torch.tensor([False, True, True, False, True, False], device=dev)
        assert torch.equal(normed.isnan().any(1), bad)
