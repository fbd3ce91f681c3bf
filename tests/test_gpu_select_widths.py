"""Selection at the numbers of blocks where another kernel, or another number of registers for a row, takes over
(128, 256, 512, 768 and 1,024), and of scores with the shapes that real ones have: peaks at a few neighbours, a few
values in all, a handful of exponents, falling with the distance."""
import numpy as np
import pytest
import torch

from test_gpu_blocks import check_select

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("nk", [127, 256, 257, 511, 512, 513, 600, 640, 767, 768, 769, 800, 1000, 1023, 1024, 1025])
def test_where_the_kernels_change(h3lib, nk):
    g = torch.Generator()
    g.manual_seed(nk)
    s = torch.randn(7, nk, generator=g)
    for most in (1, nk // 10, nk // 2, nk - 1, nk):
        check_select(h3lib, s, most)
        check_select(h3lib, (s * 4).round() / 4, most, 1 if most > 2 else 0, 1 if most > 2 else 0)


@pytest.mark.parametrize("nk", [130, 460, 700, 919, 1500])
def test_scores_as_video_has_them(h3lib, nk):
    g = torch.Generator()
    g.manual_seed(nk)
    rows = 12
    at = torch.arange(nk).float()
    here = torch.rand(rows, 1, generator=g) * nk
    near = torch.exp(-(at - here).abs() / 5) * 8 + torch.randn(rows, nk, generator=g) * 0.01
    frames = torch.cos(at * 2 * np.pi / 30) * 3 - (at - here).abs() / nk
    skew = torch.exp(3 * torch.randn(rows, nk, generator=g))
    two = (torch.rand(rows, nk, generator=g) < 0.03).float() * 100
    for s in (near, frames, skew, -skew, two, near.to(torch.bfloat16).float(), near * 1e30, near * 1e-38):
        for most in (1, nk // 10, nk // 3):
            check_select(h3lib, s, most)
