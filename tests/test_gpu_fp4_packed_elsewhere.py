"""4-bit rows whose codes and scales a program fills in itself, at the places that the layout gives them and nowhere
else: rows whose length is no multiple of 64, so that a product goes past their last block."""
import pytest
import torch

from test_gpu_fp4 import BLOCK, values

pytestmark = pytest.mark.gpu
dev = "cuda"


@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("S,N,K", [(3, 8, 32), (40, 264, 96), (130, 256, 160), (300, 128, 352), (22, 520, 4128)])
def test_packed_rows(h3lib, S, N, K, fmt):
    g = torch.Generator()
    g.manual_seed(S + K)
    n = BLOCK[fmt]

    def operand(R):
        was = torch.are_deterministic_algorithms_enabled()
        torch.use_deterministic_algorithms(True)      # memory that nothing wrote holds 0xff: NaN in both formats
        q = h3lib.fp4_rows(R, K, format=fmt)
        torch.use_deterministic_algorithms(was)
        codes = torch.randint(0, 16, (R, K), generator=g)
        codes = torch.where(codes & 7 > 2, codes & 8, codes)       # 0, +-0.5, +-1
        codes = torch.where(torch.rand(R, K, generator=g) < 0.1, codes, 0)
        q.codes.copy_((codes[:, ::2] | codes[:, 1::2] << 4).to(torch.uint8))
        nb = K // n
        e = torch.randint(-1, 2, (R, nb), generator=g)
        r, b = torch.arange(R)[:, None], torch.arange(nb)[None]
        at = ((r // 128) * -(-nb // 4) + b // 4) * 512 + r % 32 * 16 + r % 128 // 32 * 4 + b % 4
        q.scales[at.flatten().to(dev)] = (((127 + e) if fmt == "mx" else (7 + e) * 8).to(torch.uint8)).flatten().to(dev)
        if fmt == "nv":
            q.row_scale.fill_(1.0)
        return q

    qx, qw = operand(S), operand(N)
    y = torch.full((S, N), -7.25, dtype=torch.bfloat16, device=dev)
    h3lib.linear_fp4(qx, qw, y)
    h3lib.check_device_error()
    (x, _), (w, _) = values(qx), values(qw)
    assert torch.equal(y.cpu(), torch.from_numpy(x @ w.T).to(torch.bfloat16))   # sums that FP32 holds exactly
