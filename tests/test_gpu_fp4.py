"""Microscaled 4-bit rows and their products against 64-bit forms of the definitions.

Quantisation: codes, scales and row scales bit for bit (every step of the definition is
exact in 64 bits or rounded to 32 as it says). Products, given the codes: the 64-bit sum,
within
  2^-8 |y|                    half a bf16 step of the result (relative to it at most 2^-8)
  + (K / 16 + 4) 2^-23 A      the FP32 sum: at least 16 values of K meet in one addition, each
                              of them off by one unit of the last place of what was summed so
                              far, A = the sum of the products' magnitudes; and the scaling
SwiGLU, given the two rounded products g and u: 2^-8 for its own rounding and 2^-20 (an exponential
off by 2 units of FP32's last place and 2^-24 |g|, a division off by 2, three roundings), relative to
SiLU(g) u; where exp(-g) passes 2^126 it may be 0 instead of less than 2^-119 |u|."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
dev = "cuda"
SENT = -7.25
E2M1 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])
E4M3 = np.array([m * 2.0 ** -9 for m in range(8)]
                + [(8 + m) * 2.0 ** (e - 10) for e in range(1, 16) for m in range(8)][:-1])
BLOCK = {"mx": 32, "nv": 16}
f32 = lambda x: np.asarray(x, np.float64).astype(np.float32).astype(np.float64)


def nearest(a, grid):
    """Places in an ascending grid of the nearest values to a >= 0, ties to the even place."""
    hi = np.clip(np.searchsorted(grid, a), 0, len(grid) - 1)
    lo = np.maximum(hi - 1, 0)
    up, down = grid[hi] - a, a - grid[lo]
    return np.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)


def reference(x, fmt):
    """(codes, scale bytes, row scales) of x [R, K] float64 by the definition."""
    R, K = x.shape
    b = x.reshape(R, -1, BLOCK[fmt])
    bad = ~np.isfinite(b).all(-1)
    z = np.where(bad[..., None], 0.0, b)
    top = np.abs(z).max(-1)
    if fmt == "mx":
        e = np.maximum(np.frexp(top)[1] - 3.0, -127)
        e[top == 0] = -127
        y = np.abs(z) * 2.0 ** -e[..., None]
        byte, row = e + 127, None
    else:
        amax = top.max(1)
        some = amax >= 2.0 ** -100
        safe = np.where(some, amax, 1.0)
        row = np.where(some, f32(amax / 2688), 0.0)
        byte = nearest(f32(top * np.where(some, f32(448 / safe), 0.0)[:, None]), E4M3)
        sf = E4M3[byte]
        inv = np.where((sf > 0) & some[:, None],
                       f32(f32(2688 / safe)[:, None] / np.where(sf > 0, sf, 1.0)), 0.0)
        y = f32(np.abs(z) * inv[..., None])
    code = nearest(y, E2M1) + 8 * np.signbit(z)
    code[bad] = 0
    byte = np.where(bad, 255 if fmt == "mx" else 0x7f, byte)
    return code.reshape(R, K).astype(np.uint8), byte.astype(np.uint8), row


def unpack(q, R=None):
    """(codes, scale bytes) of an Fp4Rows as [R, K] and [R, blocks], by the documented layout."""
    R = q.R if R is None else R
    c = q.codes[:R].cpu().numpy()
    codes = np.stack([c & 15, c >> 4], -1).reshape(R, q.K)
    nb = q.K // BLOCK[q.format]
    r, b = np.arange(R)[:, None], np.arange(nb)[None]
    at = ((r // 128) * -(-nb // 4) + b // 4) * 512 + r % 32 * 16 + r % 128 // 32 * 4 + b % 4
    return codes, q.scales.cpu().numpy()[at]


def values(q, R=None):
    """The values that an Fp4Rows stands for, without its row scales, and those."""
    codes, byte = unpack(q, R)
    v = E2M1[codes & 7] * np.where(codes & 8, -1.0, 1.0)
    s = 2.0 ** (byte.astype(np.float64) - 127) if q.format == "mx" else E4M3[np.minimum(byte, 126)]
    v = v * np.repeat(s, BLOCK[q.format], 1)
    return v, 1.0 if q.format == "mx" else q.row_scale[:len(v)].double().cpu().numpy()


def draw(*shape, seed=0, std=1.0, wide=True):
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    x = torch.randn(*shape, generator=g, device=dev) * std
    if wide:
        x = x * torch.exp2(torch.randint(-3, 4, shape[:1] + (1,), generator=g, device=dev).float())
        x[:, ::29] *= 8
    return x.to(torch.bfloat16)


def quantize(h3lib, x, fmt, L=None):
    q = h3lib.fp4_rows(*x.shape, format=fmt)
    h3lib.quantize_fp4_rows(x, q, L)
    h3lib.check_device_error()
    return q


@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("R,K", [(1, 32), (7, 96), (129, 160), (250, 512), (300, 1056), (64, 5376),
                                 (33, 14336), (5, 16384), (3, 8192), (2, 12320)])
def test_quantize_matches_definition_bitwise(h3lib, R, K, fmt):
    x = draw(R, K, seed=R + K)
    x[0, : K // 2] = 0
    if R > 2:
        x[2] = 0
        x[1] = x[1].sign() * 5.0  # ties and equal values
    q = quantize(h3lib, x, fmt)
    code, byte, row = reference(x.double().cpu().numpy(), fmt)
    got, scales = unpack(q)
    assert np.array_equal(scales, byte)
    assert np.array_equal(got, code)
    if row is not None:
        assert np.array_equal(q.row_scale.double().cpu().numpy(), row)


@pytest.mark.parametrize("fmt", ["mx", "nv"])
def test_quantize_every_bf16_value_and_tie(h3lib, fmt):
    # every finite bf16 magnitude next to a fixed largest one of its block, and blocks of
    # multiples of a sixteenth, where every tie of E2M1 occurs
    bits = torch.arange(0x7f80, dtype=torch.int32)
    x = torch.cat([bits, bits + 0x8000]).to(torch.int16).view(torch.bfloat16)
    x = x[: x.numel() // 480 * 480].view(-1, 480)
    t = (torch.arange(480) % 97 / 16 - 3).to(torch.bfloat16).expand(8, 480).clone()
    t *= torch.exp2(torch.arange(8.0)).to(torch.bfloat16)[:, None]
    x = torch.cat([x, t]).to(dev)
    q = quantize(h3lib, x, fmt)
    code, byte, row = reference(x.double().cpu().numpy(), fmt)
    got, scales = unpack(q)
    assert np.array_equal(scales, byte) and np.array_equal(got, code)
    if row is not None:
        assert np.array_equal(q.row_scale.double().cpu().numpy(), row)


@pytest.mark.parametrize("fmt", ["mx", "nv"])
def test_quantize_rows_at_the_ends_of_the_range(h3lib, fmt):
    x = draw(6, 256, seed=2).float()
    x[0] *= 2.0 ** -126 / x[0].abs().max()
    x[1] *= 2.0 ** -101 / x[1].abs().max()
    x[2] *= 2.0 ** -99
    x[3] *= 3e38 / x[3].abs().max()
    x[4, :240] *= 2.0 ** -20   # blocks far below their row's largest
    x = x.to(torch.bfloat16)
    q = quantize(h3lib, x, fmt)
    code, byte, row = reference(x.double().cpu().numpy(), fmt)
    got, scales = unpack(q)
    assert np.array_equal(scales, byte) and np.array_equal(got, code)
    if row is not None:
        assert np.array_equal(q.row_scale.double().cpu().numpy(), row)


@pytest.mark.parametrize("fmt", ["mx", "nv"])
def test_nonfinite_blocks_show_in_the_product(h3lib, fmt):
    x = draw(40, 160, seed=4, wide=False)
    x[3, 70] = float("nan")
    x[7, 1] = float("inf")
    x[9, 159] = -float("inf")
    w = draw(64, 160, seed=5, std=0.1, wide=False)
    q, qw = quantize(h3lib, x, fmt), quantize(h3lib, w, fmt)
    code, byte, row = reference(x.double().cpu().numpy(), fmt)
    got, scales = unpack(q)
    assert np.array_equal(scales, byte) and np.array_equal(got, code)
    y = torch.empty(40, 64, dtype=torch.bfloat16, device=dev)
    h3lib.linear_fp4(q, qw, y)
    h3lib.check_device_error()
    nan = torch.zeros(40, dtype=torch.bool)
    nan[[3, 7, 9]] = True
    assert torch.equal(y.isnan().all(1).cpu(), nan) and torch.equal(y.isnan().any(1).cpu(), nan)


@pytest.mark.parametrize("fmt", ["mx", "nv"])
def test_quantize_strided_rows_and_rows_left_alone(h3lib, fmt):
    wide = draw(300, 1024, seed=6)
    x = wide[:, 256:768]
    q = h3lib.fp4_rows(300, 512, format=fmt)
    q.codes.fill_(0xa5)
    q.scales.fill_(0xa5)
    h3lib.quantize_fp4_rows(x, q, 200)
    p = quantize(h3lib, x.contiguous(), fmt)
    a, b = unpack(q), unpack(p)
    assert np.array_equal(a[0][:200], b[0][:200]) and np.array_equal(a[1][:200], b[1][:200])
    assert (q.codes[200:] == 0xa5).all() and (a[1][200:] == 0xa5).all()


def check_linear(y, qx, qw, rows, what):
    (x, rx), (w, rw) = values(qx), values(qw)
    x, rx = x[rows], (rx if np.isscalar(rx) else rx[rows, None])
    s = rx * (rw if np.isscalar(rw) else rw[None])
    ref, mag = x @ w.T * s, np.abs(x) @ np.abs(w).T * s
    err = np.abs(y[rows].double().cpu().numpy() - ref)
    bound = 2.0 ** -8 * np.abs(ref) + (qx.K / 16 + 4) * 2.0 ** -23 * mag + 1e-38
    assert np.all(err <= bound), f"{what}: {np.max(err / bound)} of the bound"


@pytest.mark.parametrize("fmt", ["mx", "nv"])
def test_linear_exact_small_integers(h3lib, fmt):
    # products and sums that FP32 and bf16 hold exactly, with a power of two of its own for
    # every block: any misplaced code or scale shows
    g = torch.Generator()
    g.manual_seed(1)
    S, N, K, n = 256, 512, 256, BLOCK[fmt]
    def operand(R, lo, hi):
        q = h3lib.fp4_rows(R, K, format=fmt)
        codes = torch.randint(0, 16, (R, K), generator=g)
        codes = torch.where(codes & 7 > 2, codes & 8, codes)       # 0, +-0.5, +-1
        keep = torch.rand(R, K, generator=g) < 0.1
        codes = torch.where(keep, codes, 0)
        q.codes.copy_((codes[:, ::2] | codes[:, 1::2] << 4).to(torch.uint8))
        e = torch.randint(lo, hi, (R, K // n), generator=g)
        r, b = torch.arange(R)[:, None], torch.arange(K // n)[None]
        at = ((r // 128) * (K // n // 4) + b // 4) * 512 + r % 32 * 16 + r % 128 // 32 * 4 + b % 4
        s = torch.zeros(q.scales.numel(), dtype=torch.uint8)
        s[at] = ((127 + e) if fmt == "mx" else (7 + e) * 8).to(torch.uint8)
        q.scales.copy_(s)
        if fmt == "nv":
            q.row_scale.copy_(torch.exp2(torch.randint(-1, 2, (R,), generator=g).float()))
        return q
    qx, qw = operand(S, -1, 2), operand(N, -1, 2)
    y = torch.full((S, N), SENT, dtype=torch.bfloat16, device=dev)
    h3lib.linear_fp4(qx, qw, y)
    h3lib.check_device_error()
    (x, rx), (w, rw) = values(qx), values(qw)
    ref = x @ w.T * (rx if np.isscalar(rx) else rx[:, None] * rw[None])
    # the sums are exact; one rounding to bf16
    assert torch.equal(y.cpu(), torch.from_numpy(ref).to(torch.bfloat16))


@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("S,L,N,K", [(1, 1, 8, 32), (3, 2, 40, 64), (22, 22, 512, 5376), (128, 128, 256, 256),
                                     (129, 129, 264, 288), (300, 257, 776, 512), (513, 512, 1000, 2080),
                                     (1999, 1999, 2816, 1056), (700, 700, 128, 14336)])
def test_linear(h3lib, S, L, N, K, fmt):
    qx = quantize(h3lib, draw(S, K, seed=S + N), fmt)
    qw = quantize(h3lib, draw(N, K, seed=K, std=0.02), fmt)
    buf = torch.full((S + 2, N), SENT, dtype=torch.bfloat16, device=dev)
    y = buf[1:S + 1]
    h3lib.linear_fp4(qx, qw, y, L)
    h3lib.check_device_error()
    check_linear(y, qx, qw, np.arange(L), f"{fmt} {S}x{N}x{K}")
    assert bool((buf[L + 1:] == SENT).all()) and bool((buf[0] == SENT).all())
    again = torch.empty_like(y)
    h3lib.linear_fp4(qx, qw, again, L)
    h3lib.check_device_error()
    assert torch.equal(again[:L], y[:L])


@pytest.mark.parametrize("fmt", ["mx", "nv"])
def test_linear_full_size(h3lib, fmt):
    S, N, K = 58758, 16128, 5376
    qx = quantize(h3lib, draw(S, K, seed=1), fmt)
    qw = quantize(h3lib, draw(N, K, seed=2, std=0.02), fmt)
    y = torch.full((S, N), SENT, dtype=torch.bfloat16, device=dev)
    h3lib.linear_fp4(qx, qw, y)
    h3lib.check_device_error()
    rows = np.unique(np.r_[0, S - 1, np.random.default_rng(3).choice(S, 60)])
    check_linear(y, qx, qw, rows, fmt)
    # every row against two of its columns, one in each half of a tile
    cols = [37, 16127]
    (x, rx), (w, rw) = values(qx), values(qw, 16128)
    ref = x @ w[cols].T * (1.0 if np.isscalar(rx) else rx[:, None] * rw[None, cols])
    mag = np.abs(x) @ np.abs(w[cols]).T * (1.0 if np.isscalar(rx) else rx[:, None] * rw[None, cols])
    err = np.abs(y[:, cols].double().cpu().numpy() - ref)
    assert np.all(err <= 2.0 ** -8 * np.abs(ref) + (K / 16 + 4) * 2.0 ** -23 * mag)


@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("S,L,F,K", [(1, 1, 128, 32), (250, 250, 256, 512), (300, 257, 384, 1056),
                                     (1999, 1999, 1408, 1056), (22, 22, 1408, 5376)])
def test_linear_swiglu_is_product_then_gate(h3lib, S, L, F, K, fmt):
    qx = quantize(h3lib, draw(S, K, seed=S), fmt)
    qw = quantize(h3lib, draw(2 * F, K, seed=F, std=0.02), fmt)
    gu = torch.empty(S, 2 * F, dtype=torch.bfloat16, device=dev)
    out = torch.full((S, F), SENT, dtype=torch.bfloat16, device=dev)
    h3lib.linear_fp4(qx, qw, gu, L)
    h3lib.linear_swiglu_fp4(qx, qw, out, L)
    h3lib.check_device_error()
    check_linear(gu, qx, qw, np.arange(L), "gate and up")
    check_swiglu(out[:L], gu[:L])
    assert bool((out[L:] == SENT).all())


def check_swiglu(out, gu):
    g, u = gu.double().chunk(2, 1)
    want = g * torch.sigmoid(g) * u
    bound = (2.0 ** -8 + 2.0 ** -20 + 2.0 ** -23 * g.abs()) * want.abs() + 2.0 ** -119 * u.abs()
    assert ((out.double() - want).abs() <= bound).all()


def test_swiglu_of_large_products(h3lib):
    # gates from -300 to 300: the exponential's overflow, and its end
    S, F, K = 64, 128, 64
    x, w = torch.zeros(S, K, device=dev), torch.zeros(2 * F, K, device=dev)
    x[:, 0] = torch.linspace(-6, 6, S, device=dev)
    x[:, 1] = 1
    w[:F, 0] = torch.linspace(0, 50, F, device=dev)
    w[F:, 1] = torch.linspace(-3, 3, F, device=dev)
    qx, qw = (quantize(h3lib, t.to(torch.bfloat16), "mx") for t in (x, w))
    gu = torch.empty(S, 2 * F, dtype=torch.bfloat16, device=dev)
    out = torch.empty(S, F, dtype=torch.bfloat16, device=dev)
    h3lib.linear_fp4(qx, qw, gu)
    h3lib.linear_swiglu_fp4(qx, qw, out)
    h3lib.check_device_error()
    assert gu[:, :F].min() < -250 and gu[:, :F].max() > 250 and torch.isfinite(out).all()
    check_swiglu(out, gu)


def test_zero_rows_and_columns(h3lib):
    for fmt in ("mx", "nv"):
        x = draw(130, 128, seed=1)
        x[5] = 0
        w = draw(136, 128, seed=2, std=0.1)
        w[9] = 0
        y = torch.empty(130, 136, dtype=torch.bfloat16, device=dev)
        h3lib.linear_fp4(quantize(h3lib, x, fmt), quantize(h3lib, w, fmt), y)
        h3lib.check_device_error()
        assert (y[5] == 0).all() and (y[:, 9] == 0).all() and torch.isfinite(y).all()


def test_graph_and_side_stream(h3lib):
    fmt, S, N, K = "nv", 300, 520, 544
    xs = [draw(S, K, seed=i) for i in (1, 2)]
    qw = quantize(h3lib, draw(N, K, seed=3, std=0.05), fmt)
    want = []
    for x in xs:
        y = torch.empty(S, N, dtype=torch.bfloat16, device=dev)
        h3lib.linear_fp4(quantize(h3lib, x, fmt), qw, y)
        want.append(y)
    x, q = xs[0].clone(), h3lib.fp4_rows(S, K, format=fmt)
    y = torch.empty(S, N, dtype=torch.bfloat16, device=dev)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        h3lib.quantize_fp4_rows(x, q)
        h3lib.linear_fp4(q, qw, y)
    for i in (1, 0):
        x.copy_(xs[i])
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want[i])
    with torch.cuda.stream(side):
        h3lib.quantize_fp4_rows(xs[1], q)
        h3lib.linear_fp4(q, qw, y)
    torch.cuda.synchronize()
    assert torch.equal(y, want[1])


@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("S,N,K", [(1, 256, 2048), (22, 2560, 4096), (128, 3840, 4128), (130, 1288, 5376),
                                   (300, 2048, 8192), (22, 5376, 5376), (256, 9216, 2080), (22, 24, 16384)])
def test_few_tiles_share_their_k(h3lib, S, N, K, fmt):
    # one tile of 256 x 256 to a cluster of two, three and four pairs, and not quite few enough
    qx = quantize(h3lib, draw(S, K, seed=S + N), fmt)
    qw = quantize(h3lib, draw(N, K, seed=K, std=0.02), fmt)
    buf = torch.full((S + 2, N), SENT, dtype=torch.bfloat16, device=dev)
    y, again = buf[1:S + 1], torch.empty(S, N, dtype=torch.bfloat16, device=dev)
    h3lib.linear_fp4(qx, qw, y)
    h3lib.linear_fp4(qx, qw, again)
    h3lib.check_device_error()
    check_linear(y, qx, qw, np.arange(S), f"{fmt} {S}x{N}x{K}")
    assert torch.equal(again, y) and (buf[0] == SENT).all() and (buf[-1] == SENT).all()
    if N % 256 == 0:
        out = torch.empty(S, N // 2, dtype=torch.bfloat16, device=dev)
        h3lib.linear_swiglu_fp4(qx, qw, out)
        h3lib.check_device_error()
        check_swiglu(out, y)
