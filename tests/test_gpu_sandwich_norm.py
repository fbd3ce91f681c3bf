"""Norms before and after a branch with its gate and the scaled residual, against the formula in
64 bits. Bounds, with e = 2^-24 (half a step of FP32) and n(x) = (x - mean) * rstd:
  a norm is off by at most 40 e (|n| + (|x| + mean |x|) rstd): sums of D values in at most 4 of
  a thread and 9 levels of partial sums, twice, and a few roundings of the value itself;
  that, times gain and gate, and 3 e of every term, is what resid_out is off by;
  normed: the same of its own norm, that of its input carried through (times rstd * (1 + scale),
  and twice for the mean and the root mean square of the row), and half a bf16 step, 2^-8 |h|."""
import pytest
import torch

pytestmark = pytest.mark.gpu
dev = "cuda"
E = 2.0 ** -24
SENT = -7.25


def norm(x, rms, eps):
    mean = torch.zeros_like(x[:, :1]) if rms else x.mean(-1, keepdim=True)
    rstd = ((x - mean).square().mean(-1, keepdim=True) + eps).rsqrt()
    n = (x - mean) * rstd
    return n, rstd, 40 * E * (n.abs() + (x.abs() + x.abs().mean(-1, keepdim=True)) * rstd)


def check(out, normed, a, L, what):
    """a: the arguments, None where left out."""
    v = lambda k, d: torch.full((1,), d, dtype=torch.float64, device=dev) if a.get(k) is None else a[k].double()
    pick = lambda t: t if t.dim() == 1 else t[a["seg"][:L].long().clamp(0, t.shape[0] - 1)]
    gate, shift, scale = pick(v("gate", 1.0)), pick(v("shift", 0.0)), pick(v("scale", 0.0))
    r = a["resid"][:L].double() * a["resid_scale"]
    er = 3 * E * r.abs()
    if a["delta"] is not None:
        p, ep = a["delta"][:L].double(), 0.0
        if a["post_norm"]:
            p, _, ep = norm(p, a["rms"], a["eps"])
            g = v("post_gain", 1.0)
            p, ep = p * g, ep * g.abs() + E * (p * g).abs()
        r = r + gate * p
        er = er + gate.abs() * ep + 3 * E * (gate * p).abs()
    if out is not None:
        d = (out[:L].double() - r).abs()
        assert (d <= er + 1e-37).all(), f"{what}: residual {float((d / (er + 1e-37)).max())} of the bound"
    if normed is not None:
        n, rstd, en = norm(r, a["rms"], a["eps"])
        m = (1 + scale) * v("pre_gain", 1.0)
        h = n * m + shift
        rms_er = er.square().mean(-1, keepdim=True).sqrt()
        eh = m.abs() * (en + rstd * (er + 2 * rms_er * (1 + n.abs()))) + 4 * E * ((n * m).abs() + shift.abs())
        d = (normed[:L].double() - h).abs()
        b = eh + 2.0 ** -8 * h.abs() + 1e-37
        assert (d <= b).all(), f"{what}: normed {float((d / b).max())} of the bound"


def draw(S, D, seed, offset=0.0, groups=0):
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    rnd = lambda *s, std=1.0: torch.randn(*s, generator=g, device=dev) * std
    a = dict(resid=rnd(S, D) + offset, delta=(rnd(S, D, std=3.0) + offset).to(torch.bfloat16),
             post_gain=1 + rnd(D, std=0.1), pre_gain=1 + rnd(D, std=0.1), post_norm=True,
             resid_scale=0.75, rms=False, eps=1e-6, seg=None)
    mod = rnd(max(groups, 1), 6, D, std=0.3)
    if groups:
        a["seg"] = torch.randint(0, groups, (S,), generator=g, device=dev, dtype=torch.int32)
    for i, k in ((2, "gate"), (3, "shift"), (4, "scale")):
        a[k] = mod[:, i] if groups else mod[0, i]
    return a


def call(h3lib, a, out, normed, L=None):
    h3lib.sandwich_norm(a["resid"], a["delta"], normed, resid_out=out, L=L,
                        **{k: v for k, v in a.items() if k not in ("resid", "delta")})
    h3lib.check_device_error()


@pytest.mark.parametrize("rms", [False, True])
@pytest.mark.parametrize("S,L,D", [(1, 1, 8), (3, 2, 24), (250, 250, 512), (22, 22, 5376), (37, 36, 1928),
                                   (9, 9, 2048), (5, 5, 2056), (64, 64, 4104), (7, 7, 6152), (300, 299, 8192),
                                   (6, 6, 1032)])
def test_against_the_formula(h3lib, S, L, D, rms):
    for seed, groups, offset in ((S, 0, 0.0), (S + 1, 3, 0.0), (S + 2, 1, 50.0)):
        a = draw(S, D, seed, offset, groups) | dict(rms=rms)
        out = torch.full((S, D), SENT, device=dev)
        normed = torch.full((S, D), SENT, device=dev, dtype=torch.bfloat16)
        call(h3lib, a, out, normed, L)
        check(out, normed, a, L, f"{S}x{D}")
        assert (out[L:] == SENT).all() and (normed[L:] == SENT).all()


@pytest.mark.parametrize("rms", [False, True])
@pytest.mark.parametrize("D", [32, 256, 264, 504, 1024, 1152, 1280, 1288, 1536, 1544, 2560, 2568, 3000, 3080,
                               4096, 4104, 5120, 5128, 6144, 7000])
def test_every_width(h3lib, D, rms):
    # each split of a row over threads, full and nearly so
    a = draw(131, D, D, 2) | dict(rms=rms)
    out = torch.full((133, D), SENT, device=dev)
    normed = torch.full((133, D), SENT, device=dev, dtype=torch.bfloat16)
    call(h3lib, a, out[1:-1], normed[1:-1], 130)
    check(out[1:-1], normed[1:-1], a, 130, f"131x{D}")
    for t in (out, normed):
        assert (t[0] == SENT).all() and (t[131:] == SENT).all()


@pytest.mark.parametrize("rms", [False, True])
def test_parts_left_out(h3lib, rms):
    S, D = 40, 640
    full = draw(S, D, 1, groups=2) | dict(rms=rms)
    plain = draw(S, D, 1) | dict(rms=rms)
    for a, gone in ((full, ("post_gain",)), (full, ("pre_gain", "shift")), (full, ("gate", "scale")),
                    (plain, ("scale", "shift", "pre_gain", "gate", "post_gain")),
                    (full, ("gate", "shift", "scale"))):
        for post in (True, False):
            b = a | {k: None for k in gone} | dict(post_norm=post)
            if not post:
                b["post_gain"] = None
            out = torch.empty(S, D, device=dev)
            normed = torch.empty(S, D, device=dev, dtype=torch.bfloat16)
            call(h3lib, b, out, normed)
            check(out, normed, b, S, f"without {gone}, post {post}")
    # only the residual
    b = plain | dict(pre_gain=None, shift=None, scale=None)
    out = torch.empty(S, D, device=dev)
    call(h3lib, b, out, None)
    check(out, None, b, S, "residual alone")
    # only the norm: with and without a residual scale
    for rs, out in ((1.0, None), (0.5, torch.empty(S, D, device=dev))):
        b = plain | dict(delta=None, gate=None, post_gain=None, post_norm=False, resid_scale=rs)
        normed = torch.empty(S, D, device=dev, dtype=torch.bfloat16)
        call(h3lib, b, out, normed)
        check(out, normed, b, S, "norm alone")


def test_in_place_and_extreme_rows(h3lib):
    S, D = 33, 1928
    for rms in (False, True):
        a = draw(S, D, 3) | dict(rms=rms)
        a["delta"][4] = 0          # a branch of zeros: eps alone under the root
        a["resid"][5] = 0
        a["delta"][5] = 0
        a["resid"][6] = 7.0        # constant rows
        a["delta"][6] = 2.0
        a["delta"][7] *= 1e15
        a["resid"][8] *= 1e-18
        a["delta"][8] *= 1e-18
        want = torch.empty(S, D, device=dev)
        normed = torch.empty(S, D, device=dev, dtype=torch.bfloat16)
        call(h3lib, a, want, normed)
        check(want, normed, a, S, "extremes")
        a["resid"] = a["resid"].clone()
        again = torch.empty_like(normed)
        call(h3lib, a, None, again)   # into resid itself
        assert torch.equal(a["resid"], want) and torch.equal(again, normed)


def test_groups_outside_the_table_are_clamped(h3lib):
    a = draw(50, 512, 9, groups=3)
    a["seg"][::7] = -5
    a["seg"][3::7] = 1 << 30
    out, normed = torch.empty(50, 512, device=dev), torch.empty(50, 512, device=dev, dtype=torch.bfloat16)
    call(h3lib, a, out, normed)
    check(out, normed, a, 50, "clamped groups")


def test_nonfinite_rows_stay_in_their_row(h3lib):
    a = draw(20, 512, 11)
    a["delta"][3, 7] = float("nan")
    a["resid"][9, 0] = float("inf")
    out, normed = torch.empty(20, 512, device=dev), torch.empty(20, 512, device=dev, dtype=torch.bfloat16)
    call(h3lib, a, out, normed)
    bad = torch.zeros(20, dtype=torch.bool, device=dev)
    bad[[3, 9]] = True
    assert torch.equal(normed.isnan().any(1), bad)
    keep = ~bad
    b = {k: (v[keep] if k in ("resid", "delta") else v) for k, v in a.items()}
    check(out[keep], normed[keep], b, 18, "the other rows")


def test_full_size(h3lib):
    S, D = 58758, 5376
    a = draw(S, D, 5, groups=2)
    out, normed = torch.empty(S, D, device=dev), torch.empty(S, D, device=dev, dtype=torch.bfloat16)
    call(h3lib, a, out, normed)
    for i in range(0, S, 8192):
        b = {k: (v[i:i + 8192] if k in ("resid", "delta", "seg") else v) for k, v in a.items()}
        check(out[i:i + 8192], normed[i:i + 8192], b, min(8192, S - i), f"rows {i}")


def test_same_as_the_modulated_norm(h3lib):
    # LayerNorm, no norm after the branch, no gains: the modulation step of the block
    S, D = 128, 5376
    a = draw(S, D, 7) | dict(post_norm=False, post_gain=None, pre_gain=None, resid_scale=1.0)
    out, normed = torch.empty(S, D, device=dev), torch.empty(S, D, device=dev, dtype=torch.bfloat16)
    call(h3lib, a, out, normed)
    r, h = a["resid"].clone(), torch.empty_like(normed)
    h3lib.mod_norm_residual(r, a["delta"], *(a[k].contiguous() for k in ("gate", "shift", "scale")), h)
    h3lib.check_device_error()
    assert torch.equal(out, r)
    step = 2.0 ** -7 * torch.maximum(h.float().abs(), normed.float().abs())
    assert ((h.float() - normed.float()).abs() <= step + 2.0 ** -22).all()


def test_graph_and_side_stream(h3lib):
    names = ("resid", "delta", "post_gain", "pre_gain", "seg")
    ins = [draw(300, 1928, seed, groups=2) for seed in (21, 22)]
    tables = [torch.stack([a["gate"], a["shift"], a["scale"]], 1) for a in ins]     # [groups, 3, D]
    live, table = {k: ins[0][k].clone() for k in names}, tables[0].clone()
    out, normed = torch.empty(300, 1928, device=dev), torch.empty(300, 1928, device=dev, dtype=torch.bfloat16)

    def run():
        h3lib.sandwich_norm(live["resid"], live["delta"], normed, resid_out=out, post_gain=live["post_gain"],
                            gate=table[:, 0], resid_scale=0.75, pre_gain=live["pre_gain"], shift=table[:, 1],
                            scale=table[:, 2], seg=live["seg"])

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        run()
    for i in (1, 0):
        for k in names:
            live[k].copy_(ins[i][k])
        table.copy_(tables[i])
        graph.replay()
        torch.cuda.synchronize()
        check(out, normed, ins[i], 300, "replayed")
        got = out.clone(), normed.clone()
        with torch.cuda.stream(side):
            run()
        torch.cuda.synchronize()
        assert torch.equal(out, got[0]) and torch.equal(normed, got[1])
