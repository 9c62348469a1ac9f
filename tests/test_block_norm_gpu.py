"""gdn2_residual_norm and gdn2_residual_norm_bwd against 64-bit plain forms (plain64.py has the bound's form).

Roundings counted for the forward: h three (scaled r, the product, the sum); a row's mean of squares at most 64
(8 or 16 in a thread, 5 shuffles, 32 warps, the scale), halved by the root, rsqrtf two steps, y three more; the
error of h enters rstd relatively and y directly.  Backward: the row's mean of products 80, the outer form 8;
weight gradients: rows of one CTA, rows of partial sums per warp, 32 warps.
"""
import itertools

import pytest
import torch

import plain64 as p64

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
TYPES = {"bf16": (BF, BF), "mixed": (F32, BF), "fp32": (F32, F32)}
SEED, OFFSET = 0x1234_5678_9ABC, (7 << 32) + 5


@pytest.fixture(scope="module")
def g():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import gated_delta_rule_111_b200 as mod
    mod.load_library()
    return mod


def draw(B, T, D, types, seed=0):
    gen = torch.Generator("cuda").manual_seed(seed)
    ts, tb = TYPES[types]
    n = lambda *s: torch.randn(*s, generator=gen, device="cuda")
    return dict(x=(2 * n(B, T, D)).to(ts), r=n(B, T, D).to(tb), dy=n(B, T, D).to(tb), dh=n(B, T, D).to(ts),
                w=1 + 0.1 * n(D), s=0.3 + 0.1 * n(D), rng=torch.tensor([SEED, OFFSET], device="cuda"))


def forward64(d, p, eps, scale, branch=True):
    B, T, D = d["x"].shape
    h = d["x"].double()
    mag = h.abs()
    if branch:
        b = d["r"].double() * p64.dropout_factor(B * T, D, p, SEED, OFFSET).view(B, T, D).cuda()
        b = b * d["s"].double() if scale else b
        h, mag = h + b, mag + b.abs()
    rstd = 1 / torch.sqrt((h * h).mean(-1) + eps)
    return h, mag, rstd, h * rstd[..., None] * d["w"].double()


def check_forward(d, h, y, rstd, p, eps, scale, branch=True):
    h64, mag, r64, y64 = forward64(d, p, eps, scale, branch)
    off = 3 * (mag.square().mean(-1).sqrt() * r64)            # h's error as a share of its size, in roundings
    if branch:
        p64.assert_close("h", h, h64, mag, 4)
    p64.assert_close("rstd", rstd, r64, r64 * (40 + off), 1)
    p64.assert_close("y", y, y64, y64.abs() * (46 + off[..., None]) + 4 * (mag * r64[..., None] * d["w"].abs().double()), 1)


def check_backward(d, h, rstd, out, p, scale, branch=True, dh=True):
    B, T, D = h.shape
    kept = p64.dropout_factor(B * T, D, p, SEED, OFFSET).view(B, T, D).cuda()
    h, dy, rs, w = h.double(), d["dy"].double(), rstd.double()[..., None], d["w"].double()
    n, t = h * rs, dy * w
    extra = d["dh"].double() if dh else torch.zeros_like(h)
    dx = rs * (t - n * (t * n).mean(-1, keepdim=True)) + extra
    mag = rs * (t.abs() + n.abs() * (t * n).abs().mean(-1, keepdim=True)) + extra.abs()
    p64.assert_close("dx", out["dx"], dx, mag, 88)
    depth = 8 + 32 + B * T / 144 + 148 * 16 / 32
    p64.assert_close("dweight", out["dweight"], (dy * n).sum((0, 1)), (dy * n).abs().sum((0, 1)), depth)
    if branch:
        f = kept * d["s"].double() if scale else kept
        p64.assert_close("dr", out["dr"], dx * f, mag * f.abs(), 92)
    if scale:
        b = d["r"].double() * kept
        p64.assert_close("dscale", out["dscale"], (dx * b).sum((0, 1)), (mag * b.abs()).sum((0, 1)), depth + 90)


SIZES = [(1, 1, 1), (1, 3, 7), (2, 5, 64), (1, 1, 2048), (3, 41, 1021), (1, 700, 512), (2, 150, 2048), (1, 33, 4104),
         (1, 9, 8192), (1, 5, 8191), (1, 160, 8187), (1, 160, 8188), (1, 2, 6001), (1, 300, 4100), (1, 3000, 96), (1, 9000, 18),
         (1, 5000, 45), (1, 1500, 515), (1, 1000, 1023), (1, 1000, 1448), (1, 1000, 1501), (1, 700, 2304), (1, 700, 2551),
         (1, 500, 5120), (1, 500, 5113), (1, 450, 6144), (1, 450, 6139), (1, 320, 7168), (1, 320, 7003), (1, 320, 8192)]


@pytest.mark.parametrize("types", TYPES)
@pytest.mark.parametrize("size", SIZES, ids=str)
@pytest.mark.parametrize("p,scale", [(0.0, False), (0.3, True)])
def test_forward_and_backward(g, types, size, p, scale):
    d = draw(*size, types, seed=size[2])
    kw = dict(scale=d["s"] if scale else None, p=p, rng=d["rng"] if p else None)
    h, y, rstd = g.gdn2_residual_norm(d["x"], d["r"], d["w"], 1e-5, **kw)
    assert h.dtype == d["x"].dtype and y.dtype == d["r"].dtype
    check_forward(d, h, y, rstd, p, 1e-5, scale)
    out = g.gdn2_residual_norm_bwd(d["dy"], h, rstd, d["w"], dh=d["dh"], r=d["r"] if scale else None, **kw)
    check_backward(d, h, rstd, out, p, scale)
    again = g.gdn2_residual_norm_bwd(d["dy"], h, rstd, d["w"], dh=d["dh"], r=d["r"] if scale else None, **kw)
    assert all(torch.equal(out[k], again[k]) for k in out if out[k] is not None)


@pytest.mark.parametrize("types", TYPES)
def test_first_norm_has_no_branch(g, types):
    d = draw(2, 17, 264, types)
    h, y, rstd = g.gdn2_residual_norm(d["x"], None, d["w"], 1e-5, y=torch.empty_like(d["r"]))
    assert h is d["x"]
    check_forward(d, h, y, rstd, 0.0, 1e-5, False, branch=False)
    out = g.gdn2_residual_norm_bwd(d["dy"], d["x"], rstd, d["w"], branch=False)
    assert out["dr"] is None and out["dscale"] is None
    check_backward(d, d["x"], rstd, out, 0.0, False, branch=False, dh=False)


def test_in_place_stream(g):
    """h over x, y over r, dx over dh give the bits of the separate buffers."""
    d = draw(2, 300, 1024, "bf16", seed=4)
    h, y, rstd = g.gdn2_residual_norm(d["x"], d["r"], d["w"], scale=d["s"])
    x, r = d["x"].clone(), d["r"].clone()
    h2, y2, _ = g.gdn2_residual_norm(x, r, d["w"], scale=d["s"], h=x, y=r)
    assert h2 is x and y2 is r and torch.equal(h, x) and torch.equal(y, r)
    a = g.gdn2_residual_norm_bwd(d["dy"], h, rstd, d["w"], dh=d["dh"])
    dh = d["dh"].clone()
    b = g.gdn2_residual_norm_bwd(d["dy"], h, rstd, d["w"], dh=dh, out={"dx": dh})
    assert b["dx"] is dh and torch.equal(a["dx"], dh) and torch.equal(a["dr"], b["dr"])


def test_mask_share_and_dropped_infinities(g):
    """A dropped element contributes nothing, whatever it holds; the share dropped is p within 6 sigma."""
    B, T, D, p = 1, 512, 640, 0.25
    d = draw(B, T, D, "bf16", seed=6)
    kept = p64.dropout_factor(T, D, p, SEED, OFFSET).view(B, T, D).cuda() > 0
    r = torch.where(kept, d["r"], torch.full_like(d["r"], float("nan")))
    r[0, ::2] = torch.where(kept[0, ::2], d["r"][0, ::2], torch.full_like(r[0, ::2], float("inf")))
    h, y, rstd = g.gdn2_residual_norm(d["x"], r, d["w"], p=p, rng=d["rng"])
    want, wy, wr = g.gdn2_residual_norm(d["x"], d["r"], d["w"], p=p, rng=d["rng"])
    assert torch.equal(h, want) and torch.equal(y, wy) and torch.equal(rstd, wr)
    out = g.gdn2_residual_norm_bwd(d["dy"], h, rstd, d["w"], dh=d["dh"], r=r, scale=d["s"], p=p, rng=d["rng"])
    assert torch.isfinite(out["dscale"]).all() and bool((out["dr"][~kept] == 0).all())
    n = kept.numel()
    assert abs(float(kept.sum()) / n - (1 - p)) < 6 * (p * (1 - p) / n) ** 0.5


@pytest.mark.parametrize("p", [2.0 ** -33, 1e-6, 0.999999, 1 - 2.0 ** -33])
def test_extreme_probabilities(g, p):
    d = draw(1, 64, 256, "fp32", seed=8)
    h, y, rstd = g.gdn2_residual_norm(d["x"], d["r"], d["w"], p=p, rng=d["rng"])
    check_forward(d, h, y, rstd, p, 1e-6, False)


def test_zero_rows_and_no_rows(g):
    z = torch.zeros(1, 4, 128, device="cuda")
    w = torch.ones(128, device="cuda")
    _, y, rstd = g.gdn2_residual_norm(z, None, w, 1e-6)
    assert bool((y == 0).all()) and torch.allclose(rstd, torch.full_like(rstd, 1e3))
    e = torch.empty(0, 4, 128, device="cuda")
    h, y, rstd = g.gdn2_residual_norm(e, e, w)
    assert h.shape == e.shape and rstd.shape == (0, 4)
    out = g.gdn2_residual_norm_bwd(e, e, rstd, w, r=e, scale=w)
    assert bool((out["dweight"] == 0).all()) and bool((out["dscale"] == 0).all())


def test_gradient_against_differences(g):
    """The gradient of sum(dy y + dh h) along a random direction against a central difference in 64 bits."""
    d = draw(1, 6, 40, "fp32", seed=9)
    h, y, rstd = g.gdn2_residual_norm(d["x"], d["r"], d["w"], 1e-5, scale=d["s"], p=0.4, rng=d["rng"])
    out = g.gdn2_residual_norm_bwd(d["dy"], h, rstd, d["w"], dh=d["dh"], r=d["r"], scale=d["s"], p=0.4, rng=d["rng"])
    gen = torch.Generator("cuda").manual_seed(1)
    for name, grad in (("x", "dx"), ("r", "dr"), ("w", "dweight"), ("s", "dscale")):
        v = torch.randn(d[name].shape, generator=gen, device="cuda", dtype=torch.float64)

        def loss(t):
            e = dict(d, **{name: d[name].double() + t * v})
            h64, _, _, y64 = forward64(e, 0.4, 1e-5, True)
            return float((d["dy"].double() * y64).sum() + (d["dh"].double() * h64).sum())
        want, got = (loss(1e-5) - loss(-1e-5)) / 2e-5, float((out[grad].double() * v).sum())
        # 64-bit difference: third-derivative and cancellation errors near 1e-9; fp32 gradients: about 100 * 2^-24
        scale = float((out[grad].double() * v).abs().sum())
        assert abs(got - want) <= 1e-5 * scale, (name, got, want)


def test_new_masks_in_a_replayed_graph(g):
    """The captured call reads rng when it runs; a side stream and a side-stream workspace too."""
    d = draw(1, 300, 520, "bf16", seed=10)
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        for _ in range(2):
            g.gdn2_residual_norm(d["x"], d["r"], d["w"], p=0.5, rng=d["rng"])
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        h, y, rstd = g.gdn2_residual_norm(d["x"], d["r"], d["w"], p=0.5, rng=d["rng"])
        out = g.gdn2_residual_norm_bwd(d["dy"], h, rstd, d["w"], dh=d["dh"], p=0.5, rng=d["rng"])
    seen = []
    for step in range(3):
        d["rng"][1] = OFFSET + step
        graph.replay()
        torch.cuda.synchronize()
        want = g.gdn2_residual_norm(d["x"], d["r"], d["w"], p=0.5, rng=d["rng"], stream=s)
        grads = g.gdn2_residual_norm_bwd(d["dy"], want[0], want[2], d["w"], dh=d["dh"], p=0.5, rng=d["rng"], stream=s)
        s.synchronize()
        assert torch.equal(h, want[0]) and torch.equal(y, want[1])
        assert all(torch.equal(out[k], grads[k]) for k in ("dx", "dr", "dweight"))
        seen.append(h.clone())
    assert not torch.equal(seen[0], seen[1]) and not torch.equal(seen[1], seen[2])


def test_more_than_2_31_elements(g):
    """Offsets past 32 bits: the last rows of a stream of 2^31 + 2^20 elements."""
    D = 8192
    rows = (1 << 18) + 128
    x = torch.zeros(1, rows, D, dtype=BF, device="cuda")
    gen = torch.Generator("cuda").manual_seed(2)
    x[0, -3:] = torch.randn(3, D, generator=gen, device="cuda").to(BF)
    w = 1 + 0.1 * torch.randn(D, generator=gen, device="cuda")
    _, y, rstd = g.gdn2_residual_norm(x, None, w, 1e-5)
    _, y2, rstd2 = g.gdn2_residual_norm(x[:, -3:].contiguous(), None, w, 1e-5)
    assert torch.equal(y[:, -3:], y2) and torch.equal(rstd[:, -3:], rstd2)
