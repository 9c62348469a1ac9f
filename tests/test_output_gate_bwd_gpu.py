"""gdn2_output_gate_bwd against its 64-bit form.

Roundings: the sigmoid's exponential carries 2 + 1.2 |g| steps (exponent scaled in 32 bits, two-step
approximation), the quotient two; each row sum at most 20 (8 channels, 5 shuffles, the scale); the outer forms
8.  Counted as 64 + 4 |g| for every element; 1 - s is bounded by its terms (1 + s), not by its value.
"""
import pytest
import torch

import plain64 as p64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def g():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import gated_delta_rule_111_b200 as mod
    mod.load_library()
    return mod


def draw(B, T, H, dv, dt, seed=0):
    gen = torch.Generator("cuda").manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=gen, device="cuda")
    return n(B, T, H, dv).to(dt), (0.5 * n(B, T, H, dv)).to(dt), (2 * n(B, T, H, dv)).to(dt), 1 + 0.1 * n(dv)


def check(out, dy, o, gl, w, eps):
    dy, o, gl, w = dy.double(), o.double(), gl.double(), w.double()
    s, rs = p64.sigmoid(gl), 1 / torch.sqrt((o * o).mean(-1, keepdim=True) + eps)
    n, t = o * rs, dy * w * s
    k = 64 + 4 * gl.abs()
    kr = k.amax(-1, keepdim=True)
    mag = rs * (t.abs() + n.abs() * (t * n).abs().mean(-1, keepdim=True))
    p64.assert_close("do", out["do"], rs * (t - n * (t * n).mean(-1, keepdim=True)), mag * kr, 1)
    p64.assert_close("dg", out["dg"], t * n * (1 - s), (t * n).abs() * (1 + s) * k, 1)
    terms = dy * n * s
    rows = dy.numel() / dy.shape[-1]
    depth = 8 + 5 + 32 + rows / (148 * 4 * 8) + 148 * 4 / 32
    p64.assert_close("dweight", out["dweight"], terms.sum((0, 1, 2)), (terms.abs() * (depth + k)).sum((0, 1, 2)), 1)


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("dv", [64, 128])
@pytest.mark.parametrize("size", [(1, 1, 1), (1, 7, 3), (2, 33, 5), (1, 257, 3), (3, 400, 16)], ids=str)
def test_matches_plain(g, dt, dv, size):
    dy, o, gl, w = draw(*size, dv, dt, seed=dv + size[1])
    out = g.gdn2_output_gate_bwd(dy, o, gl, w, 1e-5)
    check(out, dy, o, gl, w, 1e-5)
    again = g.gdn2_output_gate_bwd(dy, o, gl, w, 1e-5)
    assert all(torch.equal(out[k], again[k]) for k in out)


def test_gate_edges_and_zero_rows(g):
    """Gates far out on both sides, a zero row (n = 0: dg = 0), upstream zeros."""
    dy, o, gl, w = draw(1, 40, 2, 128, torch.float32, seed=3)
    gl[0, :10], gl[0, 10:20], o[0, 20], dy[0, 21] = 60.0, -60.0, 0.0, 0.0
    out = g.gdn2_output_gate_bwd(dy, o, gl, w, 1e-5)
    check(out, dy, o, gl, w, 1e-5)
    assert bool((out["dg"][0, 20] == 0).all()) and bool((out["do"][0, 21] == 0).all())
    gl[0, 0], gl[0, 1] = float("inf"), float("-inf")
    out = g.gdn2_output_gate_bwd(dy, o, gl, w, 1e-5)
    assert all(bool(torch.isfinite(t).all()) for t in out.values())
    assert bool((out["dg"][0, :2] == 0).all()) and bool((out["do"][0, 1] == 0).all())


def test_no_rows(g):
    e, w = torch.empty(0, 3, 2, 64, device="cuda"), torch.ones(64, device="cuda")
    assert bool((g.gdn2_output_gate_bwd(e, e, e, w)["dweight"] == 0).all())


def test_gradient_against_differences(g):
    dy, o, gl, w = draw(1, 5, 2, 64, torch.float32, seed=5)
    out = g.gdn2_output_gate_bwd(dy, o, gl, w, 1e-5)
    gen = torch.Generator("cuda").manual_seed(1)
    base = {"do": o, "dg": gl, "dweight": w}
    for name, x in base.items():
        v = torch.randn(x.shape, generator=gen, device="cuda", dtype=torch.float64)

        def loss(t):
            a = {k: (b.double() + (t * v if k == name else 0)) for k, b in base.items()}
            y = a["do"] / torch.sqrt((a["do"] ** 2).mean(-1, keepdim=True) + 1e-5) * a["dweight"] * p64.sigmoid(a["dg"])
            return float((dy.double() * y).sum())
        want, got = (loss(1e-5) - loss(-1e-5)) / 2e-5, float((out[name].double() * v).sum())
        scale = float((out[name].double() * v).abs().sum())
        assert abs(got - want) <= 1e-5 * scale, (name, got, want)       # 64-bit difference 1e-9, fp32 about 100 * 2^-24


def test_caller_buffers_and_stream(g):
    dy, o, gl, w = draw(2, 900, 4, 128, torch.bfloat16, seed=7)
    ws = torch.full((g.gdn2_output_gate_bwd_workspace_size(128),), 255, dtype=torch.uint8, device="cuda")
    bufs = {"do": torch.empty_like(dy), "dg": torch.empty_like(dy), "dweight": torch.full((128,), 7.0, device="cuda")}
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    out = g.gdn2_output_gate_bwd(dy, o, gl, w, 1e-5, workspace=ws, out=bufs, stream=s)
    s.synchronize()
    assert all(out[k] is bufs[k] for k in bufs)
    check(out, dy, o, gl, w, 1e-5)
