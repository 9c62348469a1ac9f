"""gdn2_output_gate_bwd where its arithmetic has no room: no epsilon, and gates that are wide open or shut.

The bounds are those of test_output_gate_bwd_gpu.py, 64 + 4 |g| roundings of 2^-24.
"""
import pytest
import torch

import plain64 as p64
from test_output_gate_bwd_gpu import check, draw, g  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("dv", [64, 128])
@pytest.mark.parametrize("size", [(1, 1, 1), (1, 7, 1), (1, 257, 3), (2, 16, 8), (1, 1801, 11)], ids=str)
def test_no_epsilon(g, dt, dv, size):  # noqa: F811
    """eps = 0 is allowed, and every row has a norm: what lies behind the last row adds nothing to dweight."""
    dy, o, gl, w = draw(*size, dv, dt, seed=dv + size[1])
    out = g.gdn2_output_gate_bwd(dy, o, gl, w, 0.0)
    assert all(bool(torch.isfinite(t).all()) for t in out.values())
    check(out, dy, o, gl, w, 0.0)


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("dv", [64, 128])
def test_gate_gradient_to_its_own_digits(g, dt, dv):  # noqa: F811
    """dg = dy n weight s (1 - s) within 64 + 4 |g| roundings of its own value, for gates from shut to open.

    e = exp(-g) is off by 2 + 1.2 |g| steps, two roundings each.  s = 1 / (1 + e) takes the share e / (1 + e) of that
    and five roundings, 1 - s = e s the rest of it and six: together 15 + 2.4 |g|.  n adds half of a row sum's 20,
    rsqrtf's four and a product, the outer form four: 34 + 2.4 |g| in all.
    """
    dy, o, gl, w = draw(2, 161, 3, dv, dt, seed=11)
    gen = torch.Generator("cuda").manual_seed(4)
    gl.copy_(torch.linspace(-80.0, 80.0, 161, device="cuda").view(1, 161, 1, 1) + torch.rand(gl.shape, generator=gen, device="cuda"))
    out = g.gdn2_output_gate_bwd(dy, o, gl, w, 1e-5)
    check(out, dy, o, gl, w, 1e-5)
    e = torch.exp(-gl.double())
    o64 = o.double()
    dg = dy.double() * o64 / torch.sqrt((o64 * o64).mean(-1, keepdim=True) + 1e-5) * w.double() * e / (1 + e) ** 2
    p64.assert_close("dg", out["dg"], dg, dg.abs() * (64 + 4 * gl.double().abs()), 1)


def test_gate_nan_stays_nan(g):  # noqa: F811
    dy, o, gl, w = draw(1, 9, 2, 64, torch.float32, seed=12)
    gl[0, 3, 1, 5] = float("nan")
    out = g.gdn2_output_gate_bwd(dy, o, gl, w, 1e-5)
    bad = torch.zeros(1, 9, 2, 64, dtype=torch.bool, device="cuda")
    bad[0, 3, 1, 5] = True
    assert torch.equal(torch.isnan(out["dg"]), bad)
    assert torch.equal(torch.isnan(out["do"]), bad.any(-1, keepdim=True).expand_as(bad))
    assert torch.equal(torch.isnan(out["dweight"]), bad.flatten(0, 2).any(0))
