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
@pytest.mark.parametrize("size", [(1, 1, 1), (1, 7, 1), (1, 257, 3), (2, 16, 8)], ids=str)
def test_no_epsilon(g, dt, dv, size):  # noqa: F811
    """eps = 0 is allowed, and every row has a norm: what lies behind the last row adds nothing to dweight."""
    dy, o, gl, w = draw(*size, dv, dt, seed=dv + size[1])
    out = g.gdn2_output_gate_bwd(dy, o, gl, w, 0.0)
    assert all(bool(torch.isfinite(t).all()) for t in out.values())
    check(out, dy, o, gl, w, 0.0)
