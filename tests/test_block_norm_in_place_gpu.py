"""gdn2_residual_norm and gdn2_residual_norm_bwd at widths that are no multiple of a vector, where a row's first
vector also reads the end of the row before it: that row may hold anything, and may be written meanwhile.
"""
import pytest
import torch

from test_block_norm_gpu import TYPES, draw, g  # noqa: F401

pytestmark = pytest.mark.gpu

# more rows than the grid has CTAs, but for the last two
SIZES = [(6000, 7), (5000, 45), (1500, 1001), (1500, 1021), (700, 2551), (400, 5113), (320, 8187), (320, 8188), (9, 1021), (1, 7)]


@pytest.mark.parametrize("types", TYPES)
@pytest.mark.parametrize("size", SIZES, ids=str)
@pytest.mark.parametrize("p", [0.0, 0.3])
def test_in_place(g, size, types, p):  # noqa: F811
    """h over x, y over r and dx over dh give the bits of separate buffers."""
    d = draw(1, *size, types, seed=size[1])
    kw = dict(scale=d["s"], p=p, rng=d["rng"] if p else None)
    h, y, rstd = g.gdn2_residual_norm(d["x"], d["r"], d["w"], **kw)
    x, r = d["x"].clone(), d["r"].clone()
    h2, y2, rstd2 = g.gdn2_residual_norm(x, r, d["w"], h=x, y=r, **kw)
    assert h2 is x and y2 is r and torch.equal(h, x) and torch.equal(y, r) and torch.equal(rstd, rstd2)
    want = g.gdn2_residual_norm_bwd(d["dy"], h, rstd, d["w"], dh=d["dh"], r=d["r"], **kw)
    dh = d["dh"].clone()
    got = g.gdn2_residual_norm_bwd(d["dy"], h, rstd, d["w"], dh=dh, r=d["r"], out={"dx": dh}, **kw)
    assert got["dx"] is dh and all(torch.equal(got[k], want[k]) for k in want)


@pytest.mark.parametrize("types", TYPES)
@pytest.mark.parametrize("size", SIZES[:-1], ids=str)
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_special_values_stay_in_their_row(g, size, types, value):  # noqa: F811
    """Every second row is NaN or infinite throughout; the others are those of the clean call, bit for bit."""
    d = draw(1, *size, types, seed=size[1] + 1)
    kw = dict(scale=d["s"], p=0.3, rng=d["rng"])
    h, y, rstd = g.gdn2_residual_norm(d["x"], d["r"], d["w"], **kw)
    want = g.gdn2_residual_norm_bwd(d["dy"], h, rstd, d["w"], dh=d["dh"], r=d["r"], **kw)
    bad = dict(d, **{n: d[n].clone() for n in ("x", "r", "dy", "dh")})
    for n in ("x", "r", "dy", "dh"):
        bad[n][:, 1::2] = value
    h2, y2, rstd2 = g.gdn2_residual_norm(bad["x"], bad["r"], d["w"], **kw)
    got = g.gdn2_residual_norm_bwd(bad["dy"], h2, rstd2, d["w"], dh=bad["dh"], r=bad["r"], **kw)
    for a, b in ((h, h2), (y, y2), (rstd, rstd2), (want["dx"], got["dx"]), (want["dr"], got["dr"])):
        assert torch.equal(a[:, ::2], b[:, ::2])
    assert not bool(torch.isfinite(h2[:, 1::2]).any()) and not bool(torch.isfinite(y2[:, 1::2]).any())
