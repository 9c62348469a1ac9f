"""What the Python binding of the operators around the recurrence refuses, and how it names it: every call here
raises before the library is entered."""
import pytest
import torch

pytestmark = pytest.mark.gpu

BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32


@pytest.fixture(scope="module")
def g():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import gated_delta_rule_111_b200 as mod
    mod.load_library()
    return mod


def spoiled(t):
    """The tensor in another dtype, shape, on another device and not contiguous."""
    other = {BF: F32, F32: BF, I32: torch.int64, torch.int64: I32}[t.dtype]
    yield t.to(other), TypeError
    yield torch.zeros(*t.shape[:-1], t.shape[-1] + 1, dtype=t.dtype, device=t.device), ValueError
    yield t.cpu(), ValueError
    if t.numel() > 1:
        yield torch.zeros(*t.shape, 2, dtype=t.dtype, device=t.device)[..., 0], ValueError


def check(call, args, names):
    call(**args)
    torch.cuda.synchronize()
    for name in names:
        for bad, error in spoiled(args[name]):
            with pytest.raises(error):
                call(**{**args, name: bad})


def z(*s, dtype=F32):
    return torch.zeros(*s, dtype=dtype, device="cuda")


def test_norm(g):
    rng = torch.tensor([1, 2], device="cuda")
    x = dict(x=z(2, 3, 64), r=z(2, 3, 64, dtype=BF), weight=z(64), scale=z(64), p=0.1, rng=rng, h=z(2, 3, 64),
             y=z(2, 3, 64, dtype=BF), rstd=z(2, 3))
    check(g.gdn2_residual_norm, x, ("weight", "scale", "rng", "h", "y", "rstd"))
    for bad in (dict(x=z(6, 64)), dict(r=None), dict(p=1.0), dict(p=-0.5), dict(rng=None), dict(x=z(2, 3, 64, dtype=BF), r=z(2, 3, 64)),
                dict(r=z(2, 3, 65, dtype=BF)), dict(x=x["x"].half()), dict(eps=-1.0)):
        with pytest.raises((ValueError, TypeError, g.Gdn2Error)):
            g.gdn2_residual_norm(**{**x, **bad})
    b = dict(dy=z(2, 3, 64, dtype=BF), h=z(2, 3, 64), rstd=z(2, 3), weight=z(64), dh=z(2, 3, 64), r=z(2, 3, 64, dtype=BF),
             scale=z(64), p=0.1, rng=rng)
    check(g.gdn2_residual_norm_bwd, b, ("rstd", "weight", "dh", "r", "scale", "rng"))
    for bad in (dict(branch=False), dict(r=None), dict(out={"dx": z(2, 3, 64, dtype=BF)}), dict(out={"dscale": z(63)}),
                dict(workspace=z(8, dtype=BF)), dict(workspace=torch.zeros(1 << 20, dtype=torch.uint8))):
        with pytest.raises((ValueError, TypeError, g.Gdn2Error)):
            g.gdn2_residual_norm_bwd(**{**b, **bad})


def test_gate(g):
    b = dict(dy=z(1, 5, 2, 64), o=z(1, 5, 2, 64), g=z(1, 5, 2, 64), weight=z(64))
    check(g.gdn2_output_gate_bwd, b, ("o", "g", "weight"))
    for bad in (dict(out={"do": z(1, 5, 2, 64, dtype=BF)}), dict(out={"dweight": z(65)}), dict(workspace=z(4))):
        with pytest.raises((ValueError, TypeError, g.Gdn2Error)):
            g.gdn2_output_gate_bwd(**{**b, **bad})
    with pytest.raises(g.Gdn2Error):
        t = z(1, 5, 2, 96)
        g.gdn2_output_gate_bwd(t, t.clone(), t.clone(), z(96))


@pytest.mark.parametrize("logits", [False, True])
def test_steps(g, logits):
    T, H, N = 5, 2, 3
    t, gt = (BF, BF) if logits else (F32, F32)
    names = ("xq", "xk", "xv", "xa", "xb", "xw") if logits else ("q", "k", "v", "alpha", "b", "w")
    a = {n: z(T, H, 64, dtype=gt if n in ("alpha", "b", "w") else t) for n in names}
    a.update(pool=z(4, H, 64, 64), slots=torch.tensor([0, 1, 2], dtype=I32, device="cuda"),
             cu_seqlens=torch.tensor([0, 2, 4, 5], dtype=I32, device="cuda"), keep=torch.ones(3, dtype=I32, device="cuda"),
             g=z(T, H, 64, dtype=t), weight=z(64), o=z(T, H, 64, dtype=t))
    call = g.gdn2_slot_steps_logits if logits else g.gdn2_slot_steps
    check(call, a, names[1:] + ("pool", "cu_seqlens", "keep", "g", "weight", "o"))
    for bad in (dict(cu_seqlens=None), dict(weight=None), dict(g=None), dict(slots=a["slots"].long()), dict(slots=a["slots"][None]),
                dict(o=a["g"]), dict(pool=a["pool"][:, :1])):
        with pytest.raises((ValueError, TypeError, g.Gdn2Error)):
            call(**{**a, **bad})


def test_copy(g):
    i = torch.tensor([0, 1], dtype=I32, device="cuda")
    a = dict(pool=z(4, 2, 64, 64), src=i, dst=i.clone(), source=z(3, 2, 64, 64))
    check(g.gdn2_state_copy, a, ("src", "dst", "source"))
    for bad in (dict(pool=z(4, 2, 64)), dict(source=z(1, 3, 2, 64, 64)), dict(pool=z(4, 2, 64, 64).half()),
                dict(src=torch.zeros(4097, dtype=I32, device="cuda"), dst=torch.zeros(4097, dtype=I32, device="cuda")),
                dict(source=a["pool"][1:])):
        with pytest.raises((ValueError, TypeError, g.Gdn2Error)):
            g.gdn2_state_copy(**{**a, **bad})
