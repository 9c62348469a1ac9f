"""Host-side refusals of the operators around the recurrence, without a GPU: every call below returns during
validation, before any CUDA call."""
import ctypes

import numpy as np
import pytest
import torch

import gated_delta_rule_111_b200 as g
import plain64 as p64

BF16, FP32 = 0, 1
A = 0x100000           # fake aligned device addresses, 1 MiB apart; never dereferenced
INVALID, UNSUPPORTED, OK = g.GDN2_ERR_INVALID_ARG, g.GDN2_ERR_UNSUPPORTED, g.GDN2_OK


@pytest.fixture(scope="module")
def lib():
    return g.load_library()


def call(fn, args, **change):
    assert set(change) <= set(args), change
    return fn(*{**args, **change}.values())


def norm_args():
    return dict(x=A, r=2 * A, weight=3 * A, scale=4 * A, p=0.1, rng=5 * A, eps=1e-6, h=6 * A, y=7 * A, rstd=8 * A, rows=4, D=128,
                sdt=BF16, dt=BF16, stream=None)


def test_residual_norm_refusals(lib):
    f, a = lib.gdn2_residual_norm, norm_args()
    for name in ("x", "weight", "h", "y", "rstd"):
        assert call(f, a, **{name: None}) == INVALID and name in lib.gdn2_last_error().decode()
    for name in ("x", "r", "weight", "scale", "rng", "h", "y", "rstd"):
        assert call(f, a, **{name: A * 20 + 4}) == INVALID and b"aligned" in lib.gdn2_last_error()
    assert call(f, a, rows=-1) == INVALID
    assert call(f, a, D=0) == UNSUPPORTED and call(f, a, D=8193) == UNSUPPORTED
    assert call(f, a, dt=7) == UNSUPPORTED and call(f, a, sdt=BF16, dt=FP32) == UNSUPPORTED
    for p in (-0.1, 1.0, 1.5, float("nan")):
        assert call(f, a, p=p) == INVALID
    assert call(f, a, rng=None) == INVALID
    for eps in (-1.0, float("inf"), float("nan")):
        assert call(f, a, eps=eps) == INVALID
    assert call(f, a, r=None) == INVALID                                     # scale, p and h need a branch
    assert call(f, a, r=None, scale=None, p=0.0) == INVALID                  # h without a branch
    for out, at in (("h", 2 * A), ("h", A + 16), ("y", A), ("y", 2 * A + 16), ("y", 6 * A), ("rstd", A), ("rstd", 7 * A), ("y", 3 * A)):
        assert call(f, a, **{out: at}) == INVALID and b"overlaps" in lib.gdn2_last_error()
    assert call(f, a, rows=0) == OK


def test_residual_norm_bwd_refusals(lib):
    f = lib.gdn2_residual_norm_bwd
    need = lib.gdn2_residual_norm_bwd_workspace_size(4, 128)
    assert need == 4 * 2 * 128 * 4                                           # a row of partial sums per CTA
    assert lib.gdn2_residual_norm_bwd_workspace_size(0, 128) == 0
    assert lib.gdn2_residual_norm_bwd_workspace_size(4, 8193) == 0
    a = dict(dy=A, h=2 * A, rstd=3 * A, weight=4 * A, dh=5 * A, r=6 * A, scale=7 * A, p=0.1, rng=8 * A, dx=9 * A, dr=10 * A,
             dweight=11 * A, dscale=12 * A, ws=13 * A, ws_bytes=need, rows=4, D=128, sdt=BF16, dt=BF16, stream=None)
    for name in ("dy", "h", "rstd", "weight", "dx", "dweight", "ws"):
        assert call(f, a, **{name: None}) == INVALID and b"null" in lib.gdn2_last_error()
    for name in ("r", "scale"):
        assert call(f, a, **{name: None}) == INVALID and b"dscale" in lib.gdn2_last_error()
    assert call(f, a, ws_bytes=need - 1) == INVALID and b"workspace" in lib.gdn2_last_error()
    assert call(f, a, rng=None) == INVALID and call(f, a, p=1.0) == INVALID and call(f, a, rows=-1) == INVALID
    assert call(f, a, D=8193) == UNSUPPORTED and call(f, a, dt=FP32) == UNSUPPORTED
    for out, at in (("dx", A), ("dx", 2 * A), ("dr", A), ("dr", 9 * A), ("dweight", 4 * A), ("dscale", 11 * A), ("ws", 6 * A), ("dx", 5 * A + 16)):
        assert call(f, a, **{out: at}) == INVALID and b"overlaps" in lib.gdn2_last_error()


def test_output_gate_bwd_refusals(lib):
    f, need = lib.gdn2_output_gate_bwd, lib.gdn2_output_gate_bwd_workspace_size(128)
    assert need > 0 and lib.gdn2_output_gate_bwd_workspace_size(96) == 0
    a = dict(dy=A, o=2 * A, g=3 * A, weight=4 * A, eps=1e-6, do=5 * A, dg=6 * A, dweight=7 * A, ws=8 * A, ws_bytes=need, B=1, T=4,
             H=2, dv=128, dt=BF16, stream=None)
    for name in ("dy", "o", "g", "weight", "do", "dg", "dweight", "ws"):
        assert call(f, a, **{name: None}) == INVALID and call(f, a, **{name: A * 20 + 8}) == INVALID
    assert call(f, a, B=-1) == INVALID and call(f, a, eps=-1.0) == INVALID and call(f, a, ws_bytes=need - 1) == INVALID
    assert call(f, a, dv=96) == UNSUPPORTED and call(f, a, dt=9) == UNSUPPORTED
    for out, at in (("do", A), ("do", 2 * A), ("dg", 3 * A), ("dg", 5 * A + 16), ("dweight", 4 * A), ("ws", 6 * A)):
        assert call(f, a, **{out: at}) == INVALID and b"overlaps" in lib.gdn2_last_error()


@pytest.mark.parametrize("logits", [False, True])
def test_slot_steps_refusals(lib, logits):
    a = dict(q=A, k=2 * A, v=3 * A, alpha=4 * A, b=5 * A, w=6 * A, pool=64 * A, slots=7 * A, cu=8 * A, keep=9 * A, g=10 * A,
             weight=11 * A, eps=1e-6, o=12 * A, N=3, T=8, H=2, n_slots=5, dk=128, dv=128)
    f = lib.gdn2_slot_steps
    if logits:
        f = lib.gdn2_slot_steps_logits
    else:
        a["dt"] = BF16
        assert call(f, dict(a, stream=None), dt=7) == UNSUPPORTED
    a["stream"] = None
    for name in ("q", "k", "v", "alpha", "b", "w", "pool", "o", "slots"):
        assert call(f, a, **{name: None}) == INVALID and b"null" in lib.gdn2_last_error()
    for name in ("q", "k", "v", "alpha", "b", "w", "pool", "o", "g", "weight"):
        assert call(f, a, **{name: 500 * A + 4}) == INVALID and b"aligned" in lib.gdn2_last_error()
    for name in ("slots", "cu", "keep"):
        assert call(f, a, **{name: 500 * A + 2}) == INVALID and b"4-byte" in lib.gdn2_last_error()
    assert call(f, a, cu=None) == INVALID                                    # eight tokens of three sequences
    assert call(f, a, g=None) == INVALID and call(f, a, weight=None) == INVALID
    assert call(f, a, eps=float("nan")) == INVALID
    assert call(f, a, N=-1) == INVALID and call(f, a, T=-1) == INVALID and call(f, a, n_slots=-1) == INVALID
    assert call(f, a, dk=96) == UNSUPPORTED and call(f, a, dv=256) == UNSUPPORTED
    assert call(f, a, N=1 << 30, H=2) == UNSUPPORTED
    for out, at in (("o", A), ("o", 10 * A), ("o", 64 * A), ("pool", 3 * A), ("pool", 7 * A)):
        assert call(f, a, **{out: at}) == INVALID and b"overlaps" in lib.gdn2_last_error()
    for empty in ("N", "H", "T"):
        assert call(f, a, **{empty: 0}) == OK


def test_state_copy_refusals(lib):
    f = lib.gdn2_state_copy
    a = dict(src_pool=64 * A, dst_pool=64 * A, src=A, dst=2 * A, n=3, layers=2, n_src=5, n_dst=5, H=2, dk=64, dv=128, stream=None)
    for name in ("src", "dst", "dst_pool", "src_pool"):
        assert call(f, a, **{name: None}) == INVALID and call(f, a, **{name: 500 * A + 2}) == INVALID
    assert call(f, a, dst_pool=64 * A + 256) == INVALID and b"overlaps" in lib.gdn2_last_error()
    assert call(f, a, dst_pool=2 * A) == INVALID
    assert call(f, a, n_src=6) == INVALID and call(f, a, n=-1) == INVALID and call(f, a, layers=-1) == INVALID
    assert call(f, a, n=4097) == UNSUPPORTED and call(f, a, dk=32) == UNSUPPORTED
    for empty in ("n", "layers", "H", "n_dst"):
        assert call(f, a, **{empty: 0}) == OK


def test_bindings_refuse_cpu_tensors_and_wrong_arguments():
    x, w = torch.zeros(1, 4, 64), torch.zeros(64)
    z = torch.zeros(4, 2, 64)
    i = torch.zeros(4, dtype=torch.int32)
    for call_ in (lambda: g.gdn2_residual_norm(x, x, w), lambda: g.gdn2_residual_norm_bwd(x, x, x[..., 0], w),
                  lambda: g.gdn2_output_gate_bwd(z[None], z[None], z[None], w),
                  lambda: g.gdn2_slot_steps(z, z, z, z, z, z, torch.zeros(4, 2, 64, 64), i),
                  lambda: g.gdn2_slot_steps_logits(z, z, z, z, z, z, torch.zeros(4, 2, 64, 64), i),
                  lambda: g.gdn2_state_copy(torch.zeros(4, 2, 64, 64), i, i)):
        with pytest.raises(ValueError, match="CUDA"):
            call_()


def test_philox_matches_the_published_vectors():
    """The generator of the tests' plain form against the known answers published with Philox4x32-10."""
    for counter, key, words in p64.PHILOX_KAT:
        assert tuple(int(w) for w in p64.philox([np.array([c], np.uint64) for c in counter], key)[:, 0]) == words
