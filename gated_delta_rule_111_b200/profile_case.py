"""Run one case of the library's kernels a few times on seeded inputs, for profilers.

    python -m gated_delta_rule_111_b200.profile_case prefill --B 2 --T 4096 --H 16 --calls 3
    python -m gated_delta_rule_111_b200.profile_case decode --B 64 --H 16 --calls 3
    python -m gated_delta_rule_111_b200.profile_case backward --B 1 --T 4096 --H 16 --calls 2
    python -m gated_delta_rule_111_b200.profile_case logits --B 2 --T 4096 --H 16 --calls 3
    python -m gated_delta_rule_111_b200.profile_case norm --B 4 --T 4096 --H 16        (and norm_bwd: H x d channels,
                                                              an FP32 stream, residual scale, dropout)
    python -m gated_delta_rule_111_b200.profile_case gate_bwd --B 4 --T 4096 --H 16
    python -m gated_delta_rule_111_b200.profile_case steps --B 256 --H 16 --T 4       (T tokens of B sequences)
    python -m gated_delta_rule_111_b200.profile_case copy --B 256 --H 16              (a permutation of B states)

Inputs come from ``gdn2_inputs`` (same recipe as the tests and ``bench.py``), are moved to the GPU
once, and every call goes through the C ABI.  Nothing is checked or timed here: this exists so that
``ncu`` can capture a chosen number of launches of a smaller case of the same kernels.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import gdn2_inputs as gi  # noqa: E402

from . import (gdn2_chunk_bwd, gdn2_chunk_bwd_workspace_size, gdn2_chunk_fwd, gdn2_chunk_fwd_logits,  # noqa: E402
               gdn2_output_gate_bwd, gdn2_recurrent_step, gdn2_residual_norm, gdn2_residual_norm_bwd,
               gdn2_slot_steps_logits, gdn2_state_copy)


def around(a, dev):
    """The operators around the recurrence: the norm and the epilogue's gradients, steps and copies of cached states."""
    gen = torch.Generator(device=dev)
    gen.manual_seed(0)
    n = lambda *s: torch.randn(*s, generator=gen, device=dev)  # noqa: E731
    tdt = torch.bfloat16 if a.dtype == "bf16" else torch.float32
    D = a.H * a.d
    if a.mode in ("norm", "norm_bwd"):
        x, r, w, s = n(a.B, a.T, D), n(a.B, a.T, D).to(tdt), n(D), n(D)
        kw = dict(scale=s, p=0.1, rng=torch.tensor([1, 2], device=dev))
        if a.mode == "norm":
            return lambda: gdn2_residual_norm(x, r, w, **kw)
        dy, dh, rstd = n(a.B, a.T, D).to(tdt), n(a.B, a.T, D), torch.rsqrt(x.square().mean(-1))
        return lambda: gdn2_residual_norm_bwd(dy, x, rstd, w, dh=dh, r=r, **kw)
    if a.mode == "gate_bwd":
        dy, o, g, w = *(n(a.B, a.T, a.H, a.d).to(tdt) for _ in range(3)), n(a.d)
        return lambda: gdn2_output_gate_bwd(dy, o, g, w)
    pool = 0.1 * n(a.B, a.H, a.d, a.d)
    order = torch.randperm(a.B, generator=gen, device=dev).int()
    if a.mode == "copy":
        return lambda: gdn2_state_copy(pool, order, order.roll(1))
    z = [n(a.B * a.T, a.H, a.d).bfloat16() for _ in range(7)]
    cu = torch.arange(0, a.B * a.T + 1, a.T, dtype=torch.int32, device=dev)
    w = n(a.d)
    return lambda: gdn2_slot_steps_logits(*z[:6], pool, order, cu, g=z[6], weight=w)


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("mode", choices=["prefill", "decode", "backward", "logits", "norm", "norm_bwd", "gate_bwd",
                                         "steps", "copy"])
    ap.add_argument("--B", type=int, default=2)
    ap.add_argument("--T", type=int, default=4096)
    ap.add_argument("--H", type=int, default=16)
    ap.add_argument("--d", type=int, default=128)
    ap.add_argument("--dtype", choices=["bf16", "fp32"], default="bf16")
    ap.add_argument("--calls", type=int, default=3)
    a = ap.parse_args(argv)
    tdt = torch.bfloat16 if a.dtype == "bf16" else torch.float32
    dev = torch.device("cuda:0")
    if a.mode in ("norm", "norm_bwd", "gate_bwd", "steps", "copy"):
        call = around(a, dev)
        for _ in range(a.calls):
            call()
        torch.cuda.synchronize()
        print(f"{a.mode} B={a.B} T={a.T} H={a.H} d={a.d} {a.dtype}: {a.calls} calls done")
        return
    if a.mode == "logits":
        x = gi.logit_inputs(a.B, a.T, a.H, a.d, a.d, seed=0)
        lg = {n: torch.from_numpy(x[n]).to(dev).to(torch.bfloat16) for n in ("xq", "xk", "xv", "xa", "xb", "xw")}
        o = torch.empty(a.B, a.T, a.H, a.d, dtype=torch.bfloat16, device=dev)
        S_T = torch.empty(a.B, a.H, a.d, a.d, dtype=torch.float32, device=dev)
        for _ in range(a.calls):
            gdn2_chunk_fwd_logits(lg["xq"], lg["xk"], lg["xv"], lg["xa"], lg["xb"], lg["xw"], o=o, S_T=S_T)
        torch.cuda.synchronize()
        print(f"logits B={a.B} T={a.T} H={a.H} d={a.d}: {a.calls} calls done")
        return
    if a.mode in ("prefill", "backward"):
        x = gi.chunk_inputs(a.B, a.T, a.H, a.d, a.d, dtype=a.dtype, seed=0)
    else:
        x = gi.decode_inputs(1, a.B, a.H, a.d, a.d, dtype=a.dtype, seed=0)
    g = {n: torch.from_numpy(x[n]).to(dev) for n in ("q", "k", "v", "alpha", "b", "w")}
    for n in ("q", "k", "v"):
        g[n] = g[n].to(tdt)
    if a.mode == "prefill":
        o = torch.empty(a.B, a.T, a.H, a.d, dtype=tdt, device=dev)
        S_T = torch.empty(a.B, a.H, a.d, a.d, dtype=torch.float32, device=dev)
        for _ in range(a.calls):
            gdn2_chunk_fwd(g["q"], g["k"], g["v"], g["alpha"], g["b"], g["w"], o=o, S_T=S_T)
    elif a.mode == "backward":
        gen = torch.Generator(device=dev)
        gen.manual_seed(1)
        dO = torch.randn(a.B, a.T, a.H, a.d, generator=gen, device=dev).to(tdt)
        ws = torch.empty(gdn2_chunk_bwd_workspace_size(a.B, a.T, a.H, a.d, a.d), dtype=torch.uint8, device=dev)
        for _ in range(a.calls):
            gdn2_chunk_bwd(g["q"], g["k"], g["v"], g["alpha"], g["b"], g["w"], None, dO, None, workspace=ws)
    else:
        S = torch.from_numpy(x["S0"]).to(dev)
        q, k, v, al, b, w = (g[n][0] for n in ("q", "k", "v", "alpha", "b", "w"))
        o = torch.empty(a.B, a.H, a.d, dtype=tdt, device=dev)
        for _ in range(a.calls):
            gdn2_recurrent_step(q, k, v, al, b, w, S, o=o)
    torch.cuda.synchronize()
    print(f"{a.mode} B={a.B} T={a.T} H={a.H} d={a.d} {a.dtype}: {a.calls} calls done")


if __name__ == "__main__":
    main()
