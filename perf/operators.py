"""Cases of the operators around the Gated DeltaNet-2 recurrence, in plain torch and through the library.

Five operators, by a case's "op":

  norm       h = x + scale * dropout(r), y = RMSNorm(h) * weight   (gdn2_residual_norm)
  norm_bwd   its gradient, the dropout mask regenerated           (gdn2_residual_norm_bwd)
  gate_bwd   the gradient of the output epilogue                  (gdn2_output_gate_bwd)
  steps      tokens of many sequences against a cache of states   (gdn2_slot_steps, gdn2_slot_steps_logits)
  copy       copy, fork, compact and free states of that cache    (gdn2_state_copy)

``listed()`` names the cases, ``draw(rng)`` gives further ones of the same ranges, ``prepare`` makes a case's
inputs on the GPU from a seed, ``run`` is one call of the operator (in plain torch, or through the library where
``own`` is true), ``work`` counts the bytes and operations the call cannot do without and ``exact`` computes the
result in 64 bits.
"""
import math

import numpy as np
import torch

own = False

EPS = 1e-6
DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp32": 4}

# Philox4x32-10: J. K. Salmon, M. A. Moraes, R. O. Dror, D. E. Shaw, "Parallel random numbers: as easy as 1, 2, 3",
# SC 2011 (multipliers and key increments of the 4x32 variant).
PHILOX_M = (0xD2511F53, 0xCD9E8D57)
PHILOX_W = (0x9E3779B9, 0xBB67AE85)


def listed():
    return [
        # The norm in front of one layer while one sequence decodes: one row of 16 heads x 128 channels; latency only.
        {"name": "norm 1x2048", "op": "norm", "rows": 1, "d": 2048, "stream": "bf16", "branch": "bf16", "r": True,
         "scale": False, "p": 0.0},
        # The same norm in a training step on the 4 x 4096-token batch, with residual scale and dropout.
        {"name": "norm 16384x2048 dropout", "op": "norm", "rows": 16384, "d": 2048, "stream": "bf16",
         "branch": "bf16", "r": True, "scale": True, "p": 0.1},
        # Its gradient on that batch, the residual stream kept in 32 bits.
        {"name": "norm bwd 16384x2048 fp32", "op": "norm_bwd", "rows": 16384, "d": 2048, "stream": "fp32",
         "branch": "bf16", "r": True, "scale": True, "p": 0.1},
        # A narrow odd width and few rows: a small model's step.
        {"name": "norm bwd 777x1021", "op": "norm_bwd", "rows": 777, "d": 1021, "stream": "bf16", "branch": "bf16",
         "r": True, "scale": False, "p": 0.0},
        # The epilogue's gradient on the 4 x 4096 x 16-head batch.
        {"name": "gate bwd 4x4096x16", "op": "gate_bwd", "B": 4, "T": 4096, "H": 16, "dv": 128, "dt": "bf16"},
        # The same in 32 bits on a short odd sequence with heads of 64.
        {"name": "gate bwd 1x257x3 fp32", "op": "gate_bwd", "B": 1, "T": 257, "H": 3, "dv": 64, "dt": "fp32"},
        # One sequence decodes one token from pre-activation logits, epilogue included: latency.
        {"name": "step 1 from logits", "op": "steps", "N": 1, "H": 16, "dk": 128, "dv": 128, "dt": "bf16",
         "most": 1, "logits": True, "gate": True, "keep": False, "slots": 64},
        # A full serving batch, one token each, states scattered over a larger cache.
        {"name": "step 256", "op": "steps", "N": 256, "H": 16, "dk": 128, "dv": 128, "dt": "bf16", "most": 1,
         "logits": False, "gate": False, "keep": False, "slots": 320},
        # Drafts of 1 to 8 tokens verified in one pass, states kept after the accepted ones.
        {"name": "verify 48 x 1..8", "op": "steps", "N": 48, "H": 16, "dk": 128, "dv": 128, "dt": "bf16", "most": 8,
         "logits": True, "gate": True, "keep": True, "slots": 64},
        # 32-bit values, heads of 64, an odd batch with two or three tokens at a time.
        {"name": "step 33 fp32 d64", "op": "steps", "N": 33, "H": 5, "dk": 64, "dv": 64, "dt": "fp32", "most": 3,
         "logits": False, "gate": False, "keep": False, "slots": 40},
        # One prompt's state forked to eight samples.
        {"name": "fork 1 to 8", "op": "copy", "L": 1, "slots": 32, "n": 8, "H": 16, "dk": 128, "dv": 128,
         "kind": "fork"},
        # The live states of four layers moved together, some slots swapped, some freed.
        {"name": "move 96 x 4 layers", "op": "copy", "L": 4, "slots": 160, "n": 96, "H": 16, "dk": 128, "dv": 128,
         "kind": "mixed"},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "norm_bwd", "gate_bwd", "steps", "steps", "copy"])
    if op in ("norm", "norm_bwd"):
        d = _log(rng, 64, 8192)
        if rng.random() < 0.6:
            d = max(64, d // 8 * 8)
        stream = rng.choice(["bf16", "bf16", "fp32"])
        branch = "bf16" if stream == "bf16" else rng.choice(["bf16", "fp32"])
        r = rng.random() < 0.85
        return {"op": op, "rows": _log(rng, 1, min(65536, (1 << 25) // d)), "d": d, "stream": stream,
                "branch": branch, "r": r, "scale": r and rng.random() < 0.5,
                "p": rng.choice([0.0, 0.1, rng.uniform(0.01, 0.7)]) if r else 0.0}
    if op == "gate_bwd":
        B, H = rng.randint(1, 8), rng.randint(1, 32)
        return {"op": op, "B": B, "T": _log(rng, 1, max(1, (1 << 18) // (B * H))), "H": H,
                "dv": rng.choice([64, 128]), "dt": rng.choice(["bf16", "bf16", "fp32"])}
    if op == "steps":
        most = rng.choice([1, 1, 1, 2, 4, 8, 16])
        H = rng.randint(1, 32)
        n = _log(rng, 1, max(1, min(256, (4096 if most < 4 else 8192 // most) // H)))
        logits = rng.random() < 0.5
        return {"op": op, "N": n, "H": H, "dk": rng.choice([64, 128, 128]), "dv": rng.choice([64, 128, 128]),
                "dt": "bf16" if logits else rng.choice(["bf16", "fp32"]), "most": most, "logits": logits,
                "gate": rng.random() < 0.6, "keep": most > 1 and rng.random() < 0.6,
                "slots": n + rng.randint(0, 64)}
    L, H = rng.choice([1, 1, 2, 4]), rng.randint(1, 16)
    n = _log(rng, 1, max(1, 384 // L * 16 // H // 2))
    return {"op": op, "L": L, "slots": n + rng.randint(1, 64), "n": n, "H": H, "dk": rng.choice([64, 128]),
            "dv": rng.choice([64, 128]), "kind": rng.choice(["fork", "mixed"])}


# ---- inputs ----------------------------------------------------------------------------------------------------


class _Draws:
    """Normal and uniform draws on the GPU from one seed."""

    def __init__(self, seed):
        self.gen = torch.Generator(device=DEV)
        self.gen.manual_seed(int(seed))

    def normal(self, *shape, std=1.0, mean=0.0, dtype=torch.float32):
        return (torch.randn(*shape, generator=self.gen, device=DEV) * std + mean).to(dtype)

    def uniform(self, lo, hi, *shape):
        return torch.rand(*shape, generator=self.gen, device=DEV) * (hi - lo) + lo

    def permutation(self, n):
        return torch.randperm(n, generator=self.gen, device=DEV)

    def integers(self, lo, hi, *shape):
        return torch.randint(lo, hi, shape, generator=self.gen, device=DEV)


def prepare(case, seed):
    g = _Draws(seed)
    return {"norm": _prepare_norm, "norm_bwd": _prepare_norm_bwd, "gate_bwd": _prepare_gate_bwd,
            "steps": _prepare_steps, "copy": _prepare_copy}[case["op"]](dict(case), g, int(seed))


def _prepare_norm(c, g, seed):
    """A layer's residual stream (grows over the layers: std 2), its block's output, learned weights near one."""
    n, d, ts, tb = c["rows"], c["d"], TYPES[c["stream"]], TYPES[c["branch"]]
    x = g.normal(n, d, std=2.0, dtype=ts).view(1, n, d)
    s = {"case": c, "x": x, "r": g.normal(n, d, dtype=tb).view(1, n, d) if c["r"] else None,
         "weight": 1.0 + g.normal(d, std=0.1), "scale": g.uniform(0.05, 0.5, d) if c["scale"] else None,
         "rng": torch.tensor([seed * 7919 + 3, (1 << 33) + seed], dtype=torch.int64, device=DEV)}
    s["out"] = {"h": torch.empty_like(x) if c["r"] else None, "y": torch.empty(1, n, d, dtype=tb, device=DEV),
                "rstd": torch.empty(1, n, device=DEV)}
    return s


def _prepare_norm_bwd(c, g, seed):
    n, d, ts, tb = c["rows"], c["d"], TYPES[c["stream"]], TYPES[c["branch"]]
    h = g.normal(n, d, std=2.0, dtype=ts).view(1, n, d)
    s = {"case": c, "h": h, "rstd": torch.rsqrt(h.float().square().mean(-1) + EPS),
         "dy": g.normal(n, d, dtype=tb).view(1, n, d), "dh": g.normal(n, d, dtype=ts).view(1, n, d),
         "r": g.normal(n, d, dtype=tb).view(1, n, d) if c["scale"] else None,
         "weight": 1.0 + g.normal(d, std=0.1), "scale": g.uniform(0.05, 0.5, d) if c["scale"] else None,
         "rng": torch.tensor([seed * 104729 + 11, (5 << 32) + seed], dtype=torch.int64, device=DEV)}
    s["out"] = {"dx": torch.empty_like(h), "dr": torch.empty_like(s["dy"]) if c["r"] else None,
                "dweight": torch.empty(d, device=DEV), "dscale": torch.empty(d, device=DEV) if c["scale"] else None}
    return s


def _prepare_gate_bwd(c, g, seed):
    shape, t = (c["B"], c["T"], c["H"], c["dv"]), TYPES[c["dt"]]
    s = {"case": c, "o": g.normal(*shape, std=0.5, dtype=t), "g": g.normal(*shape, dtype=t),
         "dy": g.normal(*shape, dtype=t), "weight": 1.0 + g.normal(c["dv"], std=0.1)}
    s["out"] = {"do": torch.empty_like(s["o"]), "dg": torch.empty_like(s["o"]),
                "dweight": torch.empty(c["dv"], device=DEV)}
    return s


def _prepare_steps(c, g, seed):
    """A cache of states, a slot for each sequence, and the tokens of this pass with the recipe's distributions."""
    N, H, dk, dv, t = c["N"], c["H"], c["dk"], c["dv"], TYPES[c["dt"]]
    rng = np.random.RandomState(seed % (1 << 31))
    lens = rng.permutation(_lengths(c))
    cu = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    T = int(cu[-1])
    s = {"case": c, "pool": g.normal(c["slots"], H, dk, dv, std=0.1),
         "slots": g.permutation(c["slots"])[:N].to(torch.int32), "longest": int(lens.max()),
         "cu": torch.from_numpy(cu).to(DEV) if c["most"] > 1 else None,
         "keep": torch.from_numpy(rng.randint(0, lens + 1).astype(np.int32)).to(DEV) if c["keep"] else None,
         "out": torch.empty(T, H, dv, dtype=t, device=DEV), "T": T}
    if c["logits"]:
        for n, d, mean in (("q", dk, 0.0), ("k", dk, 0.0), ("v", dv, 0.0), ("a", dk, -2.0), ("b", dk, 0.0),
                           ("w", dv, 0.0)):
            s[n] = g.normal(T, H, d, mean=mean, dtype=t)
    else:
        for n in ("q", "k"):
            x = g.normal(T, H, dk)
            s[n] = (x / x.norm(dim=-1, keepdim=True)).to(t)
        x = g.normal(T, H, dv)
        s["v"] = (x * torch.sigmoid(x)).to(t)
        s["a"] = torch.sigmoid(-g.normal(T, H, dk, mean=-2.0))
        s["b"], s["w"] = torch.sigmoid(g.normal(T, H, dk)), torch.sigmoid(g.normal(T, H, dv))
    s["gate"] = g.normal(T, H, dv, dtype=t) if c["gate"] else None
    s["weight"] = 1.0 + g.normal(dv, std=0.1) if c["gate"] else None
    return s


def _prepare_copy(c, g, seed):
    """fork: one source, n other destinations.  mixed: half of the pairs move states into free slots or swap them,
    the rest free slots (a source of -1)."""
    n, slots = c["n"], c["slots"]
    p = g.permutation(slots)
    if c["kind"] == "fork":
        src, dst = p[:1].expand(n).clone(), p[1:n + 1]
    else:
        dst = p[:n]
        src = dst[g.permutation(n)].clone()               # a permutation: swaps and longer cycles
        src[: n // 4] = p[(torch.arange(n // 4, device=DEV) + n) % slots]   # plain moves
        src[n - n // 8:] = -1                              # freed slots
    return {"case": c, "pool": g.normal(c["L"], slots, c["H"], c["dk"], c["dv"], std=0.1),
            "src": src.to(torch.int32), "dst": dst.to(torch.int32)}


# ---- one pass --------------------------------------------------------------------------------------------------


def run(s):
    c = s["case"]
    if own:
        import gated_delta_rule_111_b200 as gdn2
        return _run_own(gdn2, c["op"], s)
    return {"norm": _plain_norm, "norm_bwd": _plain_norm_bwd, "gate_bwd": _plain_gate_bwd, "steps": _plain_steps,
            "copy": _plain_copy}[c["op"]](s, c)


def _run_own(gdn2, op, s):
    c = s["case"]
    if op == "norm":
        h, y, rstd = gdn2.gdn2_residual_norm(s["x"], s["r"], s["weight"], EPS, scale=s["scale"], p=c["p"],
                                             rng=s["rng"] if c["p"] else None, **s["out"])
        return {"h": h, "y": y, "rstd": rstd} if c["r"] else {"y": y, "rstd": rstd}
    if op == "norm_bwd":
        g = gdn2.gdn2_residual_norm_bwd(s["dy"], s["h"], s["rstd"], s["weight"], dh=s["dh"], r=s["r"],
                                        scale=s["scale"], p=c["p"], rng=s["rng"] if c["p"] else None,
                                        branch=c["r"], out=s["out"])
        return {k: g[k] for k in ("dx", "dr", "dweight", "dscale") if g[k] is not None}
    if op == "gate_bwd":
        return gdn2.gdn2_output_gate_bwd(s["dy"], s["o"], s["g"], s["weight"], EPS, out=s["out"])
    if op == "steps":
        step = gdn2.gdn2_slot_steps_logits if c["logits"] else gdn2.gdn2_slot_steps
        o = step(s["q"], s["k"], s["v"], s["a"], s["b"], s["w"], s["pool"], s["slots"], s["cu"], keep=s["keep"],
                 g=s["gate"], weight=s["weight"], eps=EPS, o=s["out"])
        return {"o": o, "pool": s["pool"]}
    return gdn2.gdn2_state_copy(s["pool"], s["src"], s["dst"])


def _words(rng, rows, groups):
    """Philox words [rows, 4 * groups] (int64 values below 2^32): counter (group, row, offset), key the seed.
    64-bit products wrap, which leaves their low 64 bits right."""
    low = 0xFFFFFFFF
    seed, offset = rng[0], rng[1]
    c0 = torch.arange(groups, device=DEV).expand(rows, groups)
    c1 = torch.arange(rows, device=DEV).unsqueeze(1).expand(rows, groups)
    c2, c3 = (offset & low).expand(rows, groups), ((offset >> 32) & low).expand(rows, groups)
    k0, k1 = seed & low, (seed >> 32) & low
    for i in range(10):
        m0, m1 = c0 * PHILOX_M[0], c2 * PHILOX_M[1]
        c0, c1, c2, c3 = ((m1 >> 32) & low) ^ c1 ^ k0, m1 & low, ((m0 >> 32) & low) ^ c3 ^ k1, m0 & low
        k0, k1 = (k0 + PHILOX_W[0]) & low, (k1 + PHILOX_W[1]) & low
    return torch.stack((c0, c1, c2, c3), dim=-1).view(rows, 4 * groups)


def _plain_drop(x, s, c):
    """x over 1 - p where kept, else zero."""
    if not c["p"]:
        return x
    d = c["d"]
    keep = _words(s["rng"], c["rows"], (d + 3) // 4)[:, :d] >= int(c["p"] * 4294967296.0)
    return torch.where(keep.view(x.shape), x * (1.0 / (1.0 - c["p"])), torch.zeros_like(x))


def _plain_norm(s, c):
    h = s["x"].float()
    if c["r"]:
        b = _plain_drop(s["r"].float(), s, c)
        h = h + (b * s["scale"] if c["scale"] else b)
    rstd = torch.rsqrt(h.square().mean(-1) + EPS)
    y = (h * rstd.unsqueeze(-1) * s["weight"]).to(TYPES[c["branch"]])
    return {"h": h.to(TYPES[c["stream"]]), "y": y, "rstd": rstd} if c["r"] else {"y": y, "rstd": rstd}


def _plain_norm_bwd(s, c):
    h, dy, rstd = s["h"].float(), s["dy"].float(), s["rstd"].unsqueeze(-1)
    n = h * rstd
    t = dy * s["weight"]
    dx = rstd * (t - n * (t * n).mean(-1, keepdim=True)) + s["dh"].float()
    out = {"dx": dx.to(TYPES[c["stream"]]), "dweight": (dy * n).flatten(0, 1).sum(0, dtype=torch.float64).float()}
    if c["r"]:
        out["dr"] = _plain_drop(dx * s["scale"] if c["scale"] else dx, s, c).to(TYPES[c["branch"]])
    if c["scale"]:
        out["dscale"] = (dx * _plain_drop(s["r"].float(), s, c)).flatten(0, 1).sum(0, dtype=torch.float64).float()
    return out


def _plain_gate_bwd(s, c):
    t = TYPES[c["dt"]]
    o, dy, sg = s["o"].float(), s["dy"].float(), torch.sigmoid(s["g"].float())
    rstd = torch.rsqrt(o.square().mean(-1, keepdim=True) + EPS)
    n = o * rstd
    dn = dy * s["weight"] * sg
    return {"do": (rstd * (dn - n * (dn * n).mean(-1, keepdim=True))).to(t), "dg": (dn * n * (1.0 - sg)).to(t),
            "dweight": (dy * n * sg).flatten(0, 2).sum(0, dtype=torch.float64).float()}


def _plain_tokens(s, c):
    """q, k, v, alpha, b, w in 32 bits, from the pre-activation logits where the case has them."""
    q, k, v, a, b, w = (s[n].float() for n in ("q", "k", "v", "a", "b", "w"))
    if c["logits"]:
        q, k, v = q * torch.sigmoid(q), k * torch.sigmoid(k), v * torch.sigmoid(v)
        q = q * torch.rsqrt(q.square().sum(-1, keepdim=True))
        k = k * torch.rsqrt(k.square().sum(-1, keepdim=True))
        a, b, w = torch.sigmoid(-a), torch.sigmoid(b), torch.sigmoid(w)
    return q, k, v, a, b, w


def _plain_steps(s, c):
    """All sequences side by side, one token of each at a time."""
    q, k, v, a, b, w = _plain_tokens(s, c)
    N = c["N"]
    start = torch.arange(N + 1, device=DEV) if s["cu"] is None else s["cu"].long()
    lens = start[1:] - start[:-1]
    keep = lens if s["keep"] is None else s["keep"].long()
    slots = s["slots"].long()
    S = s["pool"][slots]
    kept = S
    o = torch.empty(s["T"], c["H"], c["dv"], device=DEV)
    for t in range(s["longest"]):
        at = torch.minimum(start[:-1] + t, start[1:] - 1)       # a sequence that has ended repeats its last token
        live = (t < lens).view(N, 1, 1, 1)
        D = S * a[at].unsqueeze(-1)
        read = (D * (b[at] * k[at]).unsqueeze(-1)).sum(-2)
        new = D + k[at].unsqueeze(-1) * (w[at] * v[at] - read).unsqueeze(-2)
        S = torch.where(live, new, S) if c["most"] > 1 else new
        kept = torch.where((t < keep).view(N, 1, 1, 1), S, kept) if c["keep"] else S
        o[at] = torch.where(live[..., 0], (S * q[at].unsqueeze(-1)).sum(-2), o[at])
    s["pool"][slots] = kept
    if c["gate"]:
        o = o * torch.rsqrt(o.square().mean(-1, keepdim=True) + EPS) * s["weight"] * torch.sigmoid(s["gate"].float())
    return {"o": o.to(TYPES[c["dt"]]), "pool": s["pool"]}


def _plain_copy(s, c):
    src, dst = s["src"].long(), s["dst"].long()
    moved = s["pool"][:, src.clamp(min=0)]
    s["pool"][:, dst] = torch.where((src >= 0).view(1, -1, 1, 1, 1), moved, torch.zeros_like(moved))
    return s["pool"]


# ---- what a pass cannot do without -----------------------------------------------------------------------------


def _lengths(c):
    """How many tokens the sequences of a pass have, in no order: 1 to most, each as often as the others."""
    return 1 + np.arange(c["N"]) % c["most"]


def work(c):
    if c["op"] == "norm":
        n, s, b = c["rows"] * c["d"], SIZE[c["stream"]], SIZE[c["branch"]]
        return {"bytes": n * (s + b + ((s + b) if c["r"] else 0)) + c["rows"] * 4 + c["d"] * (8 if c["scale"] else 4),
                "flops": n * (9 if c["r"] else 5)}
    if c["op"] == "norm_bwd":
        n, s, b = c["rows"] * c["d"], SIZE[c["stream"]], SIZE[c["branch"]]
        read = b + 2 * s + (b if c["scale"] else 0)
        return {"bytes": n * (read + s + (b if c["r"] else 0)) + c["rows"] * 4 + c["d"] * (16 if c["scale"] else 8),
                "flops": n * 14}
    if c["op"] == "gate_bwd":
        n = c["B"] * c["T"] * c["H"] * c["dv"]
        return {"bytes": 5 * n * SIZE[c["dt"]] + 8 * c["dv"], "flops": n * 20}
    if c["op"] == "steps":
        T, H, dk, dv = int(_lengths(c).sum()), c["H"], c["dk"], c["dv"]
        e, f = SIZE[c["dt"]], 2 if c["logits"] else 4
        token = (2 * dk + dv) * e + (2 * dk + dv) * f + dv * e * (2 if c["gate"] else 1)
        # `keep` is uniform in 0..length, and a state of which no token is kept is not written
        written = 1.0 - float((1.0 / (1.0 + _lengths(c))).mean()) if c["keep"] else 1.0
        return {"bytes": c["N"] * H * dk * dv * 4 * (1.0 + written) + T * H * token, "flops": T * H * dk * dv * 7}
    row = c["H"] * c["dk"] * c["dv"] * 4
    reads = 1 if c["kind"] == "fork" else c["n"] - c["n"] // 8
    return {"bytes": c["L"] * row * (reads + c["n"]), "flops": 0}


# ---- 64 bits ---------------------------------------------------------------------------------------------------


def exact(case, seed):
    s = prepare(case, seed)
    return {"norm": _exact_norm, "norm_bwd": _exact_norm_bwd, "gate_bwd": _exact_gate_bwd, "steps": _exact_steps,
            "copy": _exact_copy}[case["op"]](s, s["case"])


def _kept(s, c):
    """The dropout mask, word by word in numpy's unsigned integers; a factor of 1 / (1 - p) or 0 per element."""
    rows, d = c["rows"], c["d"]
    if not c["p"]:
        return torch.ones(1, rows, d, dtype=torch.float64, device=DEV)
    u32 = np.uint64(0xFFFFFFFF)
    seed, offset = (int(v) & (2**64 - 1) for v in s["rng"].cpu().numpy())
    x = np.empty((4, rows, (d + 3) // 4), dtype=np.uint64)
    x[0], x[1] = np.arange(x.shape[2], dtype=np.uint64)[None, :], np.arange(rows, dtype=np.uint64)[:, None]
    x[2], x[3] = offset & 0xFFFFFFFF, offset >> 32
    key = [seed & 0xFFFFFFFF, seed >> 32]
    for _ in range(10):
        a, b = x[0] * np.uint64(PHILOX_M[0]), x[2] * np.uint64(PHILOX_M[1])
        x[0], x[2] = (b >> np.uint64(32)) ^ x[1] ^ np.uint64(key[0]), (a >> np.uint64(32)) ^ x[3] ^ np.uint64(key[1])
        x[1], x[3] = b & u32, a & u32
        key = [(key[i] + PHILOX_W[i]) & 0xFFFFFFFF for i in range(2)]
    words = np.moveaxis(x, 0, -1).reshape(rows, -1)[:, :d]
    keep = torch.from_numpy(words >= np.uint64(math.floor(c["p"] * 2**32))).to(DEV)
    return keep.double().view(1, rows, d) / (1.0 - c["p"])


def _exact_norm(s, c):
    h = s["x"].double()
    if c["r"]:
        branch = s["r"].double() * _kept(s, c)
        h += branch * s["scale"].double() if c["scale"] else branch
    rms = torch.sqrt((h * h).sum(-1) / c["d"] + EPS)
    out = {"y": h / rms[..., None] * s["weight"].double(), "rstd": 1.0 / rms}
    return {"h": h, **out} if c["r"] else out


def _exact_norm_bwd(s, c):
    h, dy, rstd, w = s["h"].double(), s["dy"].double(), s["rstd"].double()[..., None], s["weight"].double()
    dot = (h * dy * w).sum(-1, keepdim=True)
    dx = s["dh"].double() + rstd * w * dy - h * rstd**3 * dot / c["d"]
    out = {"dx": dx, "dweight": (dy * h * rstd).sum((0, 1))}
    if c["r"]:
        kept = _kept(s, c)
        out["dr"] = dx * kept * s["scale"].double() if c["scale"] else dx * kept
        if c["scale"]:
            out["dscale"] = (dx * kept * s["r"].double()).sum((0, 1))
    return out


def _exact_gate_bwd(s, c):
    o, g, dy, w = s["o"].double(), s["g"].double(), s["dy"].double(), s["weight"].double()
    rms = torch.sqrt((o * o).sum(-1, keepdim=True) / c["dv"] + EPS)
    e = torch.exp(-g)
    sg = 1.0 / (1.0 + e)
    dot = (o * dy * w * sg).sum(-1, keepdim=True)
    return {"do": dy * w * sg / rms - o * dot / (c["dv"] * rms**3), "dg": dy * o / rms * w * e / (1.0 + e) ** 2,
            "dweight": (dy * o / rms * sg).sum((0, 1, 2))}


def _exact_steps(s, c):
    """One token of one sequence at a time."""
    H, dk, dv = c["H"], c["dk"], c["dv"]
    q, k, v, a, b, w = (s[n].double() for n in ("q", "k", "v", "a", "b", "w"))
    if c["logits"]:
        q, k, v = (x / (1.0 + torch.exp(-x)) for x in (q, k, v))
        q, k = (x / torch.linalg.vector_norm(x, dim=-1, keepdim=True) for x in (q, k))
        a, b, w = 1.0 / (1.0 + torch.exp(a)), 1.0 / (1.0 + torch.exp(-b)), 1.0 / (1.0 + torch.exp(-w))
    cu = list(range(c["N"] + 1)) if s["cu"] is None else s["cu"].tolist()
    slots = s["slots"].tolist()
    keep = None if s["keep"] is None else s["keep"].tolist()
    pool, o = s["pool"], torch.empty(s["T"], H, dv, dtype=torch.float64, device=DEV)
    for n in range(c["N"]):
        S = pool[slots[n]].double()
        done = cu[n + 1] - cu[n] if keep is None else keep[n]
        for i, t in enumerate(range(cu[n], cu[n + 1])):
            gain = w[t] * v[t] - torch.einsum("hk,hkv->hv", a[t] * b[t] * k[t], S)
            S = a[t][:, :, None] * S + k[t][:, :, None] * gain[:, None, :]
            o[t] = torch.einsum("hk,hkv->hv", q[t], S)
            if i + 1 == done:
                pool[slots[n]] = S.float()
    if c["gate"]:
        o = o / torch.sqrt((o * o).sum(-1, keepdim=True) / dv + EPS) * s["weight"].double()
        o = o / (1.0 + torch.exp(-s["gate"].double()))
    return {"o": o, "pool": pool}


def _exact_copy(s, c):
    before, src, dst = s["pool"].clone(), s["src"].tolist(), s["dst"].tolist()
    for i, j in zip(src, dst):
        s["pool"][:, j] = before[:, i] if i >= 0 else 0.0
    return s["pool"].double()
