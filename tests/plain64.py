"""Plain 64-bit forms of the operators around the recurrence, with a-priori rounding bounds, for the tests.

A comparison allows |x - ref| <= half a step of x's type at |ref| plus k * 2^-24 * scale, where ``scale`` is the
sum of the magnitudes that the 32-bit arithmetic adds up for that element and k counts its roundings.
"""
import numpy as np
import torch

U = 2.0 ** -24                                   # half a step of fp32, relative


def half_step(t):
    return torch.finfo(t).eps / 2


def assert_close(name, x, ref, scale, k):
    """|x - ref| <= half a step of x's type at |ref| + k roundings of ``scale`` in 32 bits (+ the denormal step)."""
    x64, ref = x.double(), ref.to(x.device)
    scale = torch.as_tensor(scale, dtype=torch.float64, device=x.device)
    bound = (half_step(x.dtype) if x.dtype != torch.float32 else 0.0) * ref.abs() + k * U * scale * (1 + 2.0 ** -7) + 2.0 ** -126
    off = (x64 - ref).abs() / bound
    worst = float(off.max()) if off.numel() else 0.0
    assert worst <= 1.0, f"{name}: {worst:.3f} of the bound at {np.unravel_index(int(off.argmax()), tuple(off.shape))}"
    return worst


PHILOX_KAT = (((0, 0, 0, 0), (0, 0), (0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8)),
              ((0xFFFFFFFF,) * 4, (0xFFFFFFFF,) * 2, (0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD)),
              ((0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344), (0xA4093822, 0x299F31D0),
               (0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1)))


def philox(counter, key):
    """Philox4x32-10 on uint64 arrays of 32-bit words; counter [4, ...], key (k0, k1)."""
    c = [np.asarray(w, dtype=np.uint64) for w in counter]
    k0, k1 = int(key[0]), int(key[1])
    lo, hi = np.uint64(0xFFFFFFFF), np.uint64(32)
    for _ in range(10):
        a, b = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        c = [(b >> hi) ^ c[1] ^ np.uint64(k0), b & lo, (a >> hi) ^ c[3] ^ np.uint64(k1), a & lo]
        k0, k1 = (k0 + 0x9E3779B9) & 0xFFFFFFFF, (k1 + 0xBB67AE85) & 0xFFFFFFFF
    return np.stack(c)


def dropout_factor(rows, D, p, seed, offset):
    """[rows, D] float64: 1 / (1 - p) where kept, else 0."""
    if p == 0.0:
        return torch.ones(rows, D, dtype=torch.float64)
    seed, offset = seed & (2**64 - 1), offset & (2**64 - 1)
    shape = (rows, (D + 3) // 4)
    words = philox((np.broadcast_to(np.arange(shape[1], dtype=np.uint64), shape),
                    np.broadcast_to(np.arange(rows, dtype=np.uint64)[:, None], shape),
                    np.full(shape, offset & 0xFFFFFFFF, np.uint64), np.full(shape, offset >> 32, np.uint64)),
                   (seed & 0xFFFFFFFF, seed >> 32))
    words = np.moveaxis(words, 0, -1).reshape(rows, -1)[:, :D]
    return torch.from_numpy((words >= np.uint64(int(p * 2.0 ** 32))).astype(np.float64)) / (1.0 - p)


def sigmoid(x):
    return 1.0 / (1.0 + torch.exp(-x))


def prepare(xq, xk, xv, xa, xb, xw):
    """The recurrence's inputs from pre-activation logits, 64 bits."""
    def unit(x):
        n = torch.linalg.vector_norm(x, dim=-1, keepdim=True)
        return torch.where(n > 0, x / n, torch.zeros_like(x))
    xq, xk, xv, xa, xb, xw = (x.double() for x in (xq, xk, xv, xa, xb, xw))
    return (unit(xq * sigmoid(xq)), unit(xk * sigmoid(xk)), xv * sigmoid(xv), sigmoid(-xa), sigmoid(xb), sigmoid(xw))


def steps(q, k, v, a, b, w, S, keep, rel_in=0.0):
    """Tokens of one sequence, all heads: q,k,a,b [T,H,dk], v,w [T,H,dv], S [H,dk,dv], 64 bits.  Returns
    (o, kept state, bound of o's error, bound of the state's error): the bounds carry every fp32 rounding of
    the recurrence forward as an absolute error, from inputs that are ``rel_in`` off (relatively)."""
    S, eS = S.double().clone(), torch.zeros_like(S, dtype=torch.float64)
    kept, e_kept = S.clone(), eS.clone()
    n = k.shape[-1] / 8 + 8                       # additions behind one column sum
    os, es = [], []
    for t in range(q.shape[0]):
        qt, kt, at, et, zt = (x[t].double() for x in (q, k, a, b, v))
        et, zt = et * kt, w[t].double() * zt
        D = at[:, :, None] * S
        eD = at[:, :, None] * eS + (U + rel_in) * D.abs()
        read, mag = (D * et[:, :, None]).sum(1), (D.abs() * et.abs()[:, :, None]).sum(1)
        e_read = (eD * et.abs()[:, :, None]).sum(1) + ((n + 2) * U + 2 * rel_in) * mag
        u = zt - read
        e_u = e_read + 3 * U * (zt.abs() + u.abs()) + 2 * rel_in * zt.abs()
        S = D + kt[:, :, None] * u[:, None, :]
        eS = eD + kt.abs()[:, :, None] * (e_u + rel_in * u.abs())[:, None, :] + 2 * U * (D.abs() + S.abs())
        kq, mkq = (kt * qt).sum(1, keepdim=True), (kt * qt).abs().sum(1, keepdim=True)
        p, mp = (D * qt[:, :, None]).sum(1), (D.abs() * qt.abs()[:, :, None]).sum(1)
        os.append(p + kq * u)
        es.append((eD * qt.abs()[:, :, None]).sum(1) + ((n + 2) * U + rel_in) * mp + mkq * e_u
                  + (10 * U + 2 * rel_in) * mkq * u.abs() + 2 * U * (p.abs() + os[-1].abs()))
        if t + 1 == keep:
            kept, e_kept = S.clone(), eS.clone()
    return torch.stack(os), kept, torch.stack(es), e_kept


def gate(o, e, g, weight, eps):
    """The output epilogue of o [..., dv] (error bound e) in 64 bits, and the bound of its result's error."""
    s = sigmoid(g.double())
    rms = torch.sqrt((o * o).mean(-1, keepdim=True) + eps)
    y = o / rms * weight.double() * s
    f = (weight.double() * s / rms).abs()
    off = e.square().mean(-1, keepdim=True).sqrt() / rms
    return y, f * e + (off + 48 * U * (1 + g.double().abs())) * y.abs()
