"""The operators around the recurrence run together, as a layer trains and as it serves.

Training: two pre-norm blocks' worth of calls (norm with residual scale and dropout, projections in torch, the FP32
recurrence, the output epilogue) and every gradient by the library's backward calls, against torch's automatic
differentiation of a plain token loop in 64 bits.  Each library gradient is within 1e-4 of its largest values (the
bound of its own tests, against RMS); five of them follow one another and their errors add, through maps that
change a vector's norm by less than two here: 1e-3 of a gradient's norm.

Serving: prompts prefilled from the cache's own slots, forked, continued by drafts of which some are kept, moved,
continued; every output against the 64-bit token loop over each branch's own tokens, bounded like the prefill that
it starts from (FP32: 1e-4 of the RMS).
"""
import pytest
import torch

import plain64 as p64

pytestmark = pytest.mark.gpu

F32 = torch.float32


@pytest.fixture(scope="module")
def g():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import gated_delta_rule_111_b200 as mod
    mod.load_library()
    return mod


def test_training_step(g):
    B, T, H, d = 2, 37, 2, 64
    D, p, eps = 96, 0.2, 1e-5
    gen = torch.Generator("cuda").manual_seed(3)
    n = lambda *s: torch.randn(*s, generator=gen, device="cuda")
    x, r0 = n(B, T, D), n(B, T, D)                          # the stream and the branch of the block before
    w1, w2, s1, s2, wo = 1 + 0.1 * n(D), 1 + 0.1 * n(D), 0.5 + 0.1 * n(D), 0.5 + 0.1 * n(D), 1 + 0.1 * n(d)
    W, Wg, Wout = n(6, D, H * d) / D ** 0.5, n(D, H * d) / D ** 0.5, n(H * d, D) / (H * d) ** 0.5
    dy, dh = n(B, T, D), n(B, T, D)
    rng = [torch.tensor([99, layer], device="cuda") for layer in range(2)]

    def prep(z):                                            # [6,B,T,H,d] logits to the recurrence's inputs
        unit = lambda t: t / torch.linalg.vector_norm(t, dim=-1, keepdim=True)
        silu = lambda t: t * torch.sigmoid(t)
        return unit(silu(z[0])), unit(silu(z[1])), silu(z[2]), torch.sigmoid(2 - z[3]), torch.sigmoid(z[4]), torch.sigmoid(z[5])

    # the library's forward and backward, the projections' by hand
    h1, y1, r1 = g.gdn2_residual_norm(x, r0, w1, eps, scale=s1, p=p, rng=rng[0])
    z = torch.einsum("btd,ndk->nbtk", y1.double(), W.double()).view(6, B, T, H, d).requires_grad_()
    rec = [t.float().contiguous() for t in prep(z)]
    o, ST = g.gdn2_chunk_fwd(*(t.detach() for t in rec))
    gl = (y1.double() @ Wg.double()).view(B, T, H, d)
    go = g.gdn2_output_gate(o, gl.float(), wo, eps)
    br = (go.double().view(B, T, H * d) @ Wout.double()).float()
    h2, y2, r2 = g.gdn2_residual_norm(h1, br, w2, eps, scale=s2, p=p, rng=rng[1])

    b2 = g.gdn2_residual_norm_bwd(dy, h2, r2, w2, dh=dh, r=br, scale=s2, p=p, rng=rng[1])
    d_go = (b2["dr"].double() @ Wout.double().T).view(B, T, H, d)
    bg = g.gdn2_output_gate_bwd(d_go.float(), o, gl.float(), wo, eps)
    bc = g.gdn2_chunk_bwd(*(t.detach() for t in rec), None, bg["do"])
    dz, = torch.autograd.grad(prep(z), z, [bc[k].double() for k in ("dq", "dk", "dv", "dalpha", "db", "dw")])
    d_y1 = torch.einsum("nbtk,ndk->btd", dz.reshape(6, B, T, H * d), W.double()) \
        + bg["dg"].double().view(B, T, H * d) @ Wg.double().T
    b1 = g.gdn2_residual_norm_bwd(d_y1.float(), h1, r1, w1, dh=b2["dx"], r=r0, scale=s1, p=p, rng=rng[0])

    # the same in 64 bits by automatic differentiation
    leaves = {k: v.double().requires_grad_() for k, v in dict(x=x, r0=r0, w1=w1, s1=s1, w2=w2, s2=s2, wo=wo).items()}
    kept = [p64.dropout_factor(B * T, D, p, 99, layer).view(B, T, D).cuda() for layer in range(2)]
    rms = lambda t: t / torch.sqrt((t * t).mean(-1, keepdim=True) + eps)
    H1 = leaves["x"] + leaves["s1"] * leaves["r0"] * kept[0]
    Y1 = rms(H1) * leaves["w1"]
    q, k, v, a, b, w = prep(torch.einsum("btd,ndk->nbtk", Y1, W.double()).view(6, B, T, H, d))
    S, outs = torch.zeros(B, H, d, d, dtype=torch.float64, device="cuda"), []
    for t in range(T):
        Sb = a[:, t, :, :, None] * S
        u = w[:, t] * v[:, t] - torch.einsum("bhk,bhkv->bhv", b[:, t] * k[:, t], Sb)
        S = Sb + k[:, t, :, :, None] * u[:, :, None, :]
        outs.append(torch.einsum("bhk,bhkv->bhv", q[:, t], S))
    go64 = rms(torch.stack(outs, 1)) * leaves["wo"] * torch.sigmoid((Y1 @ Wg.double()).view(B, T, H, d))
    H2 = H1 + leaves["s2"] * (go64.reshape(B, T, H * d) @ Wout.double()) * kept[1]
    Y2 = rms(H2) * leaves["w2"]
    ((dy.double() * Y2).sum() + (dh.double() * H2).sum()).backward()

    assert float((y2.double() - Y2.detach()).norm() / Y2.detach().norm()) < 1e-3
    got = dict(x=b1["dx"], r0=b1["dr"], w1=b1["dweight"], s1=b1["dscale"], w2=b2["dweight"], s2=b2["dscale"], wo=bg["dweight"])
    for name, t in got.items():
        ref = leaves[name].grad
        off = float((t.double() - ref).norm() / ref.norm())
        assert off < 1e-3, f"gradient of {name}: {off:.2e}"


def test_backward_captured_beside_a_live_eager_graph(g):
    """The backward calls captured while a torch graph of the same leaves is alive, then replayed on new values."""
    B, T, D = 2, 64, 256
    gen = torch.Generator("cuda").manual_seed(4)
    n = lambda *s: torch.randn(*s, generator=gen, device="cuda")
    x, r, w, dy = n(B, T, D).requires_grad_(), n(B, T, D).requires_grad_(), torch.ones(D, device="cuda").requires_grad_(), n(B, T, D)
    eager = (torch.nn.functional.rms_norm(x + r, (D,), w, 1e-6) * dy).sum()
    call = lambda: g.gdn2_residual_norm_bwd(dy, *(t for i, t in enumerate(g.gdn2_residual_norm(
        x.detach(), r.detach(), w.detach())) if i != 1), w.detach())
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = call()
    eager.backward()
    for _ in range(2):
        graph.replay()
        torch.cuda.synchronize()
        assert float((out["dx"] - x.grad).norm() / x.grad.norm()) < 1e-5
        assert float((out["dweight"] - w.grad).norm() / w.grad.norm()) < 1e-5
        with torch.no_grad():
            dy.mul_(2.0), x.grad.mul_(2.0), w.grad.mul_(2.0)


def test_serving_loop(g):
    H, d, slots = 2, 64, 12
    gen = torch.Generator("cuda").manual_seed(5)
    n = lambda *s: torch.randn(*s, generator=gen, device="cuda")

    def tokens(T):
        unit = lambda t: t / t.norm(dim=-1, keepdim=True)
        return [unit(n(T, H, d)), unit(n(T, H, d)), n(T, H, d), torch.sigmoid(2 - n(T, H, d)), torch.sigmoid(n(T, H, d)),
                torch.sigmoid(n(T, H, d))]

    def index(v):
        return torch.tensor(v, dtype=torch.int32, device="cuda")

    def same(x, ref):
        assert float((x.double() - ref).abs().max() / ref.square().mean().sqrt()) < 1e-4

    def loop(ts, S):
        o, S, _, _ = p64.steps(*ts, S, ts[0].shape[0])
        return o, S

    pool = n(slots, H, d, d)                                # whatever earlier requests left there
    ref = pool.double()
    # two prompts of 70 and 33 tokens: their slots are freed, read as start states, and take the end states
    g.gdn2_state_copy(pool, index([-1, -1]), index([7, 2]))
    start = torch.empty(2, H, d, d, device="cuda")
    g.gdn2_state_copy(start, index([7, 2]), index([0, 1]), source=pool)
    prompt = tokens(103)
    o, ST = g.gdn2_chunk_fwd_varlen(*prompt, index([0, 70, 103]), start)
    g.gdn2_state_copy(pool, index([0, 1]), index([7, 2]), source=ST)
    ref[7], ref[2] = 0.0, 0.0
    for rows, s in ((slice(0, 70), 7), (slice(70, 103), 2)):
        y, ref[s] = loop([t[rows] for t in prompt], ref[s])
        same(o[rows], y)
        same(pool[s], ref[s])
    # the first is forked twice; each branch gets a token of its own
    g.gdn2_state_copy(pool, index([7, 7]), index([0, 5]))
    ref[0], ref[5] = ref[7], ref[7]
    ts, at = tokens(4), [7, 0, 5, 2]
    o = g.gdn2_slot_steps(*ts, pool, index(at))
    for i, s in enumerate(at):
        y, ref[s] = loop([t[i:i + 1] for t in ts], ref[s])
        same(o[i:i + 1], y)
    # drafts of 4, 2, 5, 3 tokens, of which 2, 2, 0, 1 are kept, with one row of padding
    ts, lens, kept = tokens(15), [4, 2, 5, 3, 1], [2, 2, 0, 1, 1]
    o = g.gdn2_slot_steps(*ts, pool, index(at + [-1]), index([0, 4, 6, 11, 14, 15]), keep=index(kept))
    row = 0
    for i, s in enumerate(at):
        part = [t[row:row + lens[i]] for t in ts]
        y, _ = loop(part, ref[s])
        same(o[row:row + lens[i]], y)
        if kept[i]:
            _, ref[s] = loop([t[:kept[i]] for t in part], ref[s])
        row += lens[i]
    # one branch ends, the others move to the front of the cache, and go on
    g.gdn2_state_copy(pool, index([7, 5, 2, -1, -1]), index([0, 1, 2, 5, 7]))
    ref[0], ref[1], ref[2], ref[5], ref[7] = ref[7].clone(), ref[5].clone(), ref[2].clone(), 0.0, 0.0
    ts = tokens(3)
    o = g.gdn2_slot_steps(*ts, pool, index([0, 1, 2]))
    for i in range(3):
        y, ref[i] = loop([t[i:i + 1] for t in ts], ref[i])
        same(o[i:i + 1], y)
    for s in range(slots):
        if s in (5, 7):
            assert bool((pool[s] == 0).all())
        else:
            same(pool[s], ref[s])


def test_logits_prefill_continued_by_steps(g):
    """gdn2_chunk_fwd_logits' end state continued by gdn2_slot_steps_logits equals the loop over all tokens, within
    the prefill's own bound for BF16 (2e-2 of the RMS beyond rounding for o, 1e-2 for the state)."""
    H, d, T, more = 2, 128, 90, 6
    gen = torch.Generator("cuda").manual_seed(6)
    n = lambda *s: torch.randn(*s, generator=gen, device="cuda")
    z = [(n(1, T + more, H, d) - (2 if i == 3 else 0)).bfloat16() for i in range(6)]
    _, ST = g.gdn2_chunk_fwd_logits(*(t[:, :T].contiguous() for t in z))
    pool = torch.zeros(3, H, d, d, device="cuda")
    g.gdn2_state_copy(pool, torch.tensor([0], dtype=torch.int32, device="cuda"),
                      torch.tensor([2], dtype=torch.int32, device="cuda"), source=ST)
    o = g.gdn2_slot_steps_logits(*(t[0, T:].contiguous() for t in z), pool,
                                 torch.tensor([2], dtype=torch.int32, device="cuda"),
                                 torch.tensor([0, more], dtype=torch.int32, device="cuda"))
    y, S, _, _ = p64.steps(*(t[0] for t in p64.prepare(*z)), torch.zeros(H, d, d, device="cuda"), T + more)
    y, rms = y[T:], y[T:].square().mean().sqrt()
    assert float(((o.double() - y).abs() - 2 ** -8 * y.abs()).max() / rms) < 2e-2
    assert float((pool[2].double() - S).abs().max() / S.square().mean().sqrt()) < 1e-2
