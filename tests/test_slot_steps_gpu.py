"""gdn2_slot_steps and gdn2_slot_steps_logits against a 64-bit token loop whose rounding bound is carried along
(plain64.steps).  Inputs prepared from logits start 100 * 2^-24 off: the sigmoid's exponential 2 + 1.2 |x| steps
(|x| up to 8 here) twice in silu, a norm of 128 squares (10 additions, rsqrtf) and the products.
"""
import pytest
import torch

import plain64 as p64

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def g():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import gated_delta_rule_111_b200 as mod
    mod.load_library()
    mod.gdn2_device_error()
    yield mod
    assert mod.gdn2_device_error() == 0


def index(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def draw(T, H, dk, dv, dt, logits, n_slots, seed=0):
    gen = torch.Generator("cuda").manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=gen, device="cuda")
    if logits:
        t = [n(T, H, dk).to(BF), n(T, H, dk).to(BF), n(T, H, dv).to(BF), (n(T, H, dk) - 2).to(BF), n(T, H, dk).to(BF),
             n(T, H, dv).to(BF)]
    else:
        unit = lambda x: x / x.norm(dim=-1, keepdim=True)
        t = [unit(n(T, H, dk)).to(dt), unit(n(T, H, dk)).to(dt), n(T, H, dv).to(dt), torch.sigmoid(2 - n(T, H, dk)),
             2 * torch.sigmoid(n(T, H, dk)), torch.sigmoid(n(T, H, dv))]
    return t, 0.2 * n(n_slots, H, dk, dv), n(T, H, dv).to(dt), 1 + 0.1 * n(dv)


def check(g, lens, slots, H=2, dk=128, dv=128, dt=BF, logits=False, gate=False, keep=None, n_slots=None, tail=0,
          seed=0, x=None):
    """One call against the loop; rows behind the last sequence and slots that no sequence has stay as they were."""
    n_slots = n_slots or max(max(slots) + 2, 1)
    T = sum(lens) + tail
    t, pool, gl, w = draw(T, H, dk, dv, dt, logits, n_slots, seed) if x is None else x
    before, o = pool.clone(), torch.full((T, H, dv), 7.0, dtype=dt, device="cuda")
    cu = index([sum(lens[:i]) for i in range(len(lens) + 1)])
    step = g.gdn2_slot_steps_logits if logits else g.gdn2_slot_steps
    kw = dict(g=gl, weight=w, eps=1e-5) if gate else {}
    out = step(*t, pool, index(slots), cu, keep=None if keep is None else index(keep), o=o, **kw)
    assert out is o
    ins = p64.prepare(*t) if logits else t
    rel = 100 * p64.U if logits else 0.0
    touched, at = set(), 0
    for i, (n, s) in enumerate(zip(lens, slots)):
        rows = slice(at, at + n)
        at += n
        if n == 0:
            continue
        if not 0 <= s < n_slots:
            assert bool((o[rows] == 0).all())
            continue
        kept = n if keep is None else min(max(keep[i], 0), n)
        y, S, ey, eS = p64.steps(*(a[rows] for a in ins), before[s], kept, rel)
        if gate:
            y, ey = p64.gate(y, ey, gl[rows], w, 1e-5)
        p64.assert_close(f"o of sequence {i}", o[rows], y, ey / p64.U, 1)
        if kept:
            p64.assert_close(f"state of sequence {i}", pool[s], S, eS / p64.U, 1)
            touched.add(s)
    assert bool((o[at:] == 7.0).all())
    rest = [s for s in range(n_slots) if s not in touched]
    assert torch.equal(pool[rest], before[rest])
    return o, pool


@pytest.mark.parametrize("gate", [False, True])
@pytest.mark.parametrize("kind", ["bf16", "fp32", "logits"])
@pytest.mark.parametrize("dims", [(128, 128), (64, 64), (128, 64), (64, 128)], ids=str)
def test_ragged_tokens(g, dims, kind, gate):
    check(g, [1, 0, 3, 8, 9, 2, 17], [4, 1, 0, 6, 2, 8, 3], 2, *dims, dt=F32 if kind == "fp32" else BF,
          logits=kind == "logits", gate=gate, tail=3, seed=sum(dims))


@pytest.mark.parametrize("logits", [False, True])
def test_kept_tokens(g, logits):
    """keep below 0, 0, inside, at and above the number of tokens."""
    check(g, [4, 4, 4, 9, 9, 1, 1, 0], [0, 2, 4, 6, 8, 1, 3, 5], keep=[-3, 0, 2, 8, 40, 0, 1, 5], logits=logits, seed=3)


def test_one_token_each_without_offsets(g):
    """cu_seqlens None; equal to the decode step on the gathered states up to the order of its sums."""
    N, H = 5, 3
    (q, k, v, a, b, w), pool, _, _ = draw(N, H, 128, 128, BF, False, 9, seed=5)
    slots = index([8, 0, 3, 1, 6])
    S = pool[slots.long()].clone()
    before = pool.clone()
    o = g.gdn2_slot_steps(q, k, v, a, b, w, pool, slots)
    for i in range(N):
        y, S64, ey, eS = p64.steps(*(x[i:i + 1] for x in (q, k, v, a, b, w)), before[slots[i]], 1)
        p64.assert_close("o", o[i:i + 1], y, ey / p64.U, 1)
        p64.assert_close("state", pool[slots[i]], S64, eS / p64.U, 1)
    o2 = g.gdn2_recurrent_step(q, k, v, a, b, w, S)
    assert float((pool[slots.long()] - S).abs().max()) < 1e-5 * float(S.abs().max())
    assert float((o.float() - o2.float()).abs().max()) <= 2 ** -7 * float(o2.float().abs().max())


def test_padding_slots(g):
    check(g, [2, 1, 3, 1], [-1, 1, 99, -2147483648], n_slots=4, gate=True, seed=6)


def test_shared_slots(g):
    """Readers may share a slot; where one of them writes, all of that slot are refused and reported."""
    check(g, [3, 2, 1, 4], [2, 2, 0, 2], keep=[0, 0, 1, 0], seed=7)
    t, pool, _, _ = draw(7, 2, 128, 128, BF, False, 4, seed=8)
    before = pool.clone()
    o = g.gdn2_slot_steps(*t, pool, index([3, 1, 3, 0]), index([0, 2, 4, 6, 7]), keep=index([0, 2, 1, 1]))
    assert g.gdn2_device_error() == 0x10000 and g.gdn2_device_error() == 0
    assert torch.equal(pool[[2, 3]], before[[2, 3]]) and not torch.equal(pool[1], before[1])
    assert bool((o[:2] == 0).all()) and bool((o[4:6] == 0).all()) and bool((o[2:4] != 0).any()) and bool((o[6] != 0).any())
    # a sequence without tokens shares nothing
    g.gdn2_slot_steps(*(x[:2] for x in t), pool, index([3, 3]), index([0, 2, 2]))
    assert g.gdn2_device_error() == 0


@pytest.mark.parametrize("shift", [0, 1])
@pytest.mark.parametrize("N", [130, 517, 1031])
def test_shared_slots_among_many(g, N, shift):
    """A slot named twice, at both ends and at every distance from a multiple of four, in an aligned slots tensor
    and in one that is not."""
    t, pool, _, _ = draw(N, 1, 64, 64, F32, False, N, seed=N)
    buffer = torch.empty(N + 1, dtype=torch.int32, device="cuda")
    slots = buffer[shift:N + shift]
    for first, second in ((0, N - 1), (N - 2, N - 1), (1, 127), (2, N // 2), (N // 2 + 3, N - 3)):
        slots.copy_(torch.arange(N, device="cuda"))
        slots[second] = first
        state = pool.clone()
        o = g.gdn2_slot_steps(*t, state, slots)
        assert g.gdn2_device_error() == 0x10000
        dead = torch.zeros(N, dtype=torch.bool, device="cuda")
        dead[[first, second]] = True
        assert torch.equal((o == 0).all(-1).flatten(), dead)
        assert torch.equal(state[first], pool[first]) and torch.equal(state[second], pool[second])
        assert bool((state != pool).flatten(1).any(1)[~dead].all())


def test_bad_offsets_stay_inside(g):
    """Offsets below zero, falling and past the end are clamped: no sequence reads or writes outside."""
    t, pool, _, _ = draw(6, 1, 64, 64, F32, False, 5, seed=9)
    o = torch.full((6, 1, 64), 7.0, device="cuda")
    g.gdn2_slot_steps(*t, pool, index([0, 1, 2, 3]), index([-5, 2, 1, 4, 1000]), o=o)
    assert bool(torch.isfinite(o).all()) and bool((o != 7.0).all())


def test_strong_and_no_decay_zero_rows_and_idle_gates(g):
    x = draw(12, 2, 128, 128, F32, False, 3, seed=10)
    (q, k, v, a, b, w), pool, gl, wt = x
    a[0], a[1], a[2, :, ::2], k[3], q[4], b[5], w[6] = 0.0, 1.0, 1e-30, 0.0, 0.0, 0.0, 0.0
    pool[1] = 0.0
    check(g, [12], [1], dt=F32, n_slots=3, x=x)
    y = draw(6, 2, 128, 128, BF, True, 3, seed=11)
    y[0][0][0], y[0][1][1], y[0][3][2], y[0][3][3], y[0][4][4], y[0][2][5] = 0.0, 0.0, 30.0, -30.0, -20.0, 0.0
    check(g, [6], [1], logits=True, n_slots=3, x=y, gate=True)


def test_special_values_stay_in_their_sequence(g):
    """NaN and infinities of one sequence, of padding and of unused slots reach no other sequence."""
    t, pool, _, _ = draw(6, 2, 128, 128, BF, False, 6, seed=12)
    clean_t, clean = [x.clone() for x in t], pool.clone()
    t[0][2:4], t[2][4], pool[5] = float("nan"), float("inf"), float("nan")
    slots, cu = index([0, 1, -1, 2]), index([0, 2, 4, 5, 6])
    o, o2 = g.gdn2_slot_steps(*t, pool, slots, cu), g.gdn2_slot_steps(*clean_t, clean, slots, cu)
    for rows, s in ((slice(0, 2), 0), (slice(5, 6), 2)):
        assert torch.equal(o[rows], o2[rows]) and torch.equal(pool[s], clean[s])
    assert bool((o[4] == 0).all()) and bool(torch.isnan(o[2:4]).all())


def test_many_sequences_and_long_ones(g):
    check(g, [1] * 300, [(7 * i) % 300 for i in range(300)], H=1, dk=64, dv=64, dt=F32, seed=13)
    check(g, [200], [0], H=1, seed=14)


def test_no_sequences_and_no_tokens(g):
    t, pool, _, _ = draw(0, 2, 128, 128, BF, False, 2)
    before = pool.clone()
    assert g.gdn2_slot_steps(*t, pool, index([])).shape == (0, 2, 128)
    g.gdn2_slot_steps(*t, pool, index([0, 1]), index([0, 0, 0]))
    assert torch.equal(pool, before)


def test_pool_past_32_bits(g):
    """A state whose floats start behind 2^31."""
    H, n = 8, 16500
    pool = torch.zeros(n, H, 128, 128, device="cuda")
    assert (n - 2) * H * 128 * 128 > 2 ** 31
    t, small, _, _ = draw(2, H, 128, 128, BF, False, 2, seed=15)
    pool[n - 1], pool[n - 2] = small[0], small[1]
    o = g.gdn2_slot_steps(*t, pool, index([n - 1, n - 2]))
    o2 = g.gdn2_slot_steps(*t, small, index([0, 1]))
    assert torch.equal(o, o2) and torch.equal(pool[n - 1], small[0]) and torch.equal(pool[n - 2], small[1])


def test_replayed_and_on_a_side_stream(g):
    """A captured batch of fixed size: slots, lengths and kept tokens change between replays."""
    t, pool, gl, w = draw(8, 2, 128, 128, BF, True, 6, seed=16)
    slots, cu, keep = index([0, 1, 2, -1]), index([0, 2, 4, 6, 8]), index([2, 2, 2, 2])
    o = torch.empty(8, 2, 128, dtype=BF, device="cuda")
    call = lambda pool, o, s=None: g.gdn2_slot_steps_logits(*t, pool, slots, cu, keep=keep, g=gl, weight=w, o=o, stream=s)
    call(pool.clone(), o)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(pool, o)
    s = torch.cuda.Stream()
    for a, b, c in (([0, 1, 2, -1], [0, 2, 4, 6, 8], [2, 2, 2, 2]), ([5, -1, 3, 4], [0, 1, 1, 5, 8], [0, 0, 3, 1])):
        slots.copy_(index(a)), cu.copy_(index(b)), keep.copy_(index(c))
        twin, o2 = pool.clone(), torch.empty_like(o)
        torch.cuda.synchronize()
        call(twin, o2, s)
        s.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(pool, twin) and torch.equal(o, o2)
