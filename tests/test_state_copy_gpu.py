"""gdn2_state_copy: every pair reads what was there before the call; bits move unchanged."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def g():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import gated_delta_rule_111_b200 as mod
    mod.load_library()
    return mod


def plain(before, src, dst, source=None):
    out, source = before.clone(), before if source is None else source
    for i, j in zip(src, dst):
        if 0 <= j < out.shape[-4] and -1 <= i < source.shape[-4]:
            out[..., j, :, :, :] = source[..., i, :, :, :] if i >= 0 else 0.0
    return out


def index(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def states(*shape, seed=0):
    return torch.randn(*shape, generator=torch.Generator("cuda").manual_seed(seed), device="cuda")


CASES = {
    "one": ([3], [5]),
    "swap": ([2, 7], [7, 2]),
    "cycle and chain": ([1, 2, 3, 5, 6], [2, 3, 1, 6, 7]),
    "fork": ([4] * 6, [0, 1, 2, 3, 5, 6]),
    "free": ([-1, -1], [0, 9]),
    "skipped": ([0, 10, -2, 1, 2], [10, 1, 2, -1, 3]),
    "last pair counts": ([1, 2, 3, -1, 5], [0, 0, 4, 4, 0]),
    "onto itself": ([3, 3, 4], [3, 5, 4]),
}


@pytest.mark.parametrize("layers", [None, 3])
@pytest.mark.parametrize("dims", [(1, 64, 64), (3, 64, 128), (2, 128, 128)], ids=str)
@pytest.mark.parametrize("case", CASES)
def test_pairs(g, case, dims, layers):
    src, dst = CASES[case]
    pool = states(*(() if layers is None else (layers,)), 10, *dims)
    want = plain(pool, src, dst)
    assert g.gdn2_state_copy(pool, index(src), index(dst)) is pool
    assert torch.equal(pool, want)


@pytest.mark.parametrize("n", [1, 2, 3, 31, 255, 700, 2049, 4096])
def test_many_pairs(g, n):
    """A random permutation of all slots with some freed, at sizes on both sides of every slice width."""
    slots = max(n, 2)
    pool = states(slots, 1, 64, 64, seed=n)
    perm = torch.randperm(slots, generator=torch.Generator().manual_seed(n)).tolist()[:n]
    src = [-1 if i % 7 == 3 else perm[(i + 1) % n] for i in range(n)]
    want = plain(pool, src, perm)
    g.gdn2_state_copy(pool, index(src), index(perm))
    assert torch.equal(pool, want)


def test_one_destination_many_times(g):
    """All pairs name two slots; the last pair of each counts (long probe sequences of equal keys)."""
    pool = states(6, 1, 64, 64, seed=4)
    src, dst = [i % 6 for i in range(1000)], [i % 2 for i in range(1000)]
    want = plain(pool, src, dst)
    g.gdn2_state_copy(pool, index(src), index(dst))
    assert torch.equal(pool, want)


def test_between_two_pools(g):
    pool, batch = states(2, 12, 2, 128, 64, seed=1), states(2, 3, 2, 128, 64, seed=2)
    want = plain(pool, [2, 0, -1], [11, 4, 0], batch)
    g.gdn2_state_copy(pool, index([2, 0, -1]), index([11, 4, 0]), source=batch)
    assert torch.equal(pool, want)
    back = torch.empty_like(batch)
    g.gdn2_state_copy(back, index([11, 4, 0]), index([2, 0, 1]), source=pool)
    assert torch.equal(back[:, 2], batch[:, 2]) and torch.equal(back[:, 0], batch[:, 0]) and bool((back[:, 1] == 0).all())


def test_nothing_to_do(g):
    pool = states(4, 1, 64, 64, seed=3)
    before = pool.clone()
    g.gdn2_state_copy(pool, index([]), index([]))
    assert torch.equal(pool, before)


def test_special_values_move_unchanged(g):
    pool = states(4, 1, 64, 64, seed=5)
    bits = pool.view(torch.int32)
    bits[1, 0, 0, :4] = torch.tensor([0x7F800001, 0x7FC12345, -1, 0x00000001], dtype=torch.int32, device="cuda")
    want = bits[1].clone()
    g.gdn2_state_copy(pool, index([1]), index([3]))
    assert torch.equal(bits[3], want)


def test_offsets_past_32_bits(g):
    """The last slots of a pool of more than 2^31 floats."""
    layers, slots = 8, 520
    big = torch.zeros(layers, slots, 64, 128, 64, device="cuda")           # 2 MiB a state
    assert big.numel() > 2 ** 31
    big[-1, slots - 1], big[:, 2] = 3.0, 5.0
    g.gdn2_state_copy(big, index([slots - 1, 2]), index([1, slots - 2]))
    assert bool((big[-1, 1] == 3.0).all()) and bool((big[:-1, 1] == 0).all()) and bool((big[:, 0] == 0).all())
    assert bool((big[:, slots - 2] == 5.0).all()) and bool((big[:, slots - 3] == 0).all())


def test_replayed_and_on_a_side_stream(g):
    pool = states(8, 2, 64, 64, seed=6)
    src, dst = index([0, 1]), index([1, 0])
    g.gdn2_state_copy(pool.clone(), src, dst)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        g.gdn2_state_copy(pool, src, dst)
    before = pool.clone()
    for a, b in (([0, 1], [1, 0]), ([2, -1], [3, 4])):
        src.copy_(index(a)), dst.copy_(index(b))
        want = plain(before, a, b)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(pool, want)
        before = want
    s = torch.cuda.Stream()
    g.gdn2_state_copy(pool, index([5]), index([6]), stream=s)
    s.synchronize()
    assert torch.equal(pool[6], before[5])
