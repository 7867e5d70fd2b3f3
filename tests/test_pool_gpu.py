"""Slots moved within a pool, against the same moves on the CPU; nothing is computed, so all is equal."""
import pytest
import torch

import kimi_delta_attention_23_b200 as kda

pytestmark = pytest.mark.gpu

SHAPES = [(1,), (3,), (2, 128, 128), (5, 37), (4, 33), (1, 128, 130)]


def status():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def pool_of(slots, shape, layers=None, seed=0):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(*([layers] if layers else []), slots, *shape, generator=g)


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("src,dst", [
    ([], []), ([0], [1]), ([2], [2]), ([0, 1], [1, 0]), ([0, 1, 2, 3], [1, 2, 3, 0]), ([0, 0, 0], [1, 2, 3]),
    ([0, 1, 2], [1, 2, 3]), ([3, 2, 1], [2, 1, 0]), ([0, 0, 1], [1, 4, 0]), ([5, -1, 6], [6, -1, 7]), ([0, 1, 1], [0, 0, 2]),
])
@pytest.mark.parametrize("layers", [None, 3])
def test_copy_is_one_assignment(shape, src, dst, layers):
    pool = pool_of(8, shape, layers)
    got, st = pool.cuda(), status()
    kda.kda_pool_copy(got, ints(src), ints(dst), stacked=layers is not None, device_status=st)
    want = pool.clone()
    at = (slice(None),) if layers else ()
    seen = set()
    for s, d in zip(src, dst):
        if d >= 0 and d not in seen:
            want[(*at, d)] = pool[(*at, s)]
        seen.add(d)
    assert torch.equal(got.cpu(), want)
    named_twice = len([d for d in dst if d >= 0]) != len({d for d in dst if d >= 0})
    assert int(st) == (kda.ERR_DEVICE_CHECK if named_twice else 0)


@pytest.mark.parametrize("shape,slots", [((1,), 5000), ((2, 3), 3000), ((128,), 2500), ((4, 128, 128), 70), ((9, 128), 1500)])
@pytest.mark.parametrize("kind", ["rotate", "permute", "disjoint"])
def test_copy_of_many(shape, slots, kind):
    g = torch.Generator().manual_seed(slots)
    pool = pool_of(slots, shape, seed=1)
    order = torch.randperm(slots, generator=g)
    if kind == "rotate":
        src, dst = order, order.roll(1)
    elif kind == "permute":
        src, dst = torch.randint(0, slots, (slots,), generator=g), order
    else:
        src, dst = order[: slots // 2], order[slots - slots // 2:]
    got, st = pool.cuda(), status()
    kda.kda_pool_copy(got, src.int().cuda(), dst.int().cuda(), device_status=st)
    want = pool.clone()
    want[dst] = pool[src]
    assert torch.equal(got.cpu(), want) and int(st) == 0


@pytest.mark.parametrize("src,dst", [([0, 9], [1, 2]), ([0, 3], [1, 9]), ([0, -1], [1, 3]), ([0, 3], [1, -1]), ([0, -2], [1, -2])])
def test_copy_reports_what_is_out_of_range(src, dst):
    pool = pool_of(8, (5, 4))
    got, st = pool.cuda(), status()
    kda.kda_pool_copy(got, ints(src), ints(dst), device_status=st)
    want = pool.clone()
    want[1] = pool[0]
    assert torch.equal(got.cpu(), want) and int(st) == kda.ERR_DEVICE_CHECK


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("layers", [None, 2])
@pytest.mark.parametrize("slots,dead,n", [(5, 2, 2), (40, 20, 13), (2300, 1500, 1400)])
def test_fork(shape, layers, slots, dead, n):
    if slots > 1000 and len(shape) > 2:
        pytest.skip("larger than it needs to be")
    g = torch.Generator().manual_seed(n)
    pool = pool_of(slots, shape, layers)
    live = torch.ones(slots, dtype=torch.int32)
    live[torch.randperm(slots, generator=g)[:dead]] = 0
    used = live.nonzero()[:, 0]
    src = used[torch.randint(0, used.numel(), (n,), generator=g)].int()
    got, marks, st = pool.cuda(), (live * 3).cuda(), status()
    dst = kda.kda_pool_fork(got, marks, src.cuda(), stacked=layers is not None, device_status=st)
    free = (live == 0).nonzero()[:n, 0]
    assert torch.equal(dst.cpu(), free.int()) and int(st) == 0
    want = pool.clone()
    if layers:
        want[:, free] = pool[:, src.long()]
    else:
        want[free] = pool[src.long()]
    live[free] = 1
    assert torch.equal(got.cpu(), want) and torch.equal((marks != 0).int().cpu(), live)


def test_fork_reports_dead_sources_and_a_full_pool():
    pool = pool_of(6, (4, 4))
    live = torch.tensor([1, 0, 1, 0, 1, 0], dtype=torch.int32)
    # padding, a dead source, one that is only being allocated by this call, out of range, then four good ones
    src = [-1, 3, 1, 6, 0, 2, 4, 0]
    got, marks, st = pool.cuda(), live.cuda(), status()
    dst = kda.kda_pool_fork(got, marks, ints(src), device_status=st)
    assert dst.tolist() == [-1, -1, -1, -1, 1, 3, 5, -1] and int(st) == kda.ERR_DEVICE_CHECK
    want = pool.clone()
    want[[1, 3, 5]] = pool[[0, 2, 4]]
    assert torch.equal(got.cpu(), want) and marks.tolist() == [1] * 6
    st = status()
    assert kda.kda_pool_fork(got, marks, ints([-1, -1]), device_status=st).tolist() == [-1, -1] and int(st) == 0
    assert torch.equal(got.cpu(), want)


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("layers", [None, 2])
def test_free(shape, layers):
    pool = pool_of(9, shape, layers)
    got, st = pool.cuda(), status()
    marks = ints([1, 1, 1, 0, 1, 1, 0, 1, 1])
    kda.kda_pool_free(got, marks, ints([8, -1, 0, 4]), stacked=layers is not None, device_status=st)
    want = pool.clone()
    for s in (8, 0, 4):
        want[(slice(None), s) if layers else s] = 0
    assert torch.equal(got.cpu(), want) and marks.tolist() == [0, 1, 1, 0, 0, 1, 0, 1, 0] and int(st) == 0
    for again in ([4], [5, 5], [9], [-2]):  # not live, named twice, out of range
        st = status()
        kda.kda_pool_free(got, marks, ints(again), stacked=layers is not None, device_status=st)
        assert int(st) == kda.ERR_DEVICE_CHECK
    want[(slice(None), 5) if layers else 5] = 0
    assert torch.equal(got.cpu(), want) and marks.tolist() == [0, 1, 1, 0, 0, 0, 0, 1, 0]


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("layers", [None, 2])
@pytest.mark.parametrize("slots,alive", [(1, 0), (1, 1), (2, 1), (9, 4), (33, 33), (64, 0), (1024, 300), (2500, 1600), (3000, 20)])
def test_compact(shape, layers, slots, alive):
    if slots > 1000 and len(shape) > 2:
        pytest.skip("larger than it needs to be")
    g = torch.Generator().manual_seed(slots + alive)
    pool = pool_of(slots, shape, layers)
    used = torch.randperm(slots, generator=g)[:alive]
    live = torch.zeros(slots, dtype=torch.int32)
    live[used] = 2
    got, marks, idx, st = pool.cuda(), live.cuda(), used.int().cuda(), status()
    count = kda.kda_pool_compact(got, marks, idx, stacked=layers is not None, device_status=st)
    assert int(count) == alive and int(st) == 0
    assert torch.equal(marks.cpu(), (torch.arange(slots) < alive).int())
    new = idx.cpu().long()
    assert sorted(new.tolist()) == list(range(alive))
    stay = used < alive
    assert torch.equal(new[stay], used[stay])
    holes = (live[:alive] == 0).nonzero()[:, 0]
    movers = (live[alive:] != 0).nonzero()[:, 0] + alive
    places = {int(m): int(h) for m, h in zip(movers, holes)}
    assert [places[int(u)] for u in used[~stay]] == new[~stay].tolist()
    lead = (slice(None),) if layers else ()
    assert torch.equal(got.cpu()[(*lead, new)], pool[(*lead, used)])


def test_compact_keeps_and_reports_indices_of_dead_slots():
    pool = pool_of(6, (3,))
    got, marks, idx, st = pool.cuda(), ints([0, 1, 0, 0, 1, 0]), ints([4, -1, 3, 1, 4, 7]), status()
    assert kda.kda_pool_compact(got, marks, idx, device_status=st).tolist() == [2]
    assert idx.tolist() == [0, -1, 3, 1, 0, 7] and int(st) == kda.ERR_DEVICE_CHECK
    assert torch.equal(got[0].cpu(), pool[4]) and torch.equal(got[1].cpu(), pool[1])


def test_offsets_past_32_bits():
    # a stack whose last slots lie beyond 2^32 elements' bytes and 2^31 elements
    pool = torch.empty(2, 5, 4, 65536, 1024, device="cuda")  # 2 x 5 slots of 1 GiB
    for layer in range(2):
        for s in range(5):
            pool[layer, s, 0, 0, 0] = 10.0 * layer + s
            pool[layer, s, 3, 65535, 1023] = 10.0 * layer + s + 0.5
    kda.kda_pool_copy(pool, ints([4, 3]), ints([3, 4]), stacked=True)
    for layer in range(2):
        for s, old in enumerate([0, 1, 2, 4, 3]):
            assert float(pool[layer, s, 0, 0, 0]) == 10.0 * layer + old
            assert float(pool[layer, s, 3, 65535, 1023]) == 10.0 * layer + old + 0.5


def test_unaligned_pool():
    flat = torch.randn(1 + 6 * 64, generator=torch.Generator().manual_seed(3))
    got = flat.cuda()
    kda.kda_pool_copy(got[1:].view(6, 64), ints([0, 5]), ints([5, 0]))
    want = flat.clone()
    want[1:].view(6, 64)[[5, 0]] = flat[1:].view(6, 64)[[0, 5]]
    assert torch.equal(got.cpu(), want)


def test_two_graphs_and_another_stream():
    pool = pool_of(16, (4, 128), seed=4)
    got, marks = pool.cuda(), ints([1] * 8 + [0] * 8)
    src = ints([0, 3])
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    outs = []
    for g in graphs:
        with torch.cuda.graph(g):
            outs.append(kda.kda_pool_fork(got, marks, src))
    for i, g in enumerate(graphs):  # each has its own workspace; the second goes on from the first
        g.replay()
        torch.cuda.synchronize()
        assert outs[i].tolist() == [8 + 2 * i, 9 + 2 * i]
    assert torch.equal(got[[8, 9, 10, 11]].cpu(), pool[[0, 3, 0, 3]])
    src.copy_(ints([1, 2]))
    graphs[0].replay()
    torch.cuda.synchronize()
    assert outs[0].tolist() == [12, 13] and torch.equal(got[[12, 13]].cpu(), pool[[1, 2]])
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    kda.kda_pool_free(got, marks, ints([12]), stream=side)
    side.synchronize()
    assert float(got[12].abs().max()) == 0.0 and marks.tolist() == [1] * 12 + [0, 1, 0, 0]
