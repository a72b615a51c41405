"""Copying, clearing and compacting slots of state pools on the GPU: bytes are moved, so every result is
compared exactly with the same moves made one after the other on the host."""
import pytest
import torch

from selective_state_space_conv1d_amd import ssd

pytestmark = pytest.mark.gpu
DEV = "cuda"


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def rand(*shape, dtype=torch.float32, seed=0):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to(dtype)


def host_copy(dst, di, src, si, axis):
    for d, s in zip(di, si):
        if 0 <= d < dst.shape[axis] and 0 <= s < src.shape[axis]:
            dst.select(axis, d).copy_(src.select(axis, s).clone())
    return dst


SLOT = [(8,), (4, 2), (131, 64), (16384,), (24, 1031, 4)]      # 16 bytes .. several workgroups, ragged ends
LISTS = [([0], [3]), ([1, 2, 9], [4, 4, 4]), ([], []), ([5, -1, 7, 10, 3], [0, 1, -2, 2, 11]),
         ([6, 6, 6], [0, 1, 2]),                  # one destination three times: the last stays
         ([1, 2, 3, 4], [0, 1, 2, 3]),            # a chain: each copies what the one before it left
         ([0, 1, 0], [1, 0, 9]), ([3, 4], [3, 3])]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("slot", SLOT)
@pytest.mark.parametrize("pair", LISTS)
def test_copy_within_a_pool(pair, slot, dtype):
    pool = rand(10, *slot, dtype=dtype)
    want = pool.clone()
    host_copy(want, pair[0], want, pair[1], 0)
    got = pool.to(DEV)
    assert ssd.ssd_pool_copy(got, i32(pair[0]), got, i32(pair[1])) is got
    assert torch.equal(got.cpu(), want)


@pytest.mark.parametrize("pair", LISTS)
def test_copy_between_pools_of_layers(pair):
    dst, src = rand(3, 10, 72, 16), rand(3, 12, 72, 16, seed=1)
    want = host_copy(dst.clone(), pair[0], src, pair[1], 1)
    got, from_ = dst.to(DEV), src.to(DEV)
    ssd.ssd_pool_copy(got, i32(pair[0]), from_, i32(pair[1]), stacked=True)
    assert torch.equal(got.cpu(), want) and torch.equal(from_.cpu(), src)


def test_copy_of_many_entries():
    """More entries than threads; slots whose numbers agree in many low bits."""
    pool = rand(20000, 4)
    g = torch.Generator().manual_seed(5)
    p = torch.randperm(20000, generator=g)
    di, si = p[:700].tolist(), p[700:1400].tolist()
    want = pool.clone()
    want[p[:700]] = pool[p[700:1400]]
    got = pool.to(DEV)
    ssd.ssd_pool_copy(got, i32(di), got, i32(si))
    assert torch.equal(got.cpu(), want)
    got = pool.to(DEV)
    ssd.ssd_pool_copy(got, i32([8192, 0, 16384]), got, i32([5, 6, 7]))
    want = pool.clone()
    want[[8192, 0, 16384]] = pool[[5, 6, 7]]
    assert torch.equal(got.cpu(), want)


@pytest.mark.parametrize("di,si", [([131077, 5, 262149, 9], [1, 2, 3, 4]),           # destinations that share a bit
                                   ([4, 131081, 7], [262153, 9, 131076]),            # a source that shares one
                                   ([131072, 299999, 131071], [299999, 131072, 0]),  # the last bit and the first; a swap
                                   ([299999, -1, 300000], [131072, 299999, 5])])
def test_pools_of_more_slots_than_the_bitmap_has_bits(di, si):
    pool = rand(300000, 4)
    want = pool.clone()
    host_copy(want, di, want, si, 0)
    got = pool.to(DEV)
    ssd.ssd_pool_copy(got, i32(di), got, i32(si))
    assert torch.equal(got.cpu(), want)


def test_source_slots_past_the_destinations():
    """One pool named twice, as destination by its first 40 slots only."""
    pool = rand(100, 4)
    want = pool.clone()
    host_copy(want[:40], [39, 7, 8, 41], want, [99, 64, 32, 3], 0)
    got = pool.to(DEV)
    ssd.ssd_pool_copy(got[:40], i32([39, 7, 8, 41]), got, i32([99, 64, 32, 3]))
    assert torch.equal(got.cpu(), want)


def test_pools_past_32_bits():
    pool = torch.zeros(2, 9, 300 << 20, dtype=torch.int8, device=DEV)      # slots of 300 MiB: layer 1 lies past 2 GiB
    pool[1, 8, ::4097] = torch.arange(pool[1, 8, ::4097].numel(), device=DEV).to(torch.int8)
    pool[0, 8, -5:] = 7
    ssd.ssd_pool_copy(pool, i32([0, 7]), pool, i32([8, 8]), stacked=True)
    for d in (0, 7):
        assert torch.equal(pool[0, d], pool[0, 8]) and torch.equal(pool[1, d], pool[1, 8])
    assert int(pool[:, 1:7].count_nonzero()) == 0
    ssd.ssd_pool_clear(pool, i32([8]), stacked=True)
    assert int(pool[:, 8].count_nonzero()) == 0


def test_infinities_and_nans_are_bytes():
    pool = torch.tensor([[float("nan"), float("inf"), -0.0, 1.0], [0.0, 0, 0, 0]])
    got = pool.to(DEV)
    ssd.ssd_pool_copy(got, i32([1]), got, i32([0]))
    assert torch.equal(got.cpu().view(torch.int32)[1], pool.view(torch.int32)[0])


@pytest.mark.parametrize("slot", SLOT)
def test_clear(slot):
    pool = torch.full((2, 6, *slot), float("nan"), device=DEV)
    ssd.ssd_pool_clear(pool, i32([4, 1, 4, -1, 6]), stacked=True)
    assert bool((pool[:, [1, 4]] == 0).all()) and bool(pool[:, [0, 2, 3, 5]].isnan().all())


def host_plan(slots, nslots):
    used = {s for s in slots if 0 <= s < nslots}
    live, count = sorted(used), len(used)
    holes = [s for s in range(count) if s not in used]
    movers = [s for s in live if s >= count]
    to = dict(zip(movers, holes))
    pad = [-1] * (len(slots) - len(movers))
    return movers + pad, holes + pad, [to.get(s, s) for s in slots], count


@pytest.mark.parametrize("slots,nslots", [([], 5), ([0], 1), ([4], 5), ([0, 1, 2], 3), ([7, 3, 5], 9), ([7, 7, -1, 2, 9, 12], 9),
                                          ([-1, -1], 4), ([3], 0)])
def test_plan(slots, nslots):
    src, dst, new, count = ssd.ssd_pool_compact(i32(slots), nslots)
    assert (src.tolist(), dst.tolist(), new.tolist(), int(count)) == host_plan(slots, nslots)


@pytest.mark.parametrize("nslots,n", [(31, 9), (32, 32), (33, 20), (1000, 400), (40000, 3000), (131072, 5000), (131072, 131072)])
def test_plan_of_random_pools(nslots, n):
    slots = torch.randperm(nslots, generator=torch.Generator().manual_seed(n))[:n].tolist()
    src, dst, new, count = ssd.ssd_pool_compact(i32(slots), nslots)
    assert (src.tolist(), dst.tolist(), new.tolist(), int(count)) == host_plan(slots, nslots)


def test_compaction_under_a_graph():
    """Plan, moves in two pools and the clearing of the freed slots as one captured graph, replayed with new
    tables: every request finds its states under its new slot, and what was free is zero."""
    table = i32([0] * 6)
    pool, conv = torch.zeros(2, 16, 40, 16, device=DEV), torch.zeros(16, 48, 4, dtype=torch.bfloat16, device=DEV)

    def step():
        src, dst, new, count = ssd.ssd_pool_compact(table, 16)
        ssd.ssd_pool_copy(pool, dst, pool, src, stacked=True)
        ssd.ssd_pool_copy(conv, dst, conv, src)
        ssd.ssd_pool_clear(pool, src, stacked=True)
        ssd.ssd_pool_clear(conv, src)
        return new, count

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        new, count = step()
    for slots in ([15, 2, 9, 0, 4, 11], [1, 2, 3, 4, 5, 6], [10, 11, 12, 13, -1, 14], [15, 15, 14, 0, 0, -1]):
        a, b = rand(2, 16, 40, 16, seed=slots[0] + 2), rand(16, 48, 4, dtype=torch.bfloat16, seed=slots[1])
        pool.copy_(a)
        conv.copy_(b)
        table.copy_(i32(slots))
        graph.replay()
        torch.cuda.synchronize()
        src, _, want, n = host_plan(slots, 16)
        assert new.tolist() == want and int(count) == n
        for s, t in zip(slots, want):
            if s >= 0:
                assert t < n and torch.equal(pool[:, t].cpu(), a[:, s]) and torch.equal(conv[t].cpu(), b[s])
        for s in src:
            assert s < 0 or (float(pool[:, s].abs().sum()) == 0 and float(conv[s].abs().sum()) == 0)


def test_copy_on_two_streams():
    pools = [rand(8, 4096, seed=i).to(DEV) for i in range(2)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in pools]
    idx = [i32([1, 2]), i32([0, 3])]
    torch.cuda.synchronize()
    for p, st in zip(pools, streams):
        ssd.ssd_pool_copy(p, idx[0], p, idx[1], stream=st)
    torch.cuda.synchronize()
    for i, p in enumerate(pools):
        want = rand(8, 4096, seed=i)
        want[[1, 2]] = want[[0, 3]]
        assert torch.equal(p.cpu(), want)
