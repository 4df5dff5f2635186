"""GPU tests of the pages of a pool of states (ssd_cache_copy, ssd_cache_compact)
against the same moves made one after another (causal_ref). Bytes only move, so
every comparison is exact."""
import random

import pytest
import torch

import causal_ref as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ssd():
    import bidirectional_mamba_ssd_b200 as m
    return m


def i32(v):
    return torch.tensor(list(v), dtype=torch.int32, device="cuda")


def pool_of(layers, nslots, page, dtype=torch.float32, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randint(0, 120, (layers, nslots, *page), generator=g, device="cuda").to(dtype)


# layers, slots, page, dtype: 16-, 4- and 1-byte elements, pages past one chunk and below one
POOLS = [(3, 20, (2, 64, 64), torch.float32), (1, 40, (5, 3), torch.float32), (2, 17, (7,), torch.uint8),
         (2, 33, (3, 64), torch.bfloat16), (1, 9, (9,), torch.bfloat16), (12, 70, (128,), torch.float32)]


@pytest.mark.parametrize("pool", POOLS, ids=lambda p: "l%d_s%d_%s_%s" % (p[0], p[1], "x".join(map(str, p[2])), str(p[3])[6:]))
def test_copy(ssd, pool):
    layers, nslots, page, dtype = pool
    rng = random.Random(nslots)
    p = list(range(nslots))
    rng.shuffle(p)
    h = nslots // 2
    lists = [
        ([p[0]], [p[1]]),
        ([p[0]] * (h - 1) , p[1:h]),                                   # a fork
        (p[:h] + [-1] * (nslots - 2 * h), p[h:]),                      # copies and cleared pages, all apart
        ([p[0], p[1], p[2], -1, p[1]], [p[1], p[2], p[3], p[0], p[1]]),   # a chain, a page onto itself
        ([p[i] for i in range(nslots)], [p[(i + 1) % nslots] for i in range(nslots)]),   # a ring, in order
        ([p[3], p[4], p[5]], [p[6], p[6], p[6]]),                      # one page written three times
        ([p[0], -1, p[2]], [-1, -1, p[4]]),                            # pairs left out
        ([rng.randrange(-1, nslots) for _ in range(50)], [rng.randrange(-1, nslots) for _ in range(50)]),
    ]
    for k, (src, dst) in enumerate(lists):
        data = pool_of(layers, nslots, page, dtype, seed=k)
        want = ref.copy(data, i32(src), i32(dst))
        got = ssd.ssd_cache_copy(data, i32(src), i32(dst))
        torch.cuda.synchronize()
        assert got is data and torch.equal(data.cpu(), want), f"list {k}"
    assert ssd.ssd_get_device_status() == 0


def test_copy_bad_indices_and_empty(ssd):
    data = pool_of(2, 6, (33,))
    want = ref.copy(data, i32([0, 6, -2, 1, 3]), i32([1, 2, 3, 7, 4]))
    ssd.ssd_cache_copy(data, i32([0, 6, -2, 1, 3]), i32([1, 2, 3, 7, 4]))
    torch.cuda.synchronize()
    assert ssd.ssd_get_device_status() == ssd.SSD_ERR_INDEX
    assert torch.equal(data.cpu(), want)
    ssd.ssd_cache_copy(data, i32([]), i32([]))
    ssd.ssd_cache_copy(pool_of(0, 3, (4,)), i32([1]), i32([2]))
    torch.cuda.synchronize()
    assert torch.equal(data.cpu(), want) and ssd.ssd_get_device_status() == 0
    with pytest.raises(ValueError):
        ssd.ssd_cache_copy(data, i32([1, 2]), i32([3]))
    with pytest.raises(ValueError):
        ssd.ssd_cache_copy(data, i32([1]).long(), i32([3]))
    with pytest.raises(ValueError):
        ssd.ssd_cache_copy(data[:, :3], i32([1]), i32([2]))
    with pytest.raises(ValueError):
        ssd.ssd_cache_copy(data[0], i32([1]), i32([2]))


@pytest.mark.parametrize("pool", POOLS, ids=lambda p: "l%d_s%d_%s_%s" % (p[0], p[1], "x".join(map(str, p[2])), str(p[3])[6:]))
def test_compact(ssd, pool):
    layers, nslots, page, dtype = pool
    rng = random.Random(nslots)
    tables = [list(range(nslots)), [], [-1, -1], [nslots - 1], [nslots - 1] * 3 + [0],
              rng.sample(range(nslots), nslots // 2), rng.sample(range(nslots), nslots // 3) + [-1] * 5,
              list(range(nslots // 2, nslots)), [s for s in range(1, nslots)]]
    tables.append(tables[5] + tables[5][:3] + [-1])
    for k, table in enumerate(tables):
        data = pool_of(layers, nslots, page, dtype, seed=k)
        want, new, live = ref.compact(data, i32(table))
        t, n = ssd.ssd_cache_compact(data, i32(table))
        torch.cuda.synchronize()
        assert n.item() == live and t.tolist() == new, f"table {k}"
        assert torch.equal(data.cpu(), want), f"table {k}"
    assert ssd.ssd_get_device_status() == 0


def test_compact_many_slots_and_bad_indices(ssd):
    """A map of several words per thread; a table entry out of range."""
    nslots = 40000
    g = torch.Generator().manual_seed(1)
    table = torch.randperm(nslots, generator=g)[:15000].to(torch.int32)
    data = pool_of(1, nslots, (4,), seed=2)
    want, new, live = ref.compact(data, table)
    t, n = ssd.ssd_cache_compact(data, table.cuda())
    torch.cuda.synchronize()
    assert n.item() == live and t.tolist() == new and torch.equal(data.cpu(), want)
    data = pool_of(2, 8, (5,))
    bad = i32([7, 8, -3, 2])
    want, new, live = ref.compact(data, bad)
    t, n = ssd.ssd_cache_compact(data, bad)
    torch.cuda.synchronize()
    assert ssd.ssd_get_device_status() == ssd.SSD_ERR_INDEX
    assert n.item() == live == 2 and t.tolist() == new and torch.equal(data.cpu(), want)


def test_in_a_graph(ssd):
    """Captured once, replayed on changing indices."""
    data = pool_of(2, 10, (64, 4))
    src, dst, table = i32([0, 1]), i32([2, 3]), i32([9, 8, 0])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        ssd.ssd_cache_copy(data, src, dst)
        new, live = ssd.ssd_cache_compact(data, table)
    for k in range(3):
        data.copy_(pool_of(2, 10, (64, 4), seed=k))
        src.copy_(i32([k, k + 1]))
        dst.copy_(i32([k + 1, k + 4]))
        table.copy_(i32([9 - k, 4, 7]))
        want, t, n = ref.compact(ref.copy(data, src, dst), table)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(data.cpu(), want) and new.tolist() == t and live.item() == n


def test_long_lists_and_empty_pools(ssd):
    """More pairs than are kept in shared memory, forks across that border; pools without layers or bytes."""
    nslots = 4000
    data = pool_of(2, nslots, (8,), seed=9)
    p = list(range(nslots))
    random.Random(4).shuffle(p)
    src = [s for s in p[:500] for _ in range(3)] + [-1] * 300
    dst = p[500:2000] + p[2000:2300]
    src[1023:1027] = [p[400]] * 4
    want = ref.copy(data, i32(src), i32(dst))
    ssd.ssd_cache_copy(data, i32(src), i32(dst))
    torch.cuda.synchronize()
    assert torch.equal(data.cpu(), want)
    # the same list over and over its own pages, in order
    src, dst = (src * 2)[:2500], (dst + p[:1000])[:2500]
    want = ref.copy(data, i32(src), i32(dst))
    ssd.ssd_cache_copy(data, i32(src), i32(dst))
    torch.cuda.synchronize()
    assert torch.equal(data.cpu(), want)
    for shape in ((0, 9, 8), (2, 9, 0), (2, 0, 8)):
        empty = torch.zeros(shape, device="cuda")
        t, live = ssd.ssd_cache_compact(empty, i32([7, 8, 2, -1]))
        ssd.ssd_cache_copy(empty, i32([1]), i32([2]))
        torch.cuda.synchronize()
        if shape[1]:
            assert t.tolist() == [0, 1, 2, -1] and live.item() == 3
            assert ssd.ssd_get_device_status() == 0
        else:
            assert t.tolist() == [-1] * 4 and live.item() == 0
            assert ssd.ssd_get_device_status() == ssd.SSD_ERR_INDEX


def test_sizes_past_32_bits_are_refused(ssd):
    """Layers and slots are 32-bit at the boundary: more of them raise instead of wrapping."""
    idx = i32([0])
    for shape in ((2**31, 1, 0), (1, 2**32 + 4, 0)):
        pool = torch.empty(shape, dtype=torch.uint8, device="cuda")
        with pytest.raises(ValueError):
            ssd.ssd_cache_copy(pool, idx, idx)
        with pytest.raises(ValueError):
            ssd.ssd_cache_compact(pool, idx)
