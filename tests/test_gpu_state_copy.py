"""GPU tests of kda_state_copy: bit-exact copies between slots, applied in order."""
import pytest
import torch

from linear_attention_kda_gb300 import kda

pytestmark = pytest.mark.gpu


def _in_order(pool, src, dst, out=None):
    """The definition, on the CPU."""
    out = pool if out is None else out
    for a, b in zip(src, dst):
        if b >= 0:
            out[b] = pool[a] if a >= 0 else torch.zeros_like(out[b])
    return out


def _pool(slots, shape, dtype, seed):
    # any bits at all, those of NaNs among them
    n = slots * torch.Size(shape).numel() * torch.empty((), dtype=dtype).element_size()
    g = torch.Generator().manual_seed(seed)
    return torch.randint(0, 256, (n,), generator=g, dtype=torch.uint8).view(dtype).view((slots,) + tuple(shape))


def _bits(t):
    return t.cpu().contiguous().view(-1).view(torch.uint8)


def _idx(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


SHAPES = [((2, 64, 64), torch.float32), ((4,), torch.float32), ((3, 128, 128), torch.float32), ((5, 8), torch.bfloat16), ((16,), torch.uint8),
          ((1, 1028), torch.float32)]


@pytest.mark.parametrize("shape,dtype", SHAPES)
@pytest.mark.parametrize("P", [1, 2, 7, 8, 9, 40, 300])
def test_random_pairs_in_order(shape, dtype, P):
    """Chains, repeated targets, cleared slots and skipped pairs among 12 slots."""
    g = torch.Generator().manual_seed(P)
    src = torch.randint(-1, 12, (P,), generator=g).tolist()
    dst = torch.randint(-1, 12, (P,), generator=g).tolist()
    pool = _pool(12, shape, dtype, P)
    got = pool.cuda()
    assert kda.state_copy(got, _idx(src), _idx(dst)) is got
    torch.cuda.synchronize()
    assert kda.get_device_error() == 0
    assert torch.equal(_bits(got), _bits(_in_order(pool, src, dst)))


@pytest.mark.parametrize("pairs", [
    [(0, 1), (0, 2), (0, 3), (0, 4)],                            # fork
    [(9, 1), (8, 3), (7, 5)],                                    # compaction into holes
    [(1, 0), (2, 1), (3, 2), (4, 3), (5, 4), (6, 5), (7, 6), (8, 7), (9, 8)],  # every slot moves down by one
    [(0, 9), (1, 0), (9, 1)],                                    # a swap through a spare slot
    [(0, 1), (1, 2), (2, 3), (3, 4), (4, 5), (5, 6), (6, 7), (7, 8), (8, 9)],  # a chain: slot 0 everywhere
    [(-1, 3), (3, 4), (3, 3)],                                   # cleared, then read
    [(2, 2)],
])
@pytest.mark.parametrize("shape", [(2, 64, 64), (32, 128, 128)])
def test_patterns(pairs, shape):
    src, dst = [p[0] for p in pairs], [p[1] for p in pairs]
    pool = _pool(10, shape, torch.float32, 5)
    got = pool.cuda()
    kda.state_copy(got, _idx(src), _idx(dst))
    torch.cuda.synchronize()
    assert kda.get_device_error() == 0
    assert torch.equal(_bits(got), _bits(_in_order(pool, src, dst)))


@pytest.mark.parametrize("P", [1, 5, 130])
def test_between_pools(P):
    """Saving states into a larger pool and back: sources never change, the last writer of a slot wins."""
    g = torch.Generator().manual_seed(P)
    a, b = _pool(7, (2, 64, 64), torch.float32, 1), _pool(150, (2, 64, 64), torch.float32, 2)
    src = torch.randint(-1, 7, (P,), generator=g).tolist()
    dst = torch.randint(-1, 150 if P > 5 else 3, (P,), generator=g).tolist()
    x, y = a.cuda(), b.cuda()
    assert kda.state_copy(x, _idx(src), _idx(dst), out_pool=y) is y
    torch.cuda.synchronize()
    assert kda.get_device_error() == 0
    assert torch.equal(_bits(x), _bits(a)) and torch.equal(_bits(y), _bits(_in_order(a, src, dst, b)))


@pytest.mark.parametrize("pairs", [
    [(i, i + 40) for i in range(40)],                                   # independent: pairs are split over blocks
    [(i, i + 40) for i in range(39)] + [(41, 0)],                       # the last one reads a target
    [(i, i + 40) for i in range(39)] + [(5, 40)],                       # a target twice
    [(i, i) for i in range(80)],                                        # onto themselves
    [(i, i + 40) for i in range(39)] + [(0, 90)],                       # one outside the pool
])
def test_pairs_of_small_slots(pairs):
    pool = _pool(80, (4, 8), torch.float32, 11)
    got = pool.cuda()
    kda.state_copy(got, _idx([p[0] for p in pairs]), _idx([p[1] for p in pairs]))
    bad = [p for p in pairs if max(p) >= 80]
    assert kda.get_device_error() == (8 if bad else 0)
    good = [p for p in pairs if max(p) < 80]
    assert torch.equal(_bits(got), _bits(_in_order(pool, [p[0] for p in good], [p[1] for p in good])))


def test_many_pairs_and_slots():
    """A permutation-like move of many small slots, more than one block's worth of pairs."""
    g = torch.Generator().manual_seed(0)
    pool = _pool(5000, (8,), torch.float32, 3)
    for src, dst in ((torch.randperm(2000, generator=g).add(3000), torch.randperm(2000, generator=g)),   # independent
                     (torch.randint(0, 5000, (4100,), generator=g), torch.randint(0, 5000, (4100,), generator=g))):
        src, dst = src.tolist(), dst.tolist()
        got = pool.cuda()
        kda.state_copy(got, _idx(src), _idx(dst))
        torch.cuda.synchronize()
        assert kda.get_device_error() == 0
        assert torch.equal(_bits(got), _bits(_in_order(pool.clone(), src, dst)))


@pytest.mark.parametrize("src,dst", [([0, 4], [1, 0]), ([0, 1], [1, 4]), ([0, -2], [1, 0]), ([0, 0], [1, -2])])
def test_bad_index_is_reported_and_skipped(src, dst):
    pool = _pool(4, (4, 16), torch.float32, 4)
    got = pool.cuda()
    kda.state_copy(got, _idx(src), _idx(dst))
    assert kda.get_device_error() == 8
    assert torch.equal(_bits(got), _bits(_in_order(pool, src[:1], dst[:1])))


def test_only_clearing_without_a_source_pool():
    empty, out = torch.empty((0, 4, 16), device="cuda"), _pool(4, (4, 16), torch.float32, 4)
    got = out.cuda()
    kda.state_copy(empty, _idx([-1, -1]), _idx([3, 1]), out_pool=got)
    torch.cuda.synchronize()
    assert kda.get_device_error() == 0
    out[3] = out[1] = 0
    assert torch.equal(_bits(got), _bits(out))


def test_offsets_past_32_bits():
    """Slots more than 2^32 bytes apart (and 2^31 elements into the pool)."""
    slots, n = 9, 1 << 27  # 512 MiB a slot
    pool = torch.zeros((slots, n), dtype=torch.float32, device="cuda")
    pool[0, :4] = 3.0
    pool[0, -4:] = 5.0
    kda.state_copy(pool, _idx([0, 8]), _idx([8, 4]))
    torch.cuda.synchronize()
    assert kda.get_device_error() == 0
    for s in (4, 8):
        assert torch.equal(pool[s], pool[0])
    assert int(pool[[1, 2, 3, 5, 6, 7], :4].abs().sum()) == 0


def test_captured_and_replayed():
    pool = _pool(10, (2, 64, 64), torch.float32, 6)
    got, src, dst = pool.cuda(), _idx([0] * 9), _idx([-1] * 9)
    kda.state_copy(got, src, dst)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kda.state_copy(got, src, dst)
    for s, d in (([1, 0, 5], [0, 5, 9]), ([5, 5, -1], [1, 2, 5])):
        s, d = s + [0] * 6, d + [-1] * 6
        src.copy_(_idx(s))
        dst.copy_(_idx(d))
        graph.replay()
        pool = _in_order(pool, s, d)
    torch.cuda.synchronize()
    assert torch.equal(_bits(got), _bits(pool))
