"""Page copies within the pools of several layers."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from programmable_paged_kv_gb300 import build
    build()


def _pools(pages, seed):
    """K, V and scale pools of odd kinds: pages of 32 KB and more, of 16, 8, 5 and 3 bytes."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    r = lambda *s: torch.randint(0, 256, (pages, *s), generator=g, device="cuda", dtype=torch.uint8)
    return [r(8, 16, 128 * 2).view(torch.int16), r(2, 8, 64), r(8), r(3), r(1, 5), r(16),
            r(40, 16, 128).view(torch.int32), r(7, 16, 16)]


@pytest.mark.parametrize("pages,pairs", [(2, 1), (64, 5), (64, 32), (700, 300)])
def test_copies_every_pool(pages, pairs):
    import programmable_paged_kv_gb300 as pk
    pools = _pools(pages, pages)
    at = torch.from_numpy(np.random.default_rng(pairs).permutation(pages).astype(np.int32)).cuda()
    src, dst = at[:pairs].contiguous(), at[pages - pairs:].contiguous()
    want = [p.clone() for p in pools]
    for w, p in zip(want, pools):
        w[dst.long()] = p[src.long()]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    pk.copy_pages(pools, src, dst, status)
    assert int(status.item()) == 0
    assert all(torch.equal(a, b) for a, b in zip(pools, want))


def test_many_pools_and_unaligned_ones():
    """More pools than one launch takes, and a pool that starts off a 16-byte boundary."""
    import programmable_paged_kv_gb300 as pk
    flat = torch.arange(200 * 40 * 64 + 3, device="cuda").to(torch.uint8)
    pools = [flat[3 + i * 40 * 64: 3 + (i + 1) * 40 * 64].view(40, 64) for i in range(200)]
    src = torch.arange(0, 10, dtype=torch.int32, device="cuda")
    dst = src + 20
    want = [p.clone() for p in pools]
    for w in want:
        w[20:30] = w[0:10]
    pk.copy_pages(pools, src, dst)
    assert all(torch.equal(a, b) for a, b in zip(pools, want))


def test_page_ids_outside_the_pools_are_skipped():
    import programmable_paged_kv_gb300 as pk
    pools = _pools(8, 1)
    want = [p.clone() for p in pools]
    for w in want:
        w[5] = w[2]
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    pk.copy_pages(pools, i32(-1, 2, 8, 3, 4), i32(1, 5, 0, -7, 2 ** 31 - 1), status)
    assert int(status.item()) == pk.PIE_STATUS_BOUNDS
    assert all(torch.equal(a, b) for a, b in zip(pools, want))
    pk.copy_pages(pools, i32(4), i32(4))  # a page onto itself
    assert all(torch.equal(a, b) for a, b in zip(pools, want))


def test_copies_beyond_32_bit_offsets():
    """A pool of more than 2^32 bytes: its last pages."""
    import programmable_paged_kv_gb300 as pk
    pages, size = 5000, 1 << 20
    pool = torch.empty((pages, size), dtype=torch.uint8, device="cuda")
    pool[0], pool[4999], pool[4998] = 7, 9, 0
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")
    pk.copy_pages([pool], i32(4999, 0), i32(1, 4998))
    assert bool((pool[1] == 9).all()) and bool((pool[4998] == 7).all())
    assert bool((pool[0] == 7).all()) and bool((pool[4999] == 9).all())


def test_fork_copies_a_shared_page_before_either_branch_writes():
    """A lane on the 8-bit cache is forked inside a page: the branch gets a copy
    of that page, shares the full ones, and each branch's next token leaves the
    other's cache as it was."""
    import workloads as W
    import programmable_paged_kv_gb300 as pk
    from oracle import cache8 as O8
    from programmable_paged_kv_gb300 import runner
    from tests import cache_cases as CC
    desc = W.Desc(4, 2, 64, 8, W.BF16)
    (kc, ks), (vc, vs) = CC.pool8(1, 12, desc), CC.pool8(2, 12, desc)
    host = [kc, vc, ks, vs]
    dev = [CC.to_dev(x) for x in host]
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")
    pk.copy_pages(dev, i32(7), i32(3))  # slots 16..19 of 20 live in page 7; the branch's copy is page 3
    for x in host:
        x[3] = x[7]
    p, _ = CC.make_pass(3, desc, [CC.tail(21, 1), CC.tail(21, 1)], sigma=9.0)
    p.page_indptr, p.page_ids = np.array([0, 3, 6], np.int32), np.array([5, 2, 7, 5, 2, 3], np.int32)
    plan = CC.plan_of(desc, p, 12, kv="e4m3")
    q, k, v = (runner.to_device(x, 1) for x in (p.q, p.k, p.v))
    plan.append_kv8(q, k, v, torch.empty_like(q), *dev, i32(20, 20))
    kr = O8.rope(CC.values(p.k, 1), p.positions, desc.rope_base)
    O8.append(desc, p, kr, host[0], host[2], [20, 20])
    O8.append(desc, p, CC.values(p.v, 1), host[1], host[3], [20, 20])
    for t, h in zip(dev, host):
        assert np.array_equal(t.cpu().numpy(), h)


def test_captured_copies_replay_on_other_pairs():
    import programmable_paged_kv_gb300 as pk
    pools = _pools(64, 2)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    src, dst = i32([0, 1, 2]), i32([10, 11, 12])
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        pk.copy_pages(pools, src, dst, stream=stream)
    for s, d in (([3, 3, 4], [20, 21, 22]), ([5, 6, 7], [5, 30, 31])):  # a source twice, a page to itself
        src.copy_(i32(s))
        dst.copy_(i32(d))
        want = [p.clone() for p in pools]
        for w in want:
            w[d] = w[s]
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(pools, want))
