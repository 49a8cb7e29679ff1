"""Sliding-window attention with sinks over caches of the pass dtype, against
the plain 64-bit restatement and against the same visibility as a mask."""
import numpy as np
import pytest

import workloads as W
from oracle import cache8 as O8
from tests import cache_cases as CC

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from programmable_paged_kv_gb300 import build
    build()


def _run(desc, p, pages, q, k, v, **cache):
    plan = CC.plan_of(desc, p, pages, **cache)
    N, Hq = len(p.slots), desc.num_q_heads
    out = torch.full((N, Hq, desc.head_dim), float("nan"), dtype=q.dtype, device="cuda")
    lse = torch.full((N, Hq), float("nan"), device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    plan.attend(q, k, v, CC.mask_dev(p), None, None, out, lse, status)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    plan.close()
    return out, lse


def _check(desc, p, pages, seed, window, sinks):
    from programmable_paged_kv_gb300 import runner
    rng = np.random.default_rng(seed)
    shape = (pages, desc.num_kv_heads, desc.page_size, desc.head_dim)
    k, v = (W.to_storage(rng.standard_normal(shape).astype(np.float32), desc.dtype) for _ in "kv")
    q = W.to_storage((2 * rng.standard_normal((len(p.slots), desc.num_q_heads, desc.head_dim))
                      ).astype(np.float32), desc.dtype)
    kv64 = [CC.values(x, desc.dtype) for x in (k, v)]
    # slots at or past kv_len and pages no row may read hold NaN
    seen = np.zeros((pages, desc.page_size), bool)
    P = desc.page_size
    for l in range(len(p.kv_len)):
        rows = range(int(p.row_indptr[l]), int(p.row_indptr[l + 1]))
        s = np.arange(int(p.kv_len[l]))
        if rows:
            # pages between the sinks' and the first window's belong to others by now
            first = max(0, min(int(p.slots[r]) for r in rows) - window + 1) // P
            s = s[(s // P >= first) | (s // P < -(-sinks // P))]
        seen[p.page_ids[p.page_indptr[l] + s // P], s % P] = True
    nan = W.to_storage(np.full(1, np.nan, np.float32), desc.dtype)
    kd, vd = k.copy(), v.copy()
    kd.transpose(0, 2, 1, 3)[~seen] = nan
    vd.transpose(0, 2, 1, 3)[~seen] = nan
    got, lse = _run(desc, p, pages, runner.to_device(q, desc.dtype), runner.to_device(kd, desc.dtype),
                    runner.to_device(vd, desc.dtype), window=window, sinks=sinks)
    got, lse = got.double().cpu().numpy(), lse.double().cpu().numpy()
    # bf16 with d 128 and no other: the tensor-core kernels round weights to bf16
    mma = desc.dtype == W.BF16 and desc.head_dim == 128
    want, wl, tol, ltol = O8.attend(desc, p, CC.values(q, desc.dtype), *kv64, window, sinks,
                                    weight_bits=8 if mma else 24)
    tol = tol + CC.half_step(desc) * (np.abs(want) + tol)
    assert np.array_equal(np.isneginf(lse), np.isneginf(wl))
    fin = ~np.isneginf(wl)
    err = np.abs(got - want)
    assert np.all(err <= tol), (float((err / np.maximum(tol, 1e-300)).max()), float(err.max()))
    assert np.all(np.abs(lse[fin] - wl[fin]) <= ltol[fin])
    assert np.all(got[~fin] == 0.0)


# tensor-core kernels (bf16, d 128; few rows, many rows), the scalar kernel (d 64,
# fp32, or a group that does not divide a query tile)
DESCS = [W.Desc(8, 2, 128, 16, W.BF16), W.Desc(4, 4, 128, 8, W.BF16), W.Desc(16, 2, 128, 32, W.BF16),
         W.Desc(6, 2, 64, 16, W.BF16), W.Desc(4, 1, 128, 8, W.F32), W.Desc(6, 2, 64, 32, W.F32)]


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 3), (17, 1), (64, 4), (200, 70), (4096, 4),
                                          (2 ** 31 - 1, 0)])
@pytest.mark.parametrize("desc", DESCS, ids=str)
def test_window(desc, window, sinks):
    lanes = [CC.tail(900, 1), CC.tail(1, 1), CC.tail(70, 6), CC.tail(333, 30), CC.tail(150, 100)]
    p, pages = CC.make_pass(50, desc, lanes)
    _check(desc, p, pages, 51, window, sinks)


@pytest.mark.parametrize("desc", DESCS, ids=str)
def test_window_ends_before_kv_len_and_past_it(desc):
    """Rows in the middle of the cache, rows whose window lies past kv_len (they
    see sinks only, or nothing), rows in falling slot order."""
    p, pages = CC.make_pass(52, desc, [(500, [100, 99, 98]), (50, [400, 10]), (40, [300]), (0, [7]),
                                       (600, list(range(399, 359, -1)))])
    _check(desc, p, pages, 53, 30, 6)
    _check(desc, p, pages, 53, 30, 0)


@pytest.mark.parametrize("rows", [1, 3, 64])
def test_window_equals_the_same_mask(rows):
    """The window as a plan's option and as mask words agree to the roundings of
    the weights (different tiles, different running maxima)."""
    from programmable_paged_kv_gb300 import runner
    desc = DESCS[0]
    lanes = [CC.tail(2000, rows), CC.tail(321, rows)]
    p, pages = CC.make_pass(54, desc, lanes)

    def vis(rng, l, r, kv):
        s, t = np.arange(kv), lanes[l][1][r]
        return (s <= t) & ((s > t - 128) | (s < 4))
    pm, _ = CC.make_pass(54, desc, lanes, mask=vis)
    rng = np.random.default_rng(55)
    k, v = (runner.to_device(W.to_storage(rng.standard_normal((pages, 2, 16, 128)).astype(np.float32), 1), 1)
            for _ in "kv")
    q = runner.to_device(p.q, 1)
    (o1, l1), (o2, l2) = _run(desc, p, pages, q, k, v, window=128, sinks=4), _run(desc, pm, pages, q, k, v)
    # either side: weights to 2^-8 each over values of |v| <= 5, outputs to 2^-8
    assert float((o1.float() - o2.float()).abs().max()) <= 2 * (2.0 ** -8 * 5 + 2.0 ** -8 * 5)
    assert float((l1 - l2).abs().max()) <= 1e-4


def test_windowed_pass_in_one_call():
    """append, windowed attention and fold in one native call, against the
    separate calls (bit for bit)."""
    import programmable_paged_kv_gb300 as pk
    from programmable_paged_kv_gb300 import runner
    desc = DESCS[0]
    p, pages = CC.make_pass(56, desc, [CC.tail(700, 1), CC.tail(90, 9)], fold=[W.FOLD_ALL] * 2)
    rng = np.random.default_rng(57)
    pool = [W.to_storage(rng.standard_normal((pages, 2, 16, 128)).astype(np.float32), 1) for _ in "kv"]
    q, k, v = (runner.to_device(x, 1) for x in (p.q, p.k, p.v))
    cache = pk.make_cache(window=100, sinks=4)
    d, m = pk.make_desc(desc), pk.make_meta(p, pages)
    res = []
    for one_call in (False, True):
        kp, vp = (runner.to_device(x, 1) for x in pool)
        frozen = CC.to_dev(np.array([699, 81], np.int32))
        q_rot, out = torch.empty_like(q), torch.empty_like(q)
        lse = torch.empty(out.shape[:2], device="cuda")
        if one_call:
            ws = torch.empty(pk.workspace_bytes(d, m, cache), dtype=torch.uint8, device="cuda")
            pk.forward_cache(d, cache, m, ws, q, k, v, q_rot, kp, vp, frozen, out_all=out, lse_all=lse)
        else:
            plan = pk.ForwardPlan(d, m, cache=cache)
            plan.append_kv(q, k, v, q_rot, kp, vp, frozen)
            plan.attend(q_rot, kp, vp, out_all=out, lse_all=lse)
            plan.fold(frozen)
        torch.cuda.synchronize()
        res.append((q_rot, kp, vp, out, lse, frozen))
    assert all(torch.equal(a, b) for a, b in zip(*res))
    assert res[0][-1].cpu().tolist() == [700, 90]


@pytest.mark.parametrize("desc", DESCS, ids=str)
def test_sinks_past_every_slot(desc):
    p, pages = CC.make_pass(58, desc, [CC.tail(400, 1), CC.tail(70, 6), CC.tail(333, 30)])
    _check(desc, p, pages, 59, 5, 2 ** 31 - 1)


@pytest.mark.parametrize("desc", DESCS[::2], ids=str)
def test_captured_windowed_attention_replays(desc):
    """One plan's windowed attention captured and replayed on other queries and
    caches: the same bits as eager calls on them."""
    p, pages = CC.make_pass(60, desc, [CC.tail(900, 1), CC.tail(70, 6), CC.tail(333, 100)])
    plan = CC.plan_of(desc, p, pages, window=50, sinks=20)
    dt = torch.float32 if desc.dtype == W.F32 else torch.bfloat16
    q = torch.empty((len(p.slots), desc.num_q_heads, desc.head_dim), dtype=dt, device="cuda")
    k, v = (torch.zeros((pages, desc.num_kv_heads, desc.page_size, desc.head_dim), dtype=dt,
                        device="cuda") for _ in "kv")
    out, lse = torch.empty_like(q), torch.empty(q.shape[:2], device="cuda")
    stream = torch.cuda.Stream()
    run = lambda: plan.attend(q, k, v, None, None, None, out, lse, stream=stream)
    torch.cuda.synchronize()
    q.zero_()
    torch.cuda.synchronize()
    run()  # (first calls set the kernels' attributes)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        run()
    for seed in range(2):
        gen = torch.Generator(device="cuda")
        gen.manual_seed(seed)
        for x in (q, k, v):
            x.copy_(torch.randn(x.shape, generator=gen, device="cuda"))
        res = []
        for replay in (True, False):
            torch.cuda.synchronize()
            graph.replay() if replay else run()
            torch.cuda.synchronize()
            res.append((out.clone(), lse.clone()))
        assert torch.equal(res[0][0], res[1][0]) and torch.equal(res[0][1], res[1][1])
    plan.close()
