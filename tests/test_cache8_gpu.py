"""The cache of 8-bit codes on the GPU against its plain 64-bit restatement:
append (codes and scales bit for bit), attention (within bounds that count
every rounding), both in one pass, and what the calls refuse."""
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


def _append(desc, p, pages, codes, scales, frozen, status=None):
    """The library's append on copies: q_rot, k codes, v codes, k scales, v scales."""
    from programmable_paged_kv_gb300 import runner
    plan = CC.plan_of(desc, p, pages, kv="e4m3")
    q, k, v = (runner.to_device(x, desc.dtype) for x in (p.q, p.k, p.v))
    q_rot = torch.empty_like(q)
    kc, vc = (CC.to_dev(c) for c in codes)
    ks, vs = (CC.to_dev(s) for s in scales)
    plan.append_kv8(q, k, v, q_rot, kc, vc, ks, vs, CC.to_dev(np.asarray(frozen, np.int32)), status)
    torch.cuda.synchronize()
    plan.close()
    return q_rot.float().cpu().numpy(), *(x.cpu().numpy() for x in (kc, vc, ks, vs))


def _check_append(desc, p, pages, codes, scales, frozen):
    got = _append(desc, p, pages, codes, scales, frozen)
    k = O8.rope(CC.values(p.k, desc.dtype), p.positions, desc.rope_base)
    q = O8.rope(CC.values(p.q, desc.dtype), p.positions, desc.rope_base)
    want = [c.copy() for c in (*codes, *scales)]
    O8.append(desc, p, k, want[0], want[2], frozen)
    O8.append(desc, p, CC.values(p.v, desc.dtype), want[1], want[3], frozen)
    for name, g, w in zip(("k_scale", "v_scale", "k codes", "v codes"),
                          (got[3], got[4], got[1], got[2]), (want[2], want[3], want[0], want[1])):
        assert np.array_equal(g, w), (name, int((g != w).sum()), g.size)
    # queries: two fp32 products and a sum of terms up to |x| + |y| <= sqrt 2
    # |(x, y)|, cos and sin to half a step: 4 half steps in all, then the type's own
    h = desc.head_dim // 2
    pair = np.hypot(q[..., :h], q[..., h:])
    tol = CC.half_step(desc) * np.abs(q) + 4 * 2.0 ** -24 * 2 ** 0.5 * np.concatenate([pair, pair], -1)
    assert np.all(np.abs(got[0] - q) <= tol)
    return got


DESCS = [W.Desc(8, 2, 128, 16, W.BF16), W.Desc(6, 6, 64, 8, W.F32), W.Desc(5, 1, 128, 32, W.BF16),
         W.Desc(24, 8, 64, 16, W.BF16), W.Desc(12, 3, 128, 8, W.F32)]


@pytest.mark.parametrize("desc", DESCS, ids=str)
def test_append_writes_the_nearest_codes(desc):
    # single rows at a page's first, middle and last slot, whole pages, several
    # pages, a lane without rows, and slots far from the start
    lanes = [CC.tail(1, 1), CC.tail(desc.page_size, 1), CC.tail(5 * desc.page_size + 3, 1), (17, []),
             CC.tail(3 * desc.page_size, 3 * desc.page_size), CC.tail(70, 41), CC.tail(33, 7)]
    p, pages = CC.make_pass(1, desc, lanes)
    (kc, ks), (vc, vs) = CC.pool8(2, pages, desc), CC.pool8(3, pages, desc)
    frozen = [kv - len(s) for kv, s in lanes]
    _check_append(desc, p, pages, (kc, vc), (ks, vs), frozen)


@pytest.mark.parametrize("sigma", [2.0 ** -60, 2.0 ** -20, 1e-3, 1.0, 300.0, 2.0 ** 40, 2.0 ** 66])
def test_append_grows_scales_and_requantises_live_codes(sigma):
    """New rows far below and far above what the page holds: live codes keep
    their scale, or shift (subnormals, and out of the codes altogether); scales
    end at 2^-40 and 2^60."""
    desc = DESCS[0]
    p, pages = CC.make_pass(4, desc, [CC.tail(21, 2), CC.tail(16, 3), CC.tail(40, 1)], sigma=sigma)
    (kc, ks), (vc, vs) = CC.pool8(5, pages, desc), CC.pool8(6, pages, desc)
    _check_append(desc, p, pages, (kc, vc), (ks, vs), [19, 13, 39])


def test_append_far_positions():
    """Angles at positions up to 2^31 - 1: the reduction drops whole turns exactly."""
    desc = W.Desc(4, 2, 64, 16, W.BF16)
    pos = [0, 1, 32767, 131071, 1 << 20, (1 << 24) + 1]
    p, pages = CC.make_pass(7, desc, [CC.tail(40, 6)], positions=pos)
    (kc, ks), (vc, vs) = CC.pool8(8, pages, desc), CC.pool8(9, pages, desc)
    _check_append(desc, p, pages, (kc, vc), (ks, vs), [34])
    p.positions = np.array([2 ** 31 - 1] * 6, np.int32)
    # there the restatement's own angle is off by 2^31 2^-53 rad and no longer
    # decides every code: the rotation keeps each pair's length instead
    q = _append(desc, p, pages, (kc, vc), (ks, vs), [34])[0]
    x = CC.values(p.q, desc.dtype)
    a, b = (np.hypot(y[..., :32], y[..., 32:]) for y in (q, x))
    assert np.all(np.abs(a - b) <= (2.0 ** -8 + 2.0 ** -20) * b)


def test_append_special_values():
    """Zeros, infinities and NaN: zeros take the smallest scale, infinities
    saturate at the largest, NaN stays NaN and does not enter the scale."""
    desc = W.Desc(2, 2, 64, 8, W.F32)
    p, pages = CC.make_pass(10, desc, [CC.tail(8, 8), CC.tail(9, 2), CC.tail(3, 1)], positions=[0] * 11)
    p.k[:8] = 0.0
    p.v[:8] = -0.0
    p.v[8, 0, 3], p.v[9, 1, 5], p.v[10, 0, 0] = np.inf, -np.inf, np.nan
    (kc, ks), (vc, vs) = CC.pool8(11, pages, desc), CC.pool8(12, pages, desc)
    got = _append(desc, p, pages, (kc, vc), (ks, vs), [0, 7, 2])
    want, wsc = vc.copy(), vs.copy()
    O8.append(desc, p, CC.values(p.v, desc.dtype), want, wsc, [0, 7, 2])
    assert np.array_equal(got[4], wsc)
    nan = lambda c: (c & 0x7F) == 0x7F
    assert np.array_equal(nan(got[2]), nan(want))
    assert np.array_equal(got[2][~nan(want)], want[~nan(want)])
    assert set(got[3][p.page_ids[0]].tolist()) == {O8.MIN_EXP + O8.BIAS}


def test_append_leaves_frozen_slots_and_other_pages():
    """A frozen slot keeps its code (rescaled with its page when that grows) and
    sets the status; slots out of order, overwritten in the middle of a page."""
    from programmable_paged_kv_gb300 import PIE_STATUS_FOLD_GAP, PIE_STATUS_FROZEN_WRITE
    desc = DESCS[0]
    p, pages = CC.make_pass(13, desc, [(40, [18, 5, 33, 20]), (0, [3]), (16, [15])], sigma=50.0)
    (kc, ks), (vc, vs) = CC.pool8(14, pages, desc), CC.pool8(15, pages, desc)
    frozen = [19, 0, 16]  # rows at slots 18 and 5, and the last lane's only row, are frozen
    _check_append(desc, p, pages, (kc, vc), (ks, vs), frozen)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    _append(desc, p, pages, (kc, vc), (ks, vs), frozen, status)
    assert int(status.item()) == PIE_STATUS_FROZEN_WRITE
    p, pages = CC.make_pass(13, desc, [CC.tail(40, 2)], fold=[W.FOLD_ALL])
    (kc, ks), (vc, vs) = CC.pool8(14, pages, desc), CC.pool8(15, pages, desc)
    _append(desc, p, pages, (kc, vc), (ks, vs), [37], status)
    assert int(status.item()) == PIE_STATUS_FROZEN_WRITE | PIE_STATUS_FOLD_GAP


# ---- attention ------------------------------------------------------------
def _attend(desc, p, pages, q, pools, scales, window=0, sinks=0):
    plan = CC.plan_of(desc, p, pages, kv="e4m3", window=window, sinks=sinks)
    N, Hq = len(p.slots), desc.num_q_heads
    dt = torch.float32 if desc.dtype == W.F32 else torch.bfloat16
    out = torch.full((N, Hq, desc.head_dim), float("nan"), dtype=dt, device="cuda")
    lse = torch.full((N, Hq), float("nan"), device="cuda")
    ro = torch.full((plan.num_readout, Hq, desc.head_dim), float("nan"), dtype=dt, device="cuda")
    lro = torch.full((plan.num_readout, Hq), float("nan"), device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    plan.attend_kv8(q, *pools, *scales, CC.mask_dev(p), ro, lro, out, lse, status)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    rows = p.readout if p.readout is not None else [r1 - 1 for r0, r1 in zip(p.row_indptr, p.row_indptr[1:])
                                                    if r1 > r0]
    assert torch.equal(ro, out[torch.as_tensor(np.asarray(rows, np.int64)).cuda()])
    assert torch.equal(lro, lse[torch.as_tensor(np.asarray(rows, np.int64)).cuda()])
    plan.close()
    return out.float().cpu().numpy().astype(np.float64), lse.cpu().numpy().astype(np.float64)


def _check_attend(desc, p, pages, seed, window=0, sinks=0, spread=3, garbage=True, qs=2.0):
    from programmable_paged_kv_gb300 import runner
    (kc, ks), (vc, vs) = CC.pool8(seed, pages, desc, spread), CC.pool8(seed + 1, pages, desc, spread)
    rng = np.random.default_rng(seed + 2)
    q = W.to_storage((qs * rng.standard_normal((len(p.slots), desc.num_q_heads, desc.head_dim))
                      ).astype(np.float32), desc.dtype)
    kd, vd = kc.copy(), vc.copy()
    if garbage:  # slots at or past kv_len, and pages no lane holds, hold NaN codes
        seen = np.zeros(kc.shape[:1] + kc.shape[2:3], bool)
        for l in range(len(p.kv_len)):
            s = np.arange(int(p.kv_len[l]))
            seen[p.page_ids[p.page_indptr[l] + s // desc.page_size], s % desc.page_size] = True
        kd.transpose(0, 2, 1, 3)[~seen] = 0x7F
        vd.transpose(0, 2, 1, 3)[~seen] = 0xFF
    got, lse = _attend(desc, p, pages, runner.to_device(q, desc.dtype), (CC.to_dev(kd), CC.to_dev(vd)),
                       (CC.to_dev(ks), CC.to_dev(vs)), window, sinks)
    f32 = desc.dtype == W.F32
    # fp32 passes: weights and queries in two fp16 halves, 2^-22 each
    want, wl, tol, ltol = O8.attend(
        desc, p, CC.values(q, desc.dtype), O8.values(kc, ks), O8.values(vc, vs), window, sinks,
        weight_bits=22 if f32 else 11, weight_floor=2.0 ** -24, query_eps=2.0 ** -22 if f32 else 0.0,
        v_scale=2.0 ** (vs.astype(np.float64) - O8.BIAS))
    tol = tol + CC.half_step(desc) * (np.abs(want) + tol)
    assert np.array_equal(np.isneginf(lse), np.isneginf(wl))
    fin = ~np.isneginf(wl)
    err = np.abs(got - want)
    assert np.all(err <= tol), (float((err / np.maximum(tol, 1e-300)).max()), float(err.max()))
    assert np.all(np.abs(lse[fin] - wl[fin]) <= ltol[fin])
    assert np.all(got[~fin] == 0.0)


# lanes by (slots, rows): one slot, ends inside and at the end of a 64-slot
# stage, several chunks, several row blocks, many rows (wide items)
LANES = [[CC.tail(1, 1)], [CC.tail(64, 1), CC.tail(65, 1), CC.tail(63, 2), (0, [2])],
         [CC.tail(700, 1), CC.tail(31, 1), CC.tail(1290, 1)], [CC.tail(130, 5), CC.tail(9, 9)],
         [CC.tail(200, 37), CC.tail(77, 1), CC.tail(300, 4)]]


@pytest.mark.parametrize("lanes", LANES, ids=["one", "stage ends", "chunks", "drafts", "mixed"])
@pytest.mark.parametrize("desc", DESCS, ids=str)
def test_attend_default_visibility(desc, lanes):
    p, pages = CC.make_pass(20, desc, lanes)
    _check_attend(desc, p, pages, 21)


def _random_mask(rng, l, r, kv):
    if rng.random() < 0.2:
        return np.zeros(kv, bool)
    return rng.random(kv) < rng.choice([0.02, 0.5, 0.98])


def _stripe_mask(rng, l, r, kv):
    """Whole stretches unseen: stages that no row sees are skipped."""
    m = np.zeros(kv, bool)
    m[kv // 3: kv // 3 + 5] = True
    m[-1:] = r % 2 == 0
    return m


@pytest.mark.parametrize("mask", [_random_mask, _stripe_mask])
@pytest.mark.parametrize("desc", DESCS, ids=str)
def test_attend_masked(desc, mask):
    p, pages = CC.make_pass(22, desc, [CC.tail(450, 3), CC.tail(33, 1), CC.tail(2700, 2), CC.tail(96, 20)],
                            mask=mask)
    _check_attend(desc, p, pages, 23)


@pytest.mark.parametrize("window,sinks", [(1, 0), (5, 1), (64, 4), (100, 70), (3000, 9), (2 ** 31 - 1, 0)])
@pytest.mark.parametrize("desc", DESCS[:3], ids=str)
def test_attend_windowed(desc, window, sinks):
    p, pages = CC.make_pass(24, desc, [CC.tail(900, 1), CC.tail(70, 6), CC.tail(3, 3), CC.tail(333, 30)])
    _check_attend(desc, p, pages, 25, window, sinks)


def test_attend_window_ends_before_kv_len_and_past_it():
    """Rows in the middle of the cache, rows whose window lies past kv_len (they
    see sinks only, or nothing), rows in falling slot order."""
    desc = DESCS[0]
    p, pages = CC.make_pass(26, desc, [(500, [100, 99, 98]), (50, [400, 10]), (40, [300]), (0, [7])])
    _check_attend(desc, p, pages, 27, 30, 6)
    _check_attend(desc, p, pages, 27, 30, 0)


def test_attend_scales_far_apart():
    """Pages whose scales differ by up to 2^24: one accumulator serves all."""
    desc = DESCS[0]
    p, pages = CC.make_pass(28, desc, [CC.tail(260, 1), CC.tail(100, 9)])
    _check_attend(desc, p, pages, 29, spread=12, qs=0.02)


def test_attend_large_and_tiny_queries():
    for qs in (1e-30, 1e-3, 3e4):
        desc = W.Desc(4, 2, 128, 16, W.BF16, sm_scale=0.09 if qs < 1 else 0.09 / qs)
        p, pages = CC.make_pass(30, desc, [CC.tail(130, 2)])
        _check_attend(desc, p, pages, 31, qs=qs)


def test_pass_on_the_8_bit_cache():
    """Prompts, then drafts and single rows, as a program runs them: append,
    attend and fold per step on one stream, each step's attention checked on
    the codes that the restatement holds; one native call gives the same bits."""
    import programmable_paged_kv_gb300 as pk
    from programmable_paged_kv_gb300 import runner
    desc = W.Desc(8, 2, 128, 16, W.BF16)
    pages_per, steps = 6, [[20, 3, 40], [1, 1, 1], [5, 1, 9], [1, 1, 1]]
    rng = np.random.default_rng(40)
    ids = rng.permutation(3 * pages_per).astype(np.int32)
    pool = lambda: torch.zeros((3 * pages_per, 2, 16, 128), dtype=torch.uint8, device="cuda")
    dev = [[pool(), pool(), *(torch.zeros((3 * pages_per, 2), dtype=torch.uint8, device="cuda") for _ in "kv"),
            torch.zeros(3, dtype=torch.int32, device="cuda")] for _ in range(2)]
    host = [np.zeros((3 * pages_per, 2, 16, 128), np.uint8) for _ in range(2)] + \
           [np.zeros((3 * pages_per, 2), np.uint8) for _ in range(2)]
    length = np.zeros(3, np.int64)
    for i, n in enumerate(steps):
        lanes = [(int(length[l] + n[l]), list(range(int(length[l]), int(length[l] + n[l])))) for l in range(3)]
        p, _ = CC.make_pass(41 + i, desc, lanes, fold=[W.FOLD_ALL] * 3)
        p.page_ids, p.page_indptr = ids, np.arange(4, dtype=np.int32) * pages_per
        q, k, v = (runner.to_device(x, desc.dtype) for x in (p.q, p.k, p.v))
        outs = []
        for one_call, (kc, vc, ks, vs, frozen) in enumerate(dev):
            q_rot, out = torch.empty_like(q), torch.empty_like(q)
            lse = torch.empty(out.shape[:2], device="cuda")
            status = torch.zeros(1, dtype=torch.int32, device="cuda")
            cache = pk.make_cache("e4m3")
            d, m = pk.make_desc(desc), pk.make_meta(p, 3 * pages_per)
            if one_call:
                ws = torch.empty(pk.workspace_bytes(d, m, cache), dtype=torch.uint8, device="cuda")
                pk.forward_cache(d, cache, m, ws, q, k, v, q_rot, kc, vc, frozen, ks, vs, out_all=out,
                                 lse_all=lse, status=status)
            else:
                plan = pk.ForwardPlan(d, m, cache=cache)
                plan.append_kv8(q, k, v, q_rot, kc, vc, ks, vs, frozen, status)
                plan.attend_kv8(q_rot, kc, vc, ks, vs, out_all=out, lse_all=lse, status=status)
                plan.fold(frozen, status=status)
                plan.close()
            torch.cuda.synchronize()
            assert int(status.item()) == 0 and frozen.cpu().tolist() == (length + n).tolist()
            outs.append((q_rot, out, lse))
        assert all(torch.equal(a, b) for a, b in zip(*outs))
        kr = O8.rope(CC.values(p.k, desc.dtype), p.positions, desc.rope_base)
        O8.append(desc, p, kr, host[0], host[2], length)
        O8.append(desc, p, CC.values(p.v, desc.dtype), host[1], host[3], length)
        for t, h in zip(dev[0], host):
            assert np.array_equal(t.cpu().numpy(), h)
        want, wl, tol, ltol = O8.attend(
            desc, p, outs[0][0].double().cpu().numpy(), O8.values(host[0], host[2]),
            O8.values(host[1], host[3]), weight_floor=2.0 ** -24,
            v_scale=2.0 ** (host[3].astype(np.float64) - O8.BIAS))
        got = outs[0][1].double().cpu().numpy()
        assert np.all(np.abs(got - want) <= tol + 2.0 ** -8 * (np.abs(want) + tol))
        assert np.all(np.abs(outs[0][2].double().cpu().numpy() - wl) <= ltol)
        length += n


def _state(seed, desc, lanes, **kw):
    """Device state of one pass: pass, pages, queries, pools and scales."""
    from programmable_paged_kv_gb300 import runner
    p, pages = CC.make_pass(seed, desc, lanes, **kw)
    (kc, ks), (vc, vs) = CC.pool8(seed + 1, pages, desc), CC.pool8(seed + 2, pages, desc)
    q, k, v = (runner.to_device(x, desc.dtype) for x in (p.q, p.k, p.v))
    return p, pages, (q, k, v), [CC.to_dev(x) for x in (kc, vc, ks, vs)]


def test_captured_pass_replays_on_changed_inputs():
    """append, attend and fold of one pass captured once (decode, wide and
    tensor-core items in one plan) and replayed on other inputs: the same bits as
    eager calls on them."""
    desc = W.Desc(8, 2, 128, 16, W.BF16)
    p, pages, (q, k, v), pool = _state(60, desc, [CC.tail(300, 1), CC.tail(90, 7), CC.tail(200, 20)],
                                       fold=[W.FOLD_ALL] * 3)
    plan = CC.plan_of(desc, p, pages, kv="e4m3")
    q_rot, out = torch.empty_like(q), torch.empty_like(q)
    lse = torch.empty(out.shape[:2], device="cuda")
    frozen = CC.to_dev(np.array([299, 83, 180], np.int32))
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    stream = torch.cuda.Stream()

    def run():
        plan.append_kv8(q, k, v, q_rot, *pool, frozen, status, stream=stream)
        plan.attend_kv8(q_rot, *pool, None, None, None, out, lse, status, stream=stream)
        plan.fold(frozen, status=status, stream=stream)

    start = [x.clone() for x in (*pool, frozen)]
    torch.cuda.synchronize()
    run()  # (first calls set the kernels' attributes)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        run()
    for i in range(3):
        gen = torch.Generator(device="cuda")
        gen.manual_seed(i)
        for x in (q, k, v):
            x.copy_(torch.randn(x.shape, generator=gen, device="cuda") * (1 + 3 * i))
        res = []
        for replay in (True, False):
            for x, x0 in zip((*pool, frozen), start):
                x.copy_(x0)
            torch.cuda.synchronize()
            graph.replay() if replay else run()
            torch.cuda.synchronize()
            res.append([x.clone() for x in (q_rot, out, lse, *pool, frozen, status)])
        assert all(torch.equal(a, b) for a, b in zip(*res))
    assert int(status.item()) == 0
    plan.close()


def test_plans_on_two_streams_at_once():
    """Two passes with workspaces of their own, attending at the same time over
    and over: each its own result."""
    desc = W.Desc(8, 2, 128, 16, W.BF16)
    runs = []
    for i, lanes in enumerate(([CC.tail(900, 1)] * 6, [CC.tail(500, 6), CC.tail(700, 40)])):
        p, pages, (q, _, _), pool = _state(70 + 10 * i, desc, lanes)
        plan = CC.plan_of(desc, p, pages, kv="e4m3")
        outs = [torch.empty_like(q) for _ in range(8)]
        runs.append((plan, q, pool, outs, torch.cuda.Stream()))
    torch.cuda.synchronize()
    for i in range(8):
        for plan, q, pool, outs, stream in runs:
            plan.attend_kv8(q, *pool, out_all=outs[i], stream=stream)
    torch.cuda.synchronize()
    for plan, q, pool, outs, _ in runs:
        assert all(torch.equal(o, outs[0]) for o in outs[1:])
        plan.close()
    assert not torch.equal(runs[0][3][0][0], runs[1][3][0][0])


def test_pool_beyond_32_bit_offsets():
    """Pages past byte 2^32 of their pool: written and read."""
    desc = W.Desc(8, 8, 128, 32, W.BF16)
    lanes = [CC.tail(70, 1), CC.tail(40, 9)]
    p, _ = CC.make_pass(80, desc, lanes)
    pages = 140000  # 32 KB each
    p.page_ids = (np.arange(len(p.page_ids)) * 37 % 900 + pages - 900).astype(np.int32)
    pool = [torch.empty((pages, 8, 32, 128), dtype=torch.uint8, device="cuda") for _ in "kv"]
    scale = [torch.empty((pages, 8), dtype=torch.uint8, device="cuda") for _ in "kv"]
    small = [CC.pool8(81 + i, 900, desc) for i in range(2)]
    for t, s, (c, e) in zip(pool, scale, small):
        t[pages - 900:].copy_(CC.to_dev(c))
        s[pages - 900:].copy_(CC.to_dev(e))
    from programmable_paged_kv_gb300 import runner
    q, k, v = (runner.to_device(x, 1) for x in (p.q, p.k, p.v))
    plan = CC.plan_of(desc, p, pages, kv="e4m3")
    q_rot, out = torch.empty_like(q), torch.empty_like(q)
    plan.append_kv8(q, k, v, q_rot, *pool, *scale, CC.to_dev(np.array([69, 31], np.int32)))
    plan.attend_kv8(q_rot, *pool, *scale, out_all=out)
    torch.cuda.synchronize()
    local = W.Pass(**{f: getattr(p, f) for f in p.__dataclass_fields__})
    local.page_ids = p.page_ids - (pages - 900)
    host = [small[0][0], small[1][0], small[0][1], small[1][1]]
    O8.append(desc, local, O8.rope(CC.values(p.k, 1), p.positions, desc.rope_base), host[0], host[2], [69, 31])
    O8.append(desc, local, CC.values(p.v, 1), host[1], host[3], [69, 31])
    for t, h in zip((*pool, *scale), host):
        assert np.array_equal(t[pages - 900:].cpu().numpy(), h)
    want, _, tol, _ = O8.attend(desc, local, q_rot.double().cpu().numpy(), O8.values(host[0], host[2]),
                                O8.values(host[1], host[3]), weight_floor=2.0 ** -24,
                                v_scale=2.0 ** (host[3].astype(np.float64) - O8.BIAS))
    got = out.double().cpu().numpy()
    assert np.all(np.abs(got - want) <= tol + 2.0 ** -8 * (np.abs(want) + tol))
    plan.close()


@pytest.mark.parametrize("rows", [1, 8])
def test_expired_wait_sets_timeout_and_the_context_stays_usable(rows):
    """The split-KV kernels' producer stops before a stage (the library's test
    hook; no copy is in flight): the waits run out, the status says so, the call
    returns, and the same plan then attends as before."""
    from programmable_paged_kv_gb300 import PIE_STATUS_TIMEOUT, abi
    lib = abi.load()
    desc = W.Desc(8, 2, 128, 16, W.BF16)
    p, pages, (q, _, _), pool = _state(90, desc, [CC.tail(1200, rows)] * 5)
    plan = CC.plan_of(desc, p, pages, kv="e4m3")
    out, again = torch.empty_like(q), torch.empty_like(q)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    plan.attend_kv8(q, *pool, out_all=out, status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    assert lib.pie_fwd_test_wait_expiry(1, 300) == abi.PIE_OK
    try:
        plan.attend_kv8(q, *pool, out_all=again, status=status)
        torch.cuda.synchronize()
    finally:
        assert lib.pie_fwd_test_wait_expiry(-1, 0) == abi.PIE_OK
    assert int(status.item()) & PIE_STATUS_TIMEOUT
    status.zero_()
    plan.attend_kv8(q, *pool, out_all=again, status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == 0 and torch.equal(out, again)
    plan.close()


def test_refused_calls():
    """Tensors of the wrong shape, type or place, and calls for the other kind of
    cache: refused before anything is launched."""
    import programmable_paged_kv_gb300 as pk
    desc = W.Desc(8, 2, 64, 16, W.BF16)
    p, pages, (q, k, v), pool = _state(95, desc, [CC.tail(40, 2)])
    frozen = CC.to_dev(np.array([38], np.int32))
    plan = CC.plan_of(desc, p, pages, kv="e4m3")
    q_rot, out = torch.empty_like(q), torch.empty_like(q)
    good = dict(q=q, k=k, v=v, q_rot=q_rot, k_pool=pool[0], v_pool=pool[1], k_scale=pool[2],
                v_scale=pool[3], frozen_len=frozen)
    for name, bad in (("q", q.float()), ("q", q[:1]), ("k", k.transpose(1, 2)), ("v", v.cpu()),
                      ("q_rot", q_rot.half()), ("k_pool", pool[0].int()), ("k_pool", pool[0][:-1]),
                      ("v_pool", pool[1].transpose(2, 3).contiguous().transpose(2, 3)),
                      ("k_scale", pool[2][:, :1]), ("v_scale", pool[3].float()),
                      ("frozen_len", frozen.long())):
        with pytest.raises(ValueError):
            plan.append_kv8(**{**good, name: bad})
    att = dict(q_rot=q, k_pool=pool[0], v_pool=pool[1], k_scale=pool[2], v_scale=pool[3], out_all=out)
    for name, bad in (("q_rot", q[..., :32]), ("out_all", out.float()), ("k_pool", pool[0].cpu()),
                      ("lse_all", torch.empty((2, 8), device="cuda", dtype=torch.float64)),
                      ("out_readout", out)):
        with pytest.raises(ValueError):
            plan.attend_kv8(**{**att, name: bad})
    with pytest.raises(pk.PieError) as e:  # no mask in the plan
        plan.attend_kv8(**att, mask_words=torch.zeros(8, dtype=torch.int32, device="cuda"))
    assert e.value.code == pk.abi.PIE_EINVAL
    for call in (lambda: plan.append_kv(q, k, v, q_rot, pool[0], pool[1], frozen),
                 lambda: plan.attend(q, pool[0], pool[1], out_all=out)):
        with pytest.raises(pk.PieError) as e:
            call()
        assert e.value.code == pk.abi.PIE_EINVAL
    # a row of codes off the 16-byte boundary
    flat = torch.empty(pool[0].numel() + 16, dtype=torch.uint8, device="cuda")
    with pytest.raises(pk.PieError):
        plan.attend_kv8(**{**att, "k_pool": flat[8:-8].view(pool[0].shape)})
    plan.close()
    plain = CC.plan_of(desc, p, pages)
    with pytest.raises(pk.PieError) as e:
        plain.append_kv8(**good)
    assert e.value.code == pk.abi.PIE_EINVAL
    plain.close()
    none = pk.ForwardPlan(pk.make_desc(desc), pk.make_meta(p, pages))
    with pytest.raises(ValueError):
        none.attend_kv8(**att)
    none.close()
    with pytest.raises(ValueError):
        pk.make_cache("int4")


def test_copy_pages_refusals():
    import programmable_paged_kv_gb300 as pk
    pool = torch.zeros((8, 32), dtype=torch.uint8, device="cuda")
    i = torch.zeros(2, dtype=torch.int32, device="cuda")
    for pools, src, dst in (([pool, pool[:4]], i, i), ([pool.t()], i, i), ([pool.cpu()], i, i),
                            ([pool], i.long(), i), ([pool], i, i[:1]), ([pool[0, 0]], i, i)):
        with pytest.raises(ValueError):
            pk.copy_pages(pools, src, dst)
    pk.copy_pages([], i, i)
    pk.copy_pages([pool], i[:0], i[:0])


def test_too_few_mask_words_and_too_many_pages_are_refused():
    import programmable_paged_kv_gb300 as pk
    desc = W.Desc(4, 2, 64, 16, W.BF16)
    p, pages, (q, k, v), pool = _state(96, desc, [CC.tail(100, 2)],
                                       mask=lambda rng, l, r, kv: np.ones(kv, bool))
    plan = CC.plan_of(desc, p, pages, kv="e4m3")
    words, out = CC.mask_dev(p), torch.empty_like(q)
    with pytest.raises(ValueError, match="mask_words"):
        plan.attend_kv8(q, *pool, words[:-1], out_all=out)
    plan.attend_kv8(q, *pool, words, out_all=out)
    plan.close()
    i = torch.zeros(1, dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError, match="32-bit"):
        pk.copy_pages([torch.empty((2 ** 31, 1), dtype=torch.uint8, device="cuda")], i, i)


@pytest.mark.parametrize("desc", DESCS[:3], ids=str)
def test_attend_sinks_past_every_slot(desc):
    p, pages = CC.make_pass(97, desc, [CC.tail(400, 1), CC.tail(70, 6), CC.tail(333, 30)])
    _check_attend(desc, p, pages, 98, 5, 2 ** 31 - 1)


@pytest.mark.parametrize("kv", [40, 3000], ids=["one chunk", "chunks"])
@pytest.mark.parametrize("rows", [1, 8], ids=["narrow", "wide"])
@pytest.mark.parametrize("desc", DESCS[:3], ids=str)
def test_outputs_asked_for_one_by_one(desc, rows, kv):
    """Every subset of the outputs is the same bits as all of them, rows that are read
    out twice or not at all included, and nothing else is written."""
    lanes = [CC.tail(kv, rows), (0, list(range(rows)))]
    p, pages, (q, _, _), pool = _state(99, desc, lanes)
    p.readout = np.array([0, 2 * rows - 1, 0], np.int32)
    plan = CC.plan_of(desc, p, pages, kv="e4m3")
    shapes = [(3, *q.shape[1:]), (3, q.shape[1]), tuple(q.shape), tuple(q.shape[:2])]
    new = lambda: [torch.full(s, 7.0, dtype=q.dtype if len(s) == 3 else torch.float32, device="cuda")
                   for s in shapes]
    want = new()
    plan.attend_kv8(q, *pool, None, *want)
    for pick in ((0,), (2,), (0, 1), (2, 3), (0, 3), (1, 2)):
        got = new()
        plan.attend_kv8(q, *pool, None, *(x if i in pick else None for i, x in enumerate(got)))
        for i in range(4):
            assert torch.equal(got[i], want[i] if i in pick else torch.full_like(got[i], 7.0))
    assert torch.equal(want[0], want[2][p.readout.tolist()]) and torch.equal(want[1], want[3][p.readout.tolist()])
    plan.close()
