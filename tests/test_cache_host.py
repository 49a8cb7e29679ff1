"""Host-side checks of the cache operators that need no GPU: what their planner
and entry points refuse before any CUDA call, and the restatement the GPU tests
compare with."""
import ctypes as C

import numpy as np
import pytest

import workloads as W
from oracle import cache8 as O8
from programmable_paged_kv_gb300 import abi, build, make_cache, make_desc, make_meta
from tests import cache_cases as CC

DESC = W.Desc(8, 2, 128, 16, W.BF16)


@pytest.fixture(scope="module")
def lib():
    build()
    return abi.load()


def _bytes(lib, p, pages, cache, desc=DESC):
    n = C.c_size_t(0)
    m = make_meta(p, pages)
    rc = lib.pie_fwd_cache_workspace_bytes(C.byref(make_desc(desc)),
                                           None if cache is None else C.byref(cache), C.byref(m.c),
                                           C.byref(n))
    return rc, n.value


def test_no_cache_is_the_plain_plan(lib):
    p, pages = CC.make_pass(1, DESC, [CC.tail(300, 1), CC.tail(70, 40)])
    n = C.c_size_t(0)
    m = make_meta(p, pages)
    assert lib.pie_fwd_workspace_bytes(C.byref(make_desc(DESC)), C.byref(m.c), C.byref(n)) == abi.PIE_OK
    assert _bytes(lib, p, pages, None) == (abi.PIE_OK, n.value)
    assert _bytes(lib, p, pages, make_cache()) == (abi.PIE_OK, n.value)


def test_cache_arguments(lib):
    p, pages = CC.make_pass(2, DESC, [CC.tail(300, 1)])
    ok = lambda **k: _bytes(lib, p, pages, make_cache(**k))[0]
    assert ok(kv="e4m3") == ok(window=1) == ok(kv="e4m3", window=7, sinks=3) == abi.PIE_OK
    assert ok(window=2 ** 31 - 1, sinks=2 ** 31 - 1) == abi.PIE_OK
    assert ok(window=-1) == ok(window=5, sinks=-1) == abi.PIE_ERANGE
    assert ok(sinks=4) == abi.PIE_EINVAL
    assert _bytes(lib, p, pages, abi.pie_fwd_cache(2, 0, 0))[0] == abi.PIE_EINVAL
    pm, pages = CC.make_pass(2, DESC, [CC.tail(300, 1)], mask=lambda rng, l, r, kv: np.ones(kv, bool))
    assert _bytes(lib, pm, pages, make_cache("e4m3"))[0] == abi.PIE_OK
    assert _bytes(lib, pm, pages, make_cache(window=4))[0] == abi.PIE_EINVAL
    for scale in (-1.0, float("inf"), float("nan")):
        bad = W.Desc(8, 2, 128, 16, W.BF16, sm_scale=scale)
        assert _bytes(lib, p, pages, make_cache("e4m3"), bad)[0] == abi.PIE_EINVAL


def test_one_writer_per_page_of_codes(lib):
    """Two lanes, or two entries of one lane's table, that write one physical page."""
    p, pages = CC.make_pass(3, DESC, [CC.tail(20, 1), CC.tail(20, 2)])
    p.page_ids[3] = p.page_ids[1]          # slots 16.. of both lanes
    p.slots = np.array([19, 17, 18], np.int32)
    p.positions = p.slots
    assert _bytes(lib, p, pages, None)[0] == abi.PIE_OK  # distinct slots of a shared page
    assert _bytes(lib, p, pages, make_cache("e4m3"))[0] == abi.PIE_EINVAL
    p.page_ids[3] = p.page_ids[0]          # read by one lane, written by the other: allowed
    assert _bytes(lib, p, pages, make_cache("e4m3"))[0] == abi.PIE_OK
    one, pages = CC.make_pass(4, DESC, [(40, [3, 20])])
    one.page_ids[1] = one.page_ids[0]
    assert _bytes(lib, one, pages, make_cache("e4m3"))[0] == abi.PIE_EINVAL


@pytest.mark.parametrize("cache", [dict(kv="e4m3"), dict(kv="e4m3", window=50, sinks=3), dict(window=1)])
def test_every_shape_plans(lib, cache):
    """Empty passes, lanes without rows or slots, and every built shape."""
    for dt in (W.F32, W.BF16):
        for d in (64, 128):
            for P in (8, 16, 32):
                for hq, hkv in ((1, 1), (8, 1), (12, 4), (40, 8)):
                    desc = W.Desc(hq, hkv, d, P, dt)
                    p, pages = CC.make_pass(5, desc, [(0, []), (5, []), CC.tail(1, 1), (0, [4]),
                                                      CC.tail(300, 90), CC.tail(5000, 1)])
                    rc, n = _bytes(lib, p, pages, make_cache(**cache), desc)
                    assert rc == abi.PIE_OK and n % 256 == 0
    p, pages = CC.make_pass(6, DESC, [])
    assert _bytes(lib, p, pages, make_cache(**cache))[0] == abi.PIE_OK


def test_a_window_reads_no_more_than_its_pages(lib):
    """The partial states of a windowed decode row count its window's chunks, not
    the cache's."""
    size = {}
    for kv in (2048, 4096, 200000):
        p, pages = CC.make_pass(7, DESC, [CC.tail(kv, 1)] * 32)
        size[kv] = [_bytes(lib, p, pages, c)[1] - 4 * len(p.page_ids)
                    for c in (make_cache("e4m3", window=1000, sinks=4), make_cache("e4m3"))]
    assert abs(size[200000][0] - size[2048][0]) < 2048
    assert size[200000][1] > 4 * size[200000][0]


def test_calls_refuse_null_before_any_launch(lib):
    buf = C.c_void_p(1 << 20)  # never dereferenced
    assert lib.pie_fwd_append_kv8(None, *[buf] * 11) == abi.PIE_EINVAL
    assert lib.pie_fwd_attend_kv8(None, *[buf] * 12) == abi.PIE_EINVAL
    assert lib.pie_fwd_cache_plan(None, None, None, buf, 1, None, None) == abi.PIE_EINVAL
    p, pages = CC.make_pass(8, DESC, [CC.tail(30, 1)])
    m, h = make_meta(p, pages), C.c_void_p()
    cache = make_cache("e4m3")
    args = (C.byref(make_desc(DESC)), C.byref(cache), C.byref(m.c))
    assert lib.pie_fwd_cache_plan(*args, buf, 16, None, C.byref(h)) == abi.PIE_ENOSPACE
    assert lib.pie_fwd_cache_plan(*args, C.c_void_p((1 << 20) + 16), 1 << 30, None,
                                  C.byref(h)) == abi.PIE_EINVAL
    assert h.value is None


def test_copy_pages_refuses_before_any_launch(lib):
    ptr = (C.c_void_p * 2)(1 << 20, 1 << 21)  # never dereferenced
    size = (C.c_int64 * 2)(64, 8)
    buf = C.c_void_p(1 << 20)
    copy = lambda n=2, pools=ptr, sizes=size, pages=4, pairs=1, src=buf, dst=buf: lib.pie_fwd_copy_pages(
        n, pools, sizes, pages, pairs, src, dst, None, None)
    assert copy(n=-1) == copy(pages=-1) == copy(pairs=-1) == abi.PIE_EINVAL
    assert copy(pools=None) == copy(sizes=None) == copy(src=None) == copy(dst=None) == abi.PIE_EINVAL
    assert copy(sizes=(C.c_int64 * 2)(64, 0)) == abi.PIE_EINVAL
    assert copy(pools=(C.c_void_p * 2)(1 << 20, None)) == abi.PIE_EINVAL
    assert copy(n=0) == copy(pairs=0) == abi.PIE_OK


def test_restatement_rounds_to_the_nearest_code():
    t = O8.TABLE[:127]
    assert t[126] == 448.0 and t[1] == 2.0 ** -9 and t[8] == 2.0 ** -6 and t[56] == 1.0
    assert np.array_equal(O8.encode(t), np.arange(127))
    mid = (t[1:] + t[:-1]) / 2  # ties go to the even code
    assert np.array_equal(O8.encode(mid), np.arange(126) + np.arange(126) % 2)
    assert np.array_equal(O8.encode(-np.nextafter(mid, 500)), np.arange(1, 127) + 128)
    assert O8.encode(np.array([1e9, np.inf, -np.inf, np.nan])).tolist() == [126, 126, 254, 127]
    assert O8.needed_exp(448.0) == 0 and O8.needed_exp(448.1) == 1 and O8.needed_exp(0.0) == -40
    assert O8.needed_exp(224.0) == -1 and O8.needed_exp(1e300) == 60


@pytest.mark.parametrize("name", ["decode_batch", "masked_window", "masked_decode_tova"])
def test_restatement_attends_as_the_forward_pass_oracle(name):
    """On pools of the pass dtype, without a window, it agrees with the library's
    main oracle."""
    import oracle as O
    sc = W.small(name, 3)
    d, p = sc.desc, sc.passes[0]
    orc = O.run_scenario(sc)
    k = np.zeros((sc.num_pool_pages,) + orc[0].shape[1:])
    v = np.zeros_like(k)
    k[sc.pool_pages], v[sc.pool_pages] = CC.values(orc[0], d.dtype), CC.values(orc[1], d.dtype)
    k, v = np.nan_to_num(k), np.nan_to_num(v)
    assert len(sc.passes) == 1
    out, lse, _, _ = O8.attend(d, p, CC.values(orc[3][0]["q_rot"], d.dtype), k, v)
    assert np.allclose(out, orc[3][0]["out"], rtol=0, atol=1e-9)
    assert np.allclose(lse, orc[3][0]["lse"], rtol=0, atol=1e-9)
