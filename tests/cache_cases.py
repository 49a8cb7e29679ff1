"""Small passes over paged caches for the tests of the 8-bit cache, windowed
attention and page copies: seeded geometry and values, no arithmetic of the
operators."""
import numpy as np

import workloads as W
from oracle import cache8 as O8


def make_pass(seed, desc, lanes, mask=None, extra_pages=3, sigma=1.0, fold=None, positions=None):
    """lanes: (kv_len, slots of its rows) per lane; mask(rng, lane, row, kv_len) ->
    bool [kv_len] or None.  Returns (Pass, number of pool pages)."""
    rng = np.random.default_rng(seed)
    P = desc.page_size
    top = [max([kv] + [s + 1 for s in slots]) for kv, slots in lanes]
    need = [-(-t // P) for t in top]
    ids = rng.permutation(sum(need) + extra_pages).astype(np.int32)
    n = [len(s) for _, s in lanes]
    N = sum(n)
    slots = np.array([s for _, ss in lanes for s in ss], np.int32)
    val = lambda h: W.to_storage((sigma * rng.standard_normal((N, h, desc.head_dim))).astype(np.float32),
                                 desc.dtype)
    p = W.Pass(row_indptr=np.cumsum([0] + n).astype(np.int32),
               positions=slots if positions is None else np.asarray(positions, np.int32), slots=slots,
               kv_len=np.array([kv for kv, _ in lanes], np.int32),
               page_indptr=np.cumsum([0] + need).astype(np.int32), page_ids=ids[:sum(need)],
               fold_mode=np.array(fold if fold is not None else [W.FOLD_NONE] * len(lanes), np.int32),
               fold_count=np.zeros(len(lanes), np.int32),
               q=val(desc.num_q_heads), k=val(desc.num_kv_heads), v=val(desc.num_kv_heads))
    if mask is not None:
        rows = [mask(rng, l, r, kv) for l, (kv, ss) in enumerate(lanes) for r in range(len(ss))]
        p.mask_word_indptr, p.mask_words = W.mask_from_visible(rows)
    return p, sum(need) + extra_pages


def tail(kv, n):
    """A lane of kv slots whose last n are the pass's rows."""
    return kv, list(range(kv - n, kv))


def pool8(seed, pages, desc, spread=3):
    """Random codes (no NaN) and scales within 2^+-spread of 2^-7."""
    rng = np.random.default_rng(seed)
    shape = (pages, desc.num_kv_heads, desc.page_size, desc.head_dim)
    codes = O8.encode(rng.standard_normal(shape) * 128.0)
    scale = (O8.BIAS - 7 + rng.integers(-spread, spread + 1, shape[:2])).astype(np.uint8)
    return codes, scale


def to_dev(a):
    import torch
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def values(x, dtype):
    return W.storage_to_f32(x, dtype).astype(np.float64)


def plan_of(desc, p, pages, **cache):
    import programmable_paged_kv_gb300 as pk
    return pk.ForwardPlan(pk.make_desc(desc), pk.make_meta(p, pages), cache=pk.make_cache(**cache))


def half_step(desc):
    return 2.0 ** -24 if desc.dtype == W.F32 else 2.0 ** -8


def mask_dev(p):
    return None if p.mask_words is None else to_dev(p.mask_words.view(np.int32))
