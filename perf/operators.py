"""The cache operators beside the ForwardPass's own: their measured cases, the
same work in elementary torch operations, and their definitions in 64 bits.

Four operators on the paged K/V cache:

  append   RoPE of the pass's rows and the write of their K/V into a cache held
           in 8 bits: e4m3 codes with one power-of-two scale per (page, kv
           head), which grows -- and the page's live codes with it -- when a
           new row needs it;
  attend8  grouped-query attention over such a cache (decode, drafts, prompts,
           per-row bitmasks);
  window   grouped-query attention with a sliding window and sink slots that
           stay visible, over a cache of the pass dtype or of 8 bits;
  copy     pages copied within the pools of several layers (a fork's last
           page, the moves of a compaction).

`run` computes them in torch (`own` false) or through the package (`own` true).
"""
import functools
import math
import types

import numpy as np
import torch

own = False

DEV = "cuda"
E_MIN, E_MAX, BIAS, TOP = -40, 60, 127, 448.0  # exponents of a scale, its bias, e4m3's largest value


# --------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------
def _case(name, op, **kw):
    c = dict(name=name, op=op, geo=1, hq=32, hkv=8, d=128, page=16, f32=False)
    c.update(kw)
    return c


def listed():
    return [
        # one decode step of a batch: every lane writes one row
        _case("append decode 64", "append", lanes=64, lo=512, hi=4096, rows=1),
        # eight prompts of 512 tokens written at once behind a cached prefix
        _case("append prompts 8x512", "append", lanes=8, lo=600, hi=1100, rows=512),
        # one short conversation's next token: latency
        _case("attend8 single", "attend8", lanes=1, lo=300, hi=300, rows=1, mask=False),
        # the benchmark's decode batch, on the 8-bit cache
        _case("attend8 decode 64", "attend8", lanes=64, lo=512, hi=4096, rows=1, mask=False),
        # speculative verify: drafts of 8 rows
        _case("attend8 verify 48x8", "attend8", lanes=48, lo=1024, hi=8192, rows=8, mask=False),
        # guidance prefill: 64 rows a lane behind a prefix of 1,024
        _case("attend8 prompts 64x64", "attend8", lanes=64, lo=1088, hi=1088, rows=64, mask=False),
        # a small fp32 model: ragged lanes, small heads and pages, random masks
        _case("attend8 f32 masked", "attend8", lanes=7, lo=33, hi=1501, rows=5, mask=True, hq=12,
              hkv=4, d=64, page=8, f32=True),
        # long conversations that keep 4 sinks and the last 4,096 slots: decode
        _case("window decode 8x32k", "window", lanes=8, lo=32768, hi=32768, rows=1, window=4096,
              sinks=4, kv8=False),
        # and 64 rows of prompt a lane
        _case("window prompts 8x64", "window", lanes=8, lo=32768, hi=32768, rows=64, window=4096,
              sinks=4, kv8=False),
        # a smaller model's window on the 8-bit cache, ragged
        _case("window 8-bit d64", "window", lanes=33, lo=700, hi=16000, rows=1, window=1024,
              sinks=9, kv8=True, hq=16, hkv=4, d=64),
        # forks of a few lanes: each copies its last, partly filled page in every layer
        _case("copy fork 12", "copy", layers=16, pool=2048, pairs=12, kv8=False),
        # a pool compacted: many pages moved to its front, 8-bit codes and scales
        _case("copy compact 4000", "copy", layers=8, pool=16384, pairs=4000, kv8=True),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "attend8", "attend8", "window", "window", "copy"])
    d = rng.choice([64, 128, 128])
    hkv, g = rng.choice([(1, 8), (2, 4), (4, 3), (8, 4), (8, 1), (4, 8), (8, 5)])
    c = dict(op=op, geo=rng.randrange(1 << 30), hq=hkv * g, hkv=hkv, d=d,
             page=rng.choice([8, 16, 16, 32]), f32=rng.random() < 0.2)
    if op == "copy":
        pool = _spread(rng, 64, 16384 * 16 // c["page"] * 8 // hkv // (4 if c["f32"] else 2))
        c.update(layers=rng.randint(1, 12), pool=pool, pairs=_spread(rng, 1, pool // 4),
                 kv8=rng.random() < 0.5)
        return c
    rows = 1 if rng.random() < 0.4 else _spread(rng, 2, 200)
    lanes = _spread(rng, 1, 64)
    if op == "append":
        hi = _spread(rng, max(16, rows + 2), 6000)
        while lanes * rows > 4096:
            lanes = (lanes + 1) // 2
        c.update(lanes=lanes, lo=max(1, hi // 3), hi=hi, rows=rows)
        return c
    # at most the largest listed case's work: rows x slots x lanes x heads
    hi = _spread(rng, max(16, rows + 1), 20000)
    most = (4.4e6 if rows > 1 else 3.0e5) * 32 / (hkv * g)
    while lanes * hi * (rows if rows > 1 else 1) > most:
        if lanes > 1:
            lanes = (lanes + 1) // 2
        else:
            hi = max(rows + 1, hi // 2)
            if hi == rows + 1:
                rows = max(1, rows // 2)
    c.update(lanes=lanes, lo=max(1, hi // 4), hi=hi, rows=rows)
    if op == "attend8":
        c["mask"] = rng.random() < 0.3
    else:
        c.update(window=_spread(rng, 1, 5000), sinks=rng.choice([0, 1, 4, 16, 70]),
                 kv8=rng.random() < 0.5)
    return c


@functools.lru_cache(maxsize=64)
def _geometry(key):
    """Lengths, rows, page tables and mask bits of a case: the same for every seed."""
    c = dict(key)
    rng = np.random.default_rng(c["geo"])
    L, P = c["lanes"], c["page"]
    kv = rng.integers(c["lo"], c["hi"] + 1, L)
    n = np.minimum(np.full(L, c["rows"]) if L <= 2 or c["rows"] in (1, 8, 64, 512)
                   else rng.integers(max(1, c["rows"] // 2), c["rows"] + 1, L), kv)
    pages = -(-kv // P)
    total = int(pages.sum()) + 3  # a few pages that no lane holds
    perm = rng.permutation(total)
    pind = np.concatenate([[0], np.cumsum(pages)])
    ids = perm[:pind[-1]]
    rind = np.concatenate([[0], np.cumsum(n)])
    lane = np.repeat(np.arange(L), n)
    slot = np.concatenate([np.arange(kv[l] - n[l], kv[l]) for l in range(L)])
    g = dict(kv=kv, n=n, pind=pind, ids=ids, rind=rind, lane=lane, slot=slot, pool=total)
    S = int(kv.max())
    table = np.zeros((L, -(-S // P)), np.int64)
    for l in range(L):
        table[l, :pages[l]] = ids[pind[l]:pind[l + 1]]
    g["table"] = table
    if c.get("mask"):
        keep = rng.random(len(lane)) < 0.9  # a tenth of the rows see nothing
        words = -(-kv[lane] // 32)
        wind = np.concatenate([[0], np.cumsum(words)])
        bits = np.zeros(int(wind[-1]) * 32, np.uint8)
        union = 0
        seen = 0
        for l in range(L):
            any_l = np.zeros(kv[l], bool)
            for r in range(rind[l], rind[l + 1]):
                b = (rng.random(kv[l]) < 0.4) & keep[r]
                bits[wind[r] * 32: wind[r] * 32 + kv[l]] = b
                any_l |= b
                seen += int(b.sum())
            union += int(any_l.sum())
        g.update(wind=wind, union=union, seen=seen,
                 words=np.packbits(bits, bitorder="little").view(np.int32))
    return g


def _geo(case):
    return _geometry(tuple(sorted((k, v) for k, v in case.items() if k != "name")))


def work(case):
    es = 4 if case["f32"] else 2
    if case["op"] == "copy":
        block = case["hkv"] * case["page"] * case["d"]
        one = block + case["hkv"] if case["kv8"] else block * es
        return {"bytes": 2.0 * 2 * case["layers"] * case["pairs"] * one, "flops": 0.0}
    g = _geo(case)
    N, hq, hkv, d = len(g["lane"]), case["hq"], case["hkv"], case["d"]
    if case["op"] == "append":
        held = len(set(zip(g["lane"].tolist(), (g["slot"] // case["page"]).tolist())))
        return {"bytes": float(N * (2 * hq + 2 * hkv) * d * es + 2 * N * hkv * d + 4 * held * hkv),
                "flops": 3.0 * N * (hq + hkv) * d}
    if case.get("mask"):
        union, seen = g["union"], g["seen"]
    else:
        w, s = case.get("window", 0) or 1 << 40, case.get("sinks", 0)
        at = g["slot"]
        lo = np.maximum(0, at - w + 1)
        seen = int((at - lo + 1 + np.minimum(s, lo)).sum())
        first = np.maximum(0, g["kv"] - g["n"] - w + 1)  # of the lane's first row
        union = int((g["kv"] - first + np.minimum(s, first)).sum())
    kv_bytes = 1 if case["op"] == "attend8" or case["kv8"] else es
    held = union / case["page"] * 2 * hkv if kv_bytes == 1 else 0
    return {"bytes": float(2 * union * hkv * d * kv_bytes + held + 2 * N * hq * d * es + 4 * N * hq),
            "flops": 4.0 * seen * hq * d}


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------
def _times2(x, e):
    """x * 2^e, the power of two made from its bits (a pow may be an ulp off)."""
    return x * ((e.long() + 1023) << 52).view(torch.float64).to(x.dtype)


def _e4m3(x):
    """float64 or float32 -> the nearest e4m3 value (ties to even), saturating."""
    a = x.abs()
    e = torch.frexp(torch.where(a > 0, a, torch.ones_like(a)))[1].clamp(min=-5) - 4
    step = _times2(torch.ones_like(a), e)
    return (torch.round(x / step) * step).clamp(-TOP, TOP)


def _need(amax):
    """The smallest exponent e with amax <= 448 * 2^e, within the scales' range."""
    m, e = torch.frexp(amax.double() / TOP)
    return torch.where(amax > 0, torch.where(m > 0.5, e, e - 1), E_MIN).clamp(E_MIN, E_MAX)


def _cache8(shape, gen):
    """Codes and scales of a cache whose pages vary in size as activations do."""
    codes = torch.empty(shape, dtype=torch.float8_e4m3fn, device=DEV)
    scale = torch.empty(shape[:2], dtype=torch.uint8, device=DEV)
    for i in range(0, shape[0], 4096):
        x = torch.randn((min(4096, shape[0] - i),) + shape[1:], generator=gen, device=DEV)
        x *= torch.exp(0.3 * torch.randn(x.shape[:2] + (1, 1), generator=gen, device=DEV))
        e = _need(x.abs().amax((2, 3)))
        scale[i:i + 4096] = (e + BIAS).to(torch.uint8)
        codes[i:i + 4096] = _e4m3(_times2(x, -e[:, :, None, None])).to(torch.float8_e4m3fn)
    return codes, scale


def _dev(a, dtype=torch.int64):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV, dtype)


def _plan(case, g):
    """The pass's plan, as a program makes it once for all of its layers."""
    import programmable_paged_kv_gb300 as pk
    desc = pk.make_desc(types.SimpleNamespace(
        num_q_heads=case["hq"], num_kv_heads=case["hkv"], head_dim=case["d"],
        page_size=case["page"], dtype=pk.PIE_F32 if case["f32"] else pk.PIE_BF16,
        rope_base=10000.0))
    kv8 = case["op"] != "window" or case["kv8"]
    cache = pk.make_cache("e4m3" if kv8 else None, window=case.get("window", 0),
                          sinks=case.get("sinks", 0))
    L = case["lanes"]
    meta = pk.make_meta(types.SimpleNamespace(
        row_indptr=g["rind"], positions=g["slot"], slots=g["slot"], kv_len=g["kv"],
        page_indptr=g["pind"], page_ids=g["ids"], fold_mode=np.full(L, pk.PIE_FOLD_ALL),
        fold_count=None, mask_word_indptr=g.get("wind"), readout=None), g["pool"])
    return pk.ForwardPlan(desc, meta, cache=cache)


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    dt = torch.float32 if case["f32"] else torch.bfloat16
    hq, hkv, d, P = case["hq"], case["hkv"], case["d"], case["page"]
    s = dict(case=case)
    if case["op"] == "copy":
        shape = (case["pool"], hkv, P, d)
        s["pools"] = []
        for _ in range(2 * case["layers"]):
            if case["kv8"]:
                s["pools"].append(torch.randint(0, 127, shape, generator=gen, device=DEV,
                                                dtype=torch.uint8))
                s["pools"].append(torch.randint(100, 140, shape[:2], generator=gen, device=DEV,
                                                dtype=torch.uint8))
            else:
                s["pools"].append(torch.randn(shape, generator=gen, device=DEV, dtype=dt))
        at = torch.randperm(case["pool"], generator=gen, device=DEV)[:2 * case["pairs"]]
        s["src"], s["dst"] = at[:case["pairs"]].int(), at[case["pairs"]:].int()
        return s
    g = _geo(case)
    N, shape = len(g["lane"]), (g["pool"], hkv, P, d)
    kv8 = case["op"] != "window" or case["kv8"]
    if kv8:
        (s["k"], s["ks"]), (s["v"], s["vs"]) = _cache8(shape, gen), _cache8(shape, gen)
    else:
        s["k"], s["v"] = (torch.randn(shape, generator=gen, device=DEV, dtype=dt) for _ in "kv")
    s["lane"], s["slot"], s["kv"], s["table"] = (_dev(g[x]) for x in ("lane", "slot", "kv", "table"))
    s["q"] = 2 * torch.randn((N, hq, d), generator=gen, device=DEV, dtype=dt)
    s["q_rot"] = torch.empty_like(s["q"])
    if case["op"] == "append":
        s["k_new"], s["v_new"] = (torch.randn((N, hkv, d), generator=gen, device=DEV, dtype=dt)
                                  for _ in "kv")
        s["frozen"] = _dev(g["kv"] - g["n"], torch.int32)
    else:
        # the row of each (lane, position within the lane's rows); lanes with fewer repeat their last
        R = int(g["n"].max())
        s["row_at"] = _dev(np.minimum(g["rind"][:-1, None] + np.arange(R), g["rind"][1:, None] - 1))
        s["nth"] = _dev(np.arange(N) - g["rind"][g["lane"]])
        s["out"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty((N, hq), dtype=torch.float32, device=DEV)
        if "wind" in g:
            s["wind"], s["words"] = _dev(g["wind"]), _dev(g["words"], torch.int32)
    if own:
        s["plan"] = _plan(case, g)
    return s


# --------------------------------------------------------------------------
# the operators in elementary operations
# --------------------------------------------------------------------------
def _rotated(x, pos, base=10000.0):
    """RoPE, in 64 bits: the angles of far positions, and values next to a code's border."""
    h = x.shape[-1] // 2
    f = base ** (-torch.arange(h, device=x.device, dtype=torch.float64) / h)
    t = pos.double()[:, None, None] * f
    c, s = torch.cos(t), torch.sin(t)
    lo, hi = x[..., :h].double(), x[..., h:].double()
    return torch.cat([lo * c - hi * s, hi * c + lo * s], -1)


def _append_plain(s):
    c = s["case"]
    P, lane, slot = c["page"], s["lane"], s["slot"]
    page, off = s["table"][lane, slot // P], slot % P
    s["q_rot"].copy_(_rotated(s["q"], slot))
    lp = torch.arange(s["table"].shape[1], device=DEV)
    limit = torch.maximum(s["kv"], s["frozen"].long())
    # live slots of the pages that the rows' pages are, and those written now
    at = (slot // P)[:, None] * P + torch.arange(P, device=DEV)
    live = at < limit[lane][:, None]
    pool = s["k"].shape[0]
    written = torch.zeros((pool, P), dtype=torch.bool, device=DEV)
    written[page, off] = True
    keep = live & ~written[page]  # by row
    fresh = ~keep.any(1)
    for codes, scale, x in ((s["k"], s["ks"], _rotated(s["k_new"], slot)),
                            (s["v"], s["vs"], s["v_new"].double())):
        need = torch.full((pool, c["hkv"]), E_MIN, device=DEV, dtype=torch.int64)
        need.scatter_reduce_(0, page[:, None].expand(-1, c["hkv"]),
                             _need(x.abs().amax(-1)).long(), "amax")
        old = scale.long() - BIAS
        new = torch.where(fresh[:, None], need[page], torch.maximum(need[page], old[page]))
        # the rows of one page all write the same kept codes and scale
        kept = _e4m3(_times2(codes[page].float(), (old[page] - new)[:, :, None, None]))
        kept = torch.where(keep[:, None, :, None], kept, codes[page].float())
        b = codes.view(torch.uint8)
        b[page] = kept.to(torch.float8_e4m3fn).view(torch.uint8)
        scale[page] = (new + BIAS).to(torch.uint8)
        b[page, :, off] = _e4m3(_times2(x, -new[:, :, None])).float().to(
            torch.float8_e4m3fn).view(torch.uint8)
    return s["q_rot"], s["k"], s["v"], s["ks"], s["vs"]


def _slots(pool, scale, table, S):
    """A lane's slots in order: [L, S, Hkv, d] in 32 bits."""
    x = pool.view(torch.uint8)[table].view(pool.dtype).float() if scale is not None else pool[table].float()
    if scale is not None:
        x = _times2(x, scale[table].int()[..., None, None] - BIAS)
    x = x.transpose(2, 3)
    return x.reshape(x.shape[0], -1, x.shape[3], x.shape[4])[:, :S]


def _visible(s, S):
    """[L, R, S]: which slots each row sees."""
    c, row = s["case"], s["row_at"]
    at = torch.arange(S, device=DEV)
    if "words" in s:
        w = s["wind"][row][..., None] + torch.minimum(at // 32, (s["kv"][:, None, None] - 1) // 32)
        seen = (s["words"][w] >> (at % 32)) & 1 == 1
        return seen & (at < s["kv"][:, None, None])
    t = s["slot"][row][..., None]
    seen = at <= t
    if c.get("window"):
        seen &= (at > t - c["window"]) | (at < c["sinks"])
    return seen


def _attend_plain(s):
    c = s["case"]
    S, g = c["hi"], c["hq"] // c["hkv"]
    S = min(S, s["table"].shape[1] * c["page"])
    k, v = (_slots(s[x], s.get(x + "s"), s["table"], S) for x in "kv")
    row = s["row_at"]
    q = s["q"][row].float().reshape(row.shape + (c["hkv"], g, c["d"]))
    z = torch.einsum("lrhgd,lshd->lhrgs", q, k) / math.sqrt(c["d"])
    z.masked_fill_(~_visible(s, S)[:, None, :, None, :], -math.inf)
    # slots behind a lane's end may hold anything: nothing of them reaches a sum
    v = torch.where((torch.arange(S, device=DEV) < s["kv"][:, None])[..., None, None], v, 0.0)
    m = z.amax(-1, keepdim=True)
    m0 = torch.where(m == -math.inf, 0.0, m)
    z.sub_(m0).exp_()
    l = z.sum(-1, keepdim=True)
    o = torch.einsum("lhrgs,lshd->lhrgd", z, v) / torch.where(l > 0, l, 1.0)
    lse = torch.where(l > 0, torch.log(l) + m0, -math.inf)[..., 0]
    o, lse = o[s["lane"], :, s["nth"]], lse[s["lane"], :, s["nth"]]
    s["out"].copy_(o.reshape(s["out"].shape))
    s["lse"].copy_(lse.reshape(s["lse"].shape))
    return s["out"], s["lse"]


def _copy_plain(s):
    for p in s["pools"]:
        p[s["dst"].long()] = p[s["src"].long()]
    return s["pools"]


# --------------------------------------------------------------------------
# the same through the package
# --------------------------------------------------------------------------
def _append_own(s):
    s["plan"].append_kv8(s["q"], s["k_new"], s["v_new"], s["q_rot"], s["k"], s["v"], s["ks"],
                         s["vs"], s["frozen"])
    return s["q_rot"], s["k"], s["v"], s["ks"], s["vs"]


def _attend_own(s):
    if "ks" in s:
        s["plan"].attend_kv8(s["q"], s["k"], s["v"], s["ks"], s["vs"], s.get("words"),
                             out_all=s["out"], lse_all=s["lse"])
    else:
        s["plan"].attend(s["q"], s["k"], s["v"], out_all=s["out"], lse_all=s["lse"])
    return s["out"], s["lse"]


def _copy_own(s):
    import programmable_paged_kv_gb300 as pk
    pk.copy_pages(s["pools"], s["src"], s["dst"])
    return s["pools"]


def run(state):
    op = state["case"]["op"]
    if op == "append":
        r = _append_own(state) if own else _append_plain(state)
    elif op == "copy":
        r = _copy_own(state) if own else _copy_plain(state)
    else:
        r = _attend_own(state) if own else _attend_plain(state)
    return list(r)


# --------------------------------------------------------------------------
# the definitions in 64 bits, lane by lane and page by page
# --------------------------------------------------------------------------
def _e4m3_values():
    v = [m / 8 * 2.0 ** -6 for m in range(8)]
    v += [(1 + m / 8) * 2.0 ** (e - 7) for e in range(1, 16) for m in range(8)][:-1]
    return torch.tensor(v, dtype=torch.float64, device=DEV)


def _two_to(e):
    """2^e in 64 bits, from a table of exact powers."""
    return torch.tensor([2.0 ** i for i in range(-130, 131)], dtype=torch.float64, device=DEV)[e.long() + 130]


def _nearest(x):
    """The e4m3 value nearest to x, the even code at a tie, by search among all of them."""
    t = _e4m3_values()
    a = x.abs().clamp(max=TOP)
    hi = torch.searchsorted(t, a.contiguous()).clamp(max=len(t) - 1)
    lo = (hi - 1).clamp(min=0)
    up, down = t[hi] - a, a - t[lo]
    pick = torch.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)
    return torch.where(x < 0, -t[pick], t[pick])


def _exact_append(s, g):
    c = s["case"]
    P, h = c["page"], c["d"] // 2

    def turned(x):
        z = torch.complex(x[..., :h].double(), x[..., h:].double())
        f = torch.tensor([10000.0 ** (-2 * i / c["d"]) for i in range(h)], dtype=torch.float64, device=DEV)
        a = s["slot"].double()[:, None, None] * f
        z = z * torch.complex(torch.cos(a), torch.sin(a))
        return torch.cat([z.real, z.imag], -1)

    out = [turned(s["q"])]
    pools, scales = [], []
    for pool, scale, x in ((s["k"], s["ks"], turned(s["k_new"])), (s["v"], s["vs"], s["v_new"].double())):
        val, exps = pool.double(), scale.long() - BIAS
        for l in range(c["lanes"]):
            r0, r1 = int(g["rind"][l]), int(g["rind"][l + 1])
            for lp in sorted(set((g["slot"][r0:r1] // P).tolist())):
                rows = [r for r in range(r0, r1) if g["slot"][r] // P == lp]
                page = int(g["table"][l, lp])
                offs = [int(g["slot"][r]) % P for r in rows]
                kept = [o for o in range(P) if o not in offs and lp * P + o < int(g["kv"][l])]
                big = x[rows].abs().amax((0, 2))
                e = torch.full_like(exps[page], E_MIN)
                for _ in range(E_MAX - E_MIN):
                    e = torch.where(big > TOP * _two_to(e), e + 1, e)
                if kept:
                    e = torch.maximum(e, exps[page])
                    moved = val[page][:, kept] * _two_to(exps[page] - e)[:, None, None]
                    val[page, :, kept] = _nearest(moved)
                val[page, :, offs] = _nearest(x[rows] / _two_to(e)[:, None]).transpose(0, 1)
                exps[page] = e
        pools.append(val)
        scales.append((exps + BIAS).to(torch.uint8))
    return out + pools + scales


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "copy":
        got = []
        for p in s["pools"]:
            q = p.clone()
            q.index_copy_(0, s["dst"].long(), p.index_select(0, s["src"].long()))
            got.append(q)
        return got
    g = _geo(case)
    if case["op"] == "append":
        return _exact_append(s, g)
    hq, hkv, d, P = case["hq"], case["hkv"], case["d"], case["page"]
    outs, lses = [], []
    for l in range(case["lanes"]):
        kv = int(g["kv"][l])
        ids = torch.from_numpy(g["table"][l, :-(-kv // P)]).to(DEV)
        kk, vv = (s[x].view(torch.uint8)[ids].view(s[x].dtype).double() if "ks" in s
                  else s[x][ids].double() for x in "kv")
        if "ks" in s:
            kk = kk * _two_to(s["ks"][ids].long() - BIAS)[:, :, None, None]
            vv = vv * _two_to(s["vs"][ids].long() - BIAS)[:, :, None, None]
        kk, vv = (x.transpose(0, 1).reshape(hkv, -1, d)[:, :kv] for x in (kk, vv))
        r0, r1 = int(g["rind"][l]), int(g["rind"][l + 1])
        q = s["q"][r0:r1].double().reshape(r1 - r0, hkv, -1, d).permute(1, 2, 0, 3)
        z = q @ kk[:, None].transpose(2, 3) / math.sqrt(d)  # [hkv, group, rows, kv]
        seen = np.zeros((r1 - r0, kv), bool)
        for i, r in enumerate(range(r0, r1)):
            if "wind" in g:
                w = g["words"][g["wind"][r]:g["wind"][r + 1]]
                seen[i] = np.unpackbits(w.view(np.uint8), bitorder="little")[:kv] != 0
            else:
                t = int(g["slot"][r])
                first = max(0, t - case["window"] + 1) if case.get("window") else 0
                seen[i, first:t + 1] = True
                seen[i, :min(case.get("sinks", 0), t + 1)] = True
        z = torch.where(torch.from_numpy(seen).to(DEV), z, -math.inf)
        lse = torch.logsumexp(z, -1)
        p = torch.exp(z - torch.where(lse == -math.inf, 0.0, lse)[..., None])
        outs.append((p @ vv[:, None]).permute(2, 0, 1, 3).reshape(r1 - r0, hq, d))
        lses.append(lse.permute(2, 0, 1).reshape(r1 - r0, hq))
    return [torch.cat(outs), torch.cat(lses)]
