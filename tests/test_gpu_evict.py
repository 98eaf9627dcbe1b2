"""spec_kv_weigh against the formula in 64 bits, spec_kv_evict against a walk over the tokens (equal bits)."""
import math

import numpy as np
import pytest
import torch

from speculative_decoding_token_temp_gb300 import _lib, api

import kv_util as U
import test_gpu_attention as A
from test_gpu_attention import Case, dev, i32  # noqa: F401 (dev: the fixture)
from test_gpu_attention_blocks import checked_build

pytestmark = pytest.mark.gpu


# ---- weights ----

def gathered(c, lse, mass, keep, taken=None, scale=None):
    """(mass, bound) [pages, kv_heads, page] in float64.

    Bound of a weight exp(s - lse): its exponent is off by what the score is off by (fp32 sums, 2^-24 a step, 128 steps at
    most: 2^-17 of sum |q k|; queries held to 2^-22 of their largest element) plus fp32's rounding of s, of the difference and
    of its product with log2(e) (2^-22 of |s| + |lse|), and exp2's own 2^-21; sums of n weights are off by n 2^-24."""
    q = c.q.double().numpy()
    R, H, D = q.shape
    cache = c.cache()
    kc, ke = U.raw(cache.k), U.raw(cache.k_exp)
    _, Hk, S, _ = kc.shape
    G, scale = H // Hk, D ** -0.5 if scale is None else scale
    new, lim = mass.astype(np.float64), np.zeros(mass.shape)
    r = 0
    for b, n_rows in enumerate(c.rows):
        n = int(c.lens[b])
        count = n_rows if taken is None else taken[b] + 1
        t = np.arange(n)
        page, slot = np.asarray(c.table[b], dtype=np.int64)[t // S], t % S
        for h in range(Hk):
            k = U.dequantise(kc[page, h, slot], ke[page, h, slot])
            add, off, most = np.zeros(n), np.zeros(n), 0
            for i in range(count):
                for g in range(G):
                    y = float(lse[r + i, h * G + g])
                    if not math.isfinite(y):
                        continue
                    x = q[r + i, h * G + g]
                    sees = t <= n - n_rows + i
                    kk = np.where(sees[:, None], k, 0)
                    s = scale * (kk @ x)
                    w = np.where(sees, np.exp(s - y), 0)
                    e = scale * (2.0 ** -17 * (np.abs(kk) @ np.abs(x)) + 2.0 ** -22 * np.abs(x).max() * np.abs(kk).sum(-1))
                    e += 2.0 ** -22 * (np.abs(s) + abs(y)) + 2.0 ** -21
                    add += w
                    off += w * e * 1.02
                    most += 1
            old = np.where(t < n - n_rows, mass[page, h, slot], 0) if keep else np.zeros(n)
            new[page, h, slot] = keep * old + add
            lim[page, h, slot] = off + (most + 4) * 2.0 ** -24 * add + 2.0 ** -23 * np.abs(keep * old) + 1e-35
        r += n_rows
    return new, lim


def weigh(c, lse, mass, **kw):
    cu = None
    if len(set(c.rows)) > 1:
        cu = i32(np.concatenate([[0], np.cumsum([r - 1 for r in c.rows])]), c.dev)
    return api.spec_kv_weigh(c.q.to(c.dev), c.cache(), i32(c.table, c.dev), i32(c.lens, c.dev), lse, mass, gamma=max(c.rows) - 1, cu_draft=cu, **kw)


def start(c, seed=0):
    """A mass whose places without a token hold NaN."""
    shape = c.cache().k_exp.shape
    m = np.full(shape, math.nan, dtype=np.float32)
    rng = np.random.default_rng(seed)
    for b, n in enumerate(c.lens):
        t = np.arange(int(n))
        m[np.asarray(c.table[b], dtype=np.int64)[t // shape[2]], :, t % shape[2]] = rng.random((int(n), shape[1]))
    return m


def check_weigh(c, keep=1.0, taken=None, lse=None, **kw):
    lse = c.call()["lse"] if lse is None else lse
    m = start(c)
    got = torch.from_numpy(m).to(c.dev)
    out = weigh(c, lse, got, keep=keep, n_accepted=None if taken is None else i32(taken, c.dev), **kw)
    assert int(out["device_status"][0]) == 0
    want, lim = gathered(c, lse.cpu().numpy(), m, keep, taken, **kw)
    got = got.cpu().numpy().astype(np.float64)
    assert np.array_equal(np.isnan(got), np.isnan(want))
    ok = ~np.isnan(want)
    off = np.abs(got - want)[ok]
    assert (off <= lim[ok]).all(), f"{(off / np.maximum(lim[ok], 1e-300)).max():.3g} of the bound"
    return got


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dim,page", [(64, 16), (128, 64), (128, 256)])
def test_one_token_at_every_edge_length(dev, dtype, dim, page):  # noqa: F811
    check_weigh(Case(dev, A.EDGE, [1] * len(A.EDGE), dim=dim, page=page, dtype=dtype))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dim,heads,kv_heads,rows", [(128, 1, 1, 1), (128, 8, 8, 5), (128, 6, 2, 9), (64, 14, 2, 17), (128, 64, 1, 3), (64, 8, 1, 129), (128, 12, 4, 33)])
def test_head_layouts_and_many_rows(dev, dtype, dim, heads, kv_heads, rows):  # noqa: F811
    check_weigh(Case(dev, [rows, rows + 131, max(0, rows - 2)], [rows] * 3, heads=heads, kv_heads=kv_heads, dim=dim, dtype=dtype), keep=0.5)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("keep", [1.0, 0.0, 0.9])
def test_ragged_rounds_and_accepted_rows(dev, dtype, keep):  # noqa: F811
    rows = [1, 2, 17, 9, 3, 5, 1, 17, 8]
    lens = [1, 300, 17, 4, 0, 129, 0, 260, 1000]
    c = Case(dev, lens, rows, heads=12, kv_heads=4, dim=64, page=16, dtype=dtype)
    check_weigh(c, keep=keep)
    check_weigh(c, keep=keep, taken=[0, 1, 5, 8, 0, 3, 0, 11, 7])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dim", [64, 128])
def test_rows_and_heads_at_every_edge_of_what_is_worked_on_at_a_time(dev, dtype, dim):  # noqa: F811
    # 16 query heads a kv head: 128, 16, 80, 64, 112, 48, 96, 32 of a sequence's rows and heads one behind another, and
    # three heads a kv head: 129, 126, 66, 63, 15, 18
    rows = [8, 1, 5, 4, 7, 3, 6, 2]
    check_weigh(Case(dev, [300 + 41 * i for i in range(8)], rows, heads=32, kv_heads=2, dim=dim, page=32, dtype=dtype), keep=0.5)
    rows = [43, 42, 22, 21, 5, 6, 86, 85]
    c = Case(dev, [600 - 17 * i for i in range(8)], rows, heads=6, kv_heads=2, dim=dim, page=32, dtype=dtype)
    check_weigh(c)
    check_weigh(c, keep=0.0, taken=[42, 20, 21, 0, 4, 2, 43, 64])


def test_weights_of_a_row_sum_to_one_behind_a_prefix_to_less(dev):  # noqa: F811
    c = Case(dev, [500, 700], [4, 4], heads=8, kv_heads=2, dim=128)
    got = check_weigh(c, keep=0.0)
    assert abs(np.nansum(got) - 2 * 4 * 8) < 1e-3
    p = Case(dev, [500, 700], [4, 4], heads=8, kv_heads=2, dim=128, prefix=300)
    assert 1 < np.nansum(check_weigh(p, keep=0.0)) < 2 * 4 * 8 - 1


def test_rows_without_a_sum_add_nothing(dev):  # noqa: F811
    c = Case(dev, [200, 150], [6, 6], heads=4, kv_heads=2, dim=64, page=32)
    lse = c.call()["lse"].clone()
    lse[1, 0], lse[3, 2], lse[7] = math.nan, math.inf, -math.inf
    check_weigh(c, lse=lse)


def test_hidden_nan_tokens_and_scales(dev):  # noqa: F811
    c = Case(dev, [200, 150], [6, 6], heads=4, kv_heads=2, dim=64, page=32)
    lse = c.call()["lse"]
    check_weigh(c, lse=lse, scale=0.05)
    c.exps[0][c.table[0][197 // 32], 0, 197 % 32] = 255  # only rows 3, 4, 5 see it
    del c._cache
    m = torch.from_numpy(start(c)).to(dev)
    weigh(c, lse, m, n_accepted=i32([2, 5], dev))
    assert not torch.isnan(m[c.table[0][197 // 32], 0, 197 % 32])


def test_bad_lengths_pages_counts_and_offsets(dev):  # noqa: F811
    c = Case(dev, [300, 350, 280], [5] * 3, heads=8, kv_heads=2, dim=64)
    lse, m0 = c.call()["lse"], torch.from_numpy(start(c)).to(dev)
    good = m0.clone()
    weigh(c, lse, good)

    def same(a, b, b_of, tokens):
        for j in range(-(-tokens // 64)):
            pg = int(c.table[b_of][j])
            assert torch.equal(torch.nan_to_num(a[pg], -1.0), torch.nan_to_num(b[pg], -1.0))

    c.lens[1] = -4
    m = m0.clone()
    assert int(weigh(c, lse, m)["device_status"][0]) == _lib.SPEC_DEV_OFFSETS
    same(m, good, 0, 300), same(m, m0, 1, 350), same(m, good, 2, 280)
    c.lens[1] = 350
    for taken in ([4, 5, 4], [4, -1, 4]):
        m = m0.clone()
        assert int(weigh(c, lse, m, n_accepted=i32(taken, dev))["device_status"][0]) == _lib.SPEC_DEV_OFFSETS
        same(m, good, 0, 300), same(m, m0, 1, 350), same(m, good, 2, 280)
    page, c.table[2][1] = c.table[2][1], -7
    m = m0.clone()
    assert int(weigh(c, lse, m)["device_status"][0]) == _lib.SPEC_DEV_PAGE
    same(m, good, 0, 300), same(m, good, 1, 350)
    assert torch.equal(torch.nan_to_num(m[page], -1.0), torch.nan_to_num(m0[page], -1.0))
    c.table[2][1] = page
    m = m0.clone()
    out = api.spec_kv_weigh(c.q.to(dev), c.cache(), i32(c.table, dev), i32(c.lens, dev), lse, m, gamma=4, cu_draft=i32([0, 5, 9, 12], dev))
    assert int(out["device_status"][0]) == _lib.SPEC_DEV_OFFSETS and torch.equal(torch.nan_to_num(m, -1.0), torch.nan_to_num(m0, -1.0))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_weigh_views_graphs_repeats_and_the_bounds_checked_build(dev, dtype):  # noqa: F811
    rng = np.random.default_rng(0)
    c = Case(dev, [int(x) for x in rng.integers(5, 900, 40)], [5] * 40, heads=8, kv_heads=2, dim=128, dtype=dtype)
    lse, m0 = c.call()["lse"], torch.from_numpy(start(c)).to(dev)
    a = m0.clone()
    weigh(c, lse, a)
    b = m0.clone()
    with checked_build():
        assert int(weigh(c, lse, b)["device_status"][0]) == 0
    q = torch.zeros(200, 8, 131, dtype=c.dtype, device=dev)[:, :, 1:129]
    q.copy_(c.q)
    d = m0.clone()
    table, lens = i32(c.table, dev), i32(c.lens, dev)
    api.spec_kv_weigh(q, c.cache(), table, lens, lse, d, gamma=4)
    e, out = m0.clone(), {"device_status": torch.zeros(1, dtype=torch.int32, device=dev)}
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        api.spec_kv_weigh(q, c.cache(), table, lens, lse, e, gamma=4, out=out)
    for _ in range(2):
        e.copy_(m0)
        graph.replay()
    for x in (b, d, e):
        assert torch.equal(torch.nan_to_num(x, -1.0), torch.nan_to_num(a, -1.0))


# ---- eviction ----

def key(x):
    return (-math.inf, -1) if math.isnan(x) else (float(x), 0)


def stays(mass, n, budget, sinks, recent):
    """The places that stay, by the definition."""
    if n <= budget:
        return list(range(n))
    free = range(sinks, n - recent)
    best = sorted(free, key=lambda t: (-(key(mass[t])[0]), -key(mass[t])[1], t))[:budget - sinks - recent]
    return sorted(list(range(sinks)) + best + list(range(n - recent, n)))


class Held:
    """A cache with random bytes, its weights, and sequences' pages."""

    def __init__(self, dev, lens, *, kv_heads=2, page=32, dim=64, seed=0, more=0, weights="plain"):
        rng = np.random.default_rng([seed, page, dim, len(lens)])
        need = list(lens) + [more] * len(lens)
        table, pages = U.pages_for(need, page, rng)
        self.table = table[:len(lens)][:, :max(1, -(-max(lens, default=1) // page))]
        self.new = table[len(lens):][:, :max(1, -(-more // page))]
        self.lens, self.page, self.dev = list(lens), page, dev
        g = torch.Generator(device=dev).manual_seed(seed)
        shape = (pages, kv_heads, page, dim)
        self.raw = [torch.randint(0, 256, s, dtype=torch.uint8, generator=g, device=dev) for s in (shape, shape, shape[:3], shape[:3])]
        m = rng.standard_normal(shape[:3]).astype(np.float32)
        if weights == "ties":
            m = rng.integers(0, 3, shape[:3]).astype(np.float32) * rng.choice([-1, 1], shape[:3]).astype(np.float32)
        if weights == "strange":
            m = rng.choice(np.array([math.nan, math.inf, -math.inf, 0.0, -0.0, 1e-40, -1e-40, 3.0], dtype=np.float32), shape[:3])
        if weights == "equal":
            m[:] = 0.25
        self.mass = torch.from_numpy(m).to(dev)

    def copies(self):
        raw, mass = [t.clone() for t in self.raw], self.mass.clone()
        return api.KVCache(raw[0].view(torch.float8_e4m3fn), raw[1].view(torch.float8_e4m3fn), raw[2], raw[3]), raw, mass

    def check(self, budget, sinks=0, recent=0, moved=False):
        cache, raw, mass = self.copies()
        new = i32(self.new, self.dev) if moved else None
        table, lens = i32(self.table, self.dev), i32(self.lens, self.dev)
        out = api.spec_kv_evict(cache, mass, table, lens, budget, sinks=sinks, recent=recent, new_table=new)
        assert int(out["device_status"][0]) == 0
        want = [t.cpu().numpy().copy() for t in self.raw] + [self.mass.cpu().numpy().copy()]
        old = [w.copy() for w in want]
        kept, n_out = out["kept"].cpu().numpy(), out["kv_len"].cpu().numpy()
        S, Hk = self.page, kept.shape[1]
        for b, n in enumerate(self.lens):
            assert n_out[b] == min(n, budget)
            src = np.asarray(self.table[b], dtype=np.int64)
            dst = np.asarray(self.new[b], dtype=np.int64) if moved else src
            t = np.arange(n)
            for h in range(Hk):
                s = np.array(stays(old[4][src[t // S], h, t % S], n, budget, sinks, recent), dtype=np.int64)
                assert np.array_equal(kept[b, h, :len(s)], s) and (kept[b, h, len(s):] == -1).all()
                j = np.arange(len(s))
                for w, o in zip(want, old):
                    w[dst[j // S], h, j % S] = o[src[s // S], h, s % S]
        for x, w in zip(raw + [mass], want):
            assert np.array_equal(x.cpu().numpy().view(np.uint8), w.view(np.uint8))
        return out


@pytest.mark.parametrize("moved", [False, True])
@pytest.mark.parametrize("weights", ["plain", "ties", "strange", "equal"])
@pytest.mark.parametrize("dim,page,kv_heads,lens,budget,sinks,recent", [
    (64, 16, 2, [0, 1, 15, 16, 17, 100, 333], 16, 0, 0), (128, 64, 1, [500, 64, 65, 1200], 64, 4, 10), (64, 256, 3, [300, 900], 1, 0, 0),
    (128, 16, 2, [700, 701], 700, 3, 5), (64, 32, 8, [1000], 333, 33, 300), (128, 32, 1, [4100, 40, 4096], 2000, 4, 100), (64, 64, 1, [90], 50, 20, 30)])
def test_the_heaviest_stay_in_their_order(dev, dim, page, kv_heads, lens, budget, sinks, recent, weights, moved):  # noqa: F811
    Held(dev, lens, kv_heads=kv_heads, page=page, dim=dim, more=min(budget, max(lens)), weights=weights).check(budget, sinks, recent, moved)


@pytest.mark.parametrize("moved", [False, True])
def test_more_tokens_than_shared_memory_holds(dev, moved):  # noqa: F811
    Held(dev, [40000, 17000], kv_heads=1, page=256, dim=64, more=21000, weights="ties").check(21000, 4, 64, moved)


def test_a_budget_past_every_length(dev):  # noqa: F811
    h = Held(dev, [100, 37], more=100)
    h.check(1000)
    h.check(1000, moved=True)


def test_eviction_bad_lengths_and_pages(dev):  # noqa: F811
    h = Held(dev, [200, 190, 180], page=32, more=64)
    for moved in (False, True):
        for what in ("length", "page", "new page"):
            if what == "new page" and not moved:
                continue
            cache, raw, mass = h.copies()
            lens, table, new = list(h.lens), h.table.copy(), h.new.copy()
            if what == "length":
                lens[1] = 32 * table.shape[1] + 1
            elif what == "page":
                table[1, 3] = -1
            else:
                new[1, 1] = 1 << 29
            out = api.spec_kv_evict(cache, mass, i32(table, dev), i32(lens, dev), 64, new_table=i32(new, dev) if moved else None)
            assert int(out["device_status"][0]) == (_lib.SPEC_DEV_OFFSETS if what == "length" else _lib.SPEC_DEV_PAGE)
            assert out["kv_len"].tolist() == [64, 0 if moved else lens[1], 64]
            assert (out["kept"][1] == -1).all() and (out["kept"][[0, 2]] >= 0).all()
            for pg in [int(x) for x in (h.new if moved else h.table)[1] if 0 <= x < raw[0].shape[0]]:
                for a, b in zip(raw + [mass], h.raw + [h.mass]):
                    assert torch.equal(a[pg].view(torch.uint8), b[pg].view(torch.uint8))


def test_eviction_in_a_graph_and_in_the_bounds_checked_build(dev):  # noqa: F811
    h = Held(dev, [900, 700, 30], kv_heads=2, page=32, dim=128, more=400)
    for new in (None, i32(h.new, dev)):
        a, raw_a, mass_a = h.copies()
        table, lens = i32(h.table, dev), i32(h.lens, dev)
        one = api.spec_kv_evict(a, mass_a, table, lens, 400, sinks=4, recent=50, new_table=new)
        b, raw_b, mass_b = h.copies()
        with checked_build():
            two = api.spec_kv_evict(b, mass_b, table, lens, 400, sinks=4, recent=50, new_table=new)
            assert int(two["device_status"][0]) == 0
        c, raw_c, mass_c = h.copies()
        out = {"device_status": torch.zeros(1, dtype=torch.int32, device=dev)}
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            api.spec_kv_evict(c, mass_c, table, lens, 400, sinks=4, recent=50, new_table=new, out=out)
        graph.replay()
        for got, raw, mass in ((two, raw_b, mass_b), (out, raw_c, mass_c)):
            assert torch.equal(got["kept"], one["kept"]) and torch.equal(got["kv_len"], one["kv_len"])
            for x, y in zip(raw + [mass], raw_a + [mass_a]):
                assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))


def test_attention_after_eviction_is_attention_over_what_stays(dev):  # noqa: F811
    """Weigh, evict, attend: as over a cache that held only the kept tokens from the beginning."""
    c = Case(dev, [300, 500], [3, 3], heads=4, kv_heads=2, dim=64, page=32)
    first = c.call()
    mass = torch.full(c.cache().k_exp.shape, math.nan, device=dev)
    weigh(c, first["lse"], mass, keep=0.0)
    kept = api.spec_kv_evict(c.cache(), mass, i32(c.table, dev), i32(c.lens, dev), 128, sinks=2, recent=3)
    old_k, old_v = [x.copy() for x in c.codes], [x.copy() for x in c.exps]
    own = Case(dev, [128, 128], [3, 3], heads=4, kv_heads=2, dim=64, page=32)
    for b in range(2):
        src = np.asarray(c.table[b], dtype=np.int64)
        dst = np.asarray(own.table[b], dtype=np.int64)
        j = np.arange(128)
        for h in range(2):
            t = kept["kept"][b, h].cpu().numpy()
            for i in range(2):
                own.codes[i][dst[j // 32], h, j % 32] = old_k[i][src[t // 32], h, t % 32]
                own.exps[i][dst[j // 32], h, j % 32] = old_v[i][src[t // 32], h, t % 32]
    own.q = c.q
    got = api.spec_attention(c.q.to(dev), c.cache(), i32(c.table, dev), kept["kv_len"], gamma=2, want_lse=True)
    want = own.call()
    assert torch.equal(got["o"], want["o"]) and torch.equal(got["lse"], want["lse"])
