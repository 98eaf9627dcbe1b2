"""spec_attention against the 64-bit restatement, with bounds derived from the roundings (kv_util.bounds)."""
import math

import numpy as np
import pytest
import torch

from speculative_decoding_token_temp_gb300 import _lib, api, synth

import kv_util as U

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()
    return torch.device("cuda:0")


def i32(a, dev):
    return torch.as_tensor(np.asarray(a, dtype=np.int32)).to(dev)


class Case:
    """A cache that holds `lens` tokens of each sequence (and a prefix) on pages in any order, every other place a NaN code
    under a NaN exponent, with queries of `rows` rows per sequence."""

    def __init__(self, dev, lens, rows, *, heads=4, kv_heads=2, dim=128, page=64, dtype="bf16", prefix=0, parent=None,
                 seed=0, extra=2, size=1.5):
        rng = np.random.default_rng([seed, dim, page, heads, prefix, sum(rows)])
        self.dev, self.lens, self.rows, self.prefix, self.parent = dev, list(lens), list(rows), prefix, parent
        table, pages = U.pages_for(list(lens) + [prefix], page, rng, extra=extra)
        self.prefix_table = table[-1][:max(1, -(-prefix // page))]
        self.table = table[:-1][:, :max(1, max((-(-n // page) for n in lens), default=1))]
        shape = (pages, kv_heads, page, dim)
        codes = [np.full(shape, 0x7f, dtype=np.uint8) for _ in range(2)]
        exps = [np.full(shape[:3], 255, dtype=np.uint8) for _ in range(2)]
        for tb, n in list(zip(self.table, lens)) + [(self.prefix_table, prefix)]:
            for j in range(-(-int(n) // page)):
                m = min(page, int(n) - j * page)
                for i in range(2):
                    c = rng.standard_normal((kv_heads, m, dim)) * (150 if i else 100)
                    g = np.clip(c, -448, 448)
                    codes[i][tb[j], :, :m] = torch.from_numpy(g).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
                    exps[i][tb[j], :, :m] = 127 - 7 + rng.integers(-2, 2, (kv_heads, m))
        self.codes, self.exps = codes, exps
        self.rng = rng
        R = sum(rows)
        self.q = torch.from_numpy(rng.standard_normal((R, heads, dim)) * size).to(DT[dtype])
        self.dtype = DT[dtype]

    def cache(self):
        if not hasattr(self, "_cache"):
            k, v = (torch.from_numpy(c).to(self.dev).view(torch.float8_e4m3fn) for c in self.codes)
            ke, ve = (torch.from_numpy(e).to(self.dev) for e in self.exps)
            self._cache = api.KVCache(k, v, ke, ve)
        return self._cache

    def call(self, q=None, **kw):
        dense = len(set(self.rows)) <= 1
        cu = None
        if not dense:
            cu = i32(np.concatenate([[0], np.cumsum([r - 1 for r in self.rows])]), self.dev)
        kw.setdefault("want_lse", True)
        pre = dict(prefix_table=i32(self.prefix_table, self.dev), prefix_len=self.prefix) if self.prefix else {}
        return api.spec_attention(self.q.to(self.dev) if q is None else q, self.cache(), i32(self.table, self.dev),
                                  i32(self.lens, self.dev), gamma=max(self.rows) - 1 if self.rows else 0, cu_draft=cu,
                                  parent=self.parent, **pre, **kw)

    def ref(self, **kw):
        return U.attention(self.q.double().numpy(), self.cache(), self.table, self.lens, self.rows, parent=self.parent,
                           prefix_table=self.prefix_table, prefix_len=self.prefix, **kw)

    def check(self, status=0, **kw):
        out = self.call(**kw)
        assert int(out["device_status"][0]) == status
        U.compare(out["o"], out.get("lse"), self.ref(**{k: v for k, v in kw.items() if k == "scale"}), self.dtype,
                  max(self.lens, default=0) + self.prefix)
        return out


EDGE = [0, 1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 255, 256, 257, 383, 500]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("page", [16, 64, 128, 256])
def test_one_token_per_sequence_at_every_edge_length(dev, dtype, dim, page):
    Case(dev, EDGE, [1] * len(EDGE), dim=dim, page=page, dtype=dtype).check()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dim,heads,kv_heads", [(128, 1, 1), (128, 8, 8), (128, 6, 2), (64, 14, 2), (128, 16, 1), (64, 40, 1), (128, 64, 1)])
def test_head_layouts(dev, dtype, dim, heads, kv_heads):
    Case(dev, [5, 130, 300], [5, 5, 5], heads=heads, kv_heads=kv_heads, dim=dim, dtype=dtype).check()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dim,page", [(64, 32), (128, 16), (128, 256)])
def test_ragged_rounds(dev, dtype, dim, page):
    """Sequences of 1 to 17 rows, some with fewer cached tokens than rows: rows that see nothing are zeros, lse -inf."""
    rows = [1, 2, 17, 9, 3, 5, 1, 17, 8]
    lens = [1, 300, 17, 4, 0, 129, 0, 260, 1000]
    c = Case(dev, lens, rows, heads=12, kv_heads=4, dim=dim, page=page, dtype=dtype)
    out = c.check()
    first = sum(rows[:3])
    assert (out["o"][first:first + 5] == 0).all() and torch.isneginf(out["lse"][first:first + 5]).all()
    assert (out["o"][first + 5] != 0).any()


@pytest.mark.parametrize("gamma", [0, 3, 15, 16, 40, 128])
def test_long_rounds(dev, gamma):
    """Up to 129 rows per sequence: several row blocks over the same keys."""
    Case(dev, [gamma + 1, 400, 129 + gamma], [gamma + 1] * 3, heads=8, kv_heads=2, dim=128).check()


TREES = {"chains": list(synth.TREE_PARENT), "star": [-1] * 20, "binary": [-1, -1] + [j // 2 for j in range(28)],
         "deep": [j - 1 for j in range(64)], "one": [-1]}


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("tree", list(TREES))
@pytest.mark.parametrize("dim", [64, 128])
def test_trees(dev, dtype, tree, dim):
    parent = [int(x) for x in TREES[tree]]
    n = len(parent) + 1
    Case(dev, [n, 200, 127 + n // 2, n // 2], [n] * 4, heads=6, kv_heads=2, dim=dim, dtype=dtype, parent=parent).check()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("prefix", [1, 127, 128, 129, 700])
@pytest.mark.parametrize("page,dim", [(16, 64), (128, 128)])
def test_shared_prefix(dev, dtype, prefix, page, dim):
    rows = [3, 1, 6, 2, 9]
    Case(dev, [3, 0, 300, 1, 64], rows, heads=8, kv_heads=2, dim=dim, page=page, dtype=dtype, prefix=prefix).check()


def test_shared_prefix_under_a_tree_and_a_large_batch(dev):
    parent = [int(x) for x in synth.TREE_PARENT]
    Case(dev, [13, 100], [13] * 2, heads=4, kv_heads=1, prefix=260, parent=parent).check()
    Case(dev, [9] * 40, [9] * 40, heads=8, kv_heads=2, prefix=513).check()


def test_prefix_equals_the_same_tokens_in_every_sequence(dev):
    """A prefix of whole pages gives what the batch gives with these pages at the head of each sequence's own."""
    c = Case(dev, [70, 9, 140], [9] * 3, heads=8, kv_heads=2, page=64, prefix=256)
    a = c.call()
    tb = np.concatenate([np.tile(c.prefix_table[:4], (3, 1)), np.where(c.table > 1 << 29, 0, c.table)], axis=1)
    b = api.spec_attention(c.q.to(dev), c.cache(), i32(tb, dev), i32([n + 256 for n in c.lens], dev), gamma=8, want_lse=True)
    ref = c.ref()
    for got in (a, b):
        U.compare(got["o"], got["lse"], ref, c.dtype, 400)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_one_long_sequence_is_split_and_joined(dev, dtype):
    """A single sequence of many tiles (its parts come from as many blocks), alone and beside short ones."""
    Case(dev, [9001], [2], heads=2, kv_heads=1, page=256, dtype=dtype).check()
    Case(dev, [3, 5000, 1, 0, 700], [1] * 5, heads=8, kv_heads=2, dtype=dtype).check()


def test_query_layouts(dev):
    """Queries cut out of a wider projection, off the 16-byte grid, head-major, four-dimensional: the packed result."""
    c = Case(dev, [40, 200], [4, 4], heads=6, kv_heads=2)
    want = c.check()["o"]
    R, H, D = c.q.shape
    wide = torch.full((R, (H + 4) * D), math.nan, dtype=c.dtype, device=dev)
    a = wide[:, :H * D].unflatten(1, (H, D))
    odd = torch.full((R * H * (D + 1) + 1,), math.nan, dtype=c.dtype, device=dev)[1:].view(R, H, D + 1)[:, :, :D]
    major = torch.empty(H, R, D, dtype=c.dtype, device=dev).transpose(0, 1)
    for q in (a, odd, major):
        q.copy_(c.q)
        assert torch.equal(c.call(q=q)["o"], want)
    assert torch.equal(c.call(q=c.q.to(dev).view(2, 4, H, D))["o"], want)


def test_scale_is_applied(dev):
    c = Case(dev, [40, 200], [4, 4])
    c.check(scale=0.5)
    c.check(scale=1e-6)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dim", [64, 128])
def test_scores_of_every_size(dev, dtype, dim):
    """One dominant token, scores that reach hundreds, rows of very different size, values of very different size."""
    c = Case(dev, [600, 77], [3, 3], heads=4, kv_heads=2, dim=dim, dtype=dtype, size=1.0)
    c.q *= torch.tensor([1e-4, 1.0, 20.0, 3.0]).view(1, 4, 1).to(c.dtype)
    for i, e in enumerate(c.exps):
        e[...] = np.where(e == 255, 255, np.clip(e.astype(int) + c.rng.integers(-12, 2, e.shape), 27, 240))
    c.check()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_values_of_zero_and_of_tiny_size(dev, dtype):
    """Tokens whose value is zero (exponent -60) or far smaller than the others' keep their weight in the sum."""
    c = Case(dev, [300], [1], heads=2, kv_heads=1, dtype=dtype)
    page = c.table[0]
    for j in range(5):
        c.codes[1][page[j], 0, ::2] = 0
        c.exps[1][page[j], 0, ::2] = 127 + U.ZERO_EXP
        c.exps[1][page[j], 0, 1::4] = np.where(c.exps[1][page[j], 0, 1::4] == 255, 255, 127 - 40)
    c.check()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("where", ["k_exp", "v_exp", "v_code", "k_code"])
def test_nan_of_a_drafted_token_reaches_only_rows_that_see_it(dev, dtype, dim, where):
    lens, rows = [135, 60, 128], [9, 9, 9]
    c = Case(dev, lens, rows, dim=dim, dtype=dtype, heads=4, kv_heads=2)
    for b in range(3):
        t = lens[b] - 4                       # the token of row 5
        pg, slot = c.table[b, t // 64], t % 64
        if where == "k_exp":
            c.exps[0][pg, 1, slot] = 255
        elif where == "v_exp":
            c.exps[1][pg, 1, slot] = 255
        else:
            c.codes[0 if where == "k_code" else 1][pg, 1, slot, 7] = 0xff
    out = c.check()
    nan = torch.isnan(out["o"]).all(-1).view(3, 9, 4).cpu()
    assert nan[:, 5:, 2:].all() and not nan[:, :5].any() and not nan[:, :, :2].any()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("what", [math.nan, math.inf])
def test_nan_of_context_and_of_queries(dev, dtype, what):
    c = Case(dev, [300, 20], [2, 2], heads=4, kv_heads=2, dtype=dtype, prefix=40)
    c.exps[0][c.table[0, 0], 1, 5] = 255      # a context token of sequence 0, kv head 1
    c.q[3, 0, 9] = what
    out = c.check()
    nan = torch.isnan(out["o"]).all(-1).cpu()
    assert nan.tolist() == [[False, False, True, True]] * 2 + [[False] * 4, [True, False, False, False]]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("prefix", [0, 100])
def test_bad_lengths_pages_and_offsets(dev, dtype, prefix):
    c = Case(dev, [100, 150, 30, 64], [2, 2, 2, 2], dtype=dtype, prefix=prefix)
    good = c.call()["o"]
    width = c.table.shape[1] * 64
    for bad, bit in ((-1, _lib.SPEC_DEV_OFFSETS), (width + 1, _lib.SPEC_DEV_OFFSETS), (-2 ** 31, _lib.SPEC_DEV_OFFSETS)):
        lens, c.lens = c.lens, [100, bad, 30, 64]
        out = c.call()
        c.lens = lens
        assert int(out["device_status"][0]) == bit
        assert torch.isnan(out["o"][2:4]).all() and torch.isnan(out["lse"][2:4]).all()
        assert torch.equal(out["o"][:2], good[:2]) and torch.equal(out["o"][4:], good[4:])
    for bad in (-1, 1 << 30, c.cache().num_pages):
        keep = c.table.copy()
        c.table[1, 1] = bad
        out = c.call()
        c.table = keep
        assert int(out["device_status"][0]) == _lib.SPEC_DEV_PAGE
        assert torch.isnan(out["o"][2:4]).all()
        assert torch.equal(out["o"][:2], good[:2]) and torch.equal(out["o"][4:], good[4:])
    if prefix:
        keep = c.prefix_table.copy()
        c.prefix_table = keep.copy()
        c.prefix_table[1] = -5
        out = c.call()
        c.prefix_table = keep
        assert int(out["device_status"][0]) == _lib.SPEC_DEV_PAGE and torch.isnan(out["o"]).all()
    for cu in ([0, 1, 2, 3, 5], [0, 2, 1, 3, 4], [1, 1, 2, 3, 4], [0, 3, 3, 4, 4], [-1, 1, 2, 3, 4]):
        out = api.spec_attention(c.q.to(dev), c.cache(), i32(c.table, dev), i32(c.lens, dev), gamma=1, cu_draft=i32(cu, dev),
                                 want_lse=True)
        assert int(out["device_status"][0]) == _lib.SPEC_DEV_OFFSETS and torch.isnan(out["o"]).all() and torch.isnan(out["lse"]).all(), cu
    out = api.spec_attention(c.q.to(dev), c.cache(), i32(c.table, dev), i32(c.lens, dev), gamma=1, cu_draft=i32([0, 1, 2, 3, 4], dev))
    assert int(out["device_status"][0]) == 0


def test_no_sequences_and_no_pages(dev):
    c = Case(dev, [5], [1])
    q = c.q.to(dev)
    out = api.spec_attention(q[:0], c.cache(), i32(np.zeros((0, 1)), dev), i32([], dev), gamma=0)
    assert out["o"].shape[0] == 0
    out = api.spec_attention(q, c.cache(), torch.zeros(1, 0, dtype=torch.int32, device=dev), i32([0], dev), gamma=0, want_lse=True)
    assert (out["o"] == 0).all() and torch.isneginf(out["lse"]).all() and int(out["device_status"][0]) == 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_places_past_32_bits(dev, dtype):
    """A sequence whose pages start beyond 2^32 codes."""
    page, heads, dim = 256, 8, 128
    n = (1 << 32) // (page * heads * dim) + 3
    c = api.KVCache.empty(n, heads, page, dim, dev)
    rng = np.random.default_rng(7)
    length = 300
    x = [torch.from_numpy(rng.standard_normal((length, heads, dim))).to(torch.bfloat16).to(dev) for _ in range(2)]
    tb = i32([[n - 1, n - 3]], dev)
    api.spec_kv_append(c, x[0], x[1], tb, torch.zeros(length, dtype=torch.int32, device=dev), torch.arange(length, dtype=torch.int32, device=dev))
    q = torch.from_numpy(rng.standard_normal((2, 16, dim))).to(DT[dtype])
    out = api.spec_attention(q.to(dev), c, tb, i32([length], dev), gamma=1, want_lse=True)
    pick = [n - 1, n - 3]
    small = api.KVCache(*(t[pick].contiguous() if t.dtype == torch.uint8 else t.view(torch.uint8)[pick].contiguous().view(torch.float8_e4m3fn)
                          for t in (c.k, c.v, c.k_exp, c.v_exp)))
    ref = U.attention(q.double().numpy(), small, np.array([[0, 1]]), [length], [2])
    U.compare(out["o"], out["lse"], ref, DT[dtype], length)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_same_bits_every_time_and_on_other_streams(dev, dtype):
    a = Case(dev, [700, 3000, 10, 64], [3] * 4, heads=8, kv_heads=2, prefix=300, dtype=dtype)
    b = Case(dev, [90, 2000], [2] * 2, heads=8, kv_heads=2, seed=3, dtype=dtype)
    want = [x.call()["o"].clone() for x in (a, b)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(dev) for _ in range(2)]
    outs = [[], []]
    for _ in range(8):
        for i, (x, s) in enumerate(zip((a, b), streams)):
            with torch.cuda.stream(s):
                outs[i].append(x.call()["o"])
    torch.cuda.synchronize()
    for w, o in zip(want, outs):
        assert all(torch.equal(w, y) for y in o)


def test_one_call_per_launch_in_a_graph(dev):
    """Append and attention captured once, replayed as the sequences grow."""
    page, heads, dim, B, steps = 16, 2, 128, 3, 20
    rng = np.random.default_rng(11)
    start = [0, 15, 130]
    table, pages = U.pages_for([n + steps for n in start], page, rng)
    table = np.where(table > 1 << 29, 0, table)
    c = api.KVCache.empty(pages, heads, page, dim, dev)
    tb = i32(table, dev)
    past = torch.from_numpy(rng.standard_normal((2, 130, heads, dim))).to(torch.bfloat16).to(dev)
    for b, n in enumerate(start):
        if n:
            api.spec_kv_append(c, past[0, :n], past[1, :n], tb, torch.full((n,), b, dtype=torch.int32, device=dev),
                               torch.arange(n, dtype=torch.int32, device=dev))
    q = torch.zeros(B, 8, dim, dtype=torch.bfloat16, device=dev)
    k, v = (torch.zeros(B, heads, dim, dtype=torch.bfloat16, device=dev) for _ in range(2))
    pos = i32(start, dev)
    seq = torch.arange(B, dtype=torch.int32, device=dev)
    length = pos + 1
    out = {}
    ws = torch.empty(api.spec_attention_workspace_bytes(q, c, tb, length, gamma=0), dtype=torch.uint8, device=dev)

    def step():
        api.spec_kv_append(c, k, v, tb, seq, pos, out=out)
        api.spec_attention(q, c, tb, length, gamma=0, out=out, workspace=ws)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(steps):
        for t in (q, k, v):
            t.copy_(torch.from_numpy(rng.standard_normal(tuple(t.shape))))
        graph.replay()
        lens = [n + i + 1 for n in start]
        ref = U.attention(q.double().cpu().numpy(), c, table, lens, [1] * B)
        U.compare(out["o"], None, ref, torch.bfloat16, max(lens))
        pos += 1
        length += 1
    assert int(out["device_status"][0]) == 0


def test_argument_checks(dev):
    c = Case(dev, [20, 30], [2, 2])
    q, cache, tb, n = c.q.to(dev), c.cache(), i32(c.table, dev), i32(c.lens, dev)
    with pytest.raises(TypeError):
        api.spec_attention(q.half(), cache, tb, n, gamma=1)
    with pytest.raises(ValueError):
        api.spec_attention(q, cache, tb, n, gamma=2)
    with pytest.raises(ValueError):
        api.spec_attention(q, cache, tb, n)
    with pytest.raises(ValueError):
        api.spec_attention(q[:, :, :64], cache, tb, n, gamma=1)
    with pytest.raises(ValueError):
        api.spec_attention(q, cache, tb, n[:1], gamma=1)
    with pytest.raises(TypeError):
        api.spec_attention(q, cache, tb.long(), n, gamma=1)
    with pytest.raises(ValueError):
        api.spec_attention(q, cache, tb, n, gamma=1, prefix_table=tb[0][:1].contiguous(), prefix_len=65)
    with pytest.raises(ValueError):
        api.spec_attention(q, cache, tb, n, gamma=1, parent=[-1, -1])
    with pytest.raises(_lib.SpecError):
        api.spec_attention(q[:, :3], cache, tb, n, gamma=1)
    with pytest.raises(ValueError):
        api.spec_attention(q, cache, tb, n, gamma=1, workspace=torch.empty(16, dtype=torch.uint8, device=dev))
    with pytest.raises(ValueError):
        api.spec_attention(q, cache, tb, n, gamma=1, out={"o": torch.empty(1, dtype=c.dtype, device=dev)})


# rows that share keys x tiles of the prefix x kv heads decide how the prefix is computed (in 128-row tiles of the widened
# prefix from 300000 on with head_dim 128, 75000 with 64); the cases below stand on both sides, with one and two row tiles
@pytest.mark.parametrize("dim,heads,kv_heads,batch,rows,prefix", [
    (64, 64, 1, 2, 1, 76_000), (64, 64, 1, 2, 9, 9001), (64, 64, 1, 4, 5, 7700), (64, 8, 8, 17, 8, 8913),
    (128, 64, 1, 2, 17, 17_700), (128, 64, 2, 33, 1, 18_200), (128, 8, 8, 32, 9, 16_777), (128, 5, 5, 60, 10, 13_000)])
def test_long_prefix_for_many_rows(dev, dim, heads, kv_heads, batch, rows, prefix):
    c = Case(dev, [rows + 3] * batch, [rows] * batch, heads=heads, kv_heads=kv_heads, dim=dim, page=256, prefix=prefix, size=0.7)
    flat, tiles = batch * rows * heads // kv_heads, -(-prefix // 128)
    assert flat >= 128 and flat * tiles * kv_heads >= (75_000 if dim == 64 else 300_000)
    out = c.call()
    assert int(out["device_status"][0]) == 0
    # the first, a middle and the last rows of some heads (the whole restatement would take minutes)
    pick = sorted({0, 1, batch * rows // 2, 127 % (batch * rows), 128 % (batch * rows), batch * rows - 1})
    o, lse, spread, dx = sampled(c, pick)
    bo, bl = U.bounds(o, spread, dx, c.dtype, prefix + rows + 3)
    got = out["o"].double().cpu().numpy()[pick]
    assert (np.abs(got - o) <= bo).all(), (np.abs(got - o) / bo).max()
    d = np.abs(out["lse"].double().cpu().numpy()[pick] - lse)
    assert (d <= bl + 2.0 ** -23 * np.abs(lse)).all()


def sampled(c, pick):
    """U.attention for some rows of a case of equally long rounds."""
    T, keep = c.rows[0], (c.lens, c.rows, c.table, c.q)
    parts = []
    for r in pick:
        b, i = divmod(r, T)
        # row i of the round alone: what it sees are the first lens - T + i + 1 tokens
        parts.append(U.attention(keep[3][r:r + 1].double().numpy(), c.cache(), keep[2][b:b + 1], [keep[0][b] - T + i + 1], [1],
                                 prefix_table=c.prefix_table, prefix_len=c.prefix))
    return [np.concatenate(x, axis=1 if k == 3 else 0) for k, x in enumerate(zip(*parts))]


def test_long_prefix_with_bad_rows_pages_and_values_of_every_size(dev):
    """The widened prefix: a NaN query row, queries off the 16-byte grid, tokens of zero value, exponents that differ much
    within a tile, a NaN token, a page outside the cache."""
    c = Case(dev, [4] * 32, [4] * 32, heads=16, kv_heads=1, dim=64, page=128, prefix=128 * 40 + 5, size=0.7)
    rng = np.random.default_rng(3)
    c.exps[1][c.prefix_table[3]] = rng.integers(127 - 20, 127, c.exps[1][c.prefix_table[3]].shape)
    c.exps[1][c.prefix_table[4], 0, ::2] = 127 + U.ZERO_EXP
    c.codes[1][c.prefix_table[4], 0, ::2] = 0
    c.q[5, 3, 7] = math.nan
    wide = torch.empty(32 * 4 * 16 * 65 + 1, dtype=c.dtype, device=dev)[1:].view(32 * 4, 16, 65)[:, :, :64]
    wide.copy_(c.q)
    out = c.call(q=wide)
    pick = [0, 5, 6, 127]
    ref = sampled(c, pick)
    bo, _ = U.bounds(np.nan_to_num(ref[0]), ref[2], ref[3], c.dtype, c.prefix)
    got = out["o"].double().cpu().numpy()
    assert np.array_equal(np.isnan(got[pick]), np.isnan(ref[0])) and np.isnan(got[5, 3]).all() and np.isnan(got).sum() == 64
    ok = ~np.isnan(ref[0])
    assert (np.abs(got[pick] - ref[0])[ok] <= bo[ok]).all()
    keep = c.prefix_table.copy()
    c.prefix_table[7] = -1
    out = c.call()
    assert int(out["device_status"][0]) == _lib.SPEC_DEV_PAGE and torch.isnan(out["o"]).all()
    c.prefix_table[7] = keep[7]
    c.cache().k_exp[int(c.prefix_table[9]), 0, 11] = 255
    assert torch.isnan(c.call()["o"]).all()
