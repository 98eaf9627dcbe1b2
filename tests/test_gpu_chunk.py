"""spec_attention_chunk against the 64-bit restatement, with the bounds of kv_util."""
import numpy as np
import pytest
import torch

from speculative_decoding_token_temp_gb300 import _lib, api

import kv_util as U
import test_gpu_attention as A
from test_gpu_attention import dev, i32  # noqa: F401 (dev: the fixture)
from test_gpu_attention_blocks import checked_build

pytestmark = pytest.mark.gpu


def visible(rows, length, parent=None):
    """kv_util.visible for chains, as arrays."""
    return np.arange(length) <= length - rows + np.arange(rows)[:, None]


class Case(A.Case):
    """The same caches, through spec_attention_chunk."""

    def call(self, q=None, **kw):
        cu = None
        if len(set(self.rows)) > 1:
            cu = i32(np.concatenate([[0], np.cumsum([r - 1 for r in self.rows])]), self.dev)
        kw.setdefault("want_lse", True)
        kw = {**(dict(prefix_table=i32(self.prefix_table, self.dev), prefix_len=self.prefix) if self.prefix else {}), **kw}
        return api.spec_attention_chunk(self.q.to(self.dev) if q is None else q, self.cache(), i32(self.table, self.dev),
                                        i32(self.lens, self.dev), gamma=max(self.rows) - 1, cu_draft=cu, **kw)

    def ref(self, **kw):
        saved, U.visible = U.visible, visible
        try:
            return super().ref(**kw)
        finally:
            U.visible = saved


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dim,page", [(64, 16), (128, 64), (128, 256)])
@pytest.mark.parametrize("rows", [1, 2, 127, 128, 129, 130, 255, 257, 300])
def test_chunks_at_every_edge_length(dev, dtype, dim, page, rows):  # noqa: F811
    """From the beginning, behind a few tokens, behind many; and fewer cached tokens than rows."""
    Case(dev, [rows, rows + 1, rows + 200, max(0, rows - 3), 0], [rows] * 5, dim=dim, page=page, dtype=dtype).check()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dim,heads,kv_heads", [(128, 1, 1), (128, 8, 8), (64, 14, 2), (128, 6, 2), (64, 40, 1), (128, 64, 1), (128, 5, 1)])
def test_head_layouts(dev, dtype, dim, heads, kv_heads):  # noqa: F811
    Case(dev, [140, 333], [140, 140], heads=heads, kv_heads=kv_heads, dim=dim, dtype=dtype).check()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("prefix", [0, 1, 128, 333])
@pytest.mark.parametrize("dim,page", [(64, 32), (128, 16)])
def test_prompts_beside_single_tokens(dev, dtype, dim, page, prefix):  # noqa: F811
    rows = [1, 400, 1, 1, 131, 2, 65, 257]
    lens = [600, 400, 1, 0, 140, 2, 500, 100]
    Case(dev, lens, rows, heads=6, kv_heads=2, dim=dim, page=page, dtype=dtype, prefix=prefix).check()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dim", [64, 128])
def test_a_long_chunk(dev, dim, dtype):  # noqa: F811
    Case(dev, [2200], [1500], heads=8, kv_heads=1, dim=dim, prefix=130, dtype=dtype).check()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_hidden_tokens_do_not_matter_and_seen_nans_do(dev, dtype):  # noqa: F811
    """A token stored as NaN inside the chunk: rows before it are as they were, rows from it on are NaN."""
    for what in ("exponent", "k", "v"):
        c = Case(dev, [350, 300], [300, 300], heads=4, kv_heads=2, dim=64, page=32, dtype=dtype, seed=2)
        page, slot = c.table[0][200 // 32], 200 % 32
        if what == "exponent":
            c.exps[1][page, 1, slot] = 255
        else:
            c.codes["kv".index(what)][page, 1, slot, 7] = 0x7f
        out = c.check()
        hurt = torch.isnan(out["o"]).any(-1)
        assert not hurt[:150].any() and hurt[150:300, 2:].all() and not hurt[150:300, :2].any() and not hurt[300:].any()


def test_bad_lengths_pages_and_offsets(dev):  # noqa: F811
    """Rows that a bad number does not concern are what they should be (not bit for bit: where the work is cut depends on all lengths)."""
    c = Case(dev, [300, 350, 280], [280] * 3, heads=8, kv_heads=2, dim=64)
    ref = c.ref()

    def right(out, rows):
        U.compare(out["o"][rows], out["lse"][rows], [x[rows] for x in ref[:3]] + [ref[3][:, rows]], c.dtype, 350)

    c.lens[1] = 10 ** 6
    out = c.call()
    assert int(out["device_status"][0]) == _lib.SPEC_DEV_OFFSETS
    assert torch.isnan(out["o"][280:560]).all()
    right(out, np.r_[0:280, 560:840])
    c.lens[1] = 350
    c.table[2][1] = 1 << 20  # tokens 64 .. 127
    out = c.call()
    assert int(out["device_status"][0]) == _lib.SPEC_DEV_PAGE
    right(out, np.r_[0:624])
    assert torch.isnan(out["o"][624:]).all()
    ragged = Case(dev, [200, 200], [140, 150], heads=4, kv_heads=2, dim=64)
    cu = i32([0, 200, 288], dev)
    out = api.spec_attention_chunk(ragged.q.to(dev), ragged.cache(), i32(ragged.table, dev), i32(ragged.lens, dev), gamma=149, cu_draft=cu)
    assert int(out["device_status"][0]) & _lib.SPEC_DEV_OFFSETS and torch.isnan(out["o"]).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_views_scales_streams_graphs_and_the_bounds_checked_build(dev, dtype):  # noqa: F811
    c = Case(dev, [500, 260], [260, 260], heads=6, kv_heads=2, dim=128, dtype=dtype, prefix=70)
    a = c.check()
    c.check(scale=0.3)
    wide = torch.zeros(520, 9 * 128 + 3, dtype=c.dtype, device=dev)
    view = wide[:, 1:1 + 6 * 128].unflatten(1, (6, 128))  # off the 16-byte grid
    view.copy_(c.q)
    assert torch.equal(c.call(q=view)["o"], a["o"])
    with checked_build():
        b = c.call()
        assert int(b["device_status"][0]) == 0
    assert torch.equal(b["o"], a["o"]) and torch.equal(b["lse"], a["lse"])
    q, table, lens, pre = c.q.to(dev), i32(c.table, dev), i32(c.lens, dev), i32(c.prefix_table, dev)
    out = [{"device_status": torch.zeros(1, dtype=torch.int32, device=dev)} for _ in range(4)]
    call = lambda o: api.spec_attention_chunk(q, c.cache(), table, lens, gamma=259, prefix_table=pre, prefix_len=70, want_lse=True, out=o)  # noqa: E731
    streams = [torch.cuda.Stream(dev) for _ in range(2)]
    torch.cuda.synchronize(dev)
    for _ in range(3):
        for s, o in zip(streams, out):
            with torch.cuda.stream(s):
                call(o)
    torch.cuda.synchronize(dev)
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    for g, o in zip(graphs, out[2:]):
        with torch.cuda.graph(g):
            call(o)
    for _ in range(2):
        for g in graphs:
            g.replay()
    torch.cuda.synchronize(dev)
    for o in out:
        assert int(o["device_status"][0]) == 0 and torch.equal(o["o"], a["o"]) and torch.equal(o["lse"], a["lse"])


def test_a_short_chunk_is_a_round(dev):  # noqa: F811
    c = Case(dev, [300, 40, 9], [9] * 3, heads=8, kv_heads=2)
    for out in (c.call(), A.Case.call(c)):
        assert int(out["device_status"][0]) == 0
        U.compare(out["o"], out["lse"], c.ref(), c.dtype, 300)


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("spread", [12, 30, 70])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_values_of_very_different_size(dev, dim, spread, dtype):  # noqa: F811
    """Tokens whose values are 2^spread times their neighbours': rows before them do not see them and keep their places."""
    c = Case(dev, [300, 420], [300, 270], heads=8, kv_heads=2, dim=dim, page=32, seed=3, dtype=dtype)
    for b, t in ((0, 100), (0, 255), (1, 333)):
        c.exps[1][c.table[b][t // 32], 1, t % 32] += spread
    c.exps[1][c.table[1][40 // 32], 0, 40 % 32] -= min(spread, 60)
    c.check()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_infinite_queries_and_rows_that_see_nothing(dev, dtype):  # noqa: F811
    c = Case(dev, [290, 200], [290, 270], heads=8, kv_heads=2, dim=64, dtype=dtype)
    c.q[5, 1, 3], c.q[100, 2, 0], c.q[300, 0, 9], c.q[500, 3, 1] = np.inf, np.nan, np.inf, -np.inf  # (row 300 sees nothing)
    out = c.call()
    assert int(out["device_status"][0]) == 0
    c.q[300, 0, 9] = 0  # what it holds does not matter (and an infinity has no bound)
    U.compare(out["o"], out["lse"], c.ref(), c.dtype, 290)
    bad = torch.isnan(out["o"]).any(-1)
    assert bad[5, 1] and bad[100, 2] and bad[500, 3] and int(bad.sum()) == 3


@pytest.mark.parametrize("dim", [64, 128])
def test_fp32_queries_of_every_size(dev, dim):  # noqa: F811
    """Elements from 2^-40 to 2^30 of one another: nothing of a query is lost that its scores' roundings keep."""
    c = Case(dev, [310, 290], [290, 290], heads=6, kv_heads=2, dim=dim, dtype="f32", seed=5)
    c.q *= torch.exp2(torch.from_numpy(c.rng.integers(-40, 4, c.q.shape)).float())
    c.q[7] *= 2.0 ** 30
    c.q[9] = 0
    c.check()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("size", [1e3, 1e6, 1e9, 1e12])
def test_scores_of_every_size(dev, dtype, size):  # noqa: F811
    """Scores of thousands to 10^13: the weights are those of the largest, nothing overflows. (Where the two largest are nearer
    than the roundings of such scores, the bounds ask for nothing; the output then lies between the values.)"""
    c = Case(dev, [290, 700], [290, 290], heads=8, kv_heads=2, dim=128, dtype=dtype, prefix=140, seed=9)
    c.q *= size
    c.q[11] = -c.q[12]
    out = c.check()
    # values are below 2^9 times their exponent's power of two
    assert float(out["o"].abs().max()) <= 2.0 ** (int(c.exps[1][c.exps[1] != 255].max()) - 127 + 9)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("batch,rows,ctx", [(40, 70, 100), (3, 900, 2000), (1100, 65, 0)])
def test_many_and_long_sequences_repeat_bit_for_bit(dev, batch, rows, ctx, dtype):  # noqa: F811
    """More sequences than threads plan at once, cut segments; some sequences against the restatement."""
    lens = [rows + ctx * (i % 3) // 2 for i in range(batch)]
    c = Case(dev, lens, [rows] * batch, heads=4, kv_heads=1, dim=64, page=16, size=0.7, dtype=dtype)
    a, b = c.call(), c.call()
    assert int(a["device_status"][0]) == 0 and torch.equal(a["o"], b["o"]) and torch.equal(a["lse"], b["lse"])
    saved, U.visible = U.visible, visible
    try:
        for i in {0, batch // 2, batch - 1}:
            at = np.arange(i * rows, (i + 1) * rows)
            ref = U.attention(c.q[at].double().numpy(), c.cache(), [c.table[i]], [lens[i]], [rows])
            U.compare(a["o"][at], a["lse"][at], ref, c.dtype, lens[i])
    finally:
        U.visible = saved


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_bounds_checked_build_of_a_ragged_batch(dev, dtype):  # noqa: F811
    rows = [1, 400, 3, 64, 1, 129]
    c = Case(dev, [900, 400, 300, 64, 1, 500], rows, heads=8, kv_heads=2, dim=128, page=64, dtype=dtype)
    a = c.check()
    with checked_build():
        b = c.call()
        assert int(b["device_status"][0]) == 0
    assert torch.equal(a["o"], b["o"]) and torch.equal(a["lse"], b["lse"])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("size", [1.0, 1e7])
def test_segments_cut_into_many_parts(dev, dtype, dim, size):  # noqa: F811
    """Few rows behind many tokens: parts of a row block's tokens in tens of blocks, joined; with a row that is NaN and a token."""
    c = Case(dev, [4500, 80], [70, 70], heads=4, kv_heads=1, dim=dim, page=64, dtype=dtype, prefix=200, seed=4)
    c.q *= size
    c.q[30, 2, 5] = np.nan
    c.exps[0][c.table[0][4460 // 64], 0, 4460 % 64] = 255  # token 4460: rows 30 to 69 of the first sequence see it
    out = c.check()
    bad = torch.isnan(out["o"]).any(-1)
    assert not bad[:30].any() and bad[30:70].all() and not bad[70:].any()
