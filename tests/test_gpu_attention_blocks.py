"""spec_attention at every size of a row block, at many sequences, in the bounds-checked build, and captured with the
binding's own workspace; against the 64-bit restatement, with the bounds of kv_util."""
import contextlib

import numpy as np
import pytest
import torch

from speculative_decoding_token_temp_gb300 import _lib, api

import kv_util as U
from test_gpu_attention import Case, dev, i32  # noqa: F401 (dev: the fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("prefix", [0, 200])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("rows", [1, 7, 8, 9, 12, 13, 15, 16, 17, 20, 23, 24, 25, 28, 31, 32, 33, 36, 39, 40, 41, 44, 47, 48, 49, 65, 73])
def test_every_row_block(dev, rows, dim, prefix):
    """Row blocks of 16 to 48 rows, full and not, several behind one another, one query head a kv head (a row of the block
    is a row of the round)."""
    Case(dev, [rows, rows + 127, 300], [rows] * 3, heads=2, kv_heads=2, dim=dim, prefix=prefix).check()


@pytest.mark.parametrize("group,rows", [(3, 8), (4, 6), (5, 8), (4, 10), (6, 4), (12, 2), (13, 3)])
@pytest.mark.parametrize("dim", [64, 128])
def test_row_blocks_of_grouped_heads(dev, group, rows, dim):
    Case(dev, [500, 1, 129, 0, 1000], [rows] * 5, heads=2 * group, kv_heads=2, dim=dim, page=16).check()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_many_sequences(dev, dtype):
    """More sequences than blocks of the grid, most of one tile, ragged."""
    rng = np.random.default_rng(3)
    B = 1300
    rows = [int(r) for r in rng.integers(1, 4, B)]
    lens = [int(n) for n in rng.integers(0, 40, B)]
    lens[7], lens[640], lens[B - 1] = 700, 129, 300
    Case(dev, lens, rows, heads=2, kv_heads=1, dim=64, page=16, dtype=dtype).check()


@contextlib.contextmanager
def checked_build():
    saved = _lib._LIB
    _lib._LIB = _lib.bounds_lib()
    try:
        yield
    finally:
        _lib._LIB = saved


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dim,page,heads,batch,prefix", [(128, 64, 8, 3, 0), (64, 16, 12, 3, 130), (128, 256, 6, 5, 0), (128, 64, 32, 40, 1300)])
def test_bounds_checked_build(dev, dtype, dim, page, heads, batch, prefix):
    """No access outside its buffer, the same outputs as the ordinary build's."""
    rows = [5 + (i % 3) for i in range(batch)]
    c = Case(dev, [5 + 97 * (i % 7) for i in range(batch)], rows, heads=heads, kv_heads=2, dim=dim, page=page, dtype=dtype, prefix=prefix)
    a = c.call()
    n = sum(rows)
    k = torch.randn(n, 2, dim, device=dev).to(c.dtype)
    rs, rp = i32(np.zeros(n), dev), i32(np.arange(n), dev)
    table = i32(np.arange(-(-n // page)).reshape(1, -1), dev)
    caches = [api.KVCache.empty(-(-n // page), 2, page, dim, dev) for _ in range(2)]
    api.spec_kv_append(caches[0], k, k, table, rs, rp)
    with checked_build():
        b = c.call()
        w = api.spec_kv_append(caches[1], k, k, table, rs, rp)
        r = api.spec_kv_read(caches[1], table, rs, rp, dtype=c.dtype)
    plain = api.spec_kv_read(caches[0], table, rs, rp, dtype=c.dtype)
    for o in (a, b, w, r):
        assert int(o["device_status"][0]) == 0
    for name in ("o", "lse"):
        assert torch.equal(a[name], b[name]), name
    for name in ("k", "v"):
        assert torch.equal(plain[name], r[name]), name


def test_captured_with_the_bindings_own_workspace(dev):
    """Two graphs of calls without a workspace, one of them captured while the other is alive, and a call between replays."""
    a = Case(dev, [300, 20, 1000], [4] * 3, dim=128)
    b = Case(dev, [700, 129], [9] * 2, dim=64, prefix=100, heads=8)
    graphs, outs = [], []
    for c in (a, b):
        q, table, lens = c.q.to(dev), i32(c.table, dev), i32(c.lens, dev)
        pre = dict(prefix_table=i32(c.prefix_table, dev), prefix_len=c.prefix) if c.prefix else {}
        out = {}

        def step(c=c, q=q, table=table, lens=lens, pre=pre, out=out):
            return api.spec_attention(q, c.cache(), table, lens, gamma=c.rows[0] - 1, want_lse=True, out=out, **pre)

        step()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step()
        graphs.append((g, q, table, lens, pre))
        outs.append(out)
    for _ in range(3):
        for (g, *_), out in zip(graphs, outs):
            out["o"].zero_()
            g.replay()
        b.check()
    torch.cuda.synchronize()
    for c, out in zip((a, b), outs):
        assert int(out["device_status"][0]) == 0
        U.compare(out["o"], out["lse"], c.ref(), c.dtype, max(c.lens) + c.prefix)
