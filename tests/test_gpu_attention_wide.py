"""The prefix that many rows share, where it is widened and computed in 128-row tiles: the bounds-checked build, equal bits
every time and on two streams, captured calls, ragged rounds, trees, sequences of bad length; and the same shapes just below
the work from which it is widened. Against the 64-bit restatement, with the bounds of kv_util."""
import numpy as np
import pytest
import torch

from speculative_decoding_token_temp_gb300 import _lib, api, synth

import kv_util as U
from test_gpu_attention import Case, dev, i32  # noqa: F401 (dev: the fixture)
from test_gpu_attention_blocks import checked_build

pytestmark = pytest.mark.gpu

# rows that share keys x tiles of the prefix x kv heads from which the prefix is widened, by head_dim
WIDE = {64: 75_000, 128: 300_000}


def work(c, heads, kv_heads):
    return sum(c.rows) * (heads // kv_heads) * -(-c.prefix // 128) * kv_heads


def case(dev, dim, rows, heads=16, kv_heads=1, prefix=None, lens=None, **kw):
    """A case just over the threshold, unless a prefix is given."""
    if prefix is None:
        tiles = -(-WIDE[dim] // (sum(rows) * heads))
        prefix = tiles * 128 - 59
    c = Case(dev, [r + 3 for r in rows] if lens is None else lens, rows, heads=heads, kv_heads=kv_heads, dim=dim, prefix=prefix, size=0.7, **kw)
    return c


def sampled(c, pick):
    """The restatement for some sequences (pick) of a case: (o, lse, spread, dx) and the rows they are."""
    first = np.concatenate([[0], np.cumsum(c.rows)])
    at = np.concatenate([np.arange(first[b], first[b + 1]) for b in pick])
    ref = U.attention(c.q[at].double().numpy(), c.cache(), [c.table[b] for b in pick], [c.lens[b] for b in pick],
                      [c.rows[b] for b in pick], parent=c.parent, prefix_table=c.prefix_table, prefix_len=c.prefix)
    return ref, at


def check(c, out, pick, status=0):
    assert int(out["device_status"][0]) == status
    ref, at = sampled(c, pick)
    U.compare(out["o"][at], out["lse"][at], ref, c.dtype, max(c.lens) + c.prefix)


@pytest.mark.parametrize("dim,n", [(64, 40), (128, 60)])
def test_bounds_checked_build(dev, dim, n):
    """No access outside its buffer, the same outputs as the ordinary build's."""
    c = case(dev, dim, [5] * n)
    assert work(c, 16, 1) >= WIDE[dim]
    a = c.call()
    with checked_build():
        b = c.call()
    assert int(a["device_status"][0]) == 0 and int(b["device_status"][0]) == 0
    assert torch.equal(a["o"], b["o"]) and torch.equal(a["lse"], b["lse"])
    check(c, b, [0, n // 2, n - 1])


@pytest.mark.parametrize("dim,n", [(64, 40), (128, 60)])
def test_same_bits_every_time_and_on_two_streams(dev, dim, n):
    a, b = case(dev, dim, [5] * n), case(dev, 64, [3] * 60, seed=3)
    want = [{k: v.clone() for k, v in x.call().items()} for x in (a, b)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(dev) for _ in range(2)]
    outs = [[], []]
    for _ in range(6):
        for i, (x, s) in enumerate(zip((a, b), streams)):
            with torch.cuda.stream(s):
                outs[i].append(x.call())
    torch.cuda.synchronize()
    for w, o in zip(want, outs):
        for y in o:
            assert torch.equal(w["o"], y["o"]) and torch.equal(w["lse"], y["lse"])


@pytest.mark.parametrize("own_workspace", [False, True])
def test_captured(dev, own_workspace):
    """A captured call replayed between others of the same and of another shape; queries and lengths change between replays."""
    c, other = case(dev, 64, [4] * 50), case(dev, 64, [2] * 70, seed=5)
    q, table, lens = c.q.to(dev), i32(c.table, dev), i32(c.lens, dev)
    args = dict(gamma=3, want_lse=True, prefix_table=i32(c.prefix_table, dev), prefix_len=c.prefix)
    ws = None
    if own_workspace:
        need = api.spec_attention_workspace_bytes(q, c.cache(), table, lens, **{k: v for k, v in args.items() if k != "want_lse"})
        ws = torch.empty(need, dtype=torch.uint8, device=dev)
    out = {}

    def step():
        api.spec_attention(q, c.cache(), table, lens, out=out, workspace=ws, **args)

    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    rng = np.random.default_rng(2)
    for i in range(3):
        c.q = torch.from_numpy(rng.standard_normal(tuple(c.q.shape)) * 0.7).to(c.dtype)
        c.lens = [int(n) for n in rng.integers(0, 8, len(c.lens))]
        q.copy_(c.q)
        lens.copy_(i32(c.lens, dev))
        out["o"].zero_()
        g.replay()
        again = other.call()
        torch.cuda.synchronize()
        check(c, out, [0, 17, 49])
        check(other, again, [i, 69])


@pytest.mark.parametrize("dim,n", [(64, 60), (128, 90)])
def test_ragged_rounds(dev, dim, n):
    rows = [1 + (7 * i) % 9 for i in range(n)]
    lens = [(13 * i) % 150 for i in range(n)]
    c = case(dev, dim, rows, lens=lens, kv_heads=1)
    assert work(c, 16, 1) >= WIDE[dim]
    check(c, c.call(), [0, 1, 8, n // 2, n - 1])


def test_trees(dev):
    parent = [int(x) for x in synth.TREE_PARENT]
    c = case(dev, 64, [len(parent) + 1] * 20, lens=[len(parent) + 1 + (31 * i) % 140 for i in range(20)], parent=parent)
    assert work(c, 16, 1) >= WIDE[64]
    check(c, c.call(), [0, 7, 19])


def test_a_bad_length_and_a_bad_page_of_one_sequence(dev):
    c = case(dev, 64, [4] * 50, lens=[70] * 50)
    good = c.call()
    lens, c.lens = c.lens, [70] * 20 + [-3] + [70] * 29
    out = c.call()
    c.lens = lens
    assert int(out["device_status"][0]) == _lib.SPEC_DEV_OFFSETS
    bad = np.arange(80, 84)
    rest = np.setdiff1d(np.arange(200), bad)
    assert torch.isnan(out["o"][bad]).all() and torch.isnan(out["lse"][bad]).all()
    assert torch.equal(out["o"][rest], good["o"][rest]) and torch.equal(out["lse"][rest], good["lse"][rest])
    table = c.table.copy()
    c.table[20, 1] = -1
    out = c.call()
    c.table = table
    assert int(out["device_status"][0]) == _lib.SPEC_DEV_PAGE
    assert torch.isnan(out["o"][bad]).all() and torch.equal(out["o"][rest], good["o"][rest])
    out = api.spec_attention(c.q.to(dev), c.cache(), i32(c.table, dev), i32(c.lens, dev), gamma=3, cu_draft=i32([0] * 50 + [150], dev),
                             prefix_table=i32(c.prefix_table, dev), prefix_len=c.prefix)
    assert int(out["device_status"][0]) == _lib.SPEC_DEV_OFFSETS and torch.isnan(out["o"]).all()


@pytest.mark.parametrize("dim,heads,kv_heads,rows", [(64, 16, 1, [5] * 40), (64, 16, 4, [3] * 50), (128, 16, 1, [5] * 60), (128, 8, 8, [9] * 30)])
def test_both_sides_of_the_threshold(dev, dim, heads, kv_heads, rows):
    """A prefix one tile too short for the widened path and one just long enough."""
    tiles = -(-WIDE[dim] // (sum(rows) * heads))
    for t in (tiles - 1, tiles):
        c = case(dev, dim, rows, heads=heads, kv_heads=kv_heads, prefix=t * 128 - 5, page=256)
        assert (work(c, heads, kv_heads) >= WIDE[dim]) == (t == tiles)
        check(c, c.call(), [0, len(rows) // 2, len(rows) - 1])
