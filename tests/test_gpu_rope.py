"""spec_qk_rope and spec_qk_rope_append against the formulas in 64 bits.

Bounds. fp32 throughout (u = 2^-24): a head's sum of squares is off by at most (D + 2) u of itself, so the norm's factor by
(D / 2 + 4) u and a normed element by (D / 2 + 6) u. The angle is right to 2^-32 of a turn and then rounded to fp32 half turns
(at most 1: pi 2^-25), sines and cosines add 2 places: each is off by at most pi 2^-25 + 2 pi 2^-32 + 2^-23 < 2^-22. A rotated
element a cos - b sin is then off by (|a| + |b|) (2^-22 + (D / 2 + 8) u), and half a step of the output's type."""
import math

import numpy as np
import pytest
import torch

from speculative_decoding_token_temp_gb300 import _lib, api

import kv_util as U
from test_gpu_attention import dev, i32  # noqa: F401 (dev: the fixture)
from test_gpu_attention_blocks import checked_build

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def formula(x, w, eps, positions, inv_freq, axis, interleaved):
    """(y, the sum of the sizes that y's error is relative to), x [rows, heads, D] in float64."""
    x = np.asarray(x, dtype=np.float64)
    if eps is not None:
        x = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * (1.0 if w is None else np.asarray(w, dtype=np.float64))
    half = len(inv_freq)
    angle = np.asarray(positions, dtype=np.float64).reshape(x.shape[0], -1)[:, axis] * np.asarray(inv_freq)
    c, s = np.cos(angle)[:, None], np.sin(angle)[:, None]
    i = np.arange(half)
    ia, ib = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
    y, size = x.copy(), np.abs(x)
    if half:
        y[..., ia] = x[..., ia] * c - x[..., ib] * s
        y[..., ib] = x[..., ib] * c + x[..., ia] * s
        size[..., ia] = size[..., ib] = np.abs(x[..., ia]) + np.abs(x[..., ib])
    return y, size


def close(got, want, size, dtype, D):
    got = got.double().cpu().numpy()
    assert np.array_equal(np.isnan(got), np.isnan(want))
    lim = size * (2.0 ** -22 + (D / 2 + 8) * 2.0 ** -24) * 1.01 + np.abs(want) * torch.finfo(dtype).eps / 2 * 1.01 + 1e-30
    off = np.abs(got - want)
    ok = ~np.isnan(want)
    assert (off[ok] <= lim[ok]).all(), f"{(off[ok] / lim[ok]).max():.3g} of the bound"


def inputs(dev, rows, heads, kv_heads, dim, dtype, layout, seed=0):
    """Queries, keys, values as tensors of the device in a layout, with sizes from very small to large."""
    rng = np.random.default_rng([seed, rows, heads, dim])
    n = heads + 2 * kv_heads
    x = torch.from_numpy(rng.standard_normal((rows, n, dim)) * 2.0 ** rng.integers(-6, 7, (rows, n, 1))).to(DT[dtype])
    if layout == "fused":
        buf = x.reshape(rows, n * dim).to(dev)
        return [t.unflatten(1, (-1, dim)) for t in buf.split([heads * dim, kv_heads * dim, kv_heads * dim], dim=1)]
    parts = x.split([heads, kv_heads, kv_heads], dim=1)
    if layout == "packed":
        return [p.contiguous().to(dev) for p in parts]
    out = []  # off the 16-byte grid, heads before rows
    for p in parts:
        h = p.shape[1]
        buf = torch.zeros(rows * h * (dim + 3) + 1, dtype=x.dtype, device=dev)
        v = buf[1:].view(h, rows, dim + 3)[:, :, :dim].transpose(0, 1)
        v.copy_(p)
        out.append(v)
    return out


def plan(dev, dim, rot, axes, interleaved):
    axis = [j * axes // (rot // 2) for j in range(rot // 2)]
    r = api.Rope(dim, dev, rot_dim=rot, axis=axis, interleaved=interleaved)
    return r, [10000.0 ** (-2.0 * j / rot) for j in range(rot // 2)], axis


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("layout", ["packed", "fused", "odd"])
@pytest.mark.parametrize("rows,heads,kv_heads,dim,rot,axes,interleaved,normed", [
    (1, 1, 1, 128, 128, 1, False, True), (5, 32, 8, 128, 128, 1, False, True), (300, 7, 1, 64, 64, 1, True, True),
    (33, 12, 4, 64, 32, 3, False, False), (67, 5, 5, 128, 48, 2, False, True), (9, 3, 1, 128, 96, 4, True, False),
    (17, 8, 2, 64, 16, 1, False, True), (4, 6, 2, 128, 0, 1, False, True), (2, 40, 40, 64, 48, 1, True, True),
    (301, 5, 3, 128, 128, 1, False, True), (700, 2, 3, 128, 64, 1, True, True), (5003, 3, 1, 128, 128, 1, False, True), (4099, 5, 2, 64, 64, 2, True, True)])
def test_norm_and_rotation(dev, dtype, layout, rows, heads, kv_heads, dim, rot, axes, interleaved, normed):  # noqa: F811
    q, k, _ = inputs(dev, rows, heads, kv_heads, dim, dtype, layout)
    rng = np.random.default_rng(rows)
    if rot:
        r, freq, axis = plan(dev, dim, rot, axes, interleaved)
    else:
        r, freq, axis = api.Rope(dim, dev, rot_dim=0), [], []
    pos = rng.integers(-50, 3001, (rows, r.axes))
    pos[0] = 2 ** 31 - 1
    if rows > 2:
        pos[1], pos[2] = -2 ** 31, 1_000_003
    w = [(torch.from_numpy(1 + 0.3 * rng.standard_normal(dim))).to(DT[dtype]) for _ in range(2)] if normed else [None, None]
    if normed and rows == 4:
        w[1] = None  # a norm without a weight
    eps = 1e-5 if normed else None
    wd = [None if x is None else x.to(dev) for x in w]
    got = api.spec_qk_rope(q, k, r, i32(pos if r.axes > 1 else pos[:, 0], dev), q_weight=wd[0], k_weight=wd[1], eps=eps)
    for name, x, weight in (("q", q, w[0]), ("k", k, w[1])):
        y, size = formula(x.double().cpu().numpy(), None if weight is None else weight.double().numpy(), eps, pos, freq, axis, interleaved)
        assert got[name].is_contiguous() and got[name].dtype == DT[dtype] and got[name].shape == x.shape
        close(got[name], y, size, DT[dtype], dim)


def fresh(pages, heads, page, dim, dev):  # noqa: F811
    c = api.KVCache.empty(pages, heads, page, dim, dev)
    for t in (c.k, c.v, c.k_exp, c.v_exp):
        t.view(torch.uint8).fill_(0x5a)
    return c


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("layout", ["fused", "odd"])
@pytest.mark.parametrize("rows,heads,kv_heads,dim,page,rot", [(1, 8, 2, 128, 64, 128), (37, 6, 3, 64, 16, 32), (520, 4, 1, 128, 256, 64),
                                                              (130, 32, 8, 128, 32, 128), (4500, 3, 2, 64, 64, 64), (5000, 4, 1, 128, 16, 128)])
def test_append_is_the_rotation_and_then_the_append(dev, dtype, layout, rows, heads, kv_heads, dim, page, rot):  # noqa: F811
    """The cache holds, bit for bit, what spec_kv_append makes of the fp32 keys and of the values; other places are left."""
    q, k, v = inputs(dev, rows, heads, kv_heads, dim, dtype, layout, seed=1)
    rng = np.random.default_rng(rows)
    seqs = 3
    seq = rng.integers(0, seqs, rows)
    at, place = rng.integers(0, 30, seqs), np.zeros(rows, dtype=np.int64)
    for n in range(rows):
        place[n] = at[seq[n]]
        at[seq[n]] += 1
    table, pages = U.pages_for(at, page, rng)
    place[rng.random(rows) < 0.2] = -1
    r, freq, axis = plan(dev, dim, rot, 1, False)
    pos = i32(rng.integers(0, 5000, rows), dev)
    w = [torch.from_numpy(1 + 0.3 * rng.standard_normal(dim)).to(DT[dtype]).to(dev) for _ in range(2)]
    tb, rs, rp = i32(table, dev), i32(seq, dev), i32(place, dev)
    a, b = fresh(pages, kv_heads, page, dim, dev), fresh(pages, kv_heads, page, dim, dev)
    got = api.spec_qk_rope_append(a, q, k, v, r, pos, tb, rs, rp, q_weight=w[0], k_weight=w[1], eps=1e-6)
    assert int(got["device_status"][0]) == 0
    apart = api.spec_qk_rope(q, k, r, pos, q_weight=w[0], k_weight=w[1], eps=1e-6)
    wide = api.spec_qk_rope(q.float(), k.float(), r, pos, q_weight=w[0].float(), k_weight=w[1].float(), eps=1e-6)
    assert torch.equal(got["q"], apart["q"]) and torch.equal(got["q"], wide["q"].to(DT[dtype]))
    api.spec_kv_append(b, wide["k"], v.float(), tb, rs, rp)
    for x, y in ((a.k, b.k), (a.v, b.v), (a.k_exp, b.k_exp), (a.v_exp, b.v_exp)):
        assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))


def test_places_that_are_none_and_numbers_that_are_none(dev):  # noqa: F811
    q, k, v = inputs(dev, 6, 4, 2, 64, "bf16", "packed")
    k[1, 0, 3], v[2, 1, 5], q[3, 2, 0] = math.nan, math.inf, math.nan
    r, freq, axis = plan(dev, 64, 64, 1, False)
    c = fresh(4, 2, 16, 64, dev)
    before = [t.view(torch.uint8).clone() for t in (c.k, c.v, c.k_exp, c.v_exp)]
    table = i32([[1, 9], [0, 2]], dev)
    pos = i32(np.arange(6), dev)
    got = api.spec_qk_rope_append(c, q, k, v, r, pos, table, i32([0, 0, 1, 1, 2, 0], dev), i32([0, 1, 2, 40, 0, 17], dev), eps=1e-6)
    want = _lib.SPEC_DEV_NONFINITE | _lib.SPEC_DEV_OFFSETS | _lib.SPEC_DEV_PAGE
    assert int(got["device_status"][0]) == want
    assert torch.isnan(got["q"][3, 2]).all() and int(torch.isnan(got["q"]).any(-1).sum()) == 1
    assert int(c.k_exp[1, 0, 1]) == 255 and int(c.k_exp[1, 1, 1]) != 255 and int(c.v_exp[0, 1, 2]) == 255
    written = torch.zeros(4, 2, 16, dtype=torch.bool, device=dev)
    written[1, :, 0] = written[1, :, 1] = written[0, :, 2] = True
    for t, b in zip((c.k, c.v, c.k_exp, c.v_exp), before):
        same = (t.view(torch.uint8) == b).view(4, 2, 16, -1).all(-1)
        assert bool(same[~written].all()) and not bool(same[written].all())


def test_axes_past_the_last_and_no_rows(dev):  # noqa: F811
    q, k, _ = inputs(dev, 3, 2, 1, 64, "f32", "packed")
    r, freq, axis = plan(dev, 64, 32, 2, False)
    pos = np.array([[5, 7], [1, 0], [9, 2]])
    a = api.spec_qk_rope(q, k, r, i32(pos, dev))["q"]
    r.axis.fill_(200)  # read as the last axis
    b = api.spec_qk_rope(q, k, r, i32(pos, dev))["q"]
    y, size = formula(q.double().cpu().numpy(), None, None, pos, freq, [1] * 16, False)
    close(b, y, size, torch.float32, 64)
    assert not torch.equal(a, b)
    none = api.spec_qk_rope(q[:0], k[:0], r, i32(pos[:0], dev))
    assert none["q"].shape == (0, 2, 64)


@pytest.mark.parametrize("dim,rows,layout", [(64, 21, "odd"), (128, 130, "fused"), (128, 4997, "fused")])
def test_bounds_checked_build_streams_and_graphs(dev, dim, rows, layout):  # noqa: F811
    q, k, v = inputs(dev, rows, 8, 2, dim, "bf16", layout)
    r, freq, axis = plan(dev, dim, dim, 1, False)
    rng = np.random.default_rng(3)
    table, pages = U.pages_for([rows], 16, rng)
    args = (q, k, v, r, i32(np.arange(rows), dev), i32(table, dev), i32(np.zeros(rows), dev), i32(np.arange(rows), dev))
    caches = [fresh(pages, 2, 16, dim, dev) for _ in range(4)]
    a = api.spec_qk_rope_append(caches[0], *args, eps=1e-6)
    with checked_build():
        b = api.spec_qk_rope_append(caches[1], *args, eps=1e-6)
        assert int(b["device_status"][0]) == 0
    side = torch.cuda.Stream(dev)
    side.wait_stream(torch.cuda.current_stream(dev))
    with torch.cuda.stream(side):
        c = api.spec_qk_rope_append(caches[2], *args, eps=1e-6)
    torch.cuda.current_stream(dev).wait_stream(side)
    graph, out = torch.cuda.CUDAGraph(), {"device_status": torch.zeros(1, dtype=torch.int32, device=dev)}
    with torch.cuda.graph(graph):
        api.spec_qk_rope_append(caches[3], *args, eps=1e-6, out=out)
    for _ in range(3):
        graph.replay()
    for got, cache in ((b, caches[1]), (c, caches[2]), (out, caches[3])):
        assert torch.equal(got["q"], a["q"])
        for x, y in zip((cache.k, cache.v, cache.k_exp, cache.v_exp), (caches[0].k, caches[0].v, caches[0].k_exp, caches[0].v_exp)):
            assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))
