"""spec_attention where single places decide: NaN codes beside what rows see, over several masked tiles; one dominant
token before a long flat tail; many tokens of the smallest and largest values."""
import numpy as np
import pytest
import torch

from speculative_decoding_token_temp_gb300 import api

import kv_util as U
from test_gpu_attention import DT, Case, dev, i32  # noqa: F401 (dev: the fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("rows,lens", [(129, [130, 257, 300, 129]), (9, [130, 132, 128, 129]), (40, [140, 290, 128, 256])])
def test_nan_codes_past_the_end_of_rounds_over_several_tiles(dev, dim, rows, lens):
    """Unwritten places hold NaN codes of values under ordinary exponents, so that nothing but the codes tells them from
    tokens; a drafted token of each sequence has one NaN code and reaches the rows after it only. The same bits every time."""
    c = Case(dev, lens, [rows] * 4, heads=4, kv_heads=2, dim=dim, page=64)
    for e in c.exps:
        e[e == 255] = 127 - 7
    token = [max(n - rows + 2, n - 3) for n in lens]  # the token of a row near the round's end
    for b in range(4):
        c.codes[1][c.table[b, token[b] // 64], 1, token[b] % 64, 5] = 0x7f
    want = c.check()["o"].clone()
    nan = torch.isnan(want).all(-1).view(4, rows, 4).cpu().numpy()
    for b in range(4):
        row = token[b] - (lens[b] - rows)
        assert nan[b, row:, 2:].all() and not nan[b, :row].any() and not nan[b, :, :2].any()
    for _ in range(30):
        got = c.call()["o"]
        assert torch.equal(torch.nan_to_num(got, nan=-1e30), torch.nan_to_num(want, nan=-1e30))


@pytest.mark.parametrize("dtype,dim,way", [("bf16", 128, "own"), ("bf16", 64, "own"), ("f32", 64, "own"), ("bf16", 64, "prefix")])
@pytest.mark.parametrize("tail", [2000, 16300])
@pytest.mark.parametrize("place", ["first", "last"])
def test_flat_tail_under_one_dominant_token(dev, dtype, dim, way, tail, place):
    """One token whose weight is 2^20.9 to 2^24 times that of each of the others, whose values are one in every element; its
    own are one in the first half of the elements, zero in a quarter, 0.01 in the last. Each of 400 sequences reads the same
    pages, so that every stretch that a block works on is long. The bound is the one of all other cases (kv_util.bounds)."""
    n, page, B = tail + 1, 256, 400
    depth = np.array([20.9, 21.0, 21.1, 22.0, 23.0, 24.0])
    pages = -(-n // page)
    at = 0 if place == "first" else n - 1
    k, v = np.zeros((pages * page, dim)), np.ones((pages * page, dim))
    k[at, 0] = 1.0
    v[at, dim // 2:3 * dim // 4] = 0.0
    v[at, 3 * dim // 4:] = 0.01
    (kc, ke), (vc, ve) = U.quantise(k), U.quantise(v)
    cache = api.KVCache(*(torch.from_numpy(c).view(pages, 1, page, dim).to(dev).view(torch.float8_e4m3fn) for c in (kc, vc)),
                        *(torch.from_numpy(e).view(pages, 1, page).to(dev) for e in (ke, ve)))
    q = torch.zeros(B, 6, dim, dtype=DT[dtype])
    q[:, :, 0] = torch.from_numpy(depth).to(DT[dtype])
    table = np.arange(pages, dtype=np.int32).reshape(1, -1)
    scale = float(np.float32(np.log(2.0)))
    ref = U.attention(q[:1].double().numpy(), cache, table, [n], [1], scale=scale)
    ref = [np.repeat(x, B, axis=1 if i == 3 else 0) for i, x in enumerate(ref)]
    if way == "own":
        out = api.spec_attention(q.to(dev), cache, i32(np.repeat(table, B, axis=0), dev), i32([n] * B, dev), gamma=0, scale=scale, want_lse=True)
    else:
        assert B * 6 * -(-n // 128) >= 75_000 or tail < 16_000  # (the longer tail: in 128-row tiles of the widened prefix)
        out = api.spec_attention(q.to(dev), cache, torch.zeros(B, 1, dtype=torch.int32, device=dev), i32([0] * B, dev), gamma=0,
                                 prefix_table=i32(table[0], dev), prefix_len=n, scale=scale, want_lse=True)
    assert int(out["device_status"][0]) == 0
    U.compare(out["o"], out["lse"], ref, DT[dtype], n)


def one_value(dev, n, dim, exponent, code, dtype, rows):
    """A page of equal tokens (keys of zero, values `code` * 2^exponent), queries, the table that names it for n tokens."""
    value = np.flatnonzero(U.VALUES == code)[0]
    codes = [torch.full((1, 1, 256, dim), int(c), dtype=torch.uint8, device=dev).view(torch.float8_e4m3fn) for c in (0, value)]
    exps = [torch.full((1, 1, 256), 127 + e, dtype=torch.uint8, device=dev) for e in (U.ZERO_EXP, exponent)]
    return api.KVCache(*codes, *exps), torch.ones(rows, 1, dim, dtype=DT[dtype], device=dev), np.zeros((1, -(-n // 256)), dtype=np.int32)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("exponent,code", [(-100, 448.0), (120, 128.0)])
def test_many_tokens_of_the_smallest_and_largest_values(dev, dtype, exponent, code):
    """270000 equal tokens: their mean is each one's value (to the type's rounding and 2^-24 a token), lse their number's logarithm."""
    n = 270_000
    cache, q, table = one_value(dev, n, 64, exponent, code, dtype, 1)
    out = api.spec_attention(q, cache, i32(table, dev), i32([n], dev), gamma=0, want_lse=True)
    want = code * 2.0 ** exponent
    rel = n * 2.0 ** -24 + (2.0 ** -8 if dtype == "bf16" else 2.0 ** -24)
    assert ((out["o"].double() / want - 1).abs() <= rel).all()
    assert abs(float(out["lse"][0, 0]) - np.log(n)) <= n * 2.0 ** -24 + 2.0 ** -18


@pytest.mark.parametrize("exponent,code", [(-100, 448.0), (120, 128.0)])
def test_many_shared_tokens_of_the_smallest_and_largest_values(dev, exponent, code):
    """The same of a prefix of 1100000 tokens that 128 rows share (in 128-row tiles of the widened prefix)."""
    n = 1_100_000
    cache, q, table = one_value(dev, n, 64, exponent, code, "bf16", 128)
    out = api.spec_attention(q, cache, torch.zeros(128, 1, dtype=torch.int32, device=dev), i32([0] * 128, dev), gamma=0,
                             prefix_table=i32(table[0], dev), prefix_len=n, want_lse=True)
    assert ((out["o"].double() / (code * 2.0 ** exponent) - 1).abs() <= n * 2.0 ** -24 + 2.0 ** -8).all()
    assert ((out["lse"].double() - np.log(n)).abs() <= n * 2.0 ** -24 + 2.0 ** -18).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("what", [float("inf"), float("-inf")])
@pytest.mark.parametrize("tokens,prefix", [(1, 0), (3, 0), (0, 2), (1, 1)])
@pytest.mark.parametrize("sign", [1, -1])
def test_infinite_queries_make_their_rows_nan(dev, dtype, what, tokens, prefix, sign):
    """Whatever the sign of the keys that the infinite element meets, all of them the same here."""
    c = Case(dev, [tokens], [1], heads=2, kv_heads=1, dim=64, dtype=dtype, prefix=prefix)
    c.codes[0][..., 9] = 56 if sign > 0 else 184  # 1 and -1
    c.q[0, 1, 9] = what
    out = c.call()
    assert torch.isnan(out["o"][0, 1]).all() and torch.isnan(out["lse"][0, 1])
    assert torch.isfinite(out["o"][0, 0].float()).all() and torch.isfinite(out["lse"][0, 0])
    c = Case(dev, [0], [1], heads=2, kv_heads=1, dim=64, dtype=dtype)
    c.q[0, 1, 9] = what
    assert (c.call()["o"] == 0).all()  # (it sees nothing)
