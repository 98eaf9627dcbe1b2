"""spec_attention where single places decide: NaN codes beside what rows see, over several masked tiles; many tokens of
the smallest and largest values."""
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
