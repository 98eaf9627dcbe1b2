"""spec_attention where single places decide: NaN codes beside what rows see, over several masked tiles."""
import pytest
import torch

from test_gpu_attention import Case, dev  # noqa: F401 (dev: the fixture)

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
