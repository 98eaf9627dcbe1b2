"""spec_attention_chunk where single places decide: infinite queries that meet keys of one sign, in rows that see one token
and in rows that see thousands."""
import numpy as np
import pytest
import torch

from speculative_decoding_token_temp_gb300 import api

import kv_util as U
from test_gpu_attention import dev  # noqa: F401 (dev: the fixture)
from test_gpu_chunk import Case, visible

pytestmark = pytest.mark.gpu

PLUS, MINUS = 56, 184  # the codes of 1 and -1


def off_the_grid(q, dev):  # noqa: F811
    """The queries as a view that starts one element into its buffer, rows off the 16-byte grid."""
    rows, heads, dim = q.shape
    buf = torch.zeros(rows, heads * dim + 3, dtype=q.dtype, device=dev)
    view = buf[:, 1:1 + heads * dim].unflatten(1, (heads, dim))
    view.copy_(q)
    return view


def check_nan_rows(c, layout, bad):
    """The rows and heads `bad`, and no others, are NaN, log-sums among them; the others are the restatement's."""
    out = c.call(q=c.q.to(c.dev) if layout == "packed" else off_the_grid(c.q, c.dev))
    assert int(out["device_status"][0]) == 0
    got = torch.isnan(out["o"]).any(-1)
    want = torch.zeros_like(got)
    for r, h in bad:
        want[r, h] = True
        c.q[r, h] = 0  # (an infinity has no bound; what such a row gives is asked for above)
    assert torch.equal(got, want) and torch.equal(torch.isnan(out["o"]).all(-1), want) and torch.equal(torch.isnan(out["lse"]), want)
    o, lse, spread, dx = c.ref()
    keep = ~want.cpu().numpy()
    U.compare(out["o"][torch.from_numpy(keep)], out["lse"][torch.from_numpy(keep)], (o[keep], lse[keep], spread[keep], dx[:, keep]), c.dtype,
              max(c.lens) + c.prefix)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("layout", ["packed", "odd"])
@pytest.mark.parametrize("code", [PLUS, MINUS])
@pytest.mark.parametrize("dim,prefix,lens", [(64, 0, [290, 290]), (128, 0, [290, 100]), (128, 1, [290, 290]), (64, 130, [290, 0]),
                                             (128, 0, [9000, 290]), (64, 257, [6000, 290])])
def test_infinite_queries_that_meet_keys_of_one_sign(dev, dtype, layout, code, dim, prefix, lens):  # noqa: F811
    """Every key has the same number in the place that the infinity meets, so that all scores of the row are one infinity:
    +inf or -inf, in the first rows, in later ones, in several heads, and in whole segments and in cut ones (the long
    contexts). Rows that see nothing are zeros whatever they hold."""
    rows = 290
    c = Case(dev, lens, [rows] * 2, heads=4, kv_heads=2, dim=dim, page=64, dtype=dtype, prefix=prefix, seed=11)
    c.codes[0][..., 9] = code
    bad = []
    for b, n in enumerate(lens):
        first = 0 if prefix else max(0, rows - n)  # the first row that sees a token
        for i, (r, h) in enumerate([(first, 0), (first, 3), (first + 1, 1), (first + 2, 2), (first + 2, 3), (rows - 1, 0), (rows - 1, 2)]):
            if r < rows:
                c.q[b * rows + r, h, 9] = np.inf if i % 2 else -np.inf
                bad.append((b * rows + r, h))
        if first:
            c.q[b * rows, 1, 9] = c.q[b * rows + first - 1, 2, 9] = -np.inf  # they see nothing
    for b, n in enumerate(lens):
        if not prefix and n < rows:
            zero = c.call()["o"][b * rows:b * rows + rows - n]
            assert (zero == 0).all()
            c.q[b * rows, 1, 9] = c.q[b * rows + rows - n - 1, 2, 9] = 0
    check_nan_rows(c, layout, bad)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("tokens", [2997, 6997])
def test_one_long_sequence_among_many_short_ones(dev, dtype, tokens):  # noqa: F811
    """More than 64 segments a block, nearly all of two tiles and some of tens (as many as to
    leave the segments whole, and so many that they are cut): the same bits every time, and rows of short and
    long sequences as the restatement has them."""
    B, long = 1250, 777
    rows, lens = [1] * B, [1 + i % 5 for i in range(B)]
    rows[long], lens[long] = 256, tokens
    c = Case(dev, lens, rows, heads=8, kv_heads=8, dim=64, page=256, dtype=dtype, prefix=3, seed=12)
    a, b = c.call(), c.call()
    assert int(a["device_status"][0]) == 0 and torch.equal(a["o"], b["o"]) and torch.equal(a["lse"], b["lse"])
    starts = np.concatenate([[0], np.cumsum(rows)])
    saved, U.visible = U.visible, visible
    try:
        for i in (0, 3, long - 1, long, long + 1, B - 1):
            at = np.arange(starts[i], starts[i] + rows[i])
            ref = U.attention(c.q[at].double().numpy(), c.cache(), [c.table[i]], [lens[i]], [rows[i]], prefix_table=c.prefix_table, prefix_len=3)
            U.compare(a["o"][at], a["lse"][at], ref, c.dtype, lens[i] + 3)
    finally:
        U.visible = saved


def test_the_longest_chunk(dev):  # noqa: F811
    """2^20 rows from the beginning: rows at both ends and between, each against the definition over its own tokens (bounds of
    kv_util for the tokens that it sees)."""
    n, page, heads, dim = 1 << 20, 256, 2, 64
    gen = torch.Generator(device=dev).manual_seed(3)
    k, v = ((torch.randn(n // page, 1, page, dim, generator=gen, device=dev) * 100).clamp(-448, 448).to(torch.float8_e4m3fn) for _ in range(2))
    ke, ve = (torch.randint(118, 122, (n // page, 1, page), generator=gen, device=dev, dtype=torch.uint8) for _ in range(2))
    order = torch.randperm(n // page, generator=gen, device=dev)
    q = torch.randn(n, heads, dim, generator=gen, device=dev).bfloat16()
    out = api.spec_attention_chunk(q, api.KVCache(k, v, ke, ve), order.to(torch.int32).view(1, -1), torch.tensor([n], dtype=torch.int32, device=dev),
                                   gamma=n - 1, want_lse=True)
    assert int(out["device_status"][0]) == 0
    keys, values = (x[order].double().view(n, dim) * torch.exp2(e[order].double().view(n, 1) - 127) for x, e in ((k, ke), (v, ve)))
    for r in (0, 1, 127, 128, 300, 65_537, 524_287, 1_000_003, n - 2, n - 1):
        s = q[r].double() @ keys[:r + 1].T * dim ** -0.5
        w = torch.softmax(s, -1)
        size = keys[:r + 1].abs()
        dx = [(q[r].double().abs() @ size.T).amax(-1) * dim ** -0.5, q[r].double().abs().amax(-1) * size.sum(-1).max() * dim ** -0.5]
        ref = [x.cpu().numpy() for x in (w @ values[:r + 1], torch.logsumexp(s, -1), w @ values[:r + 1].abs(), torch.stack(dx))]
        U.compare(out["o"][r], out["lse"][r], ref, torch.bfloat16, r + 1)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("depth", [4.0, 12.0, 25.0])
def test_a_value_of_zeros_that_takes_nearly_all_weight(dev, dim, dtype, depth):  # noqa: F811
    """The first token's value is zeros and its weight about e^depth times that of each of the others, which are what is left of the
    output and keep their places: zeros are stored under 2^-60, and a weight counts with its token's power of two. Other zeros,
    of both signs, stand among the tokens, and a whole tile is of them."""
    c = Case(dev, [300, 420], [300, 270], heads=8, kv_heads=2, dim=dim, page=32, seed=13, dtype=dtype)
    c.q.mul_(0.2)
    c.q[..., 0] = depth * dim ** 0.5 / 4
    codes, exps = c.codes, c.exps
    for b, n in enumerate(c.lens):
        for t in range(n):
            page, slot = c.table[b][t // 32], t % 32
            codes[0][page, :, slot, 0] = 0
            if t == 0 or t % 29 == 7 or 128 <= t < 256 and b == 1:
                codes[1][page, :, slot], exps[1][page, :, slot] = (0x80 if t % 2 else 0), 127 + U.ZERO_EXP
    for b in (0, 1):
        page = c.table[b][0]
        codes[0][page, :, 0], exps[0][page, :, 0] = 0, 127
        codes[0][page, :, 0, 0] = 0x48  # 4
    c.check()


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("apart", [11, 15, 20, 30])
def test_light_tokens_of_larger_values_with_fp32_queries(dev, dim, apart):  # noqa: F811
    """One token of small values has nearly all weight; every fourth of the others has a weight of 2^-27 to 2^-25 of it and values
    2^apart times as large, and is all that half of the output's elements hold: these keep fp32's places too."""
    c = Case(dev, [420], [300], heads=8, kv_heads=2, dim=dim, page=32, seed=14, dtype="f32")
    codes, exps = c.codes, c.exps
    c.q.zero_()
    c.q[..., 0], c.q[..., 1] = 1.0, 1.3
    rng = np.random.default_rng(15)
    for t in range(420):
        page, slot = c.table[0][t // 32], t % 32
        codes[0][page, :, slot], exps[0][page, :, slot] = 0, 127
        light = t % 4 == 1
        codes[0][page, :, slot, 0] = 0 if light else 0xe0  # -32: far below
        codes[0][page, :, slot, 1] = 0x20 + t % 23 if light else 0  # 0.125 to 0.9: no power of two
        codes[1][page, :, slot] = 0x30 + rng.integers(0, 64, (2, dim))
        exps[1][page, :, slot] = 120 + (apart if light else 0)
        if t == 0:
            codes[0][page, :, slot, 0] = 0x5b  # 22
            codes[1][page, :, slot, :dim // 2] = 0
        elif not light:
            codes[1][page, :, slot, :dim // 2] = 0
    c.check(scale=27 * np.log(2) / 22)
