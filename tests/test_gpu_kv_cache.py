"""spec_kv_append and spec_kv_read against the 64-bit restatement: codes, exponents and values are exact."""
import numpy as np
import pytest
import torch

from speculative_decoding_token_temp_gb300 import _lib, api

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


def fresh(num_pages, heads, page, dim, dev, fill=0x7f):
    """A cache whose unwritten places hold NaN codes and NaN exponents."""
    c = api.KVCache.empty(num_pages, heads, page, dim, dev)
    for t in (c.k, c.v, c.k_exp, c.v_exp):
        t.view(torch.uint8).fill_(fill if t.dtype != torch.uint8 else 255)
    return c


def i32(a, dev):
    return torch.as_tensor(np.asarray(a, dtype=np.int32)).to(dev)


def special_rows(n, heads, dim, rng):
    """Vectors of all sizes: ordinary, tiny, huge, zeros (of both signs), a maximum at the code's border."""
    x = rng.standard_normal((n, heads, dim)) * 2.0 ** rng.integers(-30, 30, (n, heads, 1))
    x[0, 0] = 0.0
    x[0, 0, 1] = -0.0
    if n > 1:
        x[1, 0, 3] = np.abs(x[1, 0]).max() * 2
        x[1, 0] *= 448.0 / np.abs(x[1, 0]).max()          # the largest element is exactly 448
        x[1, 0, 3] = 448.0
        x[1, -1] *= 2.0 ** -110 / np.abs(x[1, -1]).max()  # below the smallest exponent
    return x


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dim,heads,page,rows", [(64, 1, 16, 1), (64, 3, 16, 37), (128, 2, 64, 130), (128, 8, 256, 9), (128, 1, 128, 300)])
@pytest.mark.parametrize("layout", ["packed", "fused", "odd"])
def test_append_writes_the_codes_and_read_gives_them_back(dev, dtype, dim, heads, page, rows, layout):
    rng = np.random.default_rng([dim, heads, page, rows])
    seqs = 3
    seq = rng.integers(0, seqs, rows)
    pos = np.zeros(rows, dtype=np.int64)
    start = rng.integers(0, 40, seqs)
    for n in range(rows):
        pos[n] = start[seq[n]]
        start[seq[n]] += 1
    table, pages = U.pages_for(start, page, rng)
    skip = rng.random(rows) < 0.2
    skip[0] = False
    x = [torch.from_numpy(special_rows(rows, heads, dim, rng)).to(DT[dtype]) for _ in range(2)]
    if layout == "fused":   # keys and values cut out of one projection
        wide = torch.zeros(rows, (2 + 2 * heads) * dim, dtype=DT[dtype], device=dev)
        kv = [wide[:, (2 + i * heads) * dim:(2 + (i + 1) * heads) * dim].unflatten(1, (heads, dim)) for i in range(2)]
    elif layout == "odd":   # vectors off the 16-byte grid, heads and rows spaced unevenly
        buf = torch.zeros(2, rows * heads * (dim + 3) + 1, dtype=DT[dtype], device=dev)
        kv = [buf[i, 1:].view(heads, rows, dim + 3)[:, :, :dim].transpose(0, 1) for i in range(2)]
    else:
        kv = [torch.zeros(rows, heads, dim, dtype=DT[dtype], device=dev) for _ in range(2)]
    for a, b in zip(kv, x):
        a.copy_(b)
    c = fresh(pages, heads, page, dim, dev)
    want = [U.raw(t).copy() for t in (c.k, c.v, c.k_exp, c.v_exp)]
    for i in range(2):
        codes, exps = U.quantise(x[i].double().numpy())
        for n in range(rows):
            if not skip[n]:
                pg = table[seq[n], pos[n] // page]
                want[i][pg, :, pos[n] % page] = codes[n]
                want[2 + i][pg, :, pos[n] % page] = exps[n]
    tb, rs, rp = i32(table, dev), i32(seq, dev), i32(np.where(skip, -1 - pos, pos), dev)
    out = api.spec_kv_append(c, kv[0], kv[1], tb, rs, rp)
    assert int(out["device_status"][0]) == 0
    for t, w in zip((c.k, c.v, c.k_exp, c.v_exp), want):
        assert np.array_equal(U.raw(t), w)
    for back in ("bf16", "f32"):
        got = api.spec_kv_read(c, tb, rs, rp, dtype=DT[back])
        assert int(got["device_status"][0]) == 0
        for i, name in enumerate("kv"):
            codes, exps = U.quantise(x[i].double().numpy())
            ref = U.dequantise(codes, exps)
            ref[skip] = 0
            y = got[name].double().cpu().numpy()
            # 4 significant bits and a power of two: exact in both types above fp32's and bf16's smallest normal number;
            # products below it are flushed or held as subnormals
            assert (np.abs(y - ref) <= 2.0 ** -126).all()
            assert np.array_equal(y[np.abs(ref) >= 2.0 ** -126], ref[np.abs(ref) >= 2.0 ** -126])
    only = api.spec_kv_read(c, tb, rs, rp, want_v=False)
    assert "v" not in only and torch.equal(only["k"], api.spec_kv_read(c, tb, rs, rp)["k"])


def test_no_rows(dev):
    c = fresh(2, 1, 16, 64, dev)
    e = torch.zeros(0, 1, 64, device=dev)
    none = i32([], dev)
    assert int(api.spec_kv_append(c, e, e, i32([[0]], dev), none, none)["device_status"][0]) == 0
    assert api.spec_kv_read(c, i32([[0]], dev), none, none)["k"].shape == (0, 1, 64)


@pytest.mark.parametrize("what", [float("nan"), float("inf"), float("-inf")])
def test_vectors_that_are_not_finite(dev, what):
    c = fresh(2, 2, 16, 64, dev, fill=0x11)
    k = torch.ones(2, 2, 64, device=dev)
    v = torch.ones(2, 2, 64, device=dev)
    k[0, 1, 63] = what
    tb, rs, rp = i32([[1]], dev), i32([0, 0], dev), i32([0, 1], dev)
    out = api.spec_kv_append(c, k, v, tb, rs, rp)
    assert int(out["device_status"][0]) == _lib.SPEC_DEV_NONFINITE
    assert U.raw(c.k_exp)[1, 1, 0] == 255 and (U.raw(c.k)[1, 1, 0] == 0).all()
    got = api.spec_kv_read(c, tb, rs, rp, dtype=torch.float32)
    assert torch.isnan(got["k"][0, 1]).all() and (got["k"][0, 0] == 1).all() and (got["k"][1] == 1).all()
    assert (got["v"] == 1).all()


def test_rows_out_of_range_are_reported_and_touch_nothing(dev):
    c = fresh(3, 1, 16, 64, dev, fill=0x22)
    before = [U.raw(t).copy() for t in (c.k, c.v, c.k_exp, c.v_exp)]
    x = torch.ones(1, 1, 64, device=dev)
    tb = i32([[0, 3], [1, -1]], dev)
    for seq, pos, bit in ((2, 0, _lib.SPEC_DEV_OFFSETS), (-1, 0, _lib.SPEC_DEV_OFFSETS), (0, 32, _lib.SPEC_DEV_OFFSETS),
                          (0, 2 ** 31 - 1, _lib.SPEC_DEV_OFFSETS), (0, 16, _lib.SPEC_DEV_PAGE), (1, 31, _lib.SPEC_DEV_PAGE)):
        rs, rp = i32([seq], dev), i32([pos], dev)
        assert int(api.spec_kv_append(c, x, x, tb, rs, rp)["device_status"][0]) == bit, (seq, pos)
        got = api.spec_kv_read(c, tb, rs, rp)
        assert int(got["device_status"][0]) == bit and torch.isnan(got["k"]).all() and torch.isnan(got["v"]).all()
    for t, w in zip((c.k, c.v, c.k_exp, c.v_exp), before):
        assert np.array_equal(U.raw(t), w)


def test_argument_checks(dev):
    c = fresh(2, 2, 16, 64, dev)
    k = torch.zeros(3, 2, 64, device=dev)
    tb, rs, rp = i32([[0]], dev), i32([0, 0, 0], dev), i32([0, 1, 2], dev)
    with pytest.raises(TypeError):
        api.spec_kv_append(c, k.half(), k.half(), tb, rs, rp)
    with pytest.raises(TypeError):
        api.spec_kv_append(c, k, k.bfloat16(), tb, rs, rp)
    with pytest.raises(ValueError):
        api.spec_kv_append(c, k[:2], k[:2], tb, rs, rp)
    with pytest.raises(ValueError):
        api.spec_kv_append(c, k.expand(3, 2, 64).transpose(1, 2).contiguous().transpose(1, 2), k, tb, rs, rp)
    with pytest.raises(TypeError):
        api.spec_kv_append(c, k, k, tb.long(), rs, rp)
    with pytest.raises(ValueError):
        api.spec_kv_append(c, k, k, tb, rs, rp[:2])
    with pytest.raises(TypeError):
        api.spec_kv_read(c, tb, rs, rp, dtype=torch.float16)
    with pytest.raises(ValueError):
        api.KVCache.empty(2, 2, 24, 64, dev)
    with pytest.raises(ValueError):
        api.KVCache.empty(2, 2, 16, 80, dev)


def test_places_past_32_bits(dev):
    """A page whose codes start beyond 2^32 elements."""
    page, heads, dim = 256, 8, 128
    n = (1 << 32) // (page * heads * dim) + 2
    c = api.KVCache.empty(n, heads, page, dim, dev)
    rng = np.random.default_rng(5)
    x = torch.from_numpy(rng.standard_normal((2, heads, dim))).to(torch.bfloat16).to(dev)
    tb, rs, rp = i32([[n - 1]], dev), i32([0, 0], dev), i32([3, 255], dev)
    assert int(api.spec_kv_append(c, x, -x, tb, rs, rp)["device_status"][0]) == 0
    codes, exps = U.quantise(x.double().cpu().numpy())
    assert np.array_equal(U.raw(c.k[n - 1])[:, [3, 255]].swapaxes(0, 1), codes)
    assert np.array_equal(U.raw(c.k_exp[n - 1])[:, [3, 255]].swapaxes(0, 1), exps)
    got = api.spec_kv_read(c, tb, rs, rp, dtype=torch.float32)
    assert torch.equal(got["v"], -got["k"]) and np.array_equal(got["k"].double().cpu().numpy(), U.dequantise(codes, exps))
