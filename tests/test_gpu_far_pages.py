"""Pages whose bytes lie past 32 bits of the cache's beginning: the same results as in a small cache."""
import numpy as np
import pytest
import torch

from speculative_decoding_token_temp_gb300 import api

from test_gpu_attention import dev, i32  # noqa: F401 (dev: the fixture)

pytestmark = pytest.mark.gpu


def test_places_past_32_bits(dev):  # noqa: F811
    heads, page, dim, far = 1, 256, 128, (1 << 32) // (256 * 128) + 7
    pages, lens, rows = far + 12, [900, 1200], 130
    small = api.KVCache.empty(12, heads, page, dim, dev)
    large = api.KVCache.empty(pages, heads, page, dim, dev)
    assert large.k.numel() > 1 << 32
    g = torch.Generator(device=dev).manual_seed(1)
    for a, b in ((small.k, large.k), (small.v, large.v), (small.k_exp, large.k_exp), (small.v_exp, large.v_exp)):
        a = a.view(torch.uint8)
        if a.dim() == 4:
            a.copy_((torch.randn(a.shape, generator=g, device=dev) * 80).clamp_(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8))
        else:
            a.fill_(120)
        b.view(torch.uint8)[far:].copy_(a)
    table = np.array([[3, 0, 7, 1, 11], [5, 2, 9, 4, 6]])
    kv_len = i32(lens, dev)
    n = 2 * rows
    qkv = torch.randn(n, 6 * dim, generator=g, device=dev).bfloat16()
    q, k, v = (x.unflatten(1, (-1, dim)) for x in qkv.split([4 * dim, dim, dim], dim=1))
    seq = i32(np.repeat([0, 1], rows), dev)
    pos = i32(np.concatenate([np.arange(m - rows, m) for m in lens]), dev)
    rope, got = api.Rope(dim, dev), []
    for cache, first in ((small, 0), (large, far)):
        t = i32(table + first, dev)
        q2 = api.spec_qk_rope_append(cache, q, k, v, rope, pos, t, seq, pos, eps=1e-6)["q"]
        o = api.spec_attention_chunk(q2, cache, t, kv_len, gamma=rows - 1, want_lse=True)
        mass = torch.zeros(cache.k_exp.shape, device=dev)
        last = q2.unflatten(0, (2, rows))[:, -20:].flatten(0, 1).contiguous()
        lse = o["lse"].unflatten(0, (2, rows))[:, -20:].flatten(0, 1).contiguous()
        api.spec_kv_weigh(last, cache, t, kv_len, lse, mass, gamma=19, keep=0.0)
        e = api.spec_kv_evict(cache, mass, t, kv_len, 700, sinks=4, recent=20)
        after = api.spec_attention(q2.unflatten(0, (2, rows))[:, -3:].contiguous(), cache, t, e["kv_len"], gamma=2)
        for x in (o, e, after):
            assert int(x["device_status"][0]) == 0
        got.append([o["o"], o["lse"], mass[first:first + 12], e["kept"], e["kv_len"], after["o"],
                    *(x.view(torch.uint8)[first:first + 12] for x in (cache.k, cache.v, cache.k_exp, cache.v_exp))])
    for a, b in zip(*got):
        assert torch.equal(a, b)
