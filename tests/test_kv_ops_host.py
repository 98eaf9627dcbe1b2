"""Refusals of the calls around the attention (norms and rotation, chunks, weights, eviction), and the rotation's plan.
No GPU: pointers are never followed."""
import ctypes
import math
from fractions import Fraction
from types import SimpleNamespace

import pytest
import torch

from speculative_decoding_token_temp_gb300 import _lib, api

from test_kv_host import BAD_CACHES, P, batch, cache, lib, rows  # noqa: F401 (lib: the fixture)

INV, OK, DTYPE, WS = _lib.SPEC_ERR_INVALID_ARG, _lib.SPEC_OK, _lib.SPEC_ERR_DTYPE, _lib.SPEC_ERR_WORKSPACE


def rope(**kw):
    d = dict(rot_dim=128, axes=1, interleaved=0, step=P, axis=None)
    d.update(kw)
    return _lib.SpecRope(*[d[f] for f, _ in _lib.SpecRope._fields_])


def norm(**kw):
    d = dict(q_weight=P, k_weight=P, eps=1e-6)
    d.update(kw)
    return _lib.SpecHeadNorm(*[d[f] for f, _ in _lib.SpecHeadNorm._fields_])


def call_rope(lib, r=None, n=None, rows=3, q_heads=8, k_heads=2, dim=128, pos=P, dtype=_lib.SPEC_BF16, q=P, qs=(1024, 128), k=P, ks=(256, 128),
              qo=P, ko=P):
    return lib.spec_qk_rope(rows, q_heads, k_heads, dim, r or rope(), n or norm(), pos, dtype, q, *qs, k, *ks, qo, ko, None)


def call_append(lib, c=None, r=None, rp=None, n=None, q_heads=8, pos=P, dtype=_lib.SPEC_BF16, q=P, qs=(1024, 128), k=P, ks=(256, 128), v=P,
                vs=(256, 128), qo=P, st=P):
    return lib.spec_qk_rope_append(c or cache(), r or rows(), q_heads, rp or rope(), n or norm(), pos, dtype, q, *qs, k, *ks, v, *vs, qo, st, None)


def chunk(lib, g, c, dtype=_lib.SPEC_BF16, q=P, qr=1024, qh=128, o=P, lse=None, st=P, ws=P, n=1 << 40):
    return lib.spec_attention_chunk(g, c, dtype, q, qr, qh, o, lse, st, ws, n, None)


def weigh(lib, g=None, c=None, dtype=_lib.SPEC_BF16, q=P, qr=1024, qh=128, lse=P, n=None, keep=1.0, mass=P, st=P):
    return lib.spec_kv_weigh(g or batch(), c or cache(), dtype, q, qr, qh, lse, n, keep, mass, st, None)


def evict_batch(**kw):
    d = dict(B=2, pages_per_seq=4, page_table=P, kv_len=P, new_pages_per_seq=0, new_page_table=None, budget=100, sinks=4, recent=10)
    d.update(kw)
    return _lib.SpecEvictBatch(*[d[f] for f, _ in _lib.SpecEvictBatch._fields_])


def evict(lib, g=None, c=None, mass=P, kept=P, out=2 * P, st=P):
    return lib.spec_kv_evict(g or evict_batch(), c or cache(), mass, kept, out, st, None)


def test_rope_refusals(lib):  # noqa: F811
    for kw in (dict(rows=-1), dict(rows=(1 << 22) + 1), dict(q_heads=0), dict(k_heads=0), dict(k_heads=257), dict(dim=96), dict(pos=None), dict(pos=P + 2),
               dict(q=None), dict(k=None), dict(q=P + 1), dict(qo=None), dict(ko=None), dict(qo=P + 8), dict(ko=P + 4),
               dict(qs=(-1, 128)), dict(qs=(1024, -1)), dict(ks=(-1, 128)), dict(ks=(256, -1))):
        assert call_rope(lib, **kw) == INV, kw
    for kw in (dict(rot_dim=8), dict(rot_dim=-16), dict(rot_dim=144), dict(axes=0), dict(axes=5), dict(step=None), dict(step=P + 4)):
        assert call_rope(lib, r=rope(**kw)) == INV, kw
        assert call_append(lib, rp=rope(**kw)) == INV, kw
    for kw in (dict(eps=math.nan), dict(eps=math.inf), dict(eps=-1.0), dict(q_weight=P + 1), dict(k_weight=P + 1)):
        assert call_rope(lib, n=norm(**kw)) == INV, kw
        assert call_append(lib, n=norm(**kw)) == INV, kw
    assert call_rope(lib, dtype=3) == DTYPE and call_append(lib, dtype=3) == DTYPE
    assert call_rope(lib, dtype=_lib.SPEC_F32, q=P + 2) == INV
    assert call_rope(lib, rows=0, q=None, k=None, qo=None, ko=None, pos=None) == OK


@pytest.mark.parametrize("bad", BAD_CACHES)
def test_bad_caches_are_refused(lib, bad):  # noqa: F811
    c = cache(**bad)
    assert call_append(lib, c=c) == INV
    assert chunk(lib, batch(), c) == INV and lib.spec_attention_chunk_workspace_bytes(batch(), c, _lib.SPEC_BF16) == 0
    assert weigh(lib, c=c) == INV and evict(lib, c=c) == INV


def test_append_refusals(lib):  # noqa: F811
    for kw in (dict(q_heads=0), dict(st=None), dict(st=P + 1), dict(v=None), dict(v=P + 1), dict(vs=(-1, 128)), dict(vs=(256, -1)), dict(q=None), dict(qo=P + 8)):
        assert call_append(lib, **kw) == INV, kw
    for kw in (dict(rows=-1), dict(sequences=-1), dict(page_table=None), dict(row_seq=None), dict(row_pos=P + 2)):
        assert call_append(lib, r=rows(**kw)) == INV, kw
    assert call_append(lib, r=rows(rows=0, row_seq=None, row_pos=None), q=None, k=None, v=None, qo=None) == OK


def test_chunk_refusals(lib):  # noqa: F811
    big = _lib.SPEC_MAX_CHUNK_GAMMA
    parent = (ctypes.c_int32 * 3)(-1, 0, 1)
    tree = ctypes.cast(parent, ctypes.c_void_p)
    for kw in (dict(B=-1), dict(gamma=-1), dict(gamma=big + 1, total_draft=2 * (big + 1)), dict(total_draft=5), dict(cu_draft=P, total_draft=7),
               dict(q_heads=7), dict(q_heads=130), dict(prefix_len=-1), dict(scale=0.0), dict(scale=math.nan), dict(parent=tree),
               dict(gamma=big, total_draft=2 * big, q_heads=1024, pages_per_seq=1 << 15)):  # (more rows than 2^30 / q_heads)
        g = batch(**kw)
        assert chunk(lib, g, cache()) == INV, kw
        assert lib.spec_attention_chunk_workspace_bytes(g, cache(), _lib.SPEC_BF16) == 0, kw
    g = batch(gamma=1000, total_draft=2000, pages_per_seq=40)
    need = lib.spec_attention_chunk_workspace_bytes(g, cache(), _lib.SPEC_BF16)
    assert need > 0
    for kw in (dict(ws=None), dict(ws=P + 64), dict(n=need - 1)):
        assert chunk(lib, g, cache(), **kw) == WS, kw
    for kw in (dict(q=None), dict(o=None), dict(o=P + 8), dict(lse=P + 2), dict(qr=-1), dict(st=None)):
        assert chunk(lib, g, cache(), **kw) == INV, kw
    assert chunk(lib, g, cache(), dtype=5) == DTYPE
    assert chunk(lib, batch(B=0, total_draft=0), cache(), ws=None, n=0) == OK


def test_weigh_refusals(lib):  # noqa: F811
    parent = (ctypes.c_int32 * 3)(-1, 0, 1)
    for kw in (dict(B=-1), dict(gamma=129, total_draft=258), dict(total_draft=5), dict(q_heads=7), dict(scale=-1.0), dict(kv_len=None), dict(kv_len=P + 2),
               dict(page_table=None), dict(cu_draft=P + 1), dict(prefix_len=5, prefix_table=P), dict(parent=ctypes.cast(parent, ctypes.c_void_p)),
               dict(pages_per_seq=1 << 25)):
        assert weigh(lib, g=batch(**kw)) == INV, kw
    for kw in (dict(q=None), dict(q=P + 1), dict(qr=-1), dict(qh=-1), dict(lse=None), dict(lse=P + 2), dict(mass=None), dict(mass=P + 2), dict(st=None),
               dict(n=P + 2), dict(keep=-0.5), dict(keep=math.nan), dict(keep=math.inf)):
        assert weigh(lib, **kw) == INV, kw
    assert weigh(lib, g=batch(pages_per_seq=1 << 23, B=1024, gamma=1, total_draft=1024)) == INV  # (a line past 2^30 tiles)
    assert weigh(lib, dtype=9) == DTYPE
    assert weigh(lib, g=batch(B=0, total_draft=0), q=None, lse=None) == OK


def test_evict_refusals(lib):  # noqa: F811
    for kw in (dict(B=-1), dict(B=65536), dict(pages_per_seq=-1), dict(pages_per_seq=1 << 26), dict(budget=0), dict(budget=-3), dict(sinks=-1),
               dict(recent=-1), dict(sinks=60, recent=41), dict(page_table=None), dict(page_table=P + 2), dict(kv_len=None), dict(kv_len=P + 1),
               dict(new_page_table=2 * P, new_pages_per_seq=1), dict(new_page_table=2 * P + 2, new_pages_per_seq=4), dict(kv_len=2 * P)):
        assert evict(lib, evict_batch(**kw)) == INV, kw
    for kw in (dict(mass=None), dict(mass=P + 2), dict(kept=None), dict(kept=P + 2), dict(out=None), dict(out=2 * P + 2), dict(st=None), dict(st=P + 2)):
        assert evict(lib, **kw) == INV, kw
    assert evict(lib, evict_batch(B=0)) == OK


def test_host_tensors_are_refused():
    x = torch.zeros(3, 2, 64)
    r = SimpleNamespace(head_dim=64, index=-1, axes=1)
    with pytest.raises(ValueError, match="CUDA"):
        api.spec_qk_rope(x, x, r, torch.zeros(3, dtype=torch.int32))
    with pytest.raises(TypeError):
        api.spec_qk_rope(x.half(), x.half(), r, torch.zeros(3, dtype=torch.int32))
    with pytest.raises(TypeError):
        api.spec_qk_rope(x, x.bfloat16(), r, torch.zeros(3, dtype=torch.int32))
    with pytest.raises(ValueError, match="CUDA"):
        api.Rope(64, "cpu")


@pytest.mark.parametrize("kw", [dict(head_dim=96), dict(rot_dim=24), dict(rot_dim=144), dict(rot_dim=-16), dict(inv_freq=[1.0] * 3),
                                dict(inv_freq=[math.nan] * 64), dict(sections=[10, 20]), dict(sections=[70, -6]), dict(axis=[0] * 63),
                                dict(axis=[-1] * 64), dict(axis=[4] * 64), dict(sections=[64], axis=[0] * 64), dict(sections=[60, 1, 1, 1, 1])])
def test_bad_plans_are_refused(kw):
    kw = {"head_dim": 128, **kw}
    with pytest.raises(ValueError):
        api.Rope(kw.pop("head_dim"), "cpu", **kw)


def test_the_plans_steps_are_the_frequencies_in_turns(monkeypatch):
    """round(f / 2 pi * 2^64) mod 2^64, with pi from Machin's series; with it position * step is the angle to 2^-33 of a turn."""
    def arctan_inverse(n):
        return sum(Fraction((-1) ** k, (2 * k + 1) * n ** (2 * k + 1)) for k in range(40))

    pi = 16 * arctan_inverse(5) - 4 * arctan_inverse(239)
    seen = {}
    real = torch.tensor

    def record(x, **kw):
        seen.setdefault(kw.get("dtype"), x)
        return real(x, **kw)

    monkeypatch.setattr(api.torch, "tensor", record)
    freq = [1.0, 0.75, 1e-4, 1e-7, -0.3, 0.0, 12.5, 3.0]
    with pytest.raises(ValueError, match="CUDA"):
        api.Rope(64, "cpu", rot_dim=16, inv_freq=freq)
    steps = [s % (1 << 64) for s in seen[torch.int64]]
    for f, s in zip(freq, steps):
        want = Fraction(f) / (2 * pi)
        for p in (1, 7, 123457, 2 ** 31 - 1, -5):
            off = (Fraction(p * s, 1 << 64) - want * p) % 1
            assert min(off, 1 - off) <= Fraction(1, 1 << 33), (f, p)
