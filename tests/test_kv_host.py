"""The cache and attention entry points' argument checks: every refusal is the host's, before anything is launched.
No GPU: the pointers are never followed."""
import ctypes

import numpy as np
import pytest
import torch

from speculative_decoding_token_temp_gb300 import _lib, api, build

import kv_util as U

P = 1 << 20  # a stand-in for a device pointer: 256-byte aligned, never followed


@pytest.fixture(scope="module")
def lib():
    build.build()
    return _lib.lib()


def cache(**kw):
    d = dict(k=P, v=P, k_exp=P, v_exp=P, num_pages=4, page_size=64, kv_heads=2, head_dim=128)
    d.update(kw)
    return _lib.SpecKvCache(*[d[f] for f, _ in _lib.SpecKvCache._fields_])


def rows(**kw):
    d = dict(rows=3, sequences=2, pages_per_seq=2, page_table=P, row_seq=P, row_pos=P)
    d.update(kw)
    return _lib.SpecKvRows(*[d[f] for f, _ in _lib.SpecKvRows._fields_])


def batch(**kw):
    d = dict(B=2, gamma=3, total_draft=6, cu_draft=None, q_heads=8, pages_per_seq=2, page_table=P, kv_len=P,
             prefix_len=0, prefix_table=None, parent=None, scale=0.1)
    d.update(kw)
    return _lib.SpecAttnBatch(*[d[f] for f, _ in _lib.SpecAttnBatch._fields_])


def append(lib, c, r, dtype=_lib.SPEC_BF16, k=P, kr=256, kh=128, v=P, vr=256, vh=128, st=P):
    return lib.spec_kv_append(c, r, dtype, k, kr, kh, v, vr, vh, st, None)


def read(lib, c, r, dtype=_lib.SPEC_BF16, k=P, v=P, st=P):
    return lib.spec_kv_read(c, r, dtype, k, v, st, None)


def attend(lib, g, c, dtype=_lib.SPEC_BF16, q=P, qr=1024, qh=128, o=P, lse=None, st=P, ws=P, n=1 << 40):
    return lib.spec_attention(g, c, dtype, q, qr, qh, o, lse, st, ws, n, None)


BAD_CACHES = [dict(num_pages=0), dict(page_size=48), dict(page_size=8), dict(page_size=512), dict(kv_heads=0),
              dict(kv_heads=257), dict(head_dim=96), dict(k=None), dict(v=None), dict(k_exp=None), dict(v_exp=None),
              dict(k=P + 8), dict(v_exp=P + 4)]


@pytest.mark.parametrize("bad", BAD_CACHES)
def test_bad_caches_are_refused(lib, bad):
    c = cache(**bad)
    assert append(lib, c, rows()) == _lib.SPEC_ERR_INVALID_ARG
    assert read(lib, c, rows()) == _lib.SPEC_ERR_INVALID_ARG
    assert attend(lib, batch(), c) == _lib.SPEC_ERR_INVALID_ARG
    assert lib.spec_attention_workspace_bytes(batch(), c, _lib.SPEC_BF16) == 0


@pytest.mark.parametrize("bad", [dict(rows=-1), dict(sequences=-1), dict(pages_per_seq=-1), dict(page_table=None),
                                 dict(row_seq=None), dict(row_pos=None), dict(row_pos=P + 2), dict(page_table=P + 1)])
def test_bad_rows_are_refused(lib, bad):
    assert append(lib, cache(), rows(**bad)) == _lib.SPEC_ERR_INVALID_ARG
    assert read(lib, cache(), rows(**bad)) == _lib.SPEC_ERR_INVALID_ARG


def test_append_and_read_refusals(lib):
    INV = _lib.SPEC_ERR_INVALID_ARG
    assert append(lib, cache(), rows(), dtype=7) == _lib.SPEC_ERR_DTYPE
    assert read(lib, cache(), rows(), dtype=7) == _lib.SPEC_ERR_DTYPE
    for kw in (dict(k=None), dict(v=None), dict(k=P + 1), dict(kr=-1), dict(vh=-1), dict(st=None), dict(st=P + 2)):
        assert append(lib, cache(), rows(), **kw) == INV, kw
    assert append(lib, cache(), rows(), dtype=_lib.SPEC_F32, v=P + 2) == INV
    for kw in (dict(k=P + 8), dict(v=P + 4), dict(st=None)):
        assert read(lib, cache(), rows(), **kw) == INV, kw
    # nothing to do is no error
    assert append(lib, cache(), rows(rows=0, row_seq=None, row_pos=None), k=None, v=None) == _lib.SPEC_OK
    assert read(lib, cache(), rows(), k=None, v=None) == _lib.SPEC_OK


def _parent(*p):
    a = (ctypes.c_int32 * len(p))(*p)
    return ctypes.cast(a, ctypes.c_void_p), a


def test_attention_refusals(lib):
    INV = _lib.SPEC_ERR_INVALID_ARG
    big = 1 << 40
    for kw in (dict(B=-1), dict(gamma=-1), dict(gamma=_lib.SPEC_MAX_GAMMA + 1, total_draft=2 * (_lib.SPEC_MAX_GAMMA + 1)),
               dict(total_draft=5), dict(total_draft=-1), dict(cu_draft=P, total_draft=7), dict(q_heads=0), dict(q_heads=7),
               dict(q_heads=130), dict(pages_per_seq=-1), dict(pages_per_seq=1 << 27), dict(prefix_len=-1),
               dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan")), dict(scale=float("inf"))):
        assert attend(lib, batch(**kw), cache(), n=big) == INV, kw
        assert lib.spec_attention_workspace_bytes(batch(**kw), cache(), _lib.SPEC_BF16) == 0, kw
    for kw in (dict(kv_len=None), dict(page_table=None), dict(prefix_len=5), dict(kv_len=P + 2), dict(cu_draft=P + 1)):
        assert attend(lib, batch(**kw), cache(), n=big) == INV, kw
    for kw in (dict(q=None), dict(o=None), dict(o=P + 8), dict(q=P + 1), dict(lse=P + 2), dict(qr=-1), dict(qh=-1),
               dict(st=None), dict(st=P + 1)):
        assert attend(lib, batch(), cache(), **kw) == INV, kw
    assert attend(lib, batch(), cache(), dtype=5) == _lib.SPEC_ERR_DTYPE
    for bad in ((-2, 0, 1), (0, 0, 1), (-1, 1, 0)):
        ptr, keep = _parent(*bad)
        assert attend(lib, batch(parent=ptr), cache(), n=big) == INV, bad
        del keep
    ptr, keep = _parent(-1, 0, 1)
    assert attend(lib, batch(parent=ptr, cu_draft=P), cache(), n=big) == INV
    ptr, keep = _parent(*[-1] * 65)
    assert attend(lib, batch(parent=ptr, gamma=65, total_draft=130), cache(), n=big) == INV
    need = lib.spec_attention_workspace_bytes(batch(), cache(), _lib.SPEC_BF16)
    assert need > 0
    for kw in (dict(ws=None), dict(ws=P + 64), dict(n=need - 1)):
        assert attend(lib, batch(), cache(), **kw) == _lib.SPEC_ERR_WORKSPACE, kw
    assert attend(lib, batch(B=0, total_draft=0), cache(), ws=None, n=0) == _lib.SPEC_OK


def test_host_tensors_are_refused():
    k = torch.zeros(2, 1, 16, 64, dtype=torch.uint8).view(torch.float8_e4m3fn)
    e = torch.zeros(2, 1, 16, dtype=torch.uint8)
    with pytest.raises(ValueError, match="CUDA"):
        api.KVCache(k, k.clone(), e, e.clone())


def test_quantiser_restatement():
    """The tests' own quantiser against hand values: 448 and just above it, ties to even, zeros, tiny and infinite vectors."""
    def q(*x):
        c, e = U.quantise(np.array([x]))
        return list(U.VALUES[c[0]]), int(e[0]) - 127
    assert q(448.0, 1.0) == ([448.0, 1.0], 0)
    assert q(448.5, 0.0) == ([224.0, 0.0], 1)
    assert q(-448.0, 17.0, 19.0) == ([-448.0, 16.0, 20.0], 0)          # ties to even: between 16 and 18, 18 and 20
    assert q(1.75, -1.0) == ([448.0, -256.0], -8)
    assert q(0.0, 0.0)[1] == U.ZERO_EXP
    assert q(2.0 ** -140, 0.0)[1] == U.MIN_EXP
    assert U.quantise(np.array([[1.0, np.inf]]))[1][0] == 255
    assert np.isnan(U.dequantise(np.zeros((1, 2), dtype=np.uint8), np.array([255], dtype=np.uint8))).all()


def test_visibility_restatement():
    assert U.visible(2, 3).tolist() == [[True, True, False], [True, True, True]]
    # a tree of two roots, the first with a child: rows are the context token and nodes 0..2
    v = U.visible(4, 5, parent=[-1, -1, 0])
    assert v[:, 0].all() and v[:, 1].all()                               # context, the row of the context token
    assert v[:, 2:].tolist() == [[False] * 3, [True, False, False], [False, True, False], [True, False, True]]
    # a cache shorter than the round: rows before its first token see nothing
    assert U.visible(3, 1).tolist() == [[False], [False], [True]]
