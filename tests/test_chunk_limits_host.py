"""How long a chunk one spec_attention_chunk call takes: the size query, without a GPU (pointers are never followed)."""
import pytest

from speculative_decoding_token_temp_gb300 import _lib

from test_kv_host import P, batch, cache, lib  # noqa: F401 (lib: the fixture)

MOST = _lib.SPEC_MAX_CHUNK_GAMMA


def one(rows, q_heads, **kw):
    """A prompt of `rows` rows from its beginning, on pages of 64 tokens."""
    return batch(B=1, gamma=rows - 1, total_draft=rows - 1, q_heads=q_heads, pages_per_seq=-(-rows // 64), **kw)


@pytest.mark.parametrize("dtype", [_lib.SPEC_BF16, _lib.SPEC_F32])
@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("q_heads,kv_heads", [(32, 8), (8, 8), (7, 1), (32, 1)])
def test_the_longest_chunk_is_taken(lib, dtype, packed, q_heads, kv_heads):  # noqa: F811
    """2^20 rows from the beginning, of which each row block sees half of the square on average; the widened cache is in the size."""
    c, kw = cache(kv_heads=kv_heads), dict(cu_draft=P) if packed else {}
    need = lib.spec_attention_chunk_workspace_bytes(one(MOST + 1, q_heads, **kw), c, dtype)
    assert need > (MOST + 1) * kv_heads * 128 * 4


def test_64_heads_and_what_passes_the_longest_line(lib):  # noqa: F811
    """Rows times heads / 256 blocks (128 with fp32 queries) of 4100 tiles on average: 1.07e9 with 64 heads, 2.15e9 with 128 or fp32."""
    c = cache(kv_heads=8)
    assert lib.spec_attention_chunk_workspace_bytes(one(MOST + 1, 64), c, _lib.SPEC_BF16) > 0
    assert lib.spec_attention_chunk_workspace_bytes(one(MOST + 1, 64), cache(kv_heads=1), _lib.SPEC_BF16) > 0
    for g, dtype in ((one(MOST + 1, 128), _lib.SPEC_BF16), (one(MOST + 1, 64), _lib.SPEC_F32)):  # (past 2^31 tiles)
        assert lib.spec_attention_chunk_workspace_bytes(g, c, dtype) == 0
        assert lib.spec_attention_chunk(g, c, dtype, P, 8192, 128, P, None, P, P, 1 << 50, None) == _lib.SPEC_ERR_INVALID_ARG
