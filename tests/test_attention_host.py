"""What the attention kernels' correctness rests on and no GPU is needed for: the order of hand-overs between warps, the
parts that weights are split into, the binding's own checks."""
import os
import re
from types import SimpleNamespace

import pytest
import torch

from speculative_decoding_token_temp_gb300 import api

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "speculative_decoding_token_temp_gb300", "csrc")


def source(name):
    with open(os.path.join(CSRC, name)) as f:
        return f.read()


def orders(buffers, tiles):
    """Every order in which the two halves of the softmax warps may pass through `tiles` masked tiles; True when each read of
    the flags (`buffers` of them, by the tile's number) finds its own tile's.

    A half's steps in tile i: the first one writes the flags, both meet, the second one reads them, each waits until the
    products of tile i - 1 are summed (which follows both halves' weights of that tile), each hands over its weights."""
    first = [(what, i) for i in range(tiles) for what in ("write", "meet", "wait", "hand")]
    second = [(what, i) for i in range(tiles) for what in ("meet", "read", "wait", "hand")]
    handed = {i: (first.index(("hand", i)), second.index(("hand", i))) for i in range(tiles)}
    todo, seen = [(0, 0, (None,) * buffers)], set()
    while todo:
        state = todo.pop()
        if state in seen:
            continue
        seen.add(state)
        a, b, flags = state

        def free(steps, at):
            what, i = steps[at]
            return what != "wait" or i == 0 or (a > handed[i - 1][0] and b > handed[i - 1][1])

        if a < len(first) and b < len(second) and first[a][0] == second[b][0] == "meet":
            todo.append((a + 1, b + 1, flags))
        if a < len(first) and first[a][0] != "meet" and free(first, a):
            what, i = first[a]
            todo.append((a + 1, b, tuple(i if what == "write" and k == i % buffers else f for k, f in enumerate(flags))))
        if b < len(second) and second[b][0] != "meet" and free(second, b):
            what, i = second[b]
            if what == "read" and flags[i % buffers] != i:
                return False
            todo.append((a, b + 1, flags))
    return True


def test_nan_flags_of_masked_tiles_are_read_before_they_are_written_again():
    text = source("kernels_attn_tc.cuh")
    declared = re.search(r"uint8_t nan_code((?:\[\w+\])+);", text).group(1)
    buffers = 1 if declared == "[kTile]" else int(re.match(r"\[(\d+)\]\[kTile\]$", declared).group(1))
    uses = re.findall(r"sh\.nan_code((?:\[[^\]]*\])+)", text)
    assert len(uses) == 2 and all(u == ("[t]" if buffers == 1 else f"[gi & {buffers - 1}][t]") for u in uses)
    assert orders(buffers, 5)
    assert not orders(1, 3)  # (one set of flags would not do)


def host_cache(kv_heads=2, page=16, dim=64, pages=4):
    """What the binding looks at of a cache, with tensors of the host in the place of the device's (device number -1)."""
    k = torch.zeros(pages, kv_heads, page, dim, dtype=torch.uint8).view(torch.float8_e4m3fn)
    return SimpleNamespace(k=k, index=-1, kv_heads=kv_heads, page_size=page, head_dim=dim, num_pages=pages, desc=None)


def test_rows_of_one_token_cut_out_of_a_fused_projection_are_taken_as_they_are():
    cache = host_cache()

    def same(got, address, row, head, B):
        return got[0] == address and got[2] == head and (B == 1 or got[1] == row)  # (one row has no stride)

    for B in (1, 2, 5):
        qkv = torch.randn(B, (4 + 2 * 2) * 64)
        q = qkv[:, :4 * 64].unflatten(1, (4, 64)).unsqueeze(1)  # [B, 1, 4, 64], whose second stride means nothing
        assert same(api._rows_view(q, "q", B, 4, cache), qkv.data_ptr(), qkv.shape[1], 64, B)
        k = qkv[:, 4 * 64:6 * 64].view(B, 1, 2, 64)
        assert same(api._rows_view(k, "k", B, 2, cache), qkv.data_ptr() + 4 * 4 * 64, qkv.shape[1], 64, B)
    wide = torch.randn(2, 4, 3, 64)
    assert api._rows_view(wide, "q", 8, 3, cache) == (wide.data_ptr(), 3 * 64, 64)
    with pytest.raises(ValueError, match="evenly spaced"):
        api._rows_view(wide[:, :3], "q", 6, 3, cache)


class Calls:
    """In the place of the library: what each call finds as the current device."""

    def __init__(self, device):
        self.device, self.seen = device, []

    def __getattr__(self, name):
        def call(*args):
            self.seen.append((name, self.device[0]))
            return 256 if name.endswith("bytes") else 0
        return call


def test_calls_launch_on_the_caches_device(monkeypatch):
    device = [3]  # the current one; the cache's is -1

    class guard:
        def __init__(self, index):
            self.index = index

        def __enter__(self):
            self.before, device[0] = device[0], self.index

        def __exit__(self, *a):
            device[0] = self.before

    lib, cache = Calls(device), host_cache()
    monkeypatch.setattr(api, "_current_device", lambda: device[0], raising=False)
    monkeypatch.setattr(api, "_stream_handle", lambda index: 0)
    monkeypatch.setattr(torch.cuda, "device", guard)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: device[0] != -1)
    monkeypatch.setattr(api._lib, "lib", lambda: lib)
    monkeypatch.setattr(api, "_need", lambda *a, **k: None)
    table, seq, pos = torch.zeros(3, 1, dtype=torch.int32), *torch.zeros(2, 3, dtype=torch.int32)
    x = torch.zeros(3, 2, 64)
    for now in (3, -1):  # (and where it is the current one)
        device[0] = now
        api.spec_kv_append(cache, x, x, table, seq, pos)
        api.spec_kv_read(cache, table, seq, pos, dtype=torch.float32)
        api.spec_attention(torch.zeros(3, 4, 64), cache, table, seq, gamma=0)
        api.spec_attention(torch.zeros(3, 4, 64), cache, table, seq, gamma=0, workspace=torch.zeros(256, dtype=torch.uint8))
        assert [d for name, d in lib.seen if not name.endswith("bytes")] == [-1] * 4, lib.seen
        assert device[0] == now
        lib.seen.clear()
    api._DEFAULT_WS.pop(("cuda", -1, 0), None)


def test_workspaces_of_other_places_are_refused(monkeypatch):
    """Memory of the host, and a view whose elements are fewer than it says: kernels would write outside it."""
    with pytest.raises(ValueError, match="CUDA"):
        api._workspace(torch.empty(512, dtype=torch.uint8), 256, torch.device("cuda", 0))
    monkeypatch.setattr(torch.Tensor, "is_cuda", True)
    with pytest.raises(ValueError, match="contiguous"):
        api._workspace(torch.empty(1, dtype=torch.uint8).expand(512), 256, torch.device("cpu"))
    ws = torch.empty(512, dtype=torch.uint8)
    assert api._workspace(ws, 256, torch.device("cpu")) is ws
    with pytest.raises(ValueError, match="needs"):
        api._workspace(ws, 513, torch.device("cpu"))


@pytest.mark.parametrize("gamma,prefix_len", [((1 << 32) + 1, 0), (1, (1 << 32) + 5), (1, -(1 << 32) + 5), (-(1 << 32) + 1, 0)])
def test_numbers_past_32_bits_are_refused(gamma, prefix_len):
    """They would arrive in the descriptor as other, valid ones."""
    cache = host_cache()
    table, n = torch.zeros(2, 1, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    pages = SimpleNamespace(numel=lambda: 1 << 32, data_ptr=lambda: 0)
    real = api._is
    with pytest.MonkeyPatch.context() as m:
        m.setattr(api, "_is", lambda t, *a: t is pages or real(t, *a))
        with pytest.raises(ValueError, match="32-bit"):
            api._attn_batch(torch.zeros(4, 2, 64), cache, table, n, gamma, torch.zeros(3, dtype=torch.int32), None, None, pages, prefix_len)
        g, *_ = api._attn_batch(torch.zeros(4, 2, 64), cache, table, n, 1, torch.zeros(3, dtype=torch.int32), None, None, pages, 16)
    assert (g.gamma, g.prefix_len) == (1, 16)
