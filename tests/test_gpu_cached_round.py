"""The example of a whole round: append, attention over the shared prefix and the cache, verification."""
import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    try:
        import cached_round
    finally:
        sys.path.pop(0)
    return cached_round


def test_rounds_decode_and_rerun_alike(example):
    a = example.run(batch=5, gamma=3, rounds=6, prefix=70, prompt=9)
    b = example.run(batch=5, gamma=3, rounds=6, prefix=70, prompt=9)
    assert int(a["device_status"][0]) == 0
    n = a["counts"]
    assert n.shape == (6, 5) and int(n.min()) >= 1 and int(n.max()) <= 4
    assert torch.equal(n, b["counts"])
    assert torch.equal(a["length"], 8 + n.sum(0).int())


def test_logits_do_not_depend_on_sharing_the_prefix(example):
    """The same tokens with the system prompt in every sequence's own pages: the same logits up to roundings that enter at
    other places (bf16 activations; two layers)."""
    dev = torch.device("cuda")
    t = example.Target()
    Hq, Hk, D = t.heads
    gen = torch.Generator(device=dev).manual_seed(4)
    system = torch.randint(0, 1000, (1, 64), generator=gen, device=dev)
    own = torch.randint(0, 1000, (3, 40), generator=gen, device=dev)
    api = example.api
    shared = [api.KVCache.empty(20, Hk, 16, D, dev) for _ in t.layers]
    pages = torch.arange(20, dtype=torch.int32, device=dev)
    t.prompt(system, shared, pages[:4].view(1, 4))
    a = t.prompt(own, shared, pages[4:16].view(3, 4).contiguous(), prefix_table=pages[:4].contiguous(), prefix_len=64)
    alone = [api.KVCache.empty(24, Hk, 16, D, dev) for _ in t.layers]
    b = t.prompt(torch.cat([system.expand(3, -1), own], 1), alone, torch.arange(21, dtype=torch.int32, device=dev).view(3, 7))
    a, b = a.float(), b[:, 64:].float()
    assert (a - b).norm() <= 0.05 * b.norm()
