"""Whole rounds with the calls together, as a user has them: norms, rotation and append in one pass, chunks, weights, eviction,
verification."""
import pytest
import torch

from test_gpu_cached_round import example  # noqa: F401 (the fixture)

pytestmark = pytest.mark.gpu


def test_rounds_within_a_budget(example):  # noqa: F811
    kw = dict(batch=5, gamma=3, rounds=7, prefix=70, prompt=60, budget=24)
    a, b = example.run(**kw), example.run(**kw)
    assert int(a["device_status"][0]) == 0
    n = a["counts"]
    assert n.shape == (7, 5) and int(n.min()) >= 1 and int(n.max()) <= 4
    assert torch.equal(n, b["counts"]) and torch.equal(a["held"], b["held"])
    assert torch.equal(a["length"], 59 + n.sum(0).int())
    assert int(a["held"].max()) <= 24 + 4 and torch.equal(a["held"], 24 + n[-1].int())


def test_a_budget_that_nothing_passes_changes_nothing(example):  # noqa: F811
    kw = dict(batch=4, gamma=3, rounds=5, prefix=40, prompt=30)
    a, b = example.run(**kw), example.run(budget=1000, **kw)
    assert torch.equal(a["counts"], b["counts"]) and torch.equal(a["length"], b["held"])


@pytest.mark.parametrize("prefix", [0, 48])
def test_a_prompt_in_one_chunk_and_in_stretches(example, prefix):  # noqa: F811
    """The same logits up to roundings that enter at other places (bf16 activations; two layers)."""
    dev, api = torch.device("cuda"), example.api
    t = example.Target()
    Hq, Hk, D = t.heads
    gen = torch.Generator(device=dev).manual_seed(7)
    tokens = torch.randint(0, 1000, (2, 300), generator=gen, device=dev)
    pages = torch.arange(50, dtype=torch.int32, device=dev)
    table, shared, common = pages[3:41].view(2, 19).contiguous(), pages[:3].contiguous(), {}
    got = []
    for step in (300, 100):
        caches = [api.KVCache.empty(50, Hk, 16, D, dev) for _ in t.layers]
        if prefix:
            t.prompt(torch.arange(prefix, device=dev).view(1, -1), caches, shared.view(1, 3))
            common = {"prefix_table": shared, "prefix_len": prefix}
        seq = torch.arange(2, dtype=torch.int32, device=dev).repeat_interleave(step)
        got.append(torch.cat([t.rows(tokens[:, a:a + step], caches, table, seq, torch.full((2,), a, dtype=torch.int32, device=dev), **common)
                              for a in range(0, 300, step)], 1).float())
    assert (got[0] - got[1]).norm() <= 0.05 * got[1].norm()
