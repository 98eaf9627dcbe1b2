"""Speculative decoding over the 8-bit key/value cache: the calls of this package around a small random target.

A few conversations share a system prompt. Its keys and values are appended once, to pages that every
sequence reads; each round then runs the target over a sequence's last token and its gamma drafts: every layer
appends their keys and values and attends over the shared prefix, the sequence's own tokens and the drafts before
each row; the logits go to spec_verify_stochastic, and the next round continues after the accepted drafts, writing
over what was rejected. Nothing returns to the host between rounds.

    python examples/cached_round.py [--batch 8] [--gamma 4] [--rounds 16] [--prefix 300]"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from speculative_decoding_token_temp_gb300 import api  # noqa: E402

MAX_ROWS = 129  # rows of one sequence in one attention call


class Target:
    """A two-layer target with random weights: attention over the cache, a feed-forward block, an output head."""

    def __init__(self, vocab=1000, width=512, q_heads=8, kv_heads=2, head_dim=64, layers=2, seed=0, device="cuda"):
        gen = torch.Generator(device=device).manual_seed(seed)

        def weight(*shape):
            return (torch.randn(*shape, generator=gen, device=device) * shape[0] ** -0.5).to(torch.bfloat16)

        self.heads = (q_heads, kv_heads, head_dim)
        self.embed = torch.randn(vocab, width, generator=gen, device=device).to(torch.bfloat16)
        self.layers = [(weight(width, (q_heads + 2 * kv_heads) * head_dim), weight(q_heads * head_dim, width),
                        weight(width, 2 * width), weight(2 * width, width)) for _ in range(layers)]
        self.head = weight(width, vocab) * 4

    def rows(self, tokens, caches, table, row_seq, start, **prefix):
        """Logits of tokens [B, T] whose first stands at position start[b] of its sequence."""
        B, T = tokens.shape
        Hq, Hk, D = self.heads
        pos = (start[:, None] + torch.arange(T, dtype=torch.int32, device=tokens.device)).flatten()
        length = start + T
        x = self.embed[tokens.long()].flatten(0, 1)
        for (qkv, proj, up, down), cache in zip(self.layers, caches):
            y = torch.nn.functional.rms_norm(x, x.shape[-1:]) @ qkv
            q, k, v = (z.unflatten(1, (-1, D)) for z in y.split([Hq * D, Hk * D, Hk * D], dim=1))
            api.spec_kv_append(cache, k, v, table, row_seq, pos)
            o = api.spec_attention(q, cache, table, length, gamma=T - 1, **prefix)["o"]
            x = x + o.flatten(1) @ proj
            x = x + torch.nn.functional.silu(torch.nn.functional.rms_norm(x, x.shape[-1:]) @ up) @ down
        return (torch.nn.functional.rms_norm(x, x.shape[-1:]) @ self.head).view(B, T, -1)

    def prompt(self, tokens, caches, table, **prefix):
        """Appends prompts [B, n], in stretches that one call takes; the logits of the last stretch."""
        B, n = tokens.shape
        logits = None
        for a in range(0, n, MAX_ROWS):
            part = tokens[:, a:a + MAX_ROWS]
            seq = torch.arange(B, dtype=torch.int32, device=tokens.device).repeat_interleave(part.shape[1])
            logits = self.rows(part, caches, table, seq, torch.full((B,), a, dtype=torch.int32, device=tokens.device), **prefix)
        return logits


def run(batch=8, gamma=4, rounds=16, prefix=300, prompt=20, page=16, temperature=0.8, seed=0, device="cuda"):
    """Rounds of speculative decoding; a dict of the emitted counts [rounds, batch], the caches, tables and lengths."""
    target = Target(seed=seed, device=device)
    Hq, Hk, D = target.heads
    V = target.embed.shape[0]
    gen = torch.Generator(device=device).manual_seed(seed + 1)
    own = -(-(prompt + rounds * (gamma + 1)) // page)
    shared = -(-prefix // page)
    pages = torch.randperm(batch * own + shared, generator=gen, device=device).to(torch.int32)
    prefix_table, table = pages[:shared], pages[shared:].view(batch, own).contiguous()
    caches = [api.KVCache.empty(pages.numel(), Hk, page, D, device) for _ in target.layers]
    system = torch.randint(0, V, (1, prefix), generator=gen, device=device)
    target.prompt(system, caches, prefix_table.view(1, -1))
    common = {"prefix_table": prefix_table, "prefix_len": prefix}
    prompts = torch.randint(0, V, (batch, prompt), generator=gen, device=device)
    if prompt > 1:
        target.prompt(prompts[:, :-1], caches, table, **common)
    last = prompts[:, -1:].int()
    start = torch.full((batch,), prompt - 1, dtype=torch.int32, device=device)
    seq = torch.arange(batch, dtype=torch.int32, device=device).repeat_interleave(gamma + 1)
    counts, status = [], torch.zeros(1, dtype=torch.int32, device=device)
    for _ in range(rounds):
        # the drafter: the target's own embeddings and head without attention, one token after the other
        drafts, rows, x = [], [], last
        for _ in range(gamma):
            z = torch.nn.functional.rms_norm(target.embed[x[:, 0].long()], (target.embed.shape[1],)) @ target.head
            rows.append(z)
            x = torch.multinomial(torch.softmax(z.float() / temperature, -1), 1, generator=gen).int()
            drafts.append(x)
        logits = target.rows(torch.cat([last] + drafts, 1), caches, table, seq, start, **common)
        got = api.spec_verify_stochastic(
            logits.contiguous(), torch.stack(rows, 1).contiguous(), torch.cat(drafts, 1).contiguous(), temperature,
            torch.rand(batch * gamma, generator=gen, device=device), torch.rand(batch, generator=gen, device=device),
            want_nkl=False, want_greedy=False, device_status=status)
        n = got["n_accepted"]
        last = got["out_tokens"].view(batch, gamma + 1).gather(1, n[:, None].long())
        start = start + n + 1
        counts.append(n + 1)
    return {"counts": torch.stack(counts), "caches": caches, "table": table, "prefix_table": prefix_table,
            "length": start, "device_status": status, "target": target}


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    for name, value in (("batch", 8), ("gamma", 4), ("rounds", 16), ("prefix", 300)):
        ap.add_argument("--" + name, type=int, default=value)
    out = run(**vars(ap.parse_args()))
    n = out["counts"].float()
    print(f"{n.numel()} rounds: {n.mean():.2f} tokens a round, lengths {out['length'].tolist()}, status {int(out['device_status'][0])}")
