"""Speculative decoding over the 8-bit key/value cache: the calls of this package around a small random target.

A few conversations share a system prompt. Its keys and values are appended once, to pages that every
sequence reads; each round then runs the target over a sequence's last token and its gamma drafts: every layer
norms and rotates the heads' queries and keys, appends keys and values in the same pass and attends over the shared
prefix, the sequence's own tokens and the drafts before each row; the logits go to spec_verify_stochastic, and the next
round continues after the accepted drafts, writing over what was rejected. With a budget the cached tokens gather the
weights that the accepted rows give them, and where a sequence may pass the budget its lightest tokens leave the cache.
Nothing returns to the host between rounds.

    python examples/cached_round.py [--batch 8] [--gamma 4] [--rounds 16] [--prefix 300] [--budget 0]"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from speculative_decoding_token_temp_gb300 import api  # noqa: E402

MAX_ROWS = 129  # rows of one sequence in one call of a round's attention, and of the weights


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
        self.rope = api.Rope(head_dim, device)
        self.norms = [torch.ones(head_dim, dtype=torch.bfloat16, device=device) for _ in range(2)]

    def rows(self, tokens, caches, table, row_seq, start, gone=0, seen=None, **prefix):
        """Logits of tokens [B, T] whose first stands at place start[b] of its sequence's cache; `gone`: tokens [B] of it that
        left the cache. Of each layer, the queries and log-sums go to the list `seen`."""
        B, T = tokens.shape
        Hq, Hk, D = self.heads
        place = start[:, None] + torch.arange(T, dtype=torch.int32, device=tokens.device)
        turn = (place + (gone[:, None] if torch.is_tensor(gone) else gone) + prefix.get("prefix_len", 0)).flatten()
        place, length = place.flatten(), start + T
        attend = api.spec_attention if T <= MAX_ROWS else api.spec_attention_chunk
        x = self.embed[tokens.long()].flatten(0, 1)
        for (qkv, proj, up, down), cache in zip(self.layers, caches):
            y = torch.nn.functional.rms_norm(x, x.shape[-1:]) @ qkv
            q, k, v = (z.unflatten(1, (-1, D)) for z in y.split([Hq * D, Hk * D, Hk * D], dim=1))
            q = api.spec_qk_rope_append(cache, q, k, v, self.rope, turn, table, row_seq, place, q_weight=self.norms[0],
                                        k_weight=self.norms[1], eps=1e-6)["q"]
            got = attend(q, cache, table, length, gamma=T - 1, want_lse=seen is not None, **prefix)
            if seen is not None:
                seen.append((q, got["lse"]))
            x = x + got["o"].flatten(1) @ proj
            x = x + torch.nn.functional.silu(torch.nn.functional.rms_norm(x, x.shape[-1:]) @ up) @ down
        return (torch.nn.functional.rms_norm(x, x.shape[-1:]) @ self.head).view(B, T, -1)

    def prompt(self, tokens, caches, table, seen=None, **prefix):
        """Appends prompts [B, n]; their logits."""
        B, n = tokens.shape
        seq = torch.arange(B, dtype=torch.int32, device=tokens.device).repeat_interleave(n)
        return self.rows(tokens, caches, table, seq, torch.zeros(B, dtype=torch.int32, device=tokens.device), seen=seen, **prefix)


def gather(seen, caches, masses, table, length, rows, n_accepted=None, keep=1.0):
    """Adds the weights that a round's last `rows` rows give the cached tokens, layer by layer."""
    for (q, lse), cache, mass in zip(seen, caches, masses):
        B = table.shape[0]
        q, lse = (x.unflatten(0, (B, -1))[:, -rows:].flatten(0, 1).contiguous() for x in (q, lse))
        api.spec_kv_weigh(q, cache, table, length, lse, mass, gamma=rows - 1, n_accepted=n_accepted, keep=keep)


def run(batch=8, gamma=4, rounds=16, prefix=300, prompt=20, page=16, temperature=0.8, budget=0, seed=0, device="cuda"):
    """Rounds of speculative decoding; a dict of the emitted counts [rounds, batch], the caches, tables and lengths.
    budget: tokens of a sequence's own that stay in the cache before a round (0: all)."""
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
    masses = [torch.empty(c.k_exp.shape, device=device) for c in caches] if budget else None
    gone = torch.zeros(batch, dtype=torch.int32, device=device)
    if prompt > 1:
        seen = [] if budget else None
        target.prompt(prompts[:, :-1], caches, table, seen=seen, **common)
        if budget:  # (keep 0: what the masses hold before is not read)
            held = torch.full((batch,), prompt - 1, dtype=torch.int32, device=device)
            gather(seen, caches, masses, table, held, min(prompt - 1, MAX_ROWS), keep=0.0)
    last = prompts[:, -1:].int()
    start = torch.full((batch,), prompt - 1, dtype=torch.int32, device=device)
    seq = torch.arange(batch, dtype=torch.int32, device=device).repeat_interleave(gamma + 1)
    counts, status = [], torch.zeros(1, dtype=torch.int32, device=device)
    for _ in range(rounds):
        if budget:  # every layer and head chooses its own tokens, as many of each
            kept = [api.spec_kv_evict(c, m, table, start, budget, sinks=min(2, budget // 2), recent=min(4, budget // 2))["kv_len"]
                    for c, m in zip(caches, masses)][0]
            gone, start = gone + start - kept, kept
        # the drafter: the target's own embeddings and head without attention, one token after the other
        drafts, rows, x = [], [], last
        for _ in range(gamma):
            z = torch.nn.functional.rms_norm(target.embed[x[:, 0].long()], (target.embed.shape[1],)) @ target.head
            rows.append(z)
            x = torch.multinomial(torch.softmax(z.float() / temperature, -1), 1, generator=gen).int()
            drafts.append(x)
        seen = [] if budget else None
        logits = target.rows(torch.cat([last] + drafts, 1), caches, table, seq, start, gone=gone, seen=seen, **common)
        got = api.spec_verify_stochastic(
            logits.contiguous(), torch.stack(rows, 1).contiguous(), torch.cat(drafts, 1).contiguous(), temperature,
            torch.rand(batch * gamma, generator=gen, device=device), torch.rand(batch, generator=gen, device=device),
            want_nkl=False, want_greedy=False, device_status=status)
        n = got["n_accepted"]
        if budget:
            gather(seen, caches, masses, table, start + gamma + 1, gamma + 1, n_accepted=n)
        last = got["out_tokens"].view(batch, gamma + 1).gather(1, n[:, None].long())
        start = start + n + 1
        counts.append(n + 1)
    return {"counts": torch.stack(counts), "caches": caches, "table": table, "prefix_table": prefix_table,
            "length": start + gone, "held": start, "device_status": status, "target": target}


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    for name, value in (("batch", 8), ("gamma", 4), ("rounds", 16), ("prefix", 300), ("budget", 0)):
        ap.add_argument("--" + name, type=int, default=value)
    out = run(**vars(ap.parse_args()))
    n = out["counts"].float()
    print(f"{n.numel()} rounds: {n.mean():.2f} tokens a round, lengths {out['length'].tolist()}, status {int(out['device_status'][0])}")
