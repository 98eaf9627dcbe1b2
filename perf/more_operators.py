"""Cases of what stands around the attention over the 8-bit key/value cache: the norms and rotations of queries and keys on
their way into it (`rope`, `append`), the attention of a chunk of new tokens over it (`chunk`), the weight that its tokens
gather (`weigh`) and the eviction of the lightest (`evict`)."""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
E4M3 = torch.float8_e4m3fn
SCALE = torch.float8_e8m0fnu  # an exponent byte as the power of two it stands for
EPS = 1e-6


def listed():
    heads = {"heads": 32, "kv_heads": 8, "dim": 128, "page": 64}
    text = {"axes": 1, "interleaved": False, "norm": True}
    return [
        # one decoding step of a few sequences: latency counts
        {"name": "append_one_token", "op": "append", "batch": 4, "gamma": 0, "lo": 0, "hi": 4096, "skip": 0.0, "start": 0,
         "rot": 128, "dtype": "bf16", **text, **heads},
        # a verification round of 8 drafts, far into long documents
        {"name": "append_round_far", "op": "append", "batch": 256, "gamma": 8, "lo": 100, "hi": 2000, "skip": 0.0,
         "start": 900000, "rot": 128, "dtype": "bf16", **text, **heads},
        # whole prompts, without a cache
        {"name": "rope_prompts", "op": "rope", "batch": 8, "gamma": 4095, "lo": 0, "hi": 0, "start": 0, "rot": 128,
         "dtype": "bf16", **text, **heads},
        # patches of a video (time, height, width), half of a head rotated, in 32 bits, no norms
        {"name": "rope_video_f32", "op": "rope", "batch": 3, "gamma": 1110, "lo": 0, "hi": 7, "start": 0, "rot": 32, "axes": 3,
         "interleaved": True, "norm": False, "dtype": "f32", "heads": 12, "kv_heads": 4, "dim": 64, "page": 16},
        # one prompt from its beginning
        {"name": "chunk_prompt", "op": "chunk", "batch": 1, "gamma": 4095, "ragged": False, "lo": 0, "hi": 0, "prefix": 0,
         "dtype": "bf16", **heads},
        # pieces of long documents behind what is already cached
        {"name": "chunk_long_context", "op": "chunk", "batch": 4, "gamma": 2047, "ragged": False, "lo": 0, "hi": 16384,
         "prefix": 0, "dtype": "bf16", **heads},
        # a batch of prompts of every length, some of a single token, behind a system prompt, small heads
        {"name": "chunk_ragged_prefix", "op": "chunk", "batch": 24, "gamma": 600, "ragged": True, "lo": 0, "hi": 900,
         "prefix": 777, "dtype": "bf16", "heads": 14, "kv_heads": 2, "dim": 64, "page": 16},
        # 32-bit queries
        {"name": "chunk_f32", "op": "chunk", "batch": 2, "gamma": 199, "ragged": False, "lo": 0, "hi": 300, "prefix": 0,
         "dtype": "f32", "heads": 8, "kv_heads": 4, "dim": 64, "page": 32},
        # single-token decoding of a large batch with long caches: every step adds to the weights
        {"name": "weigh_one_token", "op": "weigh", "batch": 256, "gamma": 0, "ragged": False, "lo": 1, "hi": 8192,
         "keep": 1.0, "partly": False, "dtype": "bf16", **heads},
        # the last rows of long prompts look back, before these are cut to a budget
        {"name": "weigh_window", "op": "weigh", "batch": 8, "gamma": 31, "ragged": False, "lo": 2000, "hi": 16384,
         "keep": 0.0, "partly": False, "dtype": "bf16", **heads},
        # a few short sequences
        {"name": "evict_few", "op": "evict", "batch": 3, "lo": 700, "hi": 1100, "budget": 500, "sinks": 4, "recent": 33,
         "heads": 4, "kv_heads": 4, "dim": 64, "page": 16},
        # a large batch of long sequences, half of the longest kept
        {"name": "evict_large_batch", "op": "evict", "batch": 64, "lo": 1000, "hi": 8192, "budget": 4096, "sinks": 4,
         "recent": 256, **heads},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kv = rng.choice([1, 2, 4, 8])
    c = {"op": rng.choice(["rope", "append", "chunk", "chunk", "weigh", "evict"]), "kv_heads": kv,
         "heads": min(kv * rng.choice([1, 2, 3, 4, 5, 7, 8]), 32 // kv * kv), "dim": rng.choice([64, 128, 128]),
         "page": rng.choice([16, 32, 64, 128, 256])}
    if c["op"] == "evict":
        c["heads"] = kv
        c["batch"] = _log(rng, 1, 64)
        c["hi"] = _log(rng, 64, min(32768, 64 * 8192 // c["batch"]))
        c["lo"] = rng.choice([1, c["hi"] // 2, c["hi"]])
        c["budget"] = max(1, int(c["hi"] * rng.choice([0.1, 0.3, 0.5, 0.9])))
        c["sinks"], c["recent"] = rng.choice([0, min(4, c["budget"] // 4)]), rng.choice([0, c["budget"] // 8])
        return c
    c["dtype"] = rng.choice(["bf16", "bf16", "bf16", "f32"])
    if c["op"] in ("rope", "append"):
        rows = _log(rng, 1, 32768)
        c["batch"] = min(rows, _log(rng, 1, 512))
        c["gamma"] = max(0, rows // c["batch"] - 1)
        c["lo"], c["hi"], c["start"] = 0, _log(rng, 1, 4096), rng.choice([0, 0, 30000, 1000000])
        c["axes"], c["interleaved"], c["norm"] = rng.choice([1, 1, 2, 3]), rng.random() < 0.3, rng.random() < 0.7
        c["rot"] = rng.choice([c["dim"], c["dim"], c["dim"] // 2, 32, 48])
        if c["op"] == "append":
            c["skip"] = rng.choice([0.0, 0.25])
        return c
    small = c["dtype"] == "f32"
    if c["op"] == "weigh":
        c["batch"], c["gamma"] = _log(rng, 1, 64 if small else 256), rng.choice([0, 0, 1, 5, 8, 31, 63])
        c["ragged"] = c["gamma"] > 1 and rng.random() < 0.4
        c["hi"] = _log(rng, 1, min(32768, 256 * 8192 // c["batch"], 8 * 32 * 16384 * 32 // (c["batch"] * (c["gamma"] + 1) * c["heads"])))
        c["lo"], c["keep"], c["partly"] = rng.choice([0, c["hi"] // 2, c["hi"]]), rng.choice([1.0, 1.0, 0.9, 0.0]), rng.random() < 0.3
        return c
    c["gamma"] = _log(rng, 1, 400 if small else 4096) - 1
    c["ragged"] = c["gamma"] > 1 and rng.random() < 0.5
    c["prefix"] = rng.choice([0, 0, _log(rng, 1, 1000)])
    c["batch"] = max(1, min(_log(rng, 1, 64), (1000 if small else 16384) // (c["gamma"] + 1)))
    c["hi"] = _log(rng, 1, 1000 if small else 16384)
    most = 4 * 2048 * 32 * 128 * 10000 // (c["batch"] * (c["gamma"] + 1) * c["heads"] * c["dim"])
    c["hi"] = max(0, min(c["hi"], most - c["prefix"] - c["gamma"]))
    c["lo"] = rng.choice([0, c["hi"] // 2, c["hi"]])
    return c


def _spread(n, lo, hi):
    """n whole numbers over lo..hi, the same for every seed."""
    return [lo + int((hi - lo + 1) * ((i * 0.6180339887498949 + 0.5) % 1.0)) for i in range(n)]


def _rows_of(c):
    """How many rows each sequence has."""
    return [g + 1 for g in _spread(c["batch"], 0, c["gamma"])] if c.get("ragged") else [c["gamma"] + 1] * c["batch"]


def _before(c):
    """Cached tokens of each sequence before the call's own rows (eviction: all of them)."""
    return _spread(c["batch"], c["lo"], c["hi"])


def work(c):
    D, Hk = c["dim"], c["kv_heads"]
    before = _before(c)
    if c["op"] == "evict":
        kept = sum(min(n, c["budget"]) for n in before)
        return {"bytes": Hk * (4 * sum(before) + kept * (2 * (2 * (D + 1) + 4) + 4)), "flops": 0}
    rows, H = _rows_of(c), c["heads"]
    size, R = 2 if c["dtype"] == "bf16" else 4, sum(rows)
    if c["op"] == "rope":
        return {"bytes": R * (2 * (H + Hk) * D * size + 4 * c["axes"]), "flops": R * (H + Hk) * (3 * c["rot"] + 4 * D * c["norm"])}
    if c["op"] == "append":
        n = R * (1.0 - c["skip"])
        return {"bytes": R * (2 * H * D * size + 4 * c["axes"] + 8) + n * 2 * Hk * (D * size + D + 1),
                "flops": R * H * (3 * c["rot"] + 4 * D * c["norm"])}
    seen = sum(r * (n + c.get("prefix", 0)) + r * (r + 1) / 2 for r, n in zip(rows, before))
    cached = sum(before) + R
    if c["op"] == "chunk":
        return {"bytes": (cached + c["prefix"]) * Hk * 2 * (D + 1) + 2 * R * H * D * size, "flops": 4.0 * seen * H * D}
    return {"bytes": cached * Hk * (D + 1 + (8 if c["keep"] else 4)) + R * H * (D * size + 4), "flops": 2.0 * seen * H * D}


def _generator(seed, device):
    return torch.Generator(device=device).manual_seed(seed)


def _power(e):
    """2^e for whole numbers -126..127, built from its bits (a power computed otherwise may be off in its last place)."""
    return (e.int() + 127).bitwise_left_shift(23).view(torch.float32)


def _values(codes, exps):
    return codes.float() * _power(exps.int() - 127).unsqueeze(-1)


def prepare(c, seed):
    dev, host = torch.device("cuda"), _generator(seed, "cpu")
    gen = _generator(seed, dev)
    H, Hk, D, S, B = c["heads"], c["kv_heads"], c["dim"], c["page"], c["batch"]
    order = torch.randperm(B, generator=host).tolist()
    rows = [_rows_of(c)[i] for i in order] if c["op"] != "evict" else [0] * B
    before = [_before(c)[i] for i in order]
    lens = [n + r for n, r in zip(before, rows)]
    R = sum(rows)
    s = {"op": c["op"], "dtype": DTYPES.get(c.get("dtype")), "out": {}}
    pre = -(-c.get("prefix", 0) // S)
    used = [-(-n // S) for n in lens]
    more = [-(-min(n, c["budget"]) // S) for n in lens] if c["op"] == "evict" else []
    pages = sum(used) + sum(more) + pre + 3
    if c["op"] != "rope":
        perm = torch.randperm(pages, generator=host, dtype=torch.int32)
        at = pre

        def tables(counts, at):
            """Each sequence's pages from the pool in any order; places past its end name page 0 and are never read."""
            table = torch.zeros(B, max(1, max(counts)), dtype=torch.int32)
            for b, n in enumerate(counts):
                table[b, :n] = perm[at:at + n]
                at += n
            return table.to(dev), at

        s["table"], at = tables(used, at)
        if c["op"] == "append":
            codes = torch.zeros(2, pages, Hk, S, D, dtype=torch.uint8, device=dev)
            exps = torch.zeros(2, pages, Hk, S, dtype=torch.uint8, device=dev)
        else:
            # tokens as a model's keys and values are: normal within a token, tokens of different size
            normal = torch.empty(pages, Hk, S, D, device=dev, dtype=torch.bfloat16)
            codes = torch.empty(2, pages, Hk, S, D, dtype=torch.uint8, device=dev)
            for i in (0, 1):
                normal.normal_(generator=gen)
                codes[i] = normal.mul_(80.0).clamp_(-448.0, 448.0).to(E4M3).view(torch.uint8)
            exps = 127 - 7 + torch.randint(0, 2, (2, pages, Hk, S), generator=gen, device=dev, dtype=torch.uint8)
            del normal
        s["k"], s["v"], s["k_exp"], s["v_exp"] = codes[0].view(E4M3), codes[1].view(E4M3), exps[0], exps[1]
        s["kv_len"] = torch.tensor(lens, dtype=torch.int32).to(dev)
    if c["op"] == "evict":
        # weights gathered over many steps: most tokens light, few heavy, some that nothing has looked at
        mass = torch.randn(pages, Hk, S, generator=gen, device=dev).mul_(2.0).exp_()
        s["mass"] = torch.where(torch.rand(pages, Hk, S, generator=gen, device=dev) < 0.05, 0.0, mass)
        s["new_table"] = tables(more, at)[0]
        s["budget"], s["sinks"], s["recent"] = c["budget"], c["sinks"], c["recent"]
        return s
    if c["op"] in ("rope", "append"):
        # one projection's rows: queries, keys, values side by side
        size = 2.0 * torch.rand(R, 1, generator=gen, device=dev).exp()
        qkv = (torch.randn(R, (H + 2 * Hk) * D, generator=gen, device=dev) * size).to(s["dtype"])
        s["q"], s["new_k"], s["new_v"] = (x.unflatten(1, (-1, D)) for x in qkv.split([H * D, Hk * D, Hk * D], dim=1))
        s["weights"] = [(1 + 0.2 * torch.randn(D, generator=gen, device=dev)).to(s["dtype"]) for _ in range(2)] if c["norm"] else [None] * 2
        seq = torch.repeat_interleave(torch.arange(B), torch.tensor(rows))
        i = torch.arange(R) - torch.cumsum(torch.tensor([0] + rows[:-1]), 0)[seq]
        first = torch.tensor(before)[seq]
        p = c["start"] + first + i
        if c["axes"] > 1:  # a grid of patches, 24 wide
            p = torch.stack([first + i // 576, i // 24 % 24, i % 24][:c["axes"]], 1) + c["start"]
        s["positions"] = p.to(torch.int32).to(dev)
        pairs = c["rot"] // 2
        s["axis"] = [j * c["axes"] // pairs for j in range(pairs)]
        s["axis_of"] = torch.tensor(s["axis"], device=dev)
        s["inv_freq"] = 10000.0 ** (-torch.arange(pairs, dtype=torch.float64, device=dev) * 2 / c["rot"])
        s["rot"], s["interleaved"] = c["rot"], c["interleaved"]
    if c["op"] == "append":
        left_out = torch.rand(R, generator=host) < c["skip"]
        s["row_seq"] = seq.to(torch.int32).to(dev)
        s["row_pos"] = torch.where(left_out, -1, first + i).to(torch.int32).to(dev)
    if c["op"] in ("chunk", "weigh"):
        s["q"] = torch.randn(R, H, D, generator=gen, device=dev).mul_(1.5).to(s["dtype"])
        s["gamma"], s["rows"] = c["gamma"], rows
        T = c["gamma"] + 1
        n_rows = torch.tensor(rows)
        cu = torch.cumsum(torch.tensor([0] + [r - 1 for r in rows]), 0).to(torch.int32)
        s["cu_draft"] = cu.to(dev) if c["ragged"] else None
        s["row_of"] = torch.where(torch.arange(T) < n_rows[:, None], (cu[:-1] + torch.arange(B))[:, None] + torch.arange(T), R).to(dev)  # [B, T], R: none
        s["n_rows"] = n_rows.to(dev)
    if c["op"] == "chunk":
        s["prefix_len"], s["prefix_table"] = c["prefix"], perm[:pre].to(dev) if pre else None
    if c["op"] == "weigh":
        # what the attention has left, and the weights of the steps before
        s["lse"] = torch.empty(R, H, device=dev)
        at = 0
        for b, (r, n) in enumerate(zip(rows, lens)):
            pg = s["table"][b, :used[b]].long()
            k = _values(s["k"].view(torch.uint8)[pg].view(E4M3), s["k_exp"][pg]).transpose(0, 1).reshape(Hk, -1, D)[:, :n]
            q = s["q"][at:at + r].float().view(r, Hk, H // Hk, D).permute(1, 2, 0, 3).reshape(Hk, -1, D)
            x = (q @ k.transpose(1, 2) / math.sqrt(D)).view(Hk, H // Hk, r, n)
            x.masked_fill_(torch.arange(n, device=dev) > n - r + torch.arange(r, device=dev)[:, None], -math.inf)
            s["lse"][at:at + r] = torch.logsumexp(x, -1).permute(2, 0, 1).reshape(r, H)
            at += r
        s["mass"] = torch.rand(pages, Hk, S, generator=gen, device=dev)
        s["keep"] = c["keep"]
        taken = (torch.rand(B, generator=host) * n_rows).to(torch.int32)
        s["n_accepted"] = taken.to(dev) if c["partly"] else None
    return s


def _plain_codes(x):
    """Codes and exponents of vectors: the smallest power of two that brings the vector into the code's range (448), at least 2^-100; -60 for a vector of zeros."""
    most = x.abs().amax(-1)
    part, e = torch.frexp(most)
    e = torch.where(part <= 0.875, e - 9, e - 8).clamp(min=-100)
    e = torch.where(most == 0, -60, e)
    return (x * _power(-e).unsqueeze(-1)).to(E4M3).view(torch.uint8), (e + 127).to(torch.uint8)


def _plain_rotated(s, x, weight, cos, sin):
    x = x.float()
    if weight is not None:
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * weight.float()
    rot = s["rot"]
    y = x[..., :rot]
    a, b = (y[..., 0::2], y[..., 1::2]) if s["interleaved"] else y.chunk(2, -1)
    a, b = a * cos - b * sin, b * cos + a * sin
    y = torch.stack([a, b], -1).flatten(-2) if s["interleaved"] else torch.cat([a, b], -1)
    return torch.cat([y, x[..., rot:]], -1)


def _plain_rope(s):
    p = s["positions"] if s["positions"].dim() == 2 else s["positions"][:, None]
    angle = p[:, s["axis_of"]].double() * s["inv_freq"]  # far positions: 64 bits
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
    return [_plain_rotated(s, x, w, cos, sin) for x, w in zip((s["q"], s["new_k"]), s["weights"])]


def _pool(s, *names):
    """The cache's buffers, an exponent byte as the power of two it stands for."""
    return {n: s[n].view(SCALE) if n.endswith("exp") else s[n] for n in names}


def _plain_append(s):
    q, k = _plain_rope(s)
    S = s["k"].shape[2]
    at = (s["row_pos"] >= 0).nonzero().squeeze(1)
    pos = s["row_pos"][at].long()
    page, slot = s["table"][s["row_seq"][at].long(), pos // S].long(), pos % S
    for x, n in ((k, "k"), (s["new_v"].float(), "v")):
        codes, exps = _plain_codes(x[at])
        s[n].view(torch.uint8)[page, :, slot] = codes
        s[n + "_exp"][page, :, slot] = exps
    return {"q": q.to(s["dtype"]), **_pool(s, "k", "v", "k_exp", "v_exp")}


def _keys(s, n, pages):
    """Cached vectors of a table's pages, [.., kv_heads, tokens, dim]."""
    return _values(s[n].view(torch.uint8)[pages].view(E4M3), s[n + "_exp"][pages]).transpose(-4, -3).flatten(-3, -2)


def _batch(s):
    """Queries [B, kv_heads, T, G, D], scaled, and what row i of each sequence sees, [B, T, L]."""
    dev, (B, T) = s["table"].device, s["row_of"].shape
    _, H, D = s["q"].shape
    Hk, S = s["k"].shape[1:3]
    q = torch.cat([s["q"].float(), torch.zeros(1, H, D, device=dev)])[s["row_of"]] * (1.0 / math.sqrt(D))
    t = torch.arange(s["table"].shape[1] * S, device=dev)
    sees = t <= (s["kv_len"] - s["n_rows"])[:, None, None] + torch.arange(T, device=dev)[:, None]
    return q.view(B, T, Hk, H // Hk, D).transpose(1, 2), sees


def _plain_chunk(s):
    q, sees = _batch(s)
    B, Hk, T, G, D = q.shape
    (R, H, _), P = s["q"].shape, s["prefix_len"]
    pages = s["table"].long()
    held = (torch.arange(sees.shape[2], device=q.device) < s["kv_len"][:, None])[:, None, :, None]
    k, v = _keys(s, "k", pages), torch.where(held, _keys(s, "v", pages), 0.0)
    if P:
        more = [_keys(s, n, s["prefix_table"].long())[:, :P].expand(B, Hk, P, D) for n in ("k", "v")]
        k, v = torch.cat([more[0], k], 2), torch.cat([more[1], v], 2)
        sees = torch.cat([torch.ones(B, T, P, dtype=torch.bool, device=q.device), sees], 2)
    x = (q.reshape(B, Hk, T * G, D) @ k.transpose(2, 3)).view(B, Hk, T, G, -1)
    x.masked_fill_(~sees[:, None, :, None], -math.inf)
    x.sub_(x.amax(-1, keepdim=True)).exp_()
    total = x.sum(-1, keepdim=True)
    o = (x.view(B, Hk, T * G, -1) @ v).view(B, Hk, T, G, D) / total
    out = torch.empty(R + 1, H, D, dtype=s["dtype"], device=q.device)
    out[s["row_of"]] = o.transpose(1, 2).reshape(B, T, H, D).to(s["dtype"])
    return {"o": out[:R]}


def _plain_weigh(s):
    q, sees = _batch(s)
    B, Hk, T, G, D = q.shape
    S, dev = s["k"].shape[2], q.device
    lse = torch.cat([s["lse"], torch.zeros(1, Hk * G, device=dev)])[s["row_of"]].view(B, T, Hk, G).transpose(1, 2)
    counts = torch.arange(T, device=dev) < (s["n_rows"] if s["n_accepted"] is None else s["n_accepted"] + 1)[:, None]
    x = (q.reshape(B, Hk, T * G, D) @ _keys(s, "k", s["table"].long()).transpose(2, 3)).view(B, Hk, T, G, -1)
    x.sub_(lse[..., None]).exp_().masked_fill_(~(sees & counts[..., None])[:, None, :, None], 0.0)
    add = x.sum((2, 3))  # [B, kv_heads, L]
    t = torch.arange(add.shape[2], device=dev)
    b, t = (t < s["kv_len"][:, None]).nonzero(as_tuple=True)
    page, slot = s["table"][b, t // S].long(), t % S
    old = torch.where((t < s["kv_len"][b] - s["n_rows"][b])[:, None], s["mass"][page, :, slot], 0.0)
    s["mass"][page, :, slot] = s["keep"] * old + add[b, :, t]
    return {"mass": s["mass"]}


def _plain_evict(s):
    S, Hk = s["k"].shape[2], s["k"].shape[1]
    n, K = s["kv_len"][:, None, None], s["budget"]
    mass = s["mass"][s["table"].long()].transpose(1, 2).flatten(2)  # [B, kv_heads, L]
    t = torch.arange(mass.shape[2], device=mass.device)
    mass = torch.where((t < s["sinks"]) | (t >= n - s["recent"]), math.inf, mass)
    mass = torch.where(t < n, mass, -1.0)
    best = torch.sort(mass, dim=2, descending=True, stable=True)[1][..., :K]
    if best.shape[2] < K:
        best = torch.nn.functional.pad(best, (0, K - best.shape[2]), value=mass.shape[2])
    kept = torch.where(best < n, best, 1 << 30).sort(-1)[0]
    b, h, j = (kept < (1 << 30)).nonzero(as_tuple=True)
    src = kept[b, h, j]
    old, new = s["table"][b, src // S].long(), s["new_table"][b, j // S].long()
    for x in (s["k"].view(torch.uint8), s["v"].view(torch.uint8), s["k_exp"], s["v_exp"], s["mass"]):
        x[new, h, j % S] = x[old, h, src % S]
    return {"kept": torch.where(kept < (1 << 30), kept, -1).int(), "kv_len": s["kv_len"].clamp(max=K), "mass": s["mass"],
            **_pool(s, "k", "v", "k_exp", "v_exp")}


def run(s):
    if not own:
        if s["op"] == "rope":
            return {n: x.to(s["dtype"]) for n, x in zip(("q", "k"), _plain_rope(s))}
        return {"append": _plain_append, "chunk": _plain_chunk, "weigh": _plain_weigh, "evict": _plain_evict}[s["op"]](s)
    from speculative_decoding_token_temp_gb300 import api
    if s["op"] in ("rope", "append"):
        if "rope" not in s:
            s["rope"] = api.Rope(s["q"].shape[2], s["q"].device, rot_dim=s["rot"], axis=s["axis"], interleaved=s["interleaved"])
        norm = {"q_weight": s["weights"][0], "k_weight": s["weights"][1], "eps": None if s["weights"][0] is None else EPS}
        if s["op"] == "rope":
            got = api.spec_qk_rope(s["q"], s["new_k"], s["rope"], s["positions"], **norm, out=s["out"])
            return {"q": got["q"], "k": got["k"]}
    if "cache" not in s:
        s["cache"] = api.KVCache(s["k"], s["v"], s["k_exp"], s["v_exp"])
    if s["op"] == "append":
        got = api.spec_qk_rope_append(s["cache"], s["q"], s["new_k"], s["new_v"], s["rope"], s["positions"], s["table"], s["row_seq"],
                                      s["row_pos"], **norm, out=s["out"])
        return {"q": got["q"], **_pool(s, "k", "v", "k_exp", "v_exp")}
    if s["op"] == "chunk":
        got = api.spec_attention_chunk(s["q"], s["cache"], s["table"], s["kv_len"], gamma=s["gamma"], cu_draft=s["cu_draft"],
                                       prefix_table=s["prefix_table"], prefix_len=s["prefix_len"], out=s["out"])
        return {"o": got["o"]}
    if s["op"] == "weigh":
        api.spec_kv_weigh(s["q"], s["cache"], s["table"], s["kv_len"], s["lse"], s["mass"], gamma=s["gamma"], cu_draft=s["cu_draft"],
                          n_accepted=s["n_accepted"], keep=s["keep"], out=s["out"])
        return {"mass": s["mass"]}
    got = api.spec_kv_evict(s["cache"], s["mass"], s["table"], s["kv_len"], s["budget"], sinks=s["sinks"], recent=s["recent"],
                            new_table=s["new_table"], out=s["out"])
    return {"kept": got["kept"], "kv_len": got["kv_len"], "mass": s["mass"], **_pool(s, "k", "v", "k_exp", "v_exp")}


def _e4m3_table(device):
    """The 256 values of the code, from its definition: sign, 4 bits of exponent (bias 7), 3 of fraction; no infinities, two NaNs."""
    v = []
    for b in range(256):
        e, f = b >> 3 & 15, b & 7
        x = math.nan if e == 15 and f == 7 else (f / 8 * 2.0 ** -6 if e == 0 else (1 + f / 8) * 2.0 ** (e - 7))
        v.append(-x if b & 128 else x)
    return torch.tensor(v, dtype=torch.float64, device=device)


def _two(e):
    """2^e in 64 bits, from its bits."""
    return (e.long() + 1023).bitwise_left_shift(52).view(torch.float64)


def _exact_rope(s):
    """Queries and keys after norm and rotation: complex numbers turned by the angle."""
    p = s["positions"].double().view(s["positions"].shape[0], -1)
    half = s["rot"] // 2
    turn = []
    for j in range(half):
        a = p[:, s["axis"][j]] * 10000.0 ** (-2.0 * j / s["rot"])
        turn.append(torch.complex(torch.cos(a), torch.sin(a)))
    turn = torch.stack(turn, 1)[:, None]
    got = []
    for x, w in ((s["q"], s["weights"][0]), (s["new_k"], s["weights"][1])):
        y = x.double()
        if w is not None:
            y = y / torch.sqrt((y * y).sum(-1, keepdim=True) / y.shape[-1] + EPS) * w.double()
        i = torch.arange(half, device=y.device)
        a, b = (2 * i, 2 * i + 1) if s["interleaved"] else (i, i + half)
        z = torch.complex(y[..., a], y[..., b]) * turn
        y[..., a], y[..., b] = z.real, z.imag
        got.append(y)
    return got


def _exact_append(s):
    dev, S = s["table"].device, s["k"].shape[2]
    value = _e4m3_table(dev)
    q, k = _exact_rope(s)
    at = torch.nonzero(s["row_pos"] >= 0)[:, 0]
    b, t = s["row_seq"][at].long(), s["row_pos"][at].long()
    page, slot = s["table"][b, t // S].long(), t % S
    grid = torch.sort(value[:127])[0]
    out = {"q": q}
    for n, new in (("k", k), ("v", s["new_v"])):
        codes, exps = value[s[n].view(torch.uint8).int()], _two(s[n + "_exp"].long() - 127)
        for part in torch.arange(at.numel(), device=dev).split(4096):
            x = new[at[part]].double()
            most = x.abs().amax(-1, keepdim=True)
            e = torch.ceil(torch.log2(most.clamp(min=2.0 ** -140) / 448))
            e = torch.where(most <= 448 * _two(e - 1), e - 1, torch.where(most > 448 * _two(e), e + 1, e)).clamp(min=-100)
            y = torch.where(most > 0, x * _two(-e), x)
            hi = torch.searchsorted(grid, y.abs().contiguous()).clamp(1, 126)
            below, above = grid[hi - 1], grid[hi]
            up = (y.abs() - below > above - y.abs()) | ((y.abs() - below == above - y.abs()) & (hi % 2 == 0))
            codes[page[part], :, slot[part]] = torch.where(up, above, below) * torch.sign(y)
            exps[page[part], :, slot[part]] = torch.where(most > 0, _two(e), 2.0 ** -60)[..., 0]
        out[n], out[n + "_exp"] = codes, exps
    return out


def _exact_tokens(s, n, pages, count):
    """The first `count` vectors of some pages, [kv_heads, count, dim]."""
    x = _e4m3_table(pages.device)[s[n].view(torch.uint8)[pages].int()] * _two(s[n + "_exp"][pages].long() - 127)[..., None]
    return x.permute(1, 0, 2, 3).reshape(x.shape[1], -1, x.shape[3])[:, :count]


def _exact_scores(s, r0, T, k, before):
    """Scores of one sequence's T rows against its keys, [kv_heads, G, T, tokens]; -inf where a row comes before a token."""
    H, D = s["q"].shape[1:]
    Hk = k.shape[0]
    q = s["q"][r0:r0 + T].double().view(T, Hk, H // Hk, D).permute(1, 2, 0, 3)
    x = torch.matmul(q, k.unsqueeze(1).transpose(-1, -2)) / math.sqrt(D)
    return x.masked_fill_(torch.ones(T, k.shape[1], dtype=torch.bool, device=k.device).triu(before + 1), -math.inf)


def exact(c, seed):
    s = prepare(c, seed)
    if c["op"] == "rope":
        return dict(zip(("q", "k"), _exact_rope(s)))
    if c["op"] == "append":
        return _exact_append(s)
    S, D, Hk = c["page"], c["dim"], c["kv_heads"]
    dev = s["table"].device
    if c["op"] == "evict":
        value = _e4m3_table(dev)
        mass = s["mass"].double()
        old = {n: value[s[n].view(torch.uint8).int()] for n in ("k", "v")} | {n: _two(s[n].long() - 127) for n in ("k_exp", "v_exp")}
        new = {n: x.clone() for n, x in old.items()}
        new["mass"] = mass.clone()
        for b, n in enumerate(s["kv_len"].tolist()):
            t = torch.arange(n, device=dev)
            place = s["table"][b, t // S].long()
            for h in range(Hk):
                free = t[s["sinks"]:max(n - s["recent"], s["sinks"])]
                take = min(n, c["budget"]) - (n - free.numel())
                m = mass[place, h, t % S][free]
                if take < free.numel():  # the border: all above it, of those on it the earliest
                    border = m.sort()[0][free.numel() - take] if take > 0 else math.inf
                    on = (m == border).nonzero()[:, 0]
                    stay = m > border
                    stay[on[:take - int(stay.sum())]] = True
                    free = free[stay]
                if n <= c["budget"]:
                    free = t[s["sinks"]:max(n - s["recent"], s["sinks"])]
                kept = torch.cat([t[:s["sinks"]], free, t[max(n - s["recent"], s["sinks"]):]])
                j = torch.arange(kept.numel(), device=dev)
                a, z = (place[kept], h, kept % S), (s["new_table"][b, j // S].long(), h, j % S)
                for name, x in new.items():
                    x[z] = (mass if name == "mass" else old[name])[a]
        return {"kept": None, "kv_len": None, **new}
    r0 = 0
    o = torch.empty(s["q"].shape, dtype=torch.float64, device=dev)
    mass = s["mass"].double() if c["op"] == "weigh" else None
    for b, (T, n) in enumerate(zip(s["rows"], s["kv_len"].tolist())):
        pages = s["table"][b, :-(-n // S)].long()
        k = _exact_tokens(s, "k", pages, n)
        if mass is not None:
            x = _exact_scores(s, r0, T, k, n - T)
            count = T if s["n_accepted"] is None else int(s["n_accepted"][b]) + 1
            w = (x - s["lse"][r0:r0 + T].double().view(T, Hk, -1).permute(1, 2, 0)[..., None]).exp()[:, :, :count].sum((1, 2))
            t = torch.arange(n, device=dev)
            place = (pages[t // S], slice(None), t % S)
            mass[place] = w.T + torch.where(t < n - T, c["keep"], 0.0)[:, None] * mass[place]
        else:
            v, P = _exact_tokens(s, "v", pages, n), s["prefix_len"]
            if P:
                k, v = (torch.cat([_exact_tokens(s, name, s["prefix_table"].long(), P), x], 1) for name, x in (("k", k), ("v", v)))
            for h in range(Hk):
                G = s["q"].shape[1] // Hk
                part = {"q": s["q"][:, h * G:(h + 1) * G]}
                w = torch.softmax(_exact_scores(part, r0, T, k[h:h + 1], P + n - T), -1)
                o[r0:r0 + T, h * G:(h + 1) * G] = torch.matmul(w, v[h])[0].transpose(0, 1)
        r0 += T
    return {"mass": mass} if mass is not None else {"o": o}
