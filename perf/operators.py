"""Cases of the score-modified attention, rotary and 8-bit cache operators.

Each case is one pass through one operator as a training or serving program
calls it: rotary positions and their tables, attention with capped or biased
scores and row masks (forward, and forward with backward), appending tokens to
a block-quantised cache, and attention of single tokens over that cache.
"""
import math

import torch

own = False

DT = {"bf16": torch.bfloat16, "fp16": torch.float16}
BLOCK = 128  # cache tokens that share one scale


# ------------------------------------------------------------------ the cases

def listed():
    return [
        # rotary positions of one new token of each of 32 running sequences, 32 query and 8 key heads together
        {"name": "rope_token", "kind": "rope", "B": 32, "H": 40, "N": 1, "d": 128, "rot": 128, "interleaved": False,
         "inverse": False, "token_major": False, "far": 32768, "dtype": "bf16"},
        # backward through the rotation of half of each head over a long training batch, into the projection's layout
        {"name": "rope_grad", "kind": "rope", "B": 2, "H": 32, "N": 8192, "d": 128, "rot": 64, "interleaved": True,
         "inverse": True, "token_major": True, "far": 0, "dtype": "fp16"},
        # the cosine and sine tables of a 131072-token context with stretched low frequencies
        {"name": "rope_tables", "kind": "tables", "positions": 131072, "first": 0, "rot": 128, "stretch": 32.0},
        # a short prompt: latency
        {"name": "fwd_short", "kind": "fwd", "B": 1, "Hq": 2, "Hkv": 2, "N": 256, "d": 64, "dtype": "bf16", "cap": 30.0,
         "slopes": False, "docs": 0, "prefix": 0, "window": -1, "causal": True, "pad": False, "gain": 2.0},
        # prompts of a model with capped scores: the grouped-query causal configuration
        {"name": "fwd_cap", "kind": "fwd", "B": 2, "Hq": 32, "Hkv": 8, "N": 8192, "d": 128, "dtype": "bf16", "cap": 50.0,
         "slopes": False, "docs": 0, "prefix": 0, "window": -1, "causal": True, "pad": False, "gain": 4.0},
        # documents packed into one long row, scores falling with the distance
        {"name": "fwd_docs", "kind": "fwd", "B": 1, "Hq": 16, "Hkv": 16, "N": 16384, "d": 64, "dtype": "fp16", "cap": 0.0,
         "slopes": True, "docs": 12, "prefix": 0, "window": -1, "causal": True, "pad": False, "gain": 1.0},
        # a training step over packed documents with capped scores
        {"name": "train_docs", "kind": "train", "B": 1, "Hq": 32, "Hkv": 8, "N": 8192, "d": 128, "dtype": "bf16",
         "cap": 50.0, "slopes": False, "docs": 5, "prefix": 0, "window": -1, "causal": True, "pad": False, "gain": 2.0},
        # a training step of a prefix model on a padded batch of odd length, with a distance bias
        {"name": "train_prefix", "kind": "train", "B": 3, "Hq": 8, "Hkv": 8, "N": 1111, "d": 64, "dtype": "fp16",
         "cap": 0.0, "slopes": True, "docs": 0, "prefix": 300, "window": -1, "causal": True, "pad": True, "gain": 1.0},
        # one new token of each of 64 sequences into a paged cache, keys rotated on the way
        {"name": "append_token", "kind": "append", "B": 64, "Hkv": 8, "d": 128, "room": 4096, "new": 1, "paged": True,
         "rot": 128, "interleaved": False, "dtype": "bf16"},
        # a ragged piece of prompt for each of 8 sequences into a contiguous cache
        {"name": "append_prompt", "kind": "append", "B": 8, "Hkv": 8, "d": 128, "room": 8192, "new": 4000, "paged": False,
         "rot": 64, "interleaved": True, "dtype": "bf16"},
        # a decode step over long contiguous caches of equal length
        {"name": "decode_long", "kind": "decode", "B": 16, "Hq": 32, "Hkv": 8, "d": 128, "room": 32768, "ragged": False,
         "paged": False, "cap": 0.0, "slopes": False, "window": -1, "dtype": "bf16"},
        # a decode step over a paged cache of ragged lengths, capped scores and a distance bias
        {"name": "decode_paged", "kind": "decode", "B": 37, "Hq": 32, "Hkv": 4, "d": 128, "room": 4500, "ragged": True,
         "paged": True, "cap": 50.0, "slopes": True, "window": -1, "dtype": "fp16"},
    ]


def _spread(rng, lo, hi):
    """A whole number from lo to hi, even over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["rope", "tables", "fwd", "fwd", "train", "train", "append", "decode", "decode"])
    dtype, d = rng.choice(["bf16", "fp16"]), rng.choice([64, 128, 128, 256])
    if kind == "rope":
        N = _spread(rng, 1, 16384)
        H = rng.choice([1, 5, 8, 32, 40])
        return {"kind": kind, "B": _spread(rng, 1, max(1, min(64, 2 ** 19 // (N * H)))), "H": H, "N": N, "d": d,
                "rot": rng.choice([16, 32, d // 2, d]), "interleaved": rng.random() < 0.5, "inverse": rng.random() < 0.5,
                "token_major": rng.random() < 0.5, "far": rng.choice([0, 1000, 100000]), "dtype": dtype}
    if kind == "tables":
        return {"kind": kind, "positions": _spread(rng, 1, 131072), "first": rng.choice([0, 7, 1 << 20]),
                "rot": rng.choice([16, 64, 128]), "stretch": rng.choice([1.0, 4.0, 32.0])}
    if kind in ("fwd", "train"):
        Hkv, group = rng.choice([1, 2, 3, 8]), rng.choice([1, 1, 2, 4])
        Hq = Hkv * group
        N = _spread(rng, 1, 8192 if kind == "fwd" else 4096)
        most = (2 ** 31 if kind == "fwd" else 2 ** 29) // (N * N * Hq * d // 64)
        B = _spread(rng, 1, max(1, min(8, most)))
        docs = rng.choice([0, 0, 1, 3, 9])
        causal = rng.random() < 0.7
        return {"kind": kind, "B": B, "Hq": Hq, "Hkv": Hkv, "N": N, "d": d, "dtype": dtype, "cap": rng.choice([0.0, 20.0, 50.0]),
                "slopes": rng.random() < 0.4, "docs": min(docs, N), "prefix": rng.choice([0, N // 3]) if causal else 0,
                "window": rng.choice([-1, -1, N // 4]), "causal": causal, "pad": rng.random() < 0.3, "gain": rng.choice([1.0, 2.0])}
    if kind == "append":
        room = _spread(rng, 200, 8192)
        return {"kind": kind, "B": _spread(rng, 1, max(1, min(64, 65536 // room))), "Hkv": rng.choice([1, 2, 8]), "d": d, "room": room,
                "new": _spread(rng, 1, max(1, room // 2)), "paged": rng.random() < 0.5, "rot": rng.choice([0, 16, d // 2, d]),
                "interleaved": rng.random() < 0.5, "dtype": dtype}
    Hkv, group = rng.choice([1, 2, 8]), rng.choice([1, 2, 4, 7, 8, 16, 20])
    room = _spread(rng, 1, 32768)
    return {"kind": kind, "B": _spread(rng, 1, max(1, min(64, 2 ** 22 // (room * Hkv)))), "Hq": Hkv * group, "Hkv": Hkv, "d": d, "room": room,
            "ragged": rng.random() < 0.6, "paged": rng.random() < 0.5, "cap": rng.choice([0.0, 50.0]), "slopes": rng.random() < 0.4,
            "window": rng.choice([-1, -1, max(0, room // 3)]), "dtype": dtype}


# ----------------------------------------------------------------- the inputs

def _slopes(H):
    return torch.tensor([2.0 ** (-8.0 * (h + 1) / H) for h in range(H)], dtype=torch.float32, device="cuda")


def _inv_freq(rot, stretch):
    """Frequencies 10000^(-2i/rot), the slow ones stretched for long contexts, in 64 bits."""
    i = torch.arange(rot // 2, dtype=torch.float64)
    f = 10000.0 ** (-2.0 * i / rot)
    if stretch > 1.0:
        turns = 4096.0 * f / (2.0 * math.pi)
        keep = ((turns - 1.0) / 31.0).clamp(0.0, 1.0)
        f = f / stretch * (1.0 - keep) + f * keep
    return f.cuda()


def _trig(first, positions, rot, device):
    a = torch.arange(first, first + positions, dtype=torch.float64, device=device)[:, None] * _inv_freq(rot, 1.0)[None, :]
    return a.cos().float().contiguous(), a.sin().float().contiguous()


def _cuts(g, N, docs, pad):
    """Document numbers of N rows: `docs` runs at random cuts, and -1 behind a random length where the row is padded."""
    ids = torch.zeros(N, dtype=torch.int32, device="cuda")
    if docs > 1 and N > 1:
        at = torch.randint(1, N, (docs - 1,), generator=g, device="cuda")
        step = torch.zeros(N, dtype=torch.int32, device="cuda")
        step[at] = 1
        ids = step.cumsum(0, dtype=torch.int32)
    if pad:
        n = int(torch.randint(max(1, N // 2), N + 1, (1,), generator=g, device="cuda"))
        ids[n:] = -1
    return ids


def _codes(x):
    """[..., rows, d] in blocks of 128 rows -> E4M3 values and factors: x * 2^e with the largest e that keeps the block within 448."""
    *lead, rows, d = x.shape
    nb = -(-rows // BLOCK)
    x = torch.nn.functional.pad(x, (0, 0, 0, nb * BLOCK - rows)).reshape(*lead, nb, BLOCK, d)
    e = _exponent(x.abs().amax((-1, -2)))
    x8 = (x * torch.exp2(e)[..., None, None]).to(torch.float8_e4m3fn).reshape(*lead, nb * BLOCK, d)[..., :rows, :]
    return x8.contiguous(), torch.exp2(-e).contiguous()


def _exponent(amax):
    m, k = torch.frexp(amax)
    e = torch.where(m <= 0.875, 9 - k, 8 - k).to(amax.dtype)
    return torch.where(amax > 0, e, torch.zeros_like(e))


def _cache(c, g):
    """A cache's codes and factors, filled with keys and values, and its block table where it is paged."""
    B, H, d, room = c["B"], c["Hkv"], c["d"], c["room"]
    nb = -(-room // BLOCK)
    rows = room if not c["paged"] else BLOCK
    lead = (B, H) if not c["paged"] else (B * nb, H)
    parts = []
    for _ in range(2):
        x8 = torch.empty(*lead, rows, d, dtype=torch.float8_e4m3fn, device="cuda")
        s = torch.empty(*lead, -(-rows // BLOCK), device="cuda")
        for at in range(0, lead[0], 64):  # in pieces: the floats are four times the codes
            n = min(64, lead[0] - at)
            x8[at:at + n], s[at:at + n] = _codes(torch.randn(n, H, rows, d, generator=g, device="cuda"))
        parts += [x8.view(torch.uint8), s if not c["paged"] else s[..., 0].contiguous()]
    table = torch.randperm(B * nb, generator=g, device="cuda").to(torch.int32).reshape(B, nb) if c["paged"] else None
    return parts[0], parts[2], parts[1], parts[3], table


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = {"case": c}

    def normal(*shape, gain=1.0):
        return (torch.randn(*shape, generator=g, device="cuda") * gain).to(DT[c["dtype"]])

    if c["kind"] == "rope":
        B, H, N, d = c["B"], c["H"], c["N"], c["d"]
        s["x"], s["y"] = normal(B, H, N, d), torch.empty(B, H, N, d, dtype=DT[c["dtype"]], device="cuda")
        if c["token_major"]:  # the projection's layout on its side: read by the forward, written by the backward
            side = "y" if c["inverse"] else "x"
            s[side] = s[side].transpose(1, 2).contiguous().transpose(1, 2)
        s["positions"] = None
        if c["far"]:
            s["positions"] = (torch.randint(0, c["far"], (B, 1), generator=g, device="cuda")
                              + torch.arange(N, device="cuda")).to(torch.int32)
        s["cos"], s["sin"] = _trig(0, c["far"] + N, c["rot"], "cuda")
    elif c["kind"] == "tables":
        # another model's frequencies for each seed: its base, as a factor on them
        s["inv_freq"] = _inv_freq(c["rot"], c["stretch"]) * (0.5 + torch.rand(1, generator=g, device="cuda", dtype=torch.float64))
        shape = (c["positions"], c["rot"] // 2)
        s["cos"], s["sin"] = torch.empty(shape, device="cuda"), torch.empty(shape, device="cuda")
    elif c["kind"] in ("fwd", "train"):
        B, Hq, Hkv, N, d = c["B"], c["Hq"], c["Hkv"], c["N"], c["d"]
        s["q"], s["k"], s["v"] = normal(B, Hq, N, d, gain=c["gain"]), normal(B, Hkv, N, d), normal(B, Hkv, N, d)
        s["slopes"] = _slopes(Hq) if c["slopes"] else None
        s["docs"] = torch.stack([_cuts(g, N, c["docs"], c["pad"]) for _ in range(B)]) if c["docs"] or c["pad"] else None
        s["prefix"] = torch.randint(0, c["prefix"] + 1, (B,), generator=g, device="cuda", dtype=torch.int32) if c["prefix"] else None
        if c["kind"] == "train":
            s["dout"] = normal(B, Hq, N, d)
    elif c["kind"] == "append":
        B, H, d, new, room = c["B"], c["Hkv"], c["d"], c["new"], c["room"]
        s["k8"], s["v8"], s["sk"], s["sv"], s["table"] = _cache(c, g)
        s["k"], s["v"] = (normal(B, new, H, d).transpose(1, 2) for _ in range(2))  # as a projection leaves them
        s["seqlens"] = torch.randint(0, room - new + 1, (B,), generator=g, device="cuda", dtype=torch.int32)
        s["new_lens"] = torch.randint((new + 1) // 2, new + 1, (B,), generator=g, device="cuda", dtype=torch.int32) if new > 1 else None
        s["cos"], s["sin"] = _trig(0, room, c["rot"], "cuda") if c["rot"] else (None, None)
    else:
        B, Hq, d, room = c["B"], c["Hq"], c["d"], c["room"]
        s["k8"], s["v8"], s["sk"], s["sv"], s["table"] = _cache(c, g)
        s["q"] = normal(B, Hq, d)
        s["seqlens"] = torch.full((B,), room, dtype=torch.int32, device="cuda")
        if c["ragged"]:
            s["seqlens"] = torch.randint(0, room + 1, (B,), generator=g, device="cuda", dtype=torch.int32)
        s["slopes"] = _slopes(Hq) if c["slopes"] else None
    return s


# --------------------------------------------------------------- the operators

def run(state):
    return _own(state) if own else _plain(state)


def _own(s):
    from exact_attention_73_gb300 import binding as L
    c = s["case"]
    if c["kind"] == "rope":
        L.attn_rope(s["x"], s["y"], s["cos"], s["sin"], positions=s["positions"], interleaved=c["interleaved"],
                    inverse=c["inverse"])
        return s["y"]
    if c["kind"] == "tables":
        L.attn_rope_tables(s["cos"], s["sin"], s["inv_freq"], first_position=c["first"])
        return s["cos"], s["sin"]
    if c["kind"] in ("fwd", "train"):
        q, k, v = s["q"], s["k"], s["v"]
        B, Hq, N, d = q.shape
        ranges = work_space = None
        if s["docs"] is not None or s["prefix"] is not None:
            ranges = torch.empty(B, N, 2, dtype=torch.int32, device="cuda")
            L.attn_mask_rows(ranges, doc_ids=s["docs"], prefix_lens=s["prefix"], causal=c["causal"])
            work_space = torch.empty(L.attn_score_workspace_size(B, N), dtype=torch.uint8, device="cuda")
        window = (c["window"], 0 if c["causal"] and ranges is None else -1)
        o, lse = torch.empty_like(q), torch.empty(B, Hq, N, device="cuda")
        mods = dict(row_ranges=ranges, slopes=s["slopes"], score_cap=c["cap"], window=window)
        L.attn_fwd_score(q, k, v, o, lse, workspace=work_space, **mods)
        if c["kind"] == "fwd":
            return o, lse
        dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
        ws = torch.empty(L.attn_bwd_score_workspace_size(B, Hq, k.shape[1], N, d), dtype=torch.uint8, device="cuda")
        L.attn_bwd_score(q, k, v, o, lse, s["dout"], dq, dk, dv, ws, **mods)
        return o, lse, dq, dk, dv
    if c["kind"] == "append":
        L.attn_cache_append_fp8(s["k"], s["v"], s["k8"], s["v8"], s["sk"], s["sv"], s["seqlens"], new_lens=s["new_lens"],
                                block_table=s["table"], rope_cos=s["cos"], rope_sin=s["sin"], interleaved=c["interleaved"])
        return s["k8"].view(torch.float8_e4m3fn), s["sk"], s["v8"].view(torch.float8_e4m3fn), s["sv"]
    q = s["q"]
    B, Hq, d = q.shape
    blocks = -(-c["room"] // BLOCK)
    splits = L.attn_decode_cache_fp8_splits(B, Hq, c["Hkv"], blocks)
    o, lse = torch.empty_like(q), torch.empty(B, Hq, device="cuda")
    ws = torch.empty(L.attn_decode_cache_fp8_workspace_size(B, Hq, d, splits), dtype=torch.uint8, device="cuda")
    L.attn_decode_cache_fp8(q, s["k8"], s["v8"], s["sk"], s["sv"], s["seqlens"], o, lse, ws, splits, block_table=s["table"],
                            slopes=s["slopes"], score_cap=c["cap"], window_left=c["window"])
    return o, lse


def _rotate(x, cos, sin, interleaved, inverse=False):
    """Pairs of the first 2 * cos.shape[-1] elements turned; x in 32 bits, cos and sin broadcast over it."""
    half = cos.shape[-1]
    part, rest = x[..., :2 * half], x[..., 2 * half:]
    a, b = (part[..., 0::2], part[..., 1::2]) if interleaved else (part[..., :half], part[..., half:])
    if inverse:
        sin = -sin
    u, w = a * cos - b * sin, b * cos + a * sin
    turned = torch.stack((u, w), -1).flatten(-2) if interleaved else torch.cat((u, w), -1)
    return torch.cat((turned, rest), -1)


def _visible(c, docs, prefix, B, N):
    """[B, N, N] truth values: row i sees key j."""
    i = torch.arange(N, device="cuda")[:, None]
    j = torch.arange(N, device="cuda")[None, :]
    see = (j <= i)[None] if c["causal"] else torch.ones(1, N, N, dtype=torch.bool, device="cuda")
    if prefix is not None:
        see = see | (j[None] < prefix[:, None, None])
    if c["window"] >= 0:
        see = see & (i - j <= c["window"])[None]
    if docs is not None:
        run = (docs[:, 1:] != docs[:, :-1]).cumsum(1)
        run = torch.cat((torch.zeros_like(docs[:, :1], dtype=run.dtype), run), 1)
        see = see & (run[:, :, None] == run[:, None, :]) & (docs >= 0)[:, :, None]
    return see.expand(B, N, N)


def _plain(s):
    c = s["case"]
    if c["kind"] == "rope":
        half = c["rot"] // 2
        at = s["positions"].long() if s["positions"] is not None else torch.arange(c["N"], device="cuda")[None]
        cos, sin = (t[:, :half][at][:, None] for t in (s["cos"], s["sin"]))
        s["y"].copy_(_rotate(s["x"].float(), cos, sin, c["interleaved"], c["inverse"]))
        return s["y"]
    if c["kind"] == "tables":
        a = torch.arange(c["first"], c["first"] + c["positions"], dtype=torch.float64, device="cuda")[:, None] * s["inv_freq"]
        s["cos"].copy_(a.cos())
        s["sin"].copy_(a.sin())
        return s["cos"], s["sin"]
    if c["kind"] in ("fwd", "train"):
        return _plain_attention(s, c)
    if c["kind"] == "append":
        return _plain_append(s, c)
    return _plain_decode(s, c)


def _plain_attention(s, c):
    q, k, v = (s[n].float() for n in ("q", "k", "v"))
    B, Hq, N, d = q.shape
    group = Hq // c["Hkv"]
    k, v = k.repeat_interleave(group, 1), v.repeat_interleave(group, 1)
    scale = 1.0 / math.sqrt(d)
    x = q @ k.transpose(-1, -2) * scale
    slope = None
    if c["cap"] > 0:
        x = torch.tanh(x / c["cap"])
        slope = 1.0 - x * x if c["kind"] == "train" else None
        x = x * c["cap"]
    if s["slopes"] is not None:
        i = torch.arange(N, device="cuda")
        x = x - s["slopes"][:, None, None] * (i[:, None] - i[None, :]).abs()
    see = _visible(c, s["docs"], s["prefix"], B, N)[:, None]
    x = x.masked_fill(~see, -math.inf)
    m = x.amax(-1, keepdim=True)
    p = torch.exp(x - m.masked_fill(m == -math.inf, 0.0))
    l = p.sum(-1, keepdim=True)
    lse = (m + torch.log(l)).squeeze(-1)
    p = p / l.masked_fill(l == 0, 1.0)
    o = p @ v
    out = o.to(s["q"].dtype), lse
    if c["kind"] == "fwd":
        return out
    do = s["dout"].float()
    dv = p.transpose(-1, -2) @ do
    ds = p * (do @ v.transpose(-1, -2) - (do * o).sum(-1, keepdim=True))
    if slope is not None:
        ds = ds * slope
    dq, dk = ds @ k * scale, ds.transpose(-1, -2) @ q * scale
    dk, dv = (t.reshape(B, c["Hkv"], group, N, d).sum(2) for t in (dk, dv))
    return *out, dq.to(s["q"].dtype), dk.to(s["q"].dtype), dv.to(s["q"].dtype)


def _plain_append(s, c):
    B, H, d, new = c["B"], c["Hkv"], c["d"], c["new"]
    start = s["seqlens"].long()
    n = s["new_lens"].long() if s["new_lens"] is not None else torch.full_like(start, new)
    nt = (new + BLOCK - 2) // BLOCK + 1  # blocks that the rows of one sequence can touch
    first = start // BLOCK
    block = first[:, None] + torch.arange(nt, device="cuda")  # [B, nt]
    touched = block <= (start + n - 1)[:, None] // BLOCK
    row = (block[:, :, None] * BLOCK + torch.arange(BLOCK, device="cuda"))  # [B, nt, 128] positions
    old, fresh = row < start[:, None, None], (row >= start[:, None, None]) & (row < (start + n)[:, None, None])
    src = (row - start[:, None, None]).clamp(0, new - 1).reshape(B, nt * BLOCK)
    seq = torch.arange(B, device="cuda")[:, None]
    for name in ("k", "v"):
        x8, sc = s[name + "8"].view(torch.float8_e4m3fn), s["s" + name]
        x = s[name].float()
        if name == "k" and s["cos"] is not None:
            at = (start[:, None] + torch.arange(new, device="cuda")).clamp(max=c["room"] - 1)
            x = _rotate(x, s["cos"][at][:, None], s["sin"][at][:, None], c["interleaved"])
        x = x.transpose(1, 2)[seq, src].reshape(B, nt, BLOCK, H, d).permute(0, 1, 3, 2, 4)  # [B, nt, H, 128, d]
        if s["table"] is not None:
            page = s["table"][seq, block.clamp(max=s["table"].shape[1] - 1)].long()
            held, held_s = x8[page].float(), sc[page]
        else:
            at = row.clamp(max=c["room"] - 1)
            held = x8.transpose(1, 2)[seq[:, :, None], at].permute(0, 1, 3, 2, 4).float()  # [B, nt, H, 128, d]
            held_s = sc.transpose(1, 2)[seq, block.clamp(max=sc.shape[2] - 1)]
        whole = torch.where(old[:, :, None, :, None], held * held_s[..., None, None], torch.where(fresh[:, :, None, :, None], x, 0.0))
        e = _exponent(whole.abs().amax((-1, -2)))
        codes = (whole * torch.exp2(e)[..., None, None]).to(torch.float8_e4m3fn).view(torch.uint8)
        write = ((old | fresh) & touched[:, :, None])
        if s["table"] is not None:
            b, t, r = write.nonzero(as_tuple=True)
            s[name + "8"][page[b, t], :, r] = codes[b, t, :, r]
            b, t = touched.nonzero(as_tuple=True)
            sc[page[b, t]] = torch.exp2(-e)[b, t]
        else:
            b, t, r = write.nonzero(as_tuple=True)
            s[name + "8"][b, :, row[b, t, r]] = codes[b, t, :, r]
            b, t = touched.nonzero(as_tuple=True)
            sc[b, :, block[b, t]] = torch.exp2(-e)[b, t]
    return s["k8"].view(torch.float8_e4m3fn), s["sk"], s["v8"].view(torch.float8_e4m3fn), s["sv"]


def _unpacked(s, c, name, dtype):
    """The cache's values [B, Hkv, rows, d], pages in their sequence's order."""
    x8, sc = s[name + "8"].view(torch.float8_e4m3fn), s["s" + name]
    B, H, d = c["B"], c["Hkv"], c["d"]
    if s["table"] is not None:
        x = x8[s["table"].long()].to(dtype) * sc[s["table"].long()].to(dtype)[..., None, None]  # [B, nb, H, 128, d]
        return x.transpose(1, 2).reshape(B, H, -1, d)
    return x8.to(dtype) * sc.to(dtype).repeat_interleave(BLOCK, 2)[:, :, :c["room"], None]


def _plain_decode(s, c):
    k, v = _unpacked(s, c, "k", torch.float32), _unpacked(s, c, "v", torch.float32)
    B, Hq, d = s["q"].shape
    group = Hq // c["Hkv"]
    x = s["q"].float().reshape(B, c["Hkv"], group, d) @ k.transpose(-1, -2) * (1.0 / math.sqrt(d))
    if c["cap"] > 0:
        x = torch.tanh(x / c["cap"]) * c["cap"]
    j = torch.arange(k.shape[2], device="cuda")
    last = (s["seqlens"].long() - 1)[:, None, None, None]
    if s["slopes"] is not None:
        x = x - s["slopes"].reshape(1, c["Hkv"], group, 1) * (last - j)
    see = j <= last
    if c["window"] >= 0:
        see = see & (last - j <= c["window"])
    x = x.masked_fill(~see, -math.inf)
    m = x.amax(-1, keepdim=True)
    p = torch.exp(x - m.masked_fill(m == -math.inf, 0.0))
    l = p.sum(-1, keepdim=True)
    o = p @ v / l.masked_fill(l == 0, 1.0)
    return o.reshape(B, Hq, d).to(s["q"].dtype), (m + torch.log(l)).reshape(B, Hq)


# --------------------------------------------------------------------- the work

def _seen_share(c):
    """Visible share of the N x N pairs, as expected: d documents at random cuts hold 2 / (d + 1) of the squares' sum."""
    N = c["N"]
    share = 0.5 * (1 + 1 / N) if c["causal"] else 1.0
    if c["prefix"]:
        share += 0.5 * (c["prefix"] / N) ** 2 / 3  # uniform prefix lengths: E[prefix^2] is a third of the square
    if c["docs"] > 1:
        share *= 2 / (c["docs"] + 1)
    if c["window"] >= 0:
        share = min(share, (c["window"] + 1) / N * (1.0 if c["causal"] else 2.0))
    if c["pad"]:
        share *= 7 / 12  # a length uniform over [N / 2, N]
    return share


def work(case):
    c = case
    if c["kind"] == "rope":
        n = c["B"] * c["H"] * c["N"]
        rows = c["B"] * c["N"] if c["far"] else c["N"]
        return {"bytes": 4 * n * c["d"] + 4 * rows * c["rot"] + (4 * rows if c["far"] else 0), "flops": 3 * n * c["rot"]}
    if c["kind"] == "tables":
        return {"bytes": 4 * c["positions"] * c["rot"] + 4 * c["rot"], "flops": c["positions"] * c["rot"]}
    if c["kind"] in ("fwd", "train"):
        B, Hq, Hkv, N, d = c["B"], c["Hq"], c["Hkv"], c["N"], c["d"]
        pairs = B * Hq * N * N * _seen_share(c)
        mask = B * N * 4 if c["docs"] or c["pad"] else 0
        if c["kind"] == "fwd":
            return {"bytes": 2 * B * N * d * (2 * Hq + 2 * Hkv) + 4 * B * Hq * N + mask, "flops": 4 * d * pairs}
        return {"bytes": 2 * B * N * d * (4 * Hq + 4 * Hkv) + 4 * B * Hq * N + mask, "flops": 14 * d * pairs}
    if c["kind"] == "append":
        mean = 0.75 * c["new"] if c["new"] > 1 else 1
        rows = 2 * c["B"] * c["Hkv"]
        # the rows of the first block that were there (64 on average) are read to know whether its factor holds
        return {"bytes": rows * (mean * c["d"] * 3 + 64 * c["d"] + 8 * (mean / BLOCK + 1)) + 4 * c["B"] * mean * c["rot"],
                "flops": rows * mean * c["d"] * 4}
    keys = c["room"] * (0.5 if c["ragged"] else 1.0)
    if c["window"] >= 0:
        keys = min(keys, c["window"] + 1)
    return {"bytes": 2 * c["B"] * c["Hkv"] * keys * c["d"] + 4 * c["B"] * c["Hq"] * c["d"] + 4 * c["B"] * c["Hq"],
            "flops": 4 * c["B"] * c["Hq"] * keys * c["d"]}


# ------------------------------------------------------------- in 64 bits, apart

def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["kind"] == "rope":
        y = s["x"].double().clone()
        half = c["rot"] // 2
        at = s["positions"].long() if s["positions"] is not None else torch.arange(c["N"], device="cuda").expand(c["B"], -1)
        w = torch.complex(s["cos"][at].double(), s["sin"][at].double() * (-1.0 if c["inverse"] else 1.0))[:, None]
        first = slice(0, c["rot"], 2) if c["interleaved"] else slice(0, half)
        second = slice(1, c["rot"], 2) if c["interleaved"] else slice(half, c["rot"])
        z = torch.complex(s["x"][..., first].double(), s["x"][..., second].double()) * w
        y[..., first], y[..., second] = z.real, z.imag
        return y
    if c["kind"] == "tables":
        p = torch.arange(c["first"], c["first"] + c["positions"], dtype=torch.float64, device="cuda")
        z = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"), torch.outer(p, s["inv_freq"]))
        return z.real.contiguous(), z.imag.contiguous()
    if c["kind"] in ("fwd", "train"):
        return _exact_attention(s, c)
    if c["kind"] == "append":
        return _exact_append(s, c)
    return _exact_decode(s, c)


def _exact_rows(c, s, b):
    """The first key and the end of the keys that each row of sequence b sees."""
    N = c["N"]
    i = torch.arange(N, device="cuda")
    lo, hi = torch.zeros(N, dtype=torch.long, device="cuda"), torch.full((N,), N, dtype=torch.long, device="cuda")
    if s["docs"] is not None:
        ids = s["docs"][b].tolist()
        starts, ends = list(range(N)), [0] * N
        for r in range(1, N):
            if ids[r] == ids[r - 1]:
                starts[r] = starts[r - 1]
        for r in range(N - 1, -1, -1):
            ends[r] = ends[r + 1] if r + 1 < N and ids[r] == ids[r + 1] else r + 1
        lo, hi = torch.tensor(starts, device="cuda"), torch.tensor(ends, device="cuda")
    if c["causal"]:
        top = i + 1
        if s["prefix"] is not None:
            top = torch.maximum(top, s["prefix"][b].long())
        hi = torch.minimum(hi, top)
    if c["window"] >= 0:
        lo = torch.maximum(lo, i - c["window"])
    if s["docs"] is not None:
        hi = torch.where(s["docs"][b] < 0, lo, hi)
    return lo[:, None], hi[:, None]


def _exact_attention(s, c):
    q, k, v = s["q"], s["k"], s["v"]
    B, Hq, N, d = q.shape
    group, scale = Hq // c["Hkv"], 1.0 / math.sqrt(d)
    new = lambda t: torch.zeros(t.shape, dtype=torch.float64, device="cuda")  # noqa: E731
    o, lse = new(q), torch.empty(B, Hq, N, dtype=torch.float64, device="cuda")
    dq, dk, dv = (new(q), new(k), new(v)) if c["kind"] == "train" else (None, None, None)
    j = torch.arange(N, device="cuda")[None, :]
    for b in range(B):
        lo, hi = _exact_rows(c, s, b)
        hidden = (j < lo) | (j >= hi)
        empty = hidden.all(1)
        for h in range(Hq):
            n = h // group
            Q, K, V = q[b, h].double(), k[b, n].double(), v[b, n].double()
            x = (Q @ K.T).mul_(scale)
            if c["cap"] > 0:
                t = torch.tanh(x / c["cap"])
                x = t * c["cap"]
            if s["slopes"] is not None:
                x = x - float(s["slopes"][h]) * (j.T - j).abs()
            x[hidden] = -math.inf
            z = torch.logsumexp(x, 1)
            lse[b, h] = z
            z = z.masked_fill(empty, 0.0)
            p = torch.exp(x - z[:, None])
            o[b, h] = p @ V
            if dq is None:
                continue
            G = s["dout"][b, h].double()
            dp = G @ V.T
            ds = p * (dp - (p * dp).sum(1, keepdim=True))
            if c["cap"] > 0:
                ds = ds * (1.0 - t.square())
            dv[b, n] += p.T @ G
            dq[b, h] = ds @ K * scale
            dk[b, n] += ds.T @ Q * scale
    return (o, lse) if dq is None else (o, lse, dq, dk, dv)


def _exact_append(s, c):
    out = []
    start = s["seqlens"].tolist()
    count = s["new_lens"].tolist() if s["new_lens"] is not None else [c["new"]] * c["B"]
    for name in ("k", "v"):
        x8, sc = s[name + "8"].view(torch.float8_e4m3fn).double(), s["s" + name].double()
        for b in range(c["B"]):
            x = s[name][b, :, :count[b]].double()  # [H, n, d]
            if name == "k" and c["rot"]:
                half = c["rot"] // 2
                w = torch.complex(s["cos"], s["sin"])[start[b]:start[b] + count[b]].to(torch.complex128)
                first = slice(0, c["rot"], 2) if c["interleaved"] else slice(0, half)
                second = slice(1, c["rot"], 2) if c["interleaved"] else slice(half, c["rot"])
                z = torch.complex(x[..., first], x[..., second]) * w
                x = x.clone()
                x[..., first], x[..., second] = z.real, z.imag
            for t in range(start[b] // BLOCK, (start[b] + count[b] - 1) // BLOCK + 1):
                lo, hi = max(start[b], t * BLOCK), min(start[b] + count[b], (t + 1) * BLOCK)
                if s["table"] is not None:
                    page = int(s["table"][b, t])
                    codes, at = x8[page], (page, slice(None))
                else:
                    codes, at = x8[b][:, t * BLOCK:(t + 1) * BLOCK], (b, slice(None), t)
                had = codes[:, :lo - t * BLOCK] * sc[at][:, None, None]
                rows = torch.cat((had, x[:, lo - start[b]:hi - start[b]]), 1)  # [H, rows, d]
                a = rows.abs().amax((1, 2))
                e = torch.where(a > 0, torch.floor(torch.log2(448.0 / a.clamp(min=1e-300))), torch.zeros_like(a))
                codes[:, :hi - t * BLOCK] = rows * torch.exp2(e)[:, None, None]
                sc[at] = torch.exp2(-e)
        out += [x8, sc]
    return out[0], out[1], out[2], out[3]


def _exact_decode(s, c):
    k, v = _unpacked(s, c, "k", torch.float64), _unpacked(s, c, "v", torch.float64)
    B, Hq, d = s["q"].shape
    group = Hq // c["Hkv"]
    o, lse = torch.zeros(B, Hq, d, dtype=torch.float64, device="cuda"), torch.full((B, Hq), -math.inf, dtype=torch.float64, device="cuda")
    for b in range(B):
        n = int(s["seqlens"][b])
        lo = max(0, n - 1 - c["window"]) if c["window"] >= 0 else 0
        if n == 0:
            continue
        Q = s["q"][b].double().reshape(c["Hkv"], group, d)
        x = torch.einsum("hgd,hnd->hgn", Q, k[b, :, lo:n]) / math.sqrt(d)
        if c["cap"] > 0:
            x = c["cap"] * torch.tanh(x / c["cap"])
        if s["slopes"] is not None:
            x = x - s["slopes"].double().reshape(c["Hkv"], group, 1) * torch.arange(n - 1 - lo, -1, -1, device="cuda")
        lse[b] = torch.logsumexp(x, -1).reshape(Hq)
        o[b] = torch.einsum("hgn,hnd->hgd", torch.softmax(x, -1), v[b, :, lo:n]).reshape(Hq, d)
    return o, lse
