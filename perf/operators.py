"""Cases of the cache and prompt operators: appending tokens (rotary positions,
bf16 or E4M3 storage), attention of a prompt or an appended chunk over the
cache, reading an E4M3 cache back, and the sparse decode over an E4M3 cache.

``run`` is one pass of one operator: with ``own`` the library's call, else the
same operator in elementary torch operations.  A case names its operator in
``op``; lengths of ragged batches follow from the case alone (``_spread``).
"""

import math

import torch

own = False

_DEV = "cuda" if torch.cuda.is_available() else "cpu"
_B = 64                       # tokens of a block (= a page)
_BASE = 10000.0               # rotary base
_SCALED = dict(factor=8.0, original_context=32768, low=1.0, high=32.0, attention_factor=1.2)


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # one decode step of a batch of 32 at 32k tokens: one token per sequence goes into a page
        # of a paged bf16 cache (the latency of a call is what counts)
        dict(name="append_step_b32", op="append", batch=32, new=1, ragged=False, start=32767,
             hq=32, hkv=8, d=128, rotary=128, interleaved=False, scaled=False, e4m3=False,
             paged=True),
        # a 4096-token append to a long sequence, stored as E4M3, rotary positions scaled for
        # the long context: the chunk-wise prompt of a 256k context
        dict(name="append_chunk_4k_e4m3", op="append", batch=1, new=4096, ragged=False,
             start=258048, hq=64, hkv=8, d=128, rotary=128, interleaved=False, scaled=True,
             e4m3=True, paged=False),
        # packed prompts of different lengths, small heads, half of the head rotated in pairs
        dict(name="append_ragged_d64", op="append", batch=13, new=1531, ragged=True, start=700,
             hq=4, hkv=1, d=64, rotary=32, interleaved=True, scaled=False, e4m3=False,
             paged=True),
        # reading one 4096-token chunk back for its block statistics
        dict(name="read_chunk_4k", op="read", batch=1, blocks=64, hkv=8, d=128, paged=False),
        # reading whole 32k sequences back from pages (attention of a prompt over an E4M3 cache)
        dict(name="read_b4_32k_paged", op="read", batch=4, blocks=512, hkv=8, d=128, paged=True),
        # a short prompt, small heads: the latency of a call
        dict(name="prompt_short_d64", op="prompt", batch=1, new=77, ragged=False, start=0,
             hq=4, hkv=1, d=64, paged=False),
        # packed prompts of different lengths, nothing in the cache before them
        dict(name="prompt_ragged_4k", op="prompt", batch=6, new=4099, ragged=True, start=0,
             hq=32, hkv=8, d=128, paged=True),
        # the last 4096-token chunk of a 32k prompt
        dict(name="prompt_chunk_4k_at_28k", op="prompt", batch=1, new=4096, ragged=False,
             start=28672, hq=32, hkv=8, d=128, paged=False),
        # a few new tokens over a long context: few rows, a long axis
        dict(name="prompt_16_at_128k", op="prompt", batch=1, new=16, ragged=False, start=131041,
             hq=64, hkv=8, d=128, paged=False),
        # single tokens of a ragged batch over pages (dense decode beside the sparse one)
        dict(name="prompt_single_b32", op="prompt", batch=32, new=1, ragged=True, start=8191,
             hq=32, hkv=8, d=128, paged=True),
        # one sequence at 32k tokens: the latency of a step
        dict(name="decode_e4m3_single_32k", op="decode", batch=1, length=32768, ragged=False,
             hq=16, hkv=4, d=128, top_k=16, local=8, paged=False),
        # the throughput setting: 32 sequences of 32k tokens
        dict(name="decode_e4m3_b32_32k", op="decode", batch=32, length=32768, ragged=False,
             hq=32, hkv=8, d=128, top_k=16, local=8, paged=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


_HEADS = [(4, 1, 64), (8, 8, 64), (16, 4, 128), (32, 8, 128), (64, 8, 128), (8, 4, 128),
          (8, 8, 128)]


def draw(rng):
    hq, hkv, d = rng.choice(_HEADS)
    op = rng.choice(["append", "read", "prompt", "decode"])
    paged, ragged = rng.random() < 0.5, rng.random() < 0.5
    if op == "append":
        new = 1 if rng.random() < 0.3 else _log(rng, 2, 4096)
        batch = min(_log(rng, 1, 48), max(1, 8192 // new))
        rotary = rng.choice([d, d, d // 2, d // 4])
        return dict(op=op, batch=batch, new=new, ragged=ragged, start=_log(rng, 1, 250000),
                    hq=hq, hkv=hkv, d=d, rotary=rotary, interleaved=rng.random() < 0.5,
                    scaled=rng.random() < 0.5, e4m3=rng.random() < 0.5, paged=True)
    if op == "read":
        blocks = _log(rng, 1, 512)
        return dict(op=op, batch=min(_log(rng, 1, 8), max(1, 2048 // blocks)), blocks=blocks,
                    hkv=hkv, d=d, paged=paged)
    if op == "prompt":
        new = 1 if rng.random() < 0.3 else _log(rng, 2, 4096)
        start = _log(rng, 1, 100000)
        cost = 4096 * 28672 * 32 / 4          # scores of a pass, a quarter of the largest
        start = max(1, min(start, int(cost / (new * hq)) - new))
        batch = max(1, min(_log(rng, 1, 24), int(cost / (new * hq * (new + start))),
                           int(1.5e8 / ((new + start) * hkv * d))))
        return dict(op=op, batch=batch, new=new, ragged=ragged, start=start, hq=hq, hkv=hkv,
                    d=d, paged=paged)
    length = _log(rng, 3000, 100000)
    batch = max(1, min(_log(rng, 1, 32), int(5e8 / (length * hkv * d))))
    return dict(op=op, batch=batch, length=length, ragged=ragged, hq=hq, hkv=hkv, d=d,
                top_k=rng.randint(1, 32 if length > 8000 else 8), local=rng.randint(1, 8),
                paged=paged)


def _spread(n, most, least, ragged):
    """n lengths in [least, most], the first of them `most`."""
    if not ragged:
        return [most] * n
    return [most if i == 0 else
            least + int((most - least + 1) * ((0.6180339887498949 * i) % 1.0)) for i in range(n)]


def _new(c):
    return _spread(c["batch"], c["new"], 1, c["ragged"])


def _starts(c):
    return _spread(c["batch"], c["start"], c["start"] // 2, c["ragged"])


def _lengths(c):
    """Tokens of every sequence once the new ones are in (prompt), or at the step (decode)."""
    if c["op"] == "decode":
        return _spread(c["batch"], c["length"], (3 * c["length"]) // 4, c["ragged"])
    return [s + n for s, n in zip(_starts(c), _new(c))]


def _n_sel(c):
    return 1 + c["top_k"] + c["local"]


def work(case):
    c = case
    op, d, hkv = c["op"], c["d"], c["hkv"]
    if op == "read":
        rows = c["batch"] * c["blocks"] * _B * hkv * 2
        return dict(bytes=rows * (d + 4 + 2 * d), flops=rows * d)
    hq, lens = c["hq"], _lengths(c)
    if op == "append":
        n = sum(_new(c))
        stored = (d + 4) if c["e4m3"] else 2 * d
        return dict(bytes=n * (2 * d * (2 * hq + 2 * hkv) + 2 * hkv * stored),
                    flops=n * 3 * c["rotary"] * (hq + hkv))
    if op == "prompt":
        new = _new(c)
        n = sum(new)
        pairs = sum(k * (length - k) + k * (k + 1) // 2 for k, length in zip(new, lens))
        return dict(bytes=n * hq * (4 * d + 4) + sum(lens) * hkv * 4 * d,
                    flops=4 * d * hq * pairs)
    tail = sum((length - 1) % _B + 1 for length in lens)
    tokens = (c["batch"] * (_n_sel(c) - 1) * _B + tail) * hkv
    return dict(bytes=tokens * 2 * (d + 4) + c["batch"] * (hq * (6 * d + 4) + hkv * _n_sel(c) * 4),
                flops=4 * d * tokens * (hq // hkv))


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _ints(v, dtype):
    return torch.tensor(v, dtype=dtype, device=_DEV)


def _rows(g, *shape):
    """Token rows as projections give them: a mean per head and unequal channels."""
    x = torch.randn(shape, generator=g, device=_DEV, dtype=torch.float32)
    x += 0.5 * torch.randn(shape[-2:], generator=g, device=_DEV)
    x *= torch.rand(shape[-1], generator=g, device=_DEV) * 1.5 + 0.25
    return x.to(torch.bfloat16)


def _blocks(g, *shape):
    """Cache rows [.., token, d]: a mean per block of 64 tokens, unequal spreads."""
    x = torch.randn(shape, generator=g, device=_DEV, dtype=torch.bfloat16)
    n = shape[-2] // _B
    m = 0.5 * torch.randn(shape[:-2] + (n, 1, shape[-1]), generator=g, device=_DEV,
                          dtype=torch.bfloat16)
    s = torch.rand(shape[:-2] + (n, 1, 1), generator=g, device=_DEV).to(torch.bfloat16) + 0.5
    x.view(m.shape[:-2] + (_B, shape[-1])).mul_(s).add_(m)
    return x


def _coded(x):
    """A cache that holds E4M3 codes and one scale per row."""
    top = torch.linalg.vector_norm(x, float("inf"), dim=-1, dtype=torch.float32)
    scale = top / 448.0
    return (x / scale.unsqueeze(-1)).to(torch.float8_e4m3fn), scale


def _table(g, counts, width, n_pages):
    """Block table [batch][width]: sequence b's blocks in counts[b] = (first, last) get pages
    in random order; the others have none (-1)."""
    order = torch.randperm(n_pages, generator=g, device=_DEV).to(torch.int32)
    table = torch.full((len(counts), width), -1, dtype=torch.int32, device=_DEV)
    used = 0
    for b, (first, last) in enumerate(counts):
        table[b, first:last] = order[used:used + last - first]
        used += last - first
    return table


def prepare(case, seed):
    c = case
    g = torch.Generator(device=_DEV)
    g.manual_seed(int(seed))
    op, batch, hkv, d = c["op"], c["batch"], c["hkv"], c["d"]
    s = dict(case=c)
    if op == "append":
        new, starts = _new(c), _starts(c)
        n, hq = sum(new), c["hq"]
        # the fused projection's output: q, k and v of a token side by side
        s["qkv"] = _rows(g, n, hq + 2 * hkv, d)
        s["cu"] = _ints([sum(new[:b]) for b in range(batch + 1)], torch.int32)
        s["start"] = _ints(starts, torch.int64)
        s["q_out"] = torch.zeros(n, hq, d, dtype=torch.bfloat16, device=_DEV)
        cap = -(-max(a + k for a, k in zip(starts, new)) // _B) * _B
        s["cap"] = cap
        if c["paged"]:
            spans = [(a // _B, -(-(a + k) // _B)) for a, k in zip(starts, new)]
            pages = sum(y - x for x, y in spans)
            s["table"] = _table(g, spans, cap // _B, pages)
            shape = (pages, hkv, _B)
        else:
            shape = (batch, hkv, cap)
        kind = torch.uint8 if c["e4m3"] else torch.bfloat16
        s["k"] = torch.zeros(shape + (d,), dtype=kind, device=_DEV)
        s["v"] = torch.zeros(shape + (d,), dtype=kind, device=_DEV)
        if c["e4m3"]:
            s["ks"] = torch.zeros(shape, dtype=torch.float32, device=_DEV)
            s["vs"] = torch.zeros(shape, dtype=torch.float32, device=_DEV)
    elif op == "read":
        nb = c["blocks"]
        if c["paged"]:
            s["table"] = _table(g, [(0, nb)] * batch, nb, batch * nb)
            shape = (batch * nb, hkv, _B, d)
        else:
            shape = (batch, hkv, nb * _B, d)
        s["cap"] = nb * _B
        (s["k"], s["ks"]), (s["v"], s["vs"]) = _coded(_blocks(g, *shape)), _coded(_blocks(g, *shape))
        s["out"] = [torch.zeros(batch * nb, hkv, _B, d, dtype=torch.bfloat16, device=_DEV)
                    for _ in range(2)]
    else:
        lens = _lengths(c)
        cap = -(-max(lens) // _B) * _B
        s["cap"] = cap
        if c["paged"]:
            spans = [(0, -(-length // _B)) for length in lens]
            pages = sum(y for _, y in spans)
            s["table"] = _table(g, spans, cap // _B, pages)
            shape = (pages, hkv, _B, d)
        else:
            shape = (batch, hkv, cap, d)
        k, v = _blocks(g, *shape), _blocks(g, *shape)
        s["lens"] = _ints(lens, torch.int64)
        if op == "prompt":
            new = _new(c)
            s["k"], s["v"] = k, v
            s["q"] = _rows(g, sum(new), c["hq"], d)
            s["cu"] = _ints([sum(new[:b]) for b in range(batch + 1)], torch.int32)
            s["out"] = torch.zeros_like(s["q"])
            s["lse"] = torch.zeros(s["q"].shape[:2], dtype=torch.float32, device=_DEV)
        else:
            (s["k"], s["ks"]), (s["v"], s["vs"]) = _coded(k), _coded(v)
            s["q"] = _rows(g, batch, c["hq"], d)
            # the sink block, top_k blocks anywhere between, the local window
            last = -(-s["lens"] // _B)
            first_local = (last - c["local"]).view(batch, 1, 1)
            j = torch.arange(cap // _B, device=_DEV)
            rank = torch.rand(batch, hkv, cap // _B, generator=g, device=_DEV)
            rank = rank.masked_fill((j < 1) | (j >= first_local), 2.0)
            mid = rank.argsort(-1)[..., :c["top_k"]]
            local = (first_local + torch.arange(c["local"], device=_DEV)).expand(batch, hkv, -1)
            s["idx"] = torch.cat([torch.zeros_like(mid[..., :1]), mid, local], -1) \
                .sort(-1).values.to(torch.int32).contiguous()
            s["n_sel"] = torch.full((batch, hkv), _n_sel(c), dtype=torch.int32, device=_DEV)
            s["out"] = torch.zeros(batch, c["hq"], d, dtype=torch.float32, device=_DEV)
            s["lse"] = torch.zeros(batch, c["hq"], dtype=torch.float32, device=_DEV)
    if own:
        s.update(_plan(c, s))
    return s


def _plan(c, s):
    """What a program keeps between calls: dimensions, cache descriptor, rotary table and
    workspace."""
    import block_sparse_long_cobs_b200 as cb
    dims = cb.cobs_dims(batch=c["batch"], num_q_heads=c.get("hq", c["hkv"]),
                        num_kv_heads=c["hkv"], head_dim=c["d"], block_size=_B, rank=0,
                        capacity_tokens=s["cap"])
    coded = "ks" in s
    pages = s["k"].shape[0] if "table" in s else 0
    cache = cb.cobs_kv_cache(
        k=s["k"], v=s["v"], k_scale=s.get("ks"), v_scale=s.get("vs"),
        block_table=s.get("table"), n_pages=pages,
        table_stride=s["table"].shape[1] if "table" in s else 0,
        format=cb.COBS_CACHE_E4M3 if coded else cb.COBS_CACHE_BF16)
    p = dict(cb=cb, dims=dims, cache=cache)
    size = 256
    if c["op"] == "append":
        p["rope"] = cb.cobs_rope_init(
            c["rotary"], c["interleaved"], _BASE,
            **(dict(scaling=cb.COBS_ROPE_BY_PARTS, **_SCALED) if c["scaled"] else {}))
    elif c["op"] == "prompt":
        size = cb.cobs_prompt_workspace_bytes(dims, s["q"].shape[0], max(_lengths(c)))
    elif c["op"] == "decode":
        size = cb.cobs_workspace_bytes(dims, _n_sel(c), 0, 0)
    p["ws"] = torch.zeros(size, dtype=torch.uint8, device=_DEV)
    return p


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(state):
    s = state
    c = s["case"]
    return {"append": _append, "read": _read, "prompt": _prompt, "decode": _decode}[c["op"]](c, s)


def _written(c, s):
    """What an append leaves: rotated queries and the cache rows it wrote (of the pages that
    the new tokens lie in, all)."""
    if c["paged"]:
        rows = [s["k"], s["v"]] + ([s["ks"], s["vs"]] if c["e4m3"] else [])
    else:
        at = slice(c["start"], c["start"] + c["new"])
        rows = [s["k"][:, :, at], s["v"][:, :, at]]
        rows += [s["ks"][:, :, at], s["vs"][:, :, at]] if c["e4m3"] else []
    if c["e4m3"]:
        rows[:2] = [x.view(torch.float8_e4m3fn) for x in rows[:2]]
    return [s["q_out"]] + rows


def _frequencies(c):
    """Radians per token of each rotated pair, in 64 bits."""
    f = _BASE ** (-torch.arange(0, c["rotary"], 2, dtype=torch.float64, device=_DEV) / c["rotary"])
    if c["scaled"]:
        turns = _SCALED["original_context"] * f / (2 * math.pi)
        keep = ((turns - _SCALED["low"]) / (_SCALED["high"] - _SCALED["low"])).clamp(0, 1)
        f = f * keep + f / _SCALED["factor"] * (1 - keep)
    return f


def _append(c, s):
    hq, hkv, d, rot = c["hq"], c["hkv"], c["d"], c["rotary"]
    qkv, n = s["qkv"], s["qkv"].shape[0]
    if own:
        cb, wide = s["cb"], (hq + 2 * hkv) * d
        cb.cobs_append_tokens(s["dims"], s["cache"], s["rope"], qkv[:, :hq], wide,
                              qkv[:, hq:hq + hkv], wide, qkv[:, hq + hkv:], wide,
                              s["cu"], n, s["start"], s["q_out"], s["ws"], s["ws"].numel())
        return _written(c, s)
    token = torch.arange(n, device=_DEV)
    seq = torch.searchsorted(s["cu"][1:].long(), token, right=True)
    pos = s["start"][seq] + token - s["cu"].long()[seq]
    # angles in 64 bits: a far position times a frequency loses its turn in 32
    angle = pos.double().unsqueeze(-1) * _frequencies(c)
    amp = _SCALED["attention_factor"] if c["scaled"] else 1.0
    cos, sin = ((f(angle) * amp).float().unsqueeze(1) for f in (torch.cos, torch.sin))
    x = qkv[:, :hq + hkv].float()
    t = x[..., :rot]
    if c["interleaved"]:
        a, b = t[..., 0::2], t[..., 1::2]
        t = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = t[..., :rot // 2], t[..., rot // 2:]
        t = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    x = torch.cat([t, x[..., rot:]], -1)
    s["q_out"].copy_(x[:, :hq].to(torch.bfloat16))
    if c["paged"]:
        row = (s["table"].long()[seq, pos // _B].unsqueeze(-1) * hkv
               + torch.arange(hkv, device=_DEV)) * _B + (pos % _B).unsqueeze(-1)
    else:
        row = (seq.unsqueeze(-1) * hkv + torch.arange(hkv, device=_DEV)) * s["cap"] \
            + pos.unsqueeze(-1)
    k, v = x[:, hq:], qkv[:, hq + hkv:].float()
    if c["e4m3"]:
        ks, vs = k.abs().amax(-1) / 448.0, v.abs().amax(-1) / 448.0
        s["ks"].view(-1)[row], s["vs"].view(-1)[row] = ks, vs
        s["k"].view(-1, d)[row] = (k / ks.unsqueeze(-1)).to(torch.float8_e4m3fn).view(torch.uint8)
        s["v"].view(-1, d)[row] = (v / vs.unsqueeze(-1)).to(torch.float8_e4m3fn).view(torch.uint8)
    else:
        s["k"].view(-1, d)[row] = k.to(torch.bfloat16)
        s["v"].view(-1, d)[row] = v.to(torch.bfloat16)
    return _written(c, s)


def _read(c, s):
    if own:
        s["cb"].cobs_read_cache(s["dims"], s["cache"], None, 0, c["blocks"], s["out"][0],
                                s["out"][1], s["ws"], s["ws"].numel())
        return s["out"]
    return [_page_rows(c, s, s["k"].float() * s["ks"].unsqueeze(-1)).to(torch.bfloat16),
            _page_rows(c, s, s["v"].float() * s["vs"].unsqueeze(-1)).to(torch.bfloat16)]


def _page_rows(c, s, x):
    """Cache rows as pages in block order: [batch x blocks][hkv][64][d]."""
    if c["paged"]:
        return x[s["table"].long().view(-1)]
    nb = s["cap"] // _B
    return x.view(c["batch"], c["hkv"], nb, _B, c["d"]).transpose(1, 2) \
        .reshape(c["batch"] * nb, c["hkv"], _B, c["d"])


def _whole(c, s, x):
    """Cache rows [batch][hkv][cap][..] (a block without a page reads some other page)."""
    if not c["paged"]:
        return x
    t = x[s["table"].long().clamp(min=0)]          # [batch][blocks][hkv][64][..]
    return t.transpose(1, 2).reshape((c["batch"], c["hkv"], -1) + tuple(x.shape[3:]))


def _prompt(c, s):
    hkv, d = c["hkv"], c["d"]
    group, scale = c["hq"] // hkv, 1.0 / math.sqrt(d)
    if own:
        s["cb"].cobs_prompt_attention(s["dims"], s["cache"], s["q"], s["cu"], s["q"].shape[0],
                                      s["lens"], max(_lengths(c)), scale, s["out"], s["lse"],
                                      s["ws"], s["ws"].numel())
        return [s["out"], s["lse"]]
    # every sequence padded to the longest, rows that no token has masked away
    n, batch, cap = s["q"].shape[0], c["batch"], s["cap"]
    cu, lens = s["cu"].long(), s["lens"]
    count = cu[1:] - cu[:-1]
    i = torch.arange(c["new"], device=_DEV)
    token = (cu[:-1, None] + i).clamp(max=n - 1)
    pos = (lens - count)[:, None] + i                                   # [batch][new]
    key = torch.arange(cap, device=_DEV)
    gone = (key >= lens[:, None])[:, None, :, None]
    k = _whole(c, s, s["k"]).float().masked_fill_(gone, 0.0)
    v = _whole(c, s, s["v"]).float().masked_fill_(gone, 0.0)
    q = s["q"][token].float().view(batch, c["new"], hkv, group, d).permute(0, 2, 3, 1, 4) * scale
    p = (q.reshape(batch, hkv, -1, d) @ k.transpose(-1, -2)).view(batch, hkv, group, c["new"], cap)
    p.masked_fill_((key > pos[..., None])[:, None, None], float("-inf"))
    top = p.amax(-1, keepdim=True)
    p.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    o = (p.view(batch, hkv, -1, cap) @ v).view(batch, hkv, group, c["new"], d) / total
    lse = (top + total.log()).squeeze(-1)
    here = torch.searchsorted(cu[1:], torch.arange(n, device=_DEV), right=True)
    at = torch.arange(n, device=_DEV) - cu[here]
    o = o.permute(0, 3, 1, 2, 4)[here, at].reshape(n, c["hq"], d)
    return [o.to(torch.bfloat16), lse.permute(0, 3, 1, 2)[here, at].reshape(n, c["hq"])]


def _decode(c, s):
    hkv, d, batch = c["hkv"], c["d"], c["batch"]
    group, scale = c["hq"] // hkv, 1.0 / math.sqrt(d)
    if own:
        s["cb"].cobs_sparse_decode_cache(s["dims"], s["cache"], s["q"], s["idx"], s["n_sel"],
                                         s["idx"].shape[-1], s["lens"] if c["ragged"] else None,
                                         c["length"], scale, s["out"], s["lse"], s["ws"],
                                         s["ws"].numel())
        return [s["out"], s["lse"]]
    block = s["idx"].long()
    token = (block.unsqueeze(-1) * _B + torch.arange(_B, device=_DEV)).flatten(2)
    head = torch.arange(hkv, device=_DEV).view(1, hkv, 1)
    seq = torch.arange(batch, device=_DEV).view(batch, 1, 1)
    if c["paged"]:
        row = (s["table"].long()[seq, token // _B] * hkv + head) * _B + token % _B
    else:
        row = (seq * hkv + head) * s["cap"] + token
    out_of = token >= s["lens"].view(batch, 1, 1)

    def rows(codes, scales):
        x = codes.view(torch.uint8).view(-1, d)[row].view(torch.float8_e4m3fn).float()
        x = x * scales.view(-1)[row].unsqueeze(-1)
        return x.masked_fill_(out_of.unsqueeze(-1), 0.0)

    q = s["q"].float().view(batch, hkv, group, d)
    p = q @ rows(s["k"], s["ks"]).transpose(-1, -2) * scale
    p = p.masked_fill(out_of.unsqueeze(2), float("-inf"))
    top = p.amax(-1, keepdim=True)
    p = (p - top).exp()
    total = p.sum(-1, keepdim=True)
    o = p @ rows(s["v"], s["vs"]) / total
    return [o.view(batch, c["hq"], d), (top + total.log()).view(batch, c["hq"])]


# ---------------------------------------------------------------------------
# the definitions in 64 bits, sequence by sequence
# ---------------------------------------------------------------------------

def exact(case, seed):
    c = case
    s = prepare(c, seed)
    if c["op"] == "append":
        return _exact_append(c, s)
    if c["op"] == "read":
        k, v = (x.double() * y.double()[..., None] for x, y in ((s["k"], s["ks"]), (s["v"], s["vs"])))
        return [torch.stack([_block64(c, s, x, b, j) for b in range(c["batch"])
                             for j in range(c["blocks"])]) for x in (k, v)]
    return (_exact_prompt if c["op"] == "prompt" else _exact_decode)(c, s)


def _block64(c, s, x, b, j):
    """Block j of sequence b for all kv-heads: [hkv][64][..]."""
    if c["paged"]:
        return x[int(s["table"][b, j])]
    return x[b, :, j * _B:(j + 1) * _B]


def _exact_append(c, s):
    d, rot, hq, hkv = c["d"], c["rotary"], c["hq"], c["hkv"]
    lo, hi = (_SCALED["low"], _SCALED["high"]) if c["scaled"] else (0.0, 1.0)
    first = 0
    q_all = []
    keep = {n: torch.zeros(s[n].shape, dtype=torch.float64, device=_DEV) for n in ("k", "v")}
    if c["e4m3"]:
        keep |= {n: torch.zeros(s[n].shape, dtype=torch.float64, device=_DEV) for n in ("ks", "vs")}
    table = s["table"].tolist() if c["paged"] else None
    for b, (count, start) in enumerate(zip(_new(c), _starts(c))):
        x = s["qkv"][first:first + count].double()
        first += count
        pos = torch.arange(start, start + count, dtype=torch.float64, device=_DEV)
        y = x.clone()
        for t in range(rot // 2):
            f = _BASE ** (-2.0 * t / rot)
            if c["scaled"]:
                r = (_SCALED["original_context"] * f / (2 * math.pi) - lo) / (hi - lo)
                r = min(1.0, max(0.0, r))
                f = r * f + (1 - r) * f / _SCALED["factor"]
            u, w = (2 * t, 2 * t + 1) if c["interleaved"] else (t, t + rot // 2)
            amp = _SCALED["attention_factor"] if c["scaled"] else 1.0
            turn = torch.polar(torch.full_like(pos, amp), pos * f).unsqueeze(-1)
            z = torch.complex(x[:, :hq + hkv, u], x[:, :hq + hkv, w]) * turn
            y[:, :hq + hkv, u], y[:, :hq + hkv, w] = z.real, z.imag
        q_all.append(y[:, :hq])
        for name, rows in (("k", y[:, hq:hq + hkv]), ("v", x[:, hq + hkv:])):
            scale = rows.abs().max(-1).values / 448.0 if c["e4m3"] else None
            if c["e4m3"]:
                rows = rows / scale[..., None]
            i = 0
            while i < count:                     # up to the end of a block at a time
                p = start + i
                m = min(count - i, _B - p % _B)
                if c["paged"]:
                    at = (table[b][p // _B], slice(None), slice(p % _B, p % _B + m))
                else:
                    at = (b, slice(None), slice(p, p + m))
                keep[name][at] = rows[i:i + m].transpose(0, 1)
                if c["e4m3"]:
                    keep[name + "s"][at] = scale[i:i + m].T
                i += m
    out = [torch.cat(q_all)]
    names = ["k", "v"] + (["ks", "vs"] if c["e4m3"] else [])
    at = slice(c["start"], c["start"] + c["new"])
    out += [keep[n] if c["paged"] else keep[n][:, :, at] for n in names]
    if c["e4m3"]:
        out[1] = out[2] = None                   # codes are choices of a grid, not computed values
    return out


def _sequence64(c, s, x, b, h, length):
    if not c["paged"]:
        return x[b, h, :length].double()
    nb = -(-length // _B)
    pages = s["table"][b, :nb].long()
    return x[pages, h].reshape((nb * _B,) + tuple(x.shape[3:]))[:length].double()


def _exact_prompt(c, s):
    d, group = c["d"], c["hq"] // c["hkv"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=_DEV)
    lse = torch.zeros(s["lse"].shape, dtype=torch.float64, device=_DEV)
    first = 0
    for b, (count, length) in enumerate(zip(_new(c), _lengths(c))):
        j = torch.arange(length, device=_DEV)
        for h in range(c["hkv"]):
            k = _sequence64(c, s, s["k"], b, h, length)
            v = _sequence64(c, s, s["v"], b, h, length)
            for q0 in range(h * group, (h + 1) * group):
                rows = s["q"][first:first + count, q0].double()
                logit = torch.einsum("id,jd->ij", rows, k) / math.sqrt(d)
                seen = j[None, :] <= (length - count + torch.arange(count, device=_DEV))[:, None]
                logit = torch.where(seen, logit, -math.inf)
                norm = torch.logsumexp(logit, 1)
                lse[first:first + count, q0] = norm
                out[first:first + count, q0] = torch.exp(logit - norm[:, None]) @ v
        first += count
    return [out, lse]


def _exact_decode(c, s):
    d, group = c["d"], c["hq"] // c["hkv"]
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device=_DEV)
    lse = torch.zeros(s["lse"].shape, dtype=torch.float64, device=_DEV)
    for b, length in enumerate(_lengths(c)):
        for h in range(c["hkv"]):
            tokens = (s["idx"][b, h].long()[:, None] * _B + torch.arange(_B, device=_DEV)).view(-1)
            tokens = tokens[tokens < length]
            if c["paged"]:
                page = s["table"][b].long()[tokens // _B]
                at = (page, h, tokens % _B)
            else:
                at = (b, h, tokens)
            k, v = (s[n].view(torch.uint8)[at].view(torch.float8_e4m3fn).double()
                    * s[n + "s"][at].double()[:, None] for n in ("k", "v"))
            for q0 in range(h * group, (h + 1) * group):
                logit = k @ s["q"][b, q0].double() / math.sqrt(d)
                lse[b, q0] = torch.logsumexp(logit, 0)
                out[b, q0] = torch.softmax(logit, 0) @ v
    return [out, lse]
