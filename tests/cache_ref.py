"""Plain 64-bit forms of the cache and prompt operators (test infrastructure),
and builders of contiguous and paged caches with poisoned unused rows."""

from __future__ import annotations

import math

import torch

import block_sparse_long_cobs_b200 as cb

B = 64
NAN_CODE = 0x7F


def ints(v, dtype=torch.int64):
    return torch.tensor(v, dtype=dtype, device="cuda")


def cu_of(counts):
    return ints([sum(counts[:i]) for i in range(len(counts) + 1)], torch.int32)


def dims_of(batch, hq, hkv, d, cap, **kw):
    return dict(dict(batch=batch, num_q_heads=hq, num_kv_heads=hkv, head_dim=d, block_size=B,
                     rank=0, capacity_tokens=cap), **kw)


def workspace(nbytes=256):
    return torch.zeros(nbytes, dtype=torch.uint8, device="cuda")


def bf16_rows(g, *shape, scale=1.0):
    x = torch.randn(shape, generator=g, device="cuda")
    return (x * scale * (torch.rand(shape[-1], generator=g, device="cuda") + 0.25)).bfloat16()


def page_table(g, blocks, spare=3, width_pad=2):
    """Random pages for `blocks[b]` blocks of each sequence, some spare pages."""
    n = sum(blocks) + spare
    order = torch.randperm(n, generator=g, device="cuda").to(torch.int32)
    table = torch.full((len(blocks), max(max(blocks), 1) + width_pad), -1, dtype=torch.int32,
                       device="cuda")
    at = 0
    for b, nb in enumerate(blocks):
        table[b, :nb] = order[at:at + nb]
        at += nb
    return table, n


class Cache:
    """A cache of `lens` tokens filled from logical rows [b][hkv][cap][d] (bf16);
    every row outside the sequences is poisoned (NaN, or a NaN code with a NaN
    scale)."""

    def __init__(self, g, k, v, lens, paged, e4m3=False, cap=None):
        batch, hkv, rows, d = k.shape
        self.batch, self.hkv, self.d, self.lens, self.paged = batch, hkv, d, lens, paged
        self.cap = cap or rows
        self.table, self.e4m3 = None, e4m3
        tok = torch.arange(rows, device="cuda")
        out = tok >= ints(lens)[:, None]                       # [b][rows]
        gone = out[:, None, :, None]
        self.parts = {}
        for name, x in (("k", k), ("v", v)):
            if e4m3:
                codes, scale = quantise(x)
                scale = scale.masked_fill(out[:, None, :], float("nan"))
                codes = codes.view(torch.uint8).masked_fill(gone, NAN_CODE)
                self.parts[name], self.parts[name + "s"] = codes, scale
            else:
                self.parts[name] = x.masked_fill(gone, float("nan"))
        if paged:
            self.table, self.n_pages = page_table(g, [-(-n // B) for n in lens])
            self.parts = {n: self._paged(x) for n, x in self.parts.items()}
        self.desc = cb.cobs_kv_cache(
            self.parts["k"], self.parts["v"], self.parts.get("ks"), self.parts.get("vs"),
            self.table, self.n_pages if paged else 0, self.table.shape[1] if paged else 0,
            cb.COBS_CACHE_E4M3 if e4m3 else cb.COBS_CACHE_BF16)

    def _paged(self, x):
        poison = NAN_CODE if x.dtype == torch.uint8 else float("nan")
        pool = torch.full((self.n_pages, self.hkv, B) + tuple(x.shape[3:]), poison,
                          dtype=x.dtype, device="cuda")
        for b, n in enumerate(self.lens):
            for j in range(-(-n // B)):
                rows = x[b, :, j * B:(j + 1) * B]
                pool[self.table[b, j], :, :rows.shape[1]] = rows
        return pool

    def part(self, name, b, h, n):
        """First n logical rows of an array of the cache."""
        x = self.parts[name]
        if self.table is None:
            return x[b, h, :n]
        nb = -(-n // B)
        return x[self.table[b, :nb].long(), h].flatten(0, 1)[:n]

    def scales(self, name, b, h, n):
        return self.part(name + "s", b, h, n).double()

    def rows(self, name, b, h, n):
        """First n logical rows of (sequence b, kv-head h), in 64 bits."""
        x = self.part(name, b, h, n)
        if self.e4m3:
            codes = x.contiguous().view(torch.float8_e4m3fn).double()
            return codes * self.scales(name, b, h, n)[:, None]
        return x.double()


def quantise(x):
    """E4M3 codes (uint8) and fp32 scales of rows."""
    top = x.float().abs().amax(-1)
    scale = top / 448.0
    safe = torch.where(scale > 0, scale, torch.ones_like(scale))
    return (x.float() / safe[..., None]).to(torch.float8_e4m3fn).view(torch.uint8), scale


def attend(q, k, v, scale):
    """Rows q [n][d] over keys k with per-row visible counts given by k being
    already cut: softmax(q k^T scale) v, lse, and the weighted mean of |v|."""
    s = q @ k.T * scale
    lse = torch.logsumexp(s, 1)
    p = torch.exp(s - lse[:, None])
    return p @ v, lse, p @ v.abs()


def frequencies(rotary, base=10000.0, scaling=0, factor=1.0, original_context=0.0, low=0.0,
                high=0.0):
    f = [base ** (-2.0 * t / rotary) for t in range(rotary // 2)]
    if scaling == cb.COBS_ROPE_LINEAR:
        f = [x / factor for x in f]
    if scaling == cb.COBS_ROPE_BY_PARTS:
        def part(x):
            g = (original_context * x / (2 * math.pi) - low) / (high - low)
            g = min(1.0, max(0.0, g))
            return x * g + x / factor * (1 - g)
        f = [part(x) for x in f]
    return torch.tensor(f, dtype=torch.float64, device="cuda")


def rotate(x, pos, f, interleaved, amp=1.0):
    """x [n][heads][d] in 64 bits, rotated; also |x1| + |x2| of each rotated pair."""
    y, size = x.clone(), x.abs()
    r = 2 * f.numel()
    a = pos.double()[:, None] * f
    cos, sin = (amp * a.cos())[:, None], (amp * a.sin())[:, None]
    one, two = (slice(0, r, 2), slice(1, r, 2)) if interleaved else (slice(0, r // 2),
                                                                     slice(r // 2, r))
    x1, x2 = x[..., one], x[..., two]
    y[..., one], y[..., two] = x1 * cos - x2 * sin, x2 * cos + x1 * sin
    size[..., one] = size[..., two] = amp * (x1.abs() + x2.abs())
    return y, size
