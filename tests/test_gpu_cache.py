"""Appending tokens and reading a cache back, on the GPU, against plain 64-bit
forms.  Cache rows outside the call are sentinels or NaN.

Tolerances.  A stored bf16 value is the fp32 result rounded once: half a step,
2^-8 of the value.  The fp32 rotation itself is two products and a sum of sines
and cosines that are off by a few 2^-24 (angle: 2^-25 half turns): at most
2^-21 (|x1| + |x2|).  An E4M3 value is off by half a step of the code, 2^-4 of
the value or 2^-10 of the scale, and the scale by 2^-22 of itself."""

import itertools

import pytest
import torch

import block_sparse_long_cobs_b200 as cb
from cache_ref import (B, Cache, bf16_rows, cu_of, dims_of, frequencies, ints, rotate,
                       workspace)

pytestmark = pytest.mark.gpu

HEADS = [(4, 1, 64), (8, 8, 64), (8, 2, 128), (8, 1, 128), (3, 3, 128)]
ROPES = {
    "half": dict(rotary_dim=1.0, interleaved=False),
    "inter": dict(rotary_dim=1.0, interleaved=True),
    "half_part_linear": dict(rotary_dim=0.5, interleaved=False, scaling=cb.COBS_ROPE_LINEAR,
                             factor=4.0),
    "inter_part_by_parts": dict(rotary_dim=0.5, interleaved=True,
                                scaling=cb.COBS_ROPE_BY_PARTS, factor=8.0,
                                original_context=8192, low=1.0, high=4.0,
                                attention_factor=1.25),
    "half_24": dict(rotary_dim=24, interleaved=False),
    "none": None,
}
LENS = {   # new tokens, tokens before them
    "ones": (None, [0, 1, 63, 262000]),
    "ragged": ([5, 0, 130, 1, 64], [63, 7, 0, 100000, 65]),
    "one_long": ([333], [31]),
}


def make_rope(kw, d):
    if kw is None:
        return None, None, False, 1.0
    kw = dict(kw)
    r = kw.pop("rotary_dim")
    r = int(r * d) if isinstance(r, float) else r
    inter, amp = kw.pop("interleaved"), kw.get("attention_factor", 1.0)
    rope = cb.cobs_rope_init(r, inter, **kw)
    kw.pop("attention_factor", None)
    return rope, frequencies(r, **kw), inter, amp


class Append:
    def __init__(self, heads, counts, starts, e4m3, paged, pad=3, seed=3):
        self.hq, self.hkv, self.d = heads
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        self.counts = counts or [1] * len(starts)
        self.starts = starts
        self.n = sum(self.counts)
        rows = self.n + (pad if counts else 0)
        self.rows = rows
        self.qkv = bf16_rows(g, rows, self.hq + 2 * self.hkv, self.d, scale=2.0)
        self.cu = cu_of(counts) if counts else None
        self.cap = -(-max(s + c for s, c in zip(starts, self.counts)) // B) * B
        # pages only for the blocks that the new tokens lie in
        batch = len(starts)
        self.table, shape = None, (batch, self.hkv, self.cap)
        if paged:
            spans = [(s // B, -(-(s + c) // B) if c else s // B)
                     for s, c in zip(starts, self.counts)]
            n_pages = sum(y - x for x, y in spans) + 2
            order = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32)
            self.table = torch.full((batch, self.cap // B), -1, dtype=torch.int32, device="cuda")
            at = 0
            for b, (x, y) in enumerate(spans):
                self.table[b, x:y] = order[at:at + y - x]
                at += y - x
            shape, self.n_pages = (n_pages, self.hkv, B), n_pages
        self.e4m3 = e4m3
        kind = torch.uint8 if e4m3 else torch.int16
        self.k = torch.full(shape + (self.d,), 0x5A, dtype=kind, device="cuda")
        self.v = torch.full(shape + (self.d,), 0x5A, dtype=kind, device="cuda")
        self.ks = torch.full(shape, -7.0, device="cuda") if e4m3 else None
        self.vs = torch.full(shape, -7.0, device="cuda") if e4m3 else None
        self.q_out = torch.full((rows, self.hq, self.d), -7.0, dtype=torch.bfloat16,
                                device="cuda")
        self.cache = cb.cobs_kv_cache(self.k, self.v, self.ks, self.vs, self.table,
                                      self.n_pages if paged else 0,
                                      self.table.shape[1] if paged else 0, int(e4m3))
        self.ws = workspace()
        self.dims = dims_of(batch, self.hq, self.hkv, self.d, self.cap)
        pos, seq = [], []
        for b, (s, c) in enumerate(zip(starts, self.counts)):
            pos += range(s, s + c)
            seq += [b] * c
        self.pos, self.seq = ints(pos), ints(seq)

    def call(self, rope, **kw):
        wide = (self.hq + 2 * self.hkv) * self.d
        hq, hkv = self.hq, self.hkv
        a = dict(q=self.qkv[:, :hq], q_stride=wide, k=self.qkv[:, hq:hq + hkv], k_stride=wide,
                 v=self.qkv[:, hq + hkv:], v_stride=wide, cu_tokens=self.cu, n_tokens=self.rows,
                 start=ints(self.starts), q_out=self.q_out)
        a.update(kw)
        cb.cobs_append_tokens(self.dims, self.cache, rope, ws=self.ws, ws_bytes=256, **a)
        return cb.cobs_read_device_status(self.ws, 256)

    def where(self):
        """Index of every new token's row in the cache arrays: [n][hkv]."""
        h = torch.arange(self.hkv, device="cuda")
        if self.table is None:
            return (self.seq[:, None], h, self.pos[:, None])
        page = self.table[self.seq, self.pos // B].long()
        return (page[:, None], h, (self.pos % B)[:, None])

    def check(self, f, inter, amp, q=True):
        hq, hkv, n = self.hq, self.hkv, self.n
        x = self.qkv[:n].double()
        y, size = x.clone(), x.abs()
        if f is not None:
            y[:, :hq + hkv], size[:, :hq + hkv] = rotate(x[:, :hq + hkv], self.pos, f, inter, amp)
        tol = 2.0 ** -8 * y.abs() + 2.0 ** -21 * size
        if q:
            assert ((self.q_out[:n].double() - y[:, :hq]).abs() <= tol[:, :hq]).all()
            assert (self.q_out[n:] == -7).all()
        else:
            assert (self.q_out == -7).all()
        at = self.where()
        for x_, s_, rows, size_ in ((self.k, self.ks, y[:, hq:hq + hkv], size[:, hq:hq + hkv]),
                                    (self.v, self.vs, y[:, hq + hkv:], size[:, hq + hkv:])):
            got = x_[at]
            if self.e4m3:
                top = rows.abs().amax(-1)
                sc = s_[at].double()
                assert ((sc - top / 448).abs() <= 2.0 ** -21 * size_.amax(-1) / 448).all()
                val = got.view(torch.float8_e4m3fn).double() * sc[..., None]
                t = 2.0 ** -4 * rows.abs() + 2.0 ** -10 * sc[..., None] + 2.0 ** -20 * size_
                assert ((val - rows).abs() <= t).all()
                s_[at] = -7.0
                assert (s_ == -7.0).all()
            else:
                t = 2.0 ** -8 * rows.abs() + 2.0 ** -21 * size_
                assert ((got.view(torch.bfloat16).double() - rows).abs() <= t).all()
            x_[at] = 0x5A
            assert (x_ == 0x5A).all()          # no other row was written


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("rope", list(ROPES))
@pytest.mark.parametrize("lens", list(LENS))
def test_append(lens, rope, e4m3):
    counts, starts = LENS[lens]
    for heads, paged in itertools.product(HEADS, (False, True)):
        if not paged and max(starts) > 1000:
            starts = [min(s, 900) for s in starts]
        p = Append(heads, counts, starts, e4m3, paged)
        r, f, inter, amp = make_rope(ROPES[rope], p.d)
        assert p.call(r) == 0
        p.check(f, inter, amp)
        starts = LENS[lens][1]


def test_append_keys_only_in_place_and_no_rows():
    p = Append((8, 2, 128), [5, 9], [60, 0], False, True)
    r, f, inter, amp = make_rope(ROPES["half"], 128)
    assert p.call(r, q=None, q_stride=0, q_out=None) == 0
    p.check(f, inter, amp, q=False)
    for kind in ("half", "inter", "half_24"):
        p = Append((8, 2, 128), [5, 9], [60, 0], False, True)
        r, f, inter, amp = make_rope(ROPES[kind], 128)
        q = p.qkv[:, :8].contiguous()
        keep = q.clone()
        assert p.call(r, q=q, q_stride=8 * 128, q_out=q) == 0
        p.q_out[:p.n] = q[:p.n]
        assert torch.equal(q[p.n:], keep[p.n:])
        p.check(f, inter, amp)
    p = Append((8, 2, 128), [5, 9], [60, 0], False, True)
    assert p.call(r, n_tokens=0) == 0
    assert (p.k == 0x5A).all() and (p.q_out == -7).all()


def test_append_of_many_sequences():
    """More sequences than a warp has lanes, empty ones among them."""
    counts = [(7 * b) % 5 for b in range(1500)]
    starts = [(13 * b) % 70 for b in range(1500)]
    p = Append((1, 1, 64), counts, starts, True, True)
    r, f, inter, amp = make_rope(ROPES["half"], 64)
    assert p.call(r) == 0
    p.check(f, inter, amp)


@pytest.mark.parametrize("e4m3", [False, True])
def test_append_outside_the_cache_is_reported(e4m3):
    for what in ("capacity", "page", "pool", "negative"):
        p = Append((4, 1, 64), [3, 2, 4], [10, 61, 64], e4m3, True)
        r, f, inter, amp = make_rope(ROPES["half"], 64)
        if what == "page":
            p.table[1, 0] = -1
        elif what == "pool":
            p.table[1, 0] = p.n_pages
        else:
            p.starts[1] = p.cap - 0 if what == "capacity" else -2
        assert p.call(r) == cb.COBS_ERR_DEVICE
        # the other sequences' tokens are stored; all queries are rotated
        keep = torch.tensor([0, 1, 2, 5, 6, 7, 8], device="cuda")
        pos = p.pos.clone()
        if what == "capacity":
            pos[3:5] = ints([p.cap, p.cap + 1])
        if what == "negative":
            pos[3:5] = ints([-2, -1])
        y, size = rotate(p.qkv[:p.n, :p.hq].double(), pos, f, inter, amp)
        err = (p.q_out[:p.n].double() - y).abs()
        assert (err <= 2.0 ** -8 * y.abs() + 2.0 ** -21 * size).all()
        p.n, p.pos, p.seq = 7, p.pos[keep], p.seq[keep]
        p.qkv, p.q_out = p.qkv[torch.cat([keep, ints([9, 10, 11])])], \
            p.q_out[torch.cat([keep, ints([9, 10, 11])])]
        p.check(f, inter, amp)


@pytest.mark.parametrize("extra", [0, 40])
def test_append_bounds_outside_the_rows_are_cut_and_reported(extra):
    """Bounds below 0 and past n_tokens, with few sequences and with more than a
    warp has lanes: every row is stored where the bounds cut to [0, n_tokens]
    put it."""
    counts, starts = [5, 0, 9] + [1] * extra, [60, 7, 0] + [3] * extra
    for first, last in ((-5, None), (None, 7), (-1, 1000), (None, None)):
        p = Append((4, 1, 64), counts, starts, False, True, pad=0)
        r, f, inter, amp = make_rope(ROPES["half"], 64)
        if first is not None:
            p.cu[0] = first
        if last is not None:
            p.cu[-1] += last
        bad = first is not None or last is not None
        assert p.call(r) == (cb.COBS_ERR_DEVICE if bad else 0)
        p.check(f, inter, amp)


@pytest.mark.parametrize("extra", [0, 40])
def test_append_rows_before_the_first_bound_are_nobodys(extra):
    """cu_tokens[0] > 0: the rows before it are neither stored nor rotated."""
    counts, starts = [5, 9] + [1] * extra, [60, 70] + [3] * extra
    p = Append((4, 1, 64), counts, starts, False, True, pad=0)
    r, f, inter, amp = make_rope(ROPES["half"], 64)
    cut = 2
    p.cu[0] = cut
    assert p.call(r) == 0
    assert (p.q_out[:cut] == -7).all()
    # what is left of the first sequence starts at its first position
    p.pos[cut:5] -= cut
    p.qkv, p.q_out, p.pos, p.seq = p.qkv[cut:], p.q_out[cut:], p.pos[cut:], p.seq[cut:]
    p.n -= cut
    p.check(f, inter, amp)


@pytest.mark.parametrize("batch", [31, 32, 33])
def test_append_around_a_warp_of_sequences(batch):
    """Batches about as large as a warp, empty sequences at the ends."""
    counts = [(5 * b + 1) % 4 for b in range(batch)]
    counts[0] = counts[-1] = 0
    starts = [(29 * b) % 130 for b in range(batch)]
    p = Append((8, 2, 128), counts, starts, False, True)
    r, f, inter, amp = make_rope(ROPES["inter"], 128)
    assert p.call(r) == 0
    p.check(f, inter, amp)


@pytest.mark.parametrize("interleaved", [False, True])
def test_append_with_given_frequencies(interleaved):
    want = [3.0, 0.0, 1.0, 0.31, 1e-3, 2.0 ** -20, 0.7, 1e-9]
    p = Append((4, 1, 64), [5, 9], [100000, 0], False, True)
    r = cb.cobs_rope_init(16, interleaved, scaling=cb.COBS_ROPE_CUSTOM, frequencies=want)
    assert p.call(r) == 0
    p.check(torch.tensor(want, dtype=torch.float64, device="cuda"), interleaved, 1.0)


@pytest.mark.parametrize("d", [64, 128])
def test_append_codes_are_those_of_the_quotient(d):
    """E4M3 values are not rotated, so that their scales and codes are those of
    max |x| / 448 and x / scale in fp32, each rounded once, bit for bit: quotients
    that lie on or beside the middle of two codes among them."""
    p = Append((1, 1, d), [2000, 300], [0, 64], True, False)
    g = torch.Generator(device="cuda").manual_seed(4)
    rows = torch.randint(128, 256, (p.rows, 1, d), generator=g, device="cuda").float() / 128.0
    rows *= 2.0 ** torch.randint(-6, 1, (p.rows, 1, d), generator=g, device="cuda").float()
    rows *= torch.randint(0, 2, (p.rows, 1, d), generator=g, device="cuda").float() * 2 - 1
    rows *= 2.0 ** torch.tensor([0.0, -115.0, -70.0, 60.0], device="cuda").repeat(
        p.rows // 4 + 1)[:p.rows, None, None]
    rows[0, 0, 0], rows[0, 0, 1:] = 1.078125, 0.80859375     # a quotient of 336, a tie
    p.qkv[:, 2:] = rows.bfloat16()
    assert (p.qkv[:, 2:].float() == rows).all()
    assert p.call(None) == 0
    scale = rows[:p.n, 0].abs().amax(-1).cpu() / 448.0
    code = (rows[:p.n, 0].cpu() / scale[:, None]).to(torch.float8_e4m3fn).view(torch.uint8)
    at = p.where()
    assert torch.equal(p.vs[at][:, 0].cpu(), scale)
    assert torch.equal(p.v[at][:, 0].cpu(), code)


def test_append_zero_tiny_and_non_finite_rows():
    """E4M3: zero rows, rows below the smallest scale, huge rows, NaN and
    infinities."""
    p = Append((4, 1, 64), [6], [2], True, False)
    x = p.qkv
    x[0, 5] = 0.0
    x[1, 5] = 2.0 ** -126
    x[2, 5] = 3.0e38
    x[3, 5, 3], x[3, 5, 7], x[3, 5, 9] = float("nan"), float("inf"), float("-inf")
    x[4, 5] = float("nan")
    assert p.call(None) == 0
    vals, sc = p.v[0, 0, 2:8], p.vs[0, 0, 2:8]
    assert sc[0] == 0 and (vals[0] == 0).all()
    assert sc[1] == 0 and ((vals[1] & 0x7F) == 0).all()
    code = vals.view(torch.float8_e4m3fn).double()
    big = x[2, 5].double()
    assert ((code[2] * sc[2].double() - big).abs() <= 2.0 ** -4 * big.abs()).all()
    bad = ~torch.isfinite(x[3, 5])
    assert torch.isnan(code[3][bad]).all() and torch.isfinite(code[3][~bad]).all()
    want = x[3, 5].double()[~bad]
    assert ((code[3][~bad] * sc[3].double() - want).abs()
            <= 2.0 ** -4 * want.abs() + 2.0 ** -10 * sc[3].double()).all()
    assert sc[4] == 0 and torch.isnan(code[4]).all()


# ---------------------------------------------------------------------------
# reading back
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("paged", [False, True])
@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("d", [64, 128])
def test_read_cache(d, e4m3, paged):
    g = torch.Generator(device="cuda")
    g.manual_seed(5)
    lens = [200, 64, 1]
    k, v = bf16_rows(g, 3, 2, 256, d), bf16_rows(g, 3, 2, 256, d)
    c = Cache(g, k, v, lens, paged, e4m3)
    dims, ws = dims_of(3, 2, 2, d, 256), workspace()
    for first, last, use_lens, only in ((0, 4, True, None), (1, 3, True, "k"), (0, 1, False, "v"),
                                        (2, 2, True, None)):
        n = last - first
        out = {x: torch.full((max(1, 3 * n), 2, B, d), -7.0, dtype=torch.bfloat16, device="cuda")
               for x in "kv"}
        cb.cobs_read_cache(dims, c.desc, ints(lens) if use_lens else None, first, last,
                           out["k"] if only != "v" else None, out["v"] if only != "k" else None,
                           ws, 256)
        assert cb.cobs_read_device_status(ws, 256) == 0
        for name in "kv":
            if only not in (None, name):
                assert (out[name] == -7).all()
                continue
            for b, j in itertools.product(range(3), range(first, last)):
                got = out[name][b * n + j - first]
                rows = min(B, max(0, lens[b] - j * B))
                if use_lens:
                    assert (got[:, rows:] == -7).all()
                for h in range(2):
                    want = c.rows(name, b, h, lens[b])[j * B:j * B + rows].float().bfloat16()
                    assert torch.equal(got[h, :rows], want)


def test_read_cache_pages_missing_or_outside_the_pool():
    g = torch.Generator(device="cuda")
    g.manual_seed(5)
    x = bf16_rows(g, 2, 1, 128, 64)
    c = Cache(g, x, x, [128, 128], True, True)
    dims, ws = dims_of(2, 1, 1, 64, 128), workspace()
    good = c.table.clone()
    for bad, want in ((-1, 0), (c.n_pages, cb.COBS_ERR_DEVICE)):
        c.table.copy_(good)
        c.table[0, 1] = bad
        out = torch.full((4, 1, B, 64), -7.0, dtype=torch.bfloat16, device="cuda")
        cb.cobs_read_cache(dims, c.desc, None, 0, 2, out, None, ws, 256)
        assert cb.cobs_read_device_status(ws, 256) == want
        assert (out[1] == -7).all()
        assert torch.isfinite(out[[0, 2, 3]]).all() and (out[[0, 2, 3]] != -7).any()


@pytest.mark.parametrize("e4m3", [False, True])
def test_append_and_read_back_in_a_graph(e4m3):
    """A captured decode step (append, read the blocks back), replayed from another
    stream with new tokens at new positions, as its inputs are then."""
    p = Append((8, 2, 128), None, [3, 70, 0, 130], e4m3, False)
    r, f, inter, amp = make_rope(ROPES["half"], 128)
    nb, wide, start = p.k.shape[2] // B, 12 * 128, ints(p.starts)
    out = torch.zeros(4 * nb, 2, B, 128, dtype=torch.bfloat16, device="cuda")
    s, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    s.wait_stream(torch.cuda.current_stream())
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=s):
        cb.cobs_append_tokens(p.dims, p.cache, r, p.qkv[:, :8], wide, p.qkv[:, 8:10], wide,
                              p.qkv[:, 10:], wide, None, 4, start, p.q_out, p.ws, 256, stream=s)
        cb.cobs_read_cache(p.dims, p.cache, None, 0, nb, None, out, p.ws, 256, stream=s)
    g = torch.Generator(device="cuda").manual_seed(8)
    for step in range(3):
        p.qkv.copy_(bf16_rows(g, 4, 12, 128, scale=2.0))
        start.copy_(ints([x + 7 * step for x in (3, 70, 0, 130)]))
        graph.replay()
        torch.cuda.synchronize()
        p.pos = start.clone()
        at = p.where()
        v = p.v[at]
        want = v.view(torch.float8_e4m3fn).float() * p.vs[at][..., None] if e4m3 \
            else v.view(torch.bfloat16)
        page, row = torch.arange(4, device="cuda") * nb + p.pos // B, p.pos % B
        assert torch.equal(out[page, :, row], want.bfloat16())
        p.check(f, inter, amp)      # (which puts the rows back as they were)
    assert cb.cobs_read_device_status(p.ws, 256) == 0
