"""Attention of packed new tokens over the cache, on the GPU, against the
softmax in 64 bits.  Everything outside the sequences is NaN.

Tolerances.  The output is rounded to bf16 once (half a step, 2^-8 of the
value), and each weight p before it meets its value (2^-8 of itself), which
moves the output by at most 2^-8 W with W = sum p |v| / sum p; the exponential
(2^-12 of itself) and a logit's fp32 sum over d products (2^-22 |q| |k| scale,
times ln 2 below 1) come on top, in p and in the normaliser, hence
2^-8 |out| + (2^-8 + 2^-10) W + 2^-20 L W, and 2^-12 + 2^-22 L (plus one fp32
rounding of the value) on lse, with L = max |q| |k| scale."""

import itertools
import math

import pytest
import torch

import block_sparse_long_cobs_b200 as cb
from cache_ref import Cache, attend, bf16_rows, cu_of, dims_of, ints, workspace

pytestmark = pytest.mark.gpu

HEADS = [(4, 1, 64), (2, 2, 64), (8, 8, 128), (4, 2, 128), (8, 2, 128), (8, 1, 128),
         (16, 2, 64)]
# new tokens of each sequence, tokens in the cache with them (None: one each)
LENS = {
    "one": ([1], [1]),
    "short": ([77], [77]),
    "odd_mix": ([5, 0, 130, 1, 64, 33], [5, 9, 130, 700, 64, 1000]),
    "tiles": ([128, 129, 127, 256, 257], [128, 129, 191, 256, 513]),
    "singles": (None, [1, 64, 65, 1023, 300]),
    "few_long": ([3, 2], [5000, 4097]),
    "more_rows_than_tokens": ([70, 9], [64, 0]),
    "chunk": ([300], [1400]),
}
PAD = 5


class Prompt:
    def __init__(self, heads, lens, paged, seed=1, kscale=1.0, pad=PAD):
        self.hq, self.hkv, self.d = heads
        counts, self.lens = LENS[lens] if isinstance(lens, str) else lens
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        self.counts = counts or [1] * len(self.lens)
        self.cu = cu_of(counts) if counts else None
        self.n = sum(self.counts)
        self.rows = self.n + (pad if counts else 0)
        batch = len(self.lens)
        self.cap = -(-max(max(self.lens), 1) // 64) * 64 + 64
        k = bf16_rows(g, batch, self.hkv, self.cap, self.d, scale=kscale)
        v = bf16_rows(g, batch, self.hkv, self.cap, self.d)
        self.cache = Cache(g, k, v, self.lens, paged)
        self.q = bf16_rows(g, self.rows, self.hq, self.d, scale=2.0)
        self.q[self.n:] = float("nan")
        self.out = torch.full_like(self.q, -7.0)
        self.lse = torch.full((self.rows, self.hq), -7.0, device="cuda")
        self.dims = dims_of(batch, self.hq, self.hkv, self.d, self.cap)
        self.max_len = max(max(self.lens), 1)
        self.ws_bytes = cb.cobs_prompt_workspace_bytes(self.dims, self.rows, self.max_len)
        self.ws = workspace(self.ws_bytes)
        self.scale = 1.0 / math.sqrt(self.d)
        self.seq_lens = ints(self.lens)

    def call(self, lse=True, stream=None):
        cb.cobs_prompt_attention(self.dims, self.cache.desc, self.q, self.cu, self.rows,
                                 self.seq_lens, self.max_len, self.scale, self.out,
                                 self.lse if lse else None, self.ws, self.ws_bytes, stream)

    def status(self):
        return cb.cobs_read_device_status(self.ws, self.ws_bytes)

    def check(self, lse=True):
        first, group = 0, self.hq // self.hkv
        for b, (c, n) in enumerate(zip(self.counts, self.lens)):
            for h in range(self.hkv if c else 0):
                k, v = (self.cache.rows(x, b, h, n) for x in "kv")
                pos = torch.arange(n - c, n, device="cuda")
                q = self.q[first:first + c, h * group:(h + 1) * group].double()
                s = torch.einsum("ihd,jd->hij", q, k) * self.scale
                s.masked_fill_(torch.arange(n, device="cuda") > pos[:, None], -math.inf)
                want_lse = torch.logsumexp(s, -1)
                p = torch.exp(s - want_lse[..., None]).nan_to_num(0.0)
                want, w = p @ v, p @ v.abs()
                big = float((q.norm(dim=-1).max() * (k.norm(dim=-1).max() if n else 0))) * self.scale
                got = self.out[first:first + c, h * group:(h + 1) * group].double().transpose(0, 1)
                tol = 2.0 ** -8 * want.abs() + (2.0 ** -8 + 2.0 ** -10 + 2.0 ** -20 * big) * w
                assert ((got - want).abs() <= tol + 1e-30).all(), (b, h)
                if lse:
                    got = self.lse[first:first + c, h * group:(h + 1) * group].double().T
                    empty = (pos < 0).expand_as(got)
                    assert (got[empty] == -math.inf).all()
                    d = (got - want_lse)[~empty].abs()
                    t = 2.0 ** -12 + 2.0 ** -22 * big + 2.0 ** -23 * want_lse[~empty].abs()
                    assert (d <= t).all(), (b, h, float(d.max()))
            first += c
        assert (self.out[self.n:] == -7).all()
        if lse:
            assert (self.lse[self.n:] == -7).all()


@pytest.mark.parametrize("lens", list(LENS))
@pytest.mark.parametrize("paged", [False, True])
def test_prompt(lens, paged):
    for i, heads in enumerate(HEADS):
        p = Prompt(heads, lens, paged, seed=i)
        p.call(lse=i % 3 != 2)
        assert p.status() == 0
        p.check(lse=i % 3 != 2)


@pytest.mark.parametrize("paged", [False, True])
def test_many_units_per_cta(paged):
    """More units than CTAs: whole ones of short sequences (single tokens and
    prompts mixed), and equal shares of long ones that cut units anywhere."""
    short = [(b * 37) % 300 + 1 for b in range(130)]
    mixed = ([1 if b % 3 else min(n, (b * 13) % 70) for b, n in enumerate(short)], short)
    for heads, lens in (((8, 8, 64), (None, short)), ((16, 4, 128), mixed), ((4, 4, 64), mixed),
                        ((16, 2, 128), ([1999, 700, 1, 350], [2100, 1500, 4000, 350])),
                        ((8, 8, 128), ([1111, 2], [1700, 3000])),
                        ((4, 2, 64), ([900, 2048, 17], [5000, 2048, 1100]))):
        p = Prompt(heads, lens, paged)
        p.call()
        assert p.status() == 0
        p.check()


def test_bounds_past_the_rows_are_cut_and_reported():
    p = Prompt((8, 2, 128), ([30, 40, 20], [300, 333, 64]), False, pad=0)
    p.cu[3] = 500                    # the last sequence claims rows that are not there
    p.out = torch.full((200, 8, 128), -7.0, dtype=torch.bfloat16, device="cuda")
    p.call()
    assert p.status() == cb.COBS_ERR_DEVICE
    p.check()
    p.cu[0] = -5
    p.call()
    assert p.status() == cb.COBS_ERR_DEVICE
    p.check()


def test_sharp_and_flat_rows():
    """Logits up to some hundreds (weights of one key) and all equal."""
    for kscale in (30.0, 0.0):
        p = Prompt((8, 2, 128), ([200, 40], [200, 333]), False, kscale=kscale)
        p.call()
        assert p.status() == 0
        p.check()


def test_rising_logits():
    """Keys whose logits rise steadily along the sequence, so that the running
    maximum moves at every tile, in either direction of travel."""
    for sign in (1.0, -1.0):
        p = Prompt((4, 1, 128), ([140], [3000]), False)
        c = p.cache.parts["k"]
        ramp = torch.linspace(0, 1, p.cap, device="cuda").bfloat16()
        c[0, 0, :3000] *= 0.25
        c[0, 0, :3000, 0] = sign * 300.0 * ramp[:3000]
        p.q[:p.n, :, 0] = 4.0
        p.call()
        assert p.status() == 0
        p.check()


@pytest.mark.parametrize("d", [64, 128])
def test_maximum_that_moves_at_every_tile(d):
    """Every tile's logits lie 16 above those of the tile before, so that each
    row's weights are formed twice at each tile: with two tiles a unit, with one,
    and one row, always the same answer."""
    for heads, lens in (((8, 1, d), ([40, 17], [2500, 700])), ((1, 1, d), ([300], [1900])),
                        ((8, 2, d), ([1, 1], [3000, 129]))):
        p = Prompt(heads, lens, False)
        for b, n in enumerate(lens[1]):
            step = torch.arange(n, device="cuda") // 128 * 16.0
            p.cache.parts["k"][b, :, :n] *= 0.25
            p.cache.parts["k"][b, :, :n, 0] = (step / (4.0 * p.scale)).bfloat16()
        p.q[:p.n] *= 0.25
        p.q[:p.n, :, 0] = 4.0
        p.call()
        assert p.status() == 0
        p.check()
        first = p.out.clone(), p.lse.clone()
        for _ in range(20):
            p.call()
            assert torch.equal(p.out[:p.n], first[0][:p.n])
            assert torch.equal(p.lse[:p.n], first[1][:p.n])
        assert p.status() == 0


def test_lengths_outside_the_bound_are_clamped_and_reported():
    for bad, used in ((-3, 0), (500, 333)):
        p = Prompt((4, 1, 64), ([10, 20], [100, 333]), False)
        p.seq_lens[0] = bad
        if bad > 0:
            p.cache.parts["k"][0] = 0.5
            p.cache.parts["v"][0] = 0.25
        p.call()
        assert p.status() == cb.COBS_ERR_DEVICE
        p.lens[0] = used
        p.check()


def test_missing_page_counts_as_no_tokens():
    for bad in (-1, 1 << 20):
        p = Prompt((8, 2, 128), ([30, 40], [300, 333]), True)
        good = int(p.cache.table[1, 2])
        p.cache.table[1, 2] = bad
        p.call()
        assert p.status() == cb.COBS_ERR_DEVICE
        # the same keys with that block's logits at -inf
        group = 4
        for h in range(2):
            p.cache.table[1, 2] = good
            k, v = (p.cache.rows(x, 1, h, 333) for x in "kv")
            q = p.q[30:70, h * group:(h + 1) * group].double()
            s = torch.einsum("ihd,jd->hij", q, k) * p.scale
            j = torch.arange(333, device="cuda")
            s.masked_fill_((j > torch.arange(293, 333, device="cuda")[:, None])
                           | ((j >= 128) & (j < 192)), -math.inf)
            want = torch.softmax(s, -1)
            got = p.out[30:70, h * group:(h + 1) * group].double().transpose(0, 1)
            tol = 2.0 ** -8 * (want @ v).abs() + 2.0 ** -7 * (want @ v.abs())
            assert ((got - want @ v).abs() <= tol).all()


def test_two_calls_on_one_workspace_and_another_stream():
    p = Prompt((8, 2, 128), "few_long", True)
    p.call()
    first = p.out.clone(), p.lse.clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    p.out.fill_(-7)
    s.wait_stream(torch.cuda.current_stream())
    p.call(stream=s)
    p.call(stream=s)
    s.synchronize()
    assert p.status() == 0
    assert torch.equal(p.out, first[0]) and torch.equal(p.lse, first[1])
    p.check()


@pytest.mark.parametrize("lens", ["few_long", "tiles", "singles"])
def test_graph_replay_with_new_inputs(lens):
    p = Prompt((8, 2, 128), lens, True)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        p.call(stream=s)
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        p.call(stream=s)
    p.q[:p.n] = bf16_rows(torch.Generator(device="cuda").manual_seed(9), p.n, p.hq, p.d)
    p.out.fill_(-7)
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert p.status() == 0
    p.check()


def test_chunked_prompt_equals_whole():
    """A prompt in pieces over the same cache: the rows of a piece do not
    depend on where it was cut (within the tolerance of both)."""
    p = Prompt((8, 2, 128), ([700], [700]), True, pad=0)
    p.call()
    p.check()
    whole = p.out.clone()
    for a, b in ((0, 1), (1, 130), (130, 131), (131, 700)):
        o = torch.full_like(p.q[a:b], -7.0)
        cb.cobs_prompt_attention(p.dims, p.cache.desc, p.q[a:b], cu_of([b - a]), b - a,
                                 ints([b]), p.max_len, p.scale, o, None, p.ws, p.ws_bytes)
        w = p.cache.rows("v", 0, 0, 700).abs().amax()
        assert ((o - whole[a:b]).double().abs() <= 2.0 ** -6 * w).all()
    assert p.status() == 0


def test_rows_equal_the_sparse_decode_over_all_blocks():
    """One token per sequence over every block: the sparse decode's answer."""
    p = Prompt((8, 2, 128), "singles", True)
    p.call()
    batch, nb = len(p.lens), -(-p.max_len // 64)
    idx = torch.arange(nb, dtype=torch.int32, device="cuda").expand(batch, 2, nb).contiguous()
    n_sel = ints([[-(-n // 64)] * 2 for n in p.lens], torch.int32)
    out = torch.zeros(batch, 8, 128, device="cuda")
    lse = torch.zeros(batch, 8, device="cuda")
    wsb = cb.cobs_workspace_bytes(p.dims, nb, 0, 0)
    ws = workspace(wsb)
    cb.cobs_sparse_decode_cache(p.dims, p.cache.desc, p.q, idx, n_sel, nb, p.seq_lens, p.max_len,
                                p.scale, out, lse, ws, wsb)
    assert cb.cobs_read_device_status(ws, wsb) == 0
    assert (lse - p.lse).abs().max() <= 2.0 ** -11
    assert ((out - p.out.float()).abs() <= 2.0 ** -6 * out.abs().amax() + 2.0 ** -7).all()


@pytest.mark.parametrize("bad", [math.nan, math.inf])
def test_query_that_is_not_finite(bad):
    """Its row is NaN, in out and lse, wherever it lies: in a first tile that is
    partly masked, in a later one, in a unit of one tile or two, whole or cut;
    every other row is what it was, bit for bit.  A row that attends to nothing
    stays 0 and -inf."""
    for heads, lens, rows in (((4, 1, 64), "short", (5, 76)),
                              ((8, 2, 128), "tiles", (50, 130, 700)),
                              ((8, 1, 128), "few_long", (0, 2, 4)),
                              ((8, 8, 128), "chunk", (0, 137, 299)),
                              ((16, 2, 64), "singles", (2, 3)),
                              ((4, 4, 64), ([900, 2048, 17], [5000, 2048, 1100]),
                               (3, 899, 950, 2000, 2964)),
                              ((4, 2, 128), "more_rows_than_tokens", (0, 40, 71))):
        p = Prompt(heads, lens, True)
        p.call()
        assert p.status() == 0
        clean = p.out.clone(), p.lse.clone()
        hit = torch.zeros(p.rows, p.hq, dtype=torch.bool, device="cuda")
        for i, r in enumerate(rows):
            h = (3 * i + 1) % p.hq
            p.q[r, h, (11 * i) % p.d] = bad
            # (not where the row has no key)
            first = [sum(p.counts[:b]) for b in range(len(p.counts) + 1)]
            b = max(b for b in range(len(p.counts)) if first[b] <= r)
            hit[r, h] = p.lens[b] - p.counts[b] + r - first[b] >= 0
        if bad == math.inf:
            # a logit of +inf for every key that such a row sees
            for b in range(len(p.lens)):
                k = p.cache.parts["k"]
                k.abs_()
            p.q.abs_()
            clean = None
        p.call()
        assert p.status() == 0
        assert torch.isnan(p.out[hit]).all() and torch.isnan(p.lse[hit]).all()
        n = slice(0, p.n)
        assert not torch.isnan(p.out[n][~hit[n]]).any() and not torch.isnan(p.lse[n][~hit[n]]).any()
        if clean:
            assert torch.equal(p.out[~hit], clean[0][~hit])
            assert torch.equal(p.lse[~hit], clean[1][~hit])
