"""Sparse decode over an E4M3 cache (and, through the same call, a bf16 one),
on the GPU, against the softmax in 64 bits over the values that the codes and
scales stand for.  Everything outside the sequences and blocks is NaN.

Tolerance.  A value's weight w = p vs (p its softmax weight, vs its row's scale)
is held as four E4M3 parts, each a sixteenth of the one before: an E4M3 number
is off by half a step, 2^-4 of itself or 2^-10 where it is below 2^-6, so four
parts leave 2^-16 of w or 2^-10 / 16^3 = 2^-22 of the unit, and the unit is at
most the largest weight of the pair (it is a power of two no larger than that).
A logit's fp32 sum is off by 2^-22 L and the exponential by 2^-21, with L = max
|q| |k| scale, in p and in the normaliser.  The output is a sum of w_j vc_j, vc
the codes: off by at most (2^-15 + 2^-20 L) sum p |v| + 2^-22 max w sum |vc|
(and the fp32 sum's roundings, below 2^-18 sum p |v|); lse by 2^-18 + 2^-20 L."""

import math

import pytest
import torch

import block_sparse_long_cobs_b200 as cb
from cache_ref import B, Cache, attend, bf16_rows, dims_of, ints, workspace

pytestmark = pytest.mark.gpu

HEADS = [(4, 1, 64), (2, 2, 64), (8, 1, 64), (2, 2, 128), (4, 2, 128), (8, 2, 128), (16, 2, 128)]


class Decode:
    def __init__(self, heads, lens, n_sel, paged, e4m3=True, ragged=True, seed=2, prep=None):
        self.hq, self.hkv, self.d = heads
        self.lens, self.paged, self.ragged = list(lens), paged, ragged
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        batch = len(lens)
        self.cap = -(-max(lens) // B) * B + B
        k, v = (bf16_rows(g, batch, self.hkv, self.cap, self.d) for _ in range(2))
        if prep:
            prep(k, v)
        self.cache = Cache(g, k, v, self.lens, paged, e4m3)
        self.q = bf16_rows(g, batch, self.hq, self.d, scale=3.0)
        self.n = [[min(n_sel, -(-n // B))] * self.hkv for n in lens]
        self.stride = n_sel + 1
        self.idx = torch.full((batch, self.hkv, self.stride), -9, dtype=torch.int32, device="cuda")
        for b, n in enumerate(lens):
            nb = -(-n // B)
            for h in range(self.hkv):
                pick = torch.randperm(nb, generator=g, device="cuda")[:n_sel].sort().values
                if nb - 1 not in pick:
                    pick[-1] = nb - 1
                self.idx[b, h, :len(pick)] = pick.to(torch.int32)
        self.n_sel = ints(self.n, torch.int32)
        self.seq_lens = ints(lens)
        self.out = torch.full((batch, self.hq, self.d), -7.0, device="cuda")
        self.lse = torch.full((batch, self.hq), -7.0, device="cuda")
        self.dims = dims_of(batch, self.hq, self.hkv, self.d, self.cap)
        self.scale = 1.0 / math.sqrt(self.d)
        self.ws_bytes = cb.cobs_workspace_bytes(self.dims, self.stride, 0, 0)
        self.ws = workspace(self.ws_bytes)

    def call(self, stream=None):
        cb.cobs_sparse_decode_cache(self.dims, self.cache.desc, self.q, self.idx, self.n_sel,
                                    self.stride, self.seq_lens if self.ragged else None,
                                    max(self.lens), self.scale, self.out, self.lse, self.ws,
                                    self.ws_bytes, stream)

    def status(self):
        return cb.cobs_read_device_status(self.ws, self.ws_bytes)

    def check(self, skip=()):
        group = self.hq // self.hkv
        for b, n in enumerate(self.lens):
            for h in range(self.hkv):
                blocks = [int(j) for j in self.idx[b, h, :self.n[b][h]]]
                blocks = [j for j in blocks if (b, j) not in skip and 0 <= j * B < n]
                at = torch.cat([torch.arange(j * B, min(n, (j + 1) * B), device="cuda")
                                for j in blocks]) if blocks else ints([])
                rows = slice(h * group, (h + 1) * group)
                if not blocks:
                    assert (self.out[b, rows] == 0).all()
                    assert (self.lse[b, rows] == -math.inf).all()
                    continue
                k, v = (self.cache.rows(x, b, h, n)[at] for x in "kv")
                q = self.q[b, rows].double()
                want, lse, w = attend(q, k, v, self.scale)
                big = float(q.norm(dim=-1).max() * k.norm(dim=-1).max()) * self.scale
                if self.cache.e4m3:
                    p = torch.exp(q @ k.T * self.scale - lse[:, None])
                    vs = self.cache.scales("v", b, h, n)[at]
                    codes = torch.where(vs[:, None] > 0, v / vs[:, None], 0.0)
                    floor = 2.0 ** -22 * (p * vs).amax(1, keepdim=True) * codes.abs().sum(0)
                else:
                    floor = 0.0
                err = (self.out[b, rows].double() - want).abs()
                tol = (2.0 ** -15 + 2.0 ** -18 + 2.0 ** -20 * big) * w + floor
                assert (err <= tol).all(), (b, h, float((err / tol).max()))
                err = (self.lse[b, rows].double() - lse).abs()
                assert (err <= 2.0 ** -18 + 2.0 ** -20 * big + 2.0 ** -23 * lse.abs()).all()


@pytest.mark.parametrize("paged", [False, True])
@pytest.mark.parametrize("heads", HEADS)
def test_decode(heads, paged):
    for lens, n_sel, ragged in (([1], 1, False), ([64, 64], 1, False), ([1000] * 3, 5, False),
                                ([1, 63, 65, 700, 4000], 7, True), ([3000], 40, False)):
        p = Decode(heads, lens, n_sel, paged, ragged=ragged)
        p.call()
        assert p.status() == 0
        p.check()


def test_many_pairs():
    """More pairs than CTAs of a wave, each one chunk of work."""
    p = Decode((16, 8, 128), [200 + 17 * b for b in range(90)], 3, True)
    p.call()
    assert p.status() == 0
    p.check()


def test_bf16_cache_is_the_existing_decode():
    for paged in (False, True):
        p = Decode((8, 2, 128), [700, 4000], 9, paged, e4m3=False)
        p.call()
        got = p.out.clone(), p.lse.clone()
        ws, c = p.ws, p.cache
        if paged:
            cb.cobs_sparse_decode_paged(p.dims, p.q, c.parts["k"], c.parts["v"], c.n_pages,
                                        c.table, c.table.shape[1], p.idx, p.n_sel, p.stride,
                                        p.seq_lens, 4000, p.scale, p.out, p.lse, ws, p.ws_bytes)
        else:
            cb.cobs_sparse_decode_varlen(p.dims, p.q, c.parts["k"], c.parts["v"], p.idx, p.n_sel,
                                         p.stride, p.seq_lens, 4000, p.scale, p.out, p.lse, ws,
                                         p.ws_bytes)
        assert p.status() == 0
        assert torch.equal(got[0], p.out) and torch.equal(got[1], p.lse)


def test_scales_far_apart():
    """Rows of very different magnitude: values by 2^24, keys by 2^6, zero rows."""
    def prep(k, v):
        n = k.shape[2]
        p = torch.arange(n, device="cuda")
        v *= (2.0 ** ((p * 7) % 25 - 12).float())[:, None].bfloat16()
        k *= (2.0 ** ((p * 5) % 7 - 4).float())[:, None].bfloat16()
        v[:, :, 3::17] = 0
        k[:, :, 5::19] = 0
    for heads in ((8, 2, 128), (8, 1, 64)):
        p = Decode(heads, [2000, 90], 12, True, prep=prep)
        p.call()
        assert p.status() == 0
        p.check()


def test_all_values_zero_and_sharp_logits():
    def zero(k, v):
        v.zero_()
    p = Decode((8, 2, 128), [500], 4, False, ragged=False, prep=zero)
    p.call()
    assert p.status() == 0 and (p.out == 0).all()
    p.check()

    def sharp(k, v):
        k *= 40.0
    p = Decode((8, 2, 128), [5000, 700], 20, False, prep=sharp)
    p.call()
    assert p.status() == 0
    p.check()


def test_queries_with_outliers():
    p = Decode((8, 2, 128), [900], 8, False, ragged=False)
    p.q[..., 7] = 300.0
    p.cache.parts["k"][..., 7] = 0
    p.q[0, 1] = 0
    p.call()
    assert p.status() == 0
    p.check()


def test_faulty_lists_and_pages_are_reported():
    for what in ("idx_high", "idx_negative", "n_sel_zero", "n_sel_high", "page", "pool", "length"):
        p = Decode((8, 2, 128), [700, 900], 5, True)
        skip = set()
        if what.startswith("idx"):
            p.idx[1, 0, 2] = 15 if what == "idx_high" else -1
        elif what == "n_sel_zero":
            p.n_sel[0, 1] = 0
            p.n[0][1] = 0
        elif what == "n_sel_high":
            p.n_sel[0, 1] = 100
            p.n[0][1] = p.stride
        elif what in ("page", "pool"):
            j = int(p.idx[1, 0, 1])
            p.idx[1, 1] = p.idx[1, 0]
            p.cache.table[1, j] = -1 if what == "page" else p.cache.n_pages
            skip.add((1, j))
        else:
            p.seq_lens[0] = 0
            p.idx[0, :, 0] = 0
            p.idx[0, :, 1:] = 1
        p.call()
        assert p.status() == cb.COBS_ERR_DEVICE, what
        if what in ("page", "pool"):
            p.cache.table[1, j] = 0          # the reference skips that block
        if what == "length":
            p.lens[0] = 1
        p.check(skip)


def test_graph_replay_and_stream():
    for lens, n_sel in (([4000], 30), ([300] * 80, 4)):
        p = Decode((16, 4, 128), lens, n_sel, True, ragged=False)
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        p.call(stream=s)
        s.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            p.call(stream=s)
        p.q.mul_(0.5)
        p.out.fill_(-7)
        graph.replay()
        graph.replay()
        torch.cuda.synchronize()
        assert p.status() == 0
        p.check()


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("heads", [(4, 1, 64), (8, 2, 128), (2, 2, 128), (16, 2, 128)])
def test_query_that_is_not_finite(heads, bad):
    """Its row is NaN, in out and lse, whether the pair's list is one chunk of
    work or cut and merged; every other row is what it was, bit for bit."""
    for lens, n_sel in (([4000], 40), ([700] * 160, 4), ([100, 1], 2)):
        p = Decode(heads, lens, n_sel, True)
        p.call()
        assert p.status() == 0
        clean = p.out.clone(), p.lse.clone()
        hit = torch.zeros(len(lens), p.hq, dtype=torch.bool, device="cuda")
        for i, b in enumerate({0, len(lens) // 2, len(lens) - 1}):
            h = (2 * i + 1) % p.hq
            p.q[b, h, (p.d - 1) // (i + 1)] = bad
            hit[b, h] = True
        p.call()
        assert p.status() == 0
        assert torch.isnan(p.out[hit]).all() and torch.isnan(p.lse[hit]).all()
        assert torch.equal(p.out[~hit], clean[0][~hit])
        assert torch.equal(p.lse[~hit], clean[1][~hit])


@pytest.mark.parametrize("heads", [(8, 2, 128), (8, 1, 64), (4, 4, 128)])
def test_small_weights_beside_a_large_one(heads):
    """One key's weight is 2^8 to 2^13 times that of a thousand others, which are
    all alike, so that whatever their rounding loses adds up: at most 2^-16 of
    each (four parts) or 2^-24 of the largest (the unit is at most a quarter of
    it, and the last part's step 2^-21 of the unit), whichever is more."""
    def prep(k, v):
        k.zero_()
        k[:, :, 3, 0] = 20.0
        v[:, :, 4:] = v[:, :, 4:5]
    # (so many pairs that none is cut)
    p = Decode(heads, [1024, 1000, 777] * (56 // heads[1]) + [900] * 6, 16, False, prep=prep)
    n = p.q.shape[0] * p.q.shape[1]
    ramp = torch.linspace(3.0, 5.0, n, device="cuda").view(p.q.shape[:2])
    p.q[..., 0] = (ramp * math.sqrt(p.d / 128)).bfloat16()
    p.call()
    assert p.status() == 0
    p.check()
    group = p.hq // p.hkv
    for b, n in enumerate(p.lens):
        for h in range(p.hkv):
            k, v = (p.cache.rows(x, b, h, n) for x in "kv")
            q = p.q[b, h * group:(h + 1) * group].double()
            want, lse, w = attend(q, k, v, p.scale)
            prob = torch.exp(q @ k.T * p.scale - lse[:, None])
            vs = p.cache.scales("v", b, h, n)
            codes = torch.where(vs[:, None] > 0, v / vs[:, None], 0.0)
            big = float(q.norm(dim=-1).max() * k.norm(dim=-1).max()) * p.scale
            tol = (2.0 ** -16 + 2.0 ** -18 + 2.0 ** -20 * big) * w \
                + 2.0 ** -24 * (prob * vs).amax(1, keepdim=True) * codes.abs().sum(0)
            err = (p.out[b, h * group:(h + 1) * group].double() - want).abs()
            assert (err <= tol).all(), float((err / tol).max())
