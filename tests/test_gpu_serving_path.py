"""The cache and prompt calls in a row, as a server makes them: prompts of
different lengths appended in chunks, the chunks' attention, the statistics of
the blocks that became complete, then decode steps (append one token, select,
decode), over a bf16 cache and over an E4M3 cache whose chunks are read back
as pages.  Every result is checked against the softmax in 64 bits over what
the cache holds, and the cache's keys against the rotated projections."""

import itertools
import math

import pytest
import torch

import block_sparse_long_cobs_b200 as cb
from cache_ref import (B, attend, bf16_rows, cu_of, frequencies, ints, page_table, quantise,
                       rotate, workspace)

pytestmark = pytest.mark.gpu

HQ, HKV, D, RANK = 8, 2, 128, 4
G = HQ // HKV
SCALE = 1.0 / math.sqrt(D)


class Server:
    def __init__(self, lens, cap, e4m3, paged, seed=7):
        self.g = torch.Generator(device="cuda")
        self.g.manual_seed(seed)
        self.batch, self.cap, self.e4m3, self.paged = len(lens), cap, e4m3, paged
        nb = cap // B
        self.table = None
        shape = (self.batch, HKV, cap)
        if paged:
            self.table, n_pages = page_table(self.g, [nb] * self.batch, spare=2, width_pad=0)
            shape = (n_pages, HKV, B)
        kind = torch.uint8 if e4m3 else torch.bfloat16
        # unused rows: a NaN code, or NaN
        self.k = torch.full(shape + (D,), 0x7F if e4m3 else float("nan"), dtype=kind, device="cuda")
        self.v = self.k.clone()
        self.ks = torch.full(shape, float("nan"), device="cuda") if e4m3 else None
        self.vs = self.ks.clone() if e4m3 else None
        self.cache = cb.cobs_kv_cache(self.k, self.v, self.ks, self.vs, self.table,
                                      shape[0] if paged else 0, nb if paged else 0, int(e4m3))
        self.dims = cb.cobs_dims(batch=self.batch, num_q_heads=HQ, num_kv_heads=HKV, head_dim=D,
                                 block_size=B, rank=RANK, capacity_tokens=cap)
        self.rope = cb.cobs_rope_init(64, False, scaling=cb.COBS_ROPE_LINEAR, factor=2.0)
        self.f = frequencies(64, scaling=cb.COBS_ROPE_LINEAR, factor=2.0)
        self.lens = [0] * self.batch
        self.stats = torch.zeros(self.batch, HKV, nb, (1 + RANK) * D, dtype=torch.bfloat16,
                                 device="cuda")
        self.ws = workspace(cb.cobs_prompt_workspace_bytes(self.dims, 512, cap))
        self.top_k, self.sink, self.local = 4, 1, 64
        self.stride = cb.cobs_selected_capacity(self.dims, self.top_k, self.sink, self.local)
        self.dws = workspace(cb.cobs_workspace_bytes(self.dims, self.top_k, self.sink, self.local))
        self.want_k = [[] for _ in range(self.batch)]      # rotated keys in 64 bits
        # pages of the read-back cache: block j of sequence b is page b * nb + j
        self.pages = torch.full((self.batch * nb, HKV, B, D), float("nan"), dtype=torch.bfloat16,
                                device="cuda")
        self.vpages = self.pages.clone()
        self.ptable = torch.arange(self.batch * nb, dtype=torch.int32, device="cuda").view(
            self.batch, nb)

    def rows(self, name, b, h):
        n = self.lens[b]
        x = {"k": (self.k, self.ks), "v": (self.v, self.vs)}[name]

        def get(t):
            if self.table is None:
                return t[b, h, :n]
            return t[self.table[b].long(), h].flatten(0, 1)[:n]
        if self.e4m3:
            return get(x[0]).contiguous().view(torch.float8_e4m3fn).double() * \
                get(x[1]).double()[:, None]
        return get(x[0]).double()

    def append(self, counts):
        n = sum(counts)
        qkv = bf16_rows(self.g, n, HQ + 2 * HKV, D, scale=1.5)
        q_out = torch.empty(n, HQ, D, dtype=torch.bfloat16, device="cuda")
        wide = (HQ + 2 * HKV) * D
        one = all(c == 1 for c in counts)
        cb.cobs_append_tokens(self.dims, self.cache, self.rope, qkv[:, :HQ], wide,
                              qkv[:, HQ:HQ + HKV], wide, qkv[:, HQ + HKV:], wide,
                              None if one else cu_of(counts), n, ints(self.lens), q_out, self.ws,
                              self.ws.numel())
        first = 0
        for b, c in enumerate(counts):
            pos = torch.arange(self.lens[b], self.lens[b] + c, device="cuda")
            x = qkv[first:first + c, HQ:HQ + HKV].double()
            self.want_k[b].append(rotate(x, pos, self.f, False)[0])
            self.lens[b] += c
            first += c
        return q_out

    def bf16_cache(self):
        """The cache that statistics and prompt attention read."""
        if not self.e4m3:
            return self.cache
        nb = self.cap // B
        cb.cobs_read_cache(self.dims, self.cache, ints(self.lens), 0, nb, self.pages, self.vpages,
                           self.ws, self.ws.numel())
        return cb.cobs_kv_cache(self.pages, self.vpages, None, None, self.ptable, self.batch * nb,
                                nb, cb.COBS_CACHE_BF16)

    def prompt(self, counts):
        q = self.append(counts)
        cache = self.bf16_cache()
        out = torch.empty_like(q)
        lse = torch.empty(q.shape[:2], device="cuda")
        cb.cobs_prompt_attention(self.dims, cache, q, cu_of(counts), q.shape[0], ints(self.lens),
                                 max(self.lens), SCALE, out, lse, self.ws, self.ws.numel())
        first = 0
        for b, c in enumerate(counts):
            for h in range(HKV if c else 0):
                k, v = self.rows("k", b, h), self.rows("v", b, h)
                if self.e4m3:
                    k, v = k.float().bfloat16().double(), v.float().bfloat16().double()
                for i, g in itertools.product((0, c // 2, c - 1), range(G)):
                    n = self.lens[b] - c + i + 1
                    qr = q[first + i, h * G + g].double()[None]
                    want, wl, w = attend(qr, k[:n], v[:n], SCALE)
                    got = out[first + i, h * G + g].double()
                    assert ((got - want[0]).abs() <= 2.0 ** -8 * want[0].abs()
                            + 2.0 ** -7 * w[0]).all()
                    assert abs(float(lse[first + i, h * G + g] - wl[0])) <= 2.0 ** -10
            first += c
        # statistics of every block that is complete by now
        done = min(self.lens) // B
        src = cache
        if src.block_table:
            pool, tab = (self.pages, self.ptable) if self.e4m3 else (self.k, self.table)
            cb.cobs_build_block_stats_paged(self.dims, pool, pool.shape[0], tab, tab.shape[1], 0,
                                            done, self.stats, self.ws, self.ws.numel())
        else:
            cb.cobs_build_block_stats(self.dims, self.k, 0, done, self.stats, self.ws,
                                      self.ws.numel())

    def decode(self):
        q = self.append([1] * self.batch)
        idx = torch.full((self.batch, HKV, self.stride), -5, dtype=torch.int32, device="cuda")
        n_sel = torch.zeros(self.batch, HKV, dtype=torch.int32, device="cuda")
        out = torch.empty(self.batch, HQ, D, device="cuda")
        lse = torch.empty(self.batch, HQ, device="cuda")
        lens, most = ints(self.lens), max(self.lens)
        cb.cobs_select_blocks_varlen(self.dims, q, self.stats, lens, most, self.top_k, self.sink,
                                     self.local, idx, self.stride, n_sel, None, self.dws,
                                     self.dws.numel())
        cb.cobs_sparse_decode_cache(self.dims, self.cache, q, idx, n_sel, self.stride, lens, most,
                                    SCALE, out, lse, self.dws, self.dws.numel())
        for b, h in itertools.product(range(self.batch), range(HKV)):
            blocks = idx[b, h, :int(n_sel[b, h])].tolist()
            n = self.lens[b]
            assert 0 in blocks and (n - 1) // B in blocks and blocks == sorted(set(blocks))
            at = torch.cat([torch.arange(j * B, min(n, j * B + B), device="cuda") for j in blocks])
            k, v = self.rows("k", b, h)[at], self.rows("v", b, h)[at]
            want, wl, w = attend(q[b, h * G:(h + 1) * G].double(), k, v, SCALE)
            got = out[b, h * G:(h + 1) * G].double()
            assert ((got - want).abs() <= 2.0 ** -13 * w + 2.0 ** -16).all()
            assert ((lse[b, h * G:(h + 1) * G].double() - wl).abs() <= 2.0 ** -13).all()

    def finish(self):
        assert cb.cobs_read_device_status(self.ws, self.ws.numel()) == 0
        assert cb.cobs_read_device_status(self.dws, self.dws.numel()) == 0
        for b, h in itertools.product(range(self.batch), range(HKV)):
            want = torch.cat(self.want_k[b])[:, h]
            got = self.rows("k", b, h)
            step = 2.0 ** -4 if self.e4m3 else 2.0 ** -8
            top = want.abs().amax(-1, keepdim=True)
            assert ((got - want).abs() <= step * want.abs() + 2.0 ** -18 * top).all()


@pytest.mark.parametrize("paged", [False, True])
@pytest.mark.parametrize("e4m3", [False, True])
def test_prompt_in_chunks_then_decode(e4m3, paged):
    s = Server([0, 0, 0], 1024, e4m3, paged)
    s.prompt([300, 129, 200])
    s.prompt([1, 70, 0])
    s.prompt([256, 100, 64])
    for _ in range(3):
        s.decode()
    s.prompt([5, 60, 130])
    s.decode()
    s.finish()


def test_wrong_memory_is_refused():
    """A host address where device memory is needed."""
    s = Server([0], 128, False, False)
    host = torch.zeros(4, HQ, D, dtype=torch.bfloat16)
    with pytest.raises(TypeError):
        cb.cobs_prompt_attention(s.dims, s.cache, host, cu_of([4]), 4, ints([4]), 64, SCALE,
                                 torch.zeros(4, HQ, D, device="cuda"), None, s.ws, s.ws.numel())
    with pytest.raises(cb.CobsError) as e:
        cb.cobs_prompt_attention(s.dims, s.cache, host.data_ptr() & ~15, cu_of([4]), 4, ints([4]),
                                 64, SCALE, torch.zeros(4, HQ, D, dtype=torch.bfloat16,
                                                        device="cuda"), None, s.ws, s.ws.numel())
    assert e.value.status == cb.COBS_ERR_INVALID_ARG
    assert "device pointer" in cb.cobs_last_error()


def test_append_then_fused_selection_and_decode():
    """Decode steps without a host wait between the calls: append, then the call
    whose decode starts while the selection still runs, against the separate
    calls on the same cache with the GPU idle in between."""
    batch, cap, n0, hkv = 40, 1024, 700, 8
    g = torch.Generator(device="cuda").manual_seed(3)
    k, v = (bf16_rows(g, batch, hkv, cap, D) for _ in range(2))
    dims = cb.cobs_dims(batch=batch, num_q_heads=4 * hkv, num_kv_heads=hkv, head_dim=D,
                        block_size=B, rank=RANK, capacity_tokens=cap)
    cache = cb.cobs_kv_cache(k, v)
    rope = cb.cobs_rope_init(D, True)
    stats = torch.zeros(batch, hkv, cap // B, (1 + RANK) * D, dtype=torch.bfloat16, device="cuda")
    stride = cb.cobs_selected_capacity(dims, 3, 1, 64)
    size = cb.cobs_workspace_bytes(dims, 3, 1, 64)
    ws, ws2 = workspace(size), workspace(size)
    cb.cobs_build_block_stats(dims, k, 0, n0 // B, stats, ws, size)

    def buffers():
        return (torch.zeros(batch, hkv, stride, dtype=torch.int32, device="cuda"),
                torch.zeros(batch, hkv, dtype=torch.int32, device="cuda"),
                torch.zeros(batch, 4 * hkv, D, device="cuda"),
                torch.zeros(batch, 4 * hkv, device="cuda"))
    steps = 6
    qkv = [bf16_rows(g, batch, 6 * hkv, D, scale=2.0) for _ in range(steps)]
    got = [buffers() for _ in range(steps)]
    q = [torch.zeros(batch, 4 * hkv, D, dtype=torch.bfloat16, device="cuda") for _ in range(steps)]
    torch.cuda.synchronize()
    starts = [ints([n0 + t] * batch) for t in range(steps)]
    torch.cuda.synchronize()
    for t in range(steps):
        x, wide = qkv[t], 6 * hkv * D
        cb.cobs_append_tokens(dims, cache, rope, x[:, :4 * hkv], wide, x[:, 4 * hkv:5 * hkv], wide,
                              x[:, 5 * hkv:], wide, None, batch, starts[t], q[t], ws, size)
        idx, n_sel, out, lse = got[t]
        cb.cobs_select_and_decode(dims, q[t], stats, k, v, n0 + t + 1, 3, 1, 64, SCALE, idx, stride,
                                  n_sel, None, out, lse, ws, size)
    assert cb.cobs_read_device_status(ws, size) == 0
    for t in range(steps):
        idx, n_sel, out, lse = buffers()
        cb.cobs_select_blocks(dims, q[t], stats, n0 + t + 1, 3, 1, 64, idx, stride, n_sel, None,
                              ws2, size)
        torch.cuda.synchronize()
        cb.cobs_sparse_decode_cache(dims, cache, q[t], idx, n_sel, stride, None, n0 + t + 1, SCALE,
                                    out, lse, ws2, size)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got[t], (idx, n_sel, out, lse)))


@pytest.mark.parametrize("e4m3", [False, True])
def test_one_workspace_for_every_call(e4m3):
    """Prompt attention whose units are cut, selection, decode and the fused
    call in turn on one workspace, against the same calls on workspaces of their
    own: no call leaves the others' counters changed."""
    batch, cap, hkv, hq = 8, 2048, 4, 16
    g = torch.Generator(device="cuda").manual_seed(11)
    k, v = (bf16_rows(g, batch, hkv, cap, D) for _ in range(2))
    dims = cb.cobs_dims(batch=batch, num_q_heads=hq, num_kv_heads=hkv, head_dim=D, block_size=B,
                        rank=RANK, capacity_tokens=cap)
    cache = cb.cobs_kv_cache(k, v)
    dcache = cache
    if e4m3:
        (kc, ks), (vc, vs) = quantise(k), quantise(v)
        dcache = cb.cobs_kv_cache(kc, vc, ks, vs, format=cb.COBS_CACHE_E4M3)
    counts, lens = [40, 1, 0, 200, 3, 17, 64, 5], [1500, 2048, 64, 1999, 1100, 700, 1280, 2000]
    n, most = sum(counts), max(lens)
    stats = torch.zeros(batch, hkv, cap // B, (1 + RANK) * D, dtype=torch.bfloat16, device="cuda")
    stride = cb.cobs_selected_capacity(dims, 5, 1, 64)
    size = cb.cobs_workspace_bytes(dims, 5, 1, 64)
    psize = cb.cobs_prompt_workspace_bytes(dims, n, most)
    cb.cobs_build_block_stats(dims, k, 0, cap // B, stats, workspace(), 256)
    pq = bf16_rows(g, n, hq, D, scale=2.0)
    q = bf16_rows(g, batch, hq, D, scale=2.0)
    cu, sl = cu_of(counts), ints(lens)
    torch.cuda.synchronize()

    def step(ws_of):
        out = torch.zeros_like(pq)
        plse = torch.zeros(n, hq, device="cuda")
        res = [out, plse]
        ws = ws_of("prompt", psize)
        cb.cobs_prompt_attention(dims, cache, pq, cu, n, sl, most, SCALE, out, plse, ws,
                                 ws.numel())
        for fused in (False, True):
            idx = torch.zeros(batch, hkv, stride, dtype=torch.int32, device="cuda")
            n_sel = torch.zeros(batch, hkv, dtype=torch.int32, device="cuda")
            o = torch.zeros(batch, hq, D, device="cuda")
            lse = torch.zeros(batch, hq, device="cuda")
            ws = ws_of("fused" if fused else "select", size)
            if fused:
                cb.cobs_select_and_decode(dims, q, stats, k, v, 1900, 5, 1, 64, SCALE, idx, stride,
                                          n_sel, None, o, lse, ws, ws.numel())
            else:
                cb.cobs_select_blocks(dims, q, stats, 1900, 5, 1, 64, idx, stride, n_sel, None, ws,
                                      ws.numel())
                ws = ws_of("decode", size)
                cb.cobs_sparse_decode_cache(dims, dcache, q, idx, n_sel, stride, None, 1900, SCALE,
                                            o, lse, ws, ws.numel())
            res += [idx, n_sel, o, lse]
        torch.cuda.synchronize()
        return res

    own = {}

    def own_ws(name, nbytes):
        own.setdefault(name, workspace(nbytes))
        return own[name]
    want = step(own_ws)
    shared = workspace(max(size, psize))
    for _ in range(4):
        got = step(lambda name, nbytes: shared)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    for ws in [shared, *own.values()]:
        assert cb.cobs_read_device_status(ws, ws.numel()) == 0


def test_every_buffer_in_host_memory_is_refused():
    """A host address in place of any buffer of a call: INVALID_ARG, no launch."""
    host = torch.zeros(1 << 16, dtype=torch.uint8).data_ptr() + 15 & ~15
    dev = torch.zeros(1 << 20, dtype=torch.uint8, device="cuda").data_ptr()
    dims = cb.cobs_dims(batch=2, num_q_heads=4, num_kv_heads=1, head_dim=64, block_size=B, rank=0,
                        capacity_tokens=64)
    rope = cb.cobs_rope_init(64)

    def append(c, q, k, v, cu, start, out, ws):
        cb.cobs_append_tokens(dims, c, rope, q, 256, k, 64, v, 64, cu, 2, start, out, ws, 1 << 16)

    def read(c, lens, k, v, ws):
        cb.cobs_read_cache(dims, c, lens, 0, 1, k, v, ws, 1 << 16)

    def prompt(c, q, cu, lens, out, lse, ws):
        cb.cobs_prompt_attention(dims, c, q, cu, 2, lens, 64, SCALE, out, lse, ws, 1 << 16)

    def decode(c, q, idx, n, lens, out, lse, ws):
        cb.cobs_sparse_decode_cache(dims, c, q, idx, n, 1, lens, 64, SCALE, out, lse, ws, 1 << 16)
    for fn, n, formats in ((append, 7, (0, 1)), (read, 4, (0, 1)), (prompt, 6, (0,)),
                           (decode, 7, (0, 1))):
        for fmt in formats:
            for bad in range(n + 5):
                if fmt == 0 and bad in (2, 3):        # scales of a bf16 cache: not looked at
                    continue
                at = [host if i == bad else dev for i in range(n + 5)]
                cache = cb.cobs_kv_cache(*at[:5], n_pages=1, table_stride=1, format=fmt)
                with pytest.raises(cb.CobsError) as e:
                    fn(cache, *at[5:])
                assert e.value.status == cb.COBS_ERR_INVALID_ARG, (fn.__name__, bad)
                assert "not a device pointer" in cb.cobs_last_error()
    torch.cuda.synchronize()
