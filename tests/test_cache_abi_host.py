"""Host-side checks of the cache and prompt calls: exported symbols, argument
checks before any launch, and the rotary table (no GPU)."""

import ctypes
import itertools
import math
import os
import re
from fractions import Fraction

import pytest

import block_sparse_long_cobs_b200 as cb

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
A = 1 << 20            # a fake address: never dereferenced, rejected first
INV, UNS, WS = cb.COBS_ERR_INVALID_ARG, cb.COBS_ERR_UNSUPPORTED, cb.COBS_ERR_WORKSPACE


def test_every_declared_symbol_is_exported():
    text = open(os.path.join(ROOT, "include", "cobs_cache.h")).read()
    names = sorted(set(re.findall(r"COBS_API\s+[\w\s\*]+?\b(cobs_\w+)\s*\(", text)))
    assert names == ["cobs_append_tokens", "cobs_prompt_attention", "cobs_prompt_workspace_bytes",
                     "cobs_read_cache", "cobs_rope_init", "cobs_sparse_decode_cache"]
    raw = ctypes.CDLL(cb.LIB_PATH)
    for n in names:
        assert hasattr(raw, n) and callable(getattr(cb, n)), n


def dims(**kw):
    return dict(dict(batch=2, num_q_heads=8, num_kv_heads=2, head_dim=128, block_size=64, rank=8,
                     capacity_tokens=4096), **kw)


def cache(**kw):
    return cb.cobs_kv_cache(**dict(dict(k=A, v=A), **kw))


E4 = dict(k_scale=A, v_scale=A, format=cb.COBS_CACHE_E4M3)
PAGED = dict(block_table=A, n_pages=100, table_stride=64)
BAD_CACHES = [
    (None, INV), (cache(k=None), INV), (cache(v=None), INV), (cache(k=A + 8), INV),
    (cache(format=2), INV), (cache(format=cb.COBS_CACHE_E4M3), INV),
    (cache(**dict(E4, k_scale=None)), INV), (cache(**dict(E4, v_scale=A + 4)), INV),
    (cache(**dict(PAGED, block_table=A + 4)), INV), (cache(**dict(PAGED, n_pages=0)), INV),
    (cache(**dict(PAGED, n_pages=1 << 24)), UNS), (cache(**dict(PAGED, table_stride=0)), INV),
]


def refuse(code, fn, **kw):
    with pytest.raises(cb.CobsError) as e:
        fn(**kw)
    assert e.value.status == code, (e.value, kw)
    assert cb.cobs_last_error()


def append(**kw):
    a = dict(dims=dims(), cache=cache(), rope=cb.cobs_rope_init(128), q=A, q_stride=1024, k=A,
             k_stride=256, v=A, v_stride=256, cu_tokens=A, n_tokens=5, start=A, q_out=A + 4096,
             ws=A, ws_bytes=256)
    a.update(kw)
    cb.cobs_append_tokens(**a)


def test_append_refusals():
    for c, code in BAD_CACHES:
        refuse(code, append, cache=c)
    for kw in (dict(k=None), dict(v=None), dict(k=A + 2), dict(k_stride=248), dict(k_stride=260),
               dict(v_stride=8), dict(q_stride=1016), dict(q=A + 8), dict(q_out=None),
               dict(q_out=A + 2), dict(q=None, q_stride=0), dict(start=None), dict(start=A + 8),
               dict(cu_tokens=A + 4), dict(n_tokens=-1), dict(cu_tokens=None),
               dict(q=A, q_out=A, q_stride=2048), dict(ws=A + 1),
               dict(rope=cb.cobs_rope_init(128), dims=dims(head_dim=64))):
        refuse(INV, append, **kw)
    bad = cb.cobs_rope_init(64)
    bad.rotary_dim = 12
    refuse(INV, append, rope=bad)
    bad.rotary_dim, bad.attention_factor = 64, math.nan
    refuse(INV, append, rope=bad)
    refuse(UNS, append, n_tokens=1 << 28)
    refuse(UNS, append, dims=dims(head_dim=96))
    refuse(WS, append, ws=None)
    refuse(WS, append, ws_bytes=128)
    append(n_tokens=0)      # nothing to do: no launch


def read(**kw):
    a = dict(dims=dims(), cache=cache(**E4), seq_lens=A, block_begin=0, block_end=4, k_out=A,
             v_out=A, ws=A, ws_bytes=256)
    a.update(kw)
    cb.cobs_read_cache(**a)


def test_read_refusals():
    for c, code in BAD_CACHES:
        refuse(code, read, cache=c)
    for kw in (dict(block_begin=-1), dict(block_end=65), dict(block_begin=5), dict(k_out=None,
               v_out=None), dict(k_out=A + 8), dict(v_out=A + 8), dict(seq_lens=A + 8),
               dict(cache=cache(**dict(PAGED, table_stride=3)))):
        refuse(INV, read, **kw)
    refuse(WS, read, ws=None)
    refuse(WS, read, ws_bytes=64)
    read(block_begin=3, block_end=3)


def prompt(**kw):
    a = dict(dims=dims(), cache=cache(), q=A, cu_tokens=A, n_tokens=40, seq_lens=A,
             max_seq_len=4096, softmax_scale=0.1, out=A, lse=A, ws=A, ws_bytes=1 << 40)
    a.update(kw)
    cb.cobs_prompt_attention(**a)


def test_prompt_refusals():
    for c, code in BAD_CACHES:
        refuse(code, prompt, cache=c)
    for kw in (dict(q=None), dict(q=A + 2), dict(out=None), dict(out=A + 8), dict(lse=A + 4),
               dict(seq_lens=None), dict(seq_lens=A + 8), dict(cu_tokens=A + 4),
               dict(cu_tokens=None), dict(n_tokens=-1), dict(max_seq_len=0),
               dict(max_seq_len=4097), dict(softmax_scale=0.0), dict(softmax_scale=math.inf),
               dict(softmax_scale=math.nan), dict(cache=cache(**dict(PAGED, table_stride=63)))):
        refuse(INV, prompt, **kw)
    refuse(UNS, prompt, cache=cache(**E4))
    refuse(UNS, prompt, n_tokens=1 << 28)
    refuse(WS, prompt, ws=None)
    need = cb.cobs_prompt_workspace_bytes(dims(), 40, 4096)
    refuse(WS, prompt, ws_bytes=need - 1)
    prompt(n_tokens=0)
    for kw in (dict(n_tokens=-1), dict(max_seq_len=0), dict(max_seq_len=5000)):
        refuse(INV, cb.cobs_prompt_workspace_bytes,
               **dict(dict(dims=dims(), n_tokens=4, max_seq_len=64), **kw))
    # a program may size its workspace once, for its largest call
    sizes = [cb.cobs_prompt_workspace_bytes(dims(), n, t) for n, t in ((1, 64), (1, 4096))]
    assert sizes == sorted(sizes)


def test_token_counts_that_overflow_are_refused():
    """Products with the head counts would wrap around to nothing."""
    for n in (1 << 62, (1 << 63) - 1, (1 << 64) // 12 + 1, (1 << 31) // 12 + 1):
        for fn in (append, prompt):
            refuse(UNS, fn, n_tokens=n)
        with pytest.raises(cb.CobsError):
            cb.cobs_prompt_workspace_bytes(dims(), n, 64)


def test_empty_calls_need_no_buffers_of_rows():
    """No token, no block: an empty tensor has no address, and nothing is done."""
    append(n_tokens=0, q=None, k=None, v=None, q_out=None)
    append(n_tokens=0, q=A, k=None, v=None, q_out=None)
    prompt(n_tokens=0, q=None, out=None, lse=None)
    read(block_begin=2, block_end=2, k_out=None, v_out=None)
    for kw in (dict(start=None), dict(ws_bytes=8), dict(cache=cache(k=None))):
        with pytest.raises(cb.CobsError):
            append(n_tokens=0, k=None, v=None, q=None, q_out=None, **kw)


def test_prompt_partials_lie_behind_the_counters():
    """One workspace may serve the prompt attention, the selection and the
    decode: the split rows of the first leave the counters of the others alone,
    which take 4 + 4 + 8 bytes per (sequence, kv-head)."""
    for hkv in (2, 8):
        need = [cb.cobs_prompt_workspace_bytes(
            dims(batch=b, num_q_heads=4 * hkv, num_kv_heads=hkv), 100000, 4096)
            for b in (1, 50, 2000)]
        for (b0, n0), (b1, n1) in itertools.pairwise(zip((1, 50, 2000), need)):
            # (each of the three arrays is padded to 256 bytes)
            assert n1 - n0 >= 16 * hkv * (b1 - b0) - 3 * 256


def decode(**kw):
    a = dict(dims=dims(), cache=cache(**E4), q=A, idx=A, n_sel=A, idx_stride=8, seq_lens=A,
             max_seq_len=4096, softmax_scale=0.1, out=A, lse=A, ws=A, ws_bytes=1 << 40)
    a.update(kw)
    cb.cobs_sparse_decode_cache(**a)


def test_decode_refusals():
    for c, code in BAD_CACHES:
        refuse(code, decode, cache=c)
    for kw in (dict(q=None), dict(idx=None), dict(n_sel=A + 4), dict(out=None), dict(lse=None),
               dict(idx_stride=0), dict(max_seq_len=0), dict(max_seq_len=4097),
               dict(softmax_scale=-1.0), dict(seq_lens=A + 8),
               dict(cache=cache(**dict(E4, **dict(PAGED, table_stride=63))))):
        refuse(INV, decode, **kw)
    refuse(WS, decode, ws_bytes=1024)


# ---------------------------------------------------------------------------
# rotary table
# ---------------------------------------------------------------------------

def test_rope_refusals():
    ok = dict(rotary_dim=64)
    for kw in (dict(rotary_dim=-8), dict(rotary_dim=12), dict(rotary_dim=136), dict(scaling=4),
               dict(base=1.0), dict(base=math.nan), dict(attention_factor=0.0),
               dict(attention_factor=math.inf), dict(scaling=cb.COBS_ROPE_LINEAR, factor=0.5),
               dict(scaling=cb.COBS_ROPE_BY_PARTS, factor=2.0, original_context=0, low=1, high=2),
               dict(scaling=cb.COBS_ROPE_BY_PARTS, factor=2.0, original_context=9, low=2, high=2),
               dict(scaling=cb.COBS_ROPE_BY_PARTS, factor=2.0, original_context=9, low=-1, high=2),
               dict(scaling=cb.COBS_ROPE_CUSTOM),
               dict(scaling=cb.COBS_ROPE_CUSTOM, frequencies=[4.0] * 32),
               dict(scaling=cb.COBS_ROPE_CUSTOM, frequencies=[-0.1] * 32)):
        refuse(INV, cb.cobs_rope_init, **dict(ok, **kw))
    with pytest.raises(ValueError):
        cb.cobs_rope_init(64, scaling=cb.COBS_ROPE_CUSTOM, frequencies=[0.1] * 31)


def turns_of(f):
    return f / (2 * math.pi)


@pytest.mark.parametrize("kw", [
    dict(), dict(base=500000.0), dict(scaling=cb.COBS_ROPE_LINEAR, factor=4.0),
    dict(scaling=cb.COBS_ROPE_BY_PARTS, factor=8.0, original_context=8192.0, low=1.0, high=4.0)])
def test_rope_table(kw):
    for r in (0, 8, 64, 128):
        t = cb.cobs_rope_init(r, **kw)
        assert t.rotary_dim == r and t.attention_factor == 1.0
        for i in range(r // 2):
            f = kw.get("base", 10000.0) ** (-2.0 * i / r)
            if kw.get("scaling") == cb.COBS_ROPE_LINEAR:
                f /= 4.0
            if kw.get("scaling") == cb.COBS_ROPE_BY_PARTS:
                g = min(1.0, max(0.0, (8192.0 * turns_of(f) - 1.0) / 3.0))
                f = f * g + f / 8.0 * (1 - g)
            assert abs(t.turns[i] / 2.0 ** 64 - turns_of(f)) <= 2.0 ** -50 * turns_of(f) + 2.0 ** -64
        assert all(t.turns[i] == 0 for i in range(r // 2, 64))


def test_rope_far_positions_keep_their_turn():
    """position x turns modulo 2^64 against the exact fraction."""
    t = cb.cobs_rope_init(16, scaling=cb.COBS_ROPE_CUSTOM,
                          frequencies=[1.0, 0.5, 1e-3, 3.0, 0.0, 1e-9, 0.1, math.pi])
    # pi to 40 digits
    pi = Fraction(31415926535897932384626433832795028841971, 10 ** 40)
    for i, f in enumerate([1.0, 0.5, 1e-3, 3.0, 0.0, 1e-9, 0.1, math.pi]):
        for p in (1, 4095, 262143, (1 << 31) - 1):
            got = Fraction((p * t.turns[i]) % (1 << 64), 1 << 64)
            want = Fraction(f) * p / (2 * pi)
            want -= want.numerator // want.denominator
            gap = abs(got - want)
            assert min(gap, 1 - gap) <= Fraction(p, 1 << 62)
