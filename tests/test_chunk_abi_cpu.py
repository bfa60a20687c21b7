"""CPU checks of the chunk calls and the windowed decode: arguments that must be refused before any launch."""
import ctypes
import os

import numpy as np
import pytest

from attention_group_quantized_gb300 import kvq

P = ctypes.byref
A = 0x10000      # an aligned address, never dereferenced: every call here ends before a launch


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(kvq.LIB_PATH):
        from attention_group_quantized_gb300 import build
        build.build()
    return kvq.lib()


def _cache(hb=(8, 8), B=2, Tcap=128, D=128, codes=A, sz=A):
    hb = np.asarray(hb, np.int8)
    c = kvq.CCache(codes, sz, hb.ctypes.data, B, len(hb), Tcap, D)
    c.keep = hb
    return c


def _chunk(start=A, lens=A, B=2, rows=10, max_chunk=0):
    return kvq.CChunk(start, lens, B, rows, max_chunk)


def _table(pages=A, B=2, max_pages=3):
    return kvq.CBlockTable(pages, B, max_pages)


BAD_CHUNKS = [
    (dict(start=None), 1), (dict(lens=None), 1), (dict(start=A + 2), 1), (dict(lens=A + 1), 1), (dict(B=3), 1),
    (dict(B=0), 1), (dict(rows=-1), 1), (dict(max_chunk=-1), 1), (dict(rows=(1 << 30)), 2),
]


@pytest.mark.parametrize("change,want", BAD_CHUNKS, ids=[str(c[0]) for c in BAD_CHUNKS])
def test_chunk_descriptions_are_refused_by_every_call(L, change, want):
    k, ch, big = _cache(), _chunk(**change), 1 << 40
    assert L.kvq_append_chunk(A, A, 256, 128, P(ch), P(k), P(k), None, None) == want
    assert L.kvq_dequantize(P(k), P(ch), A, 0, None, None) == want
    assert L.kvq_chunk_attention(A, 1024, 128, P(ch), P(k), P(k), 8, 0.0, 0, 0, A, 0, A, big, None, None) == want
    pool, bt = _cache(B=9, Tcap=64), _table()
    assert L.kvq_append_chunk_paged(A, A, 256, 128, P(ch), P(pool), P(pool), P(bt), None, None) == want
    assert L.kvq_dequantize_paged(P(pool), P(ch), P(bt), A, 0, None, None) == want
    assert L.kvq_chunk_attention_paged(A, 1024, 128, P(ch), P(pool), P(pool), P(bt), 8, 0.0, 0, 0, A, 0, A, big, None,
                                       None) == want


def test_no_rows_is_nothing_to_do(L):
    k, ch = _cache(), _chunk(rows=0)
    assert L.kvq_append_chunk(A, A, 256, 128, P(ch), P(k), P(k), None, None) == 0
    assert L.kvq_dequantize(P(k), P(ch), A, 0, None, None) == 0
    assert L.kvq_chunk_attention(A, 1024, 128, P(ch), P(k), P(k), 8, 0.0, 0, 0, A, 0, A, 1 << 40, None, None) == 0


def test_no_rows_need_no_row_buffers(L):
    """An empty tensor has no address."""
    k, ch = _cache(), _chunk(rows=0)
    assert L.kvq_append_chunk(None, None, 256, 128, P(ch), P(k), P(k), None, None) == 0
    assert L.kvq_dequantize(P(k), P(ch), None, 0, None, None) == 0
    assert L.kvq_chunk_attention(None, 1024, 128, P(ch), P(k), P(k), 8, 0.0, 0, 0, None, 0, A, 1 << 40, None, None) == 0
    pool, bt = _cache(B=9, Tcap=64), _table()
    assert L.kvq_dequantize_paged(P(pool), P(ch), P(bt), None, 1, None, None) == 0
    assert L.kvq_append_chunk(A, None, 256, 128, P(_chunk()), P(k), P(k), None, None) == 1


def test_more_sequences_than_the_tables_hold(L):
    k, ch = _cache(B=4097), _chunk(B=4097)
    assert L.kvq_append_chunk(A, A, 256, 128, P(ch), P(k), P(k), None, None) == 2
    assert L.kvq_dequantize(P(k), P(ch), A, 0, None, None) == 2
    assert L.kvq_chunk_attention(A, 1024, 128, P(ch), P(k), P(k), 8, 0.0, 0, 0, A, 0, A, 1 << 40, None, None) == 2
    assert L.kvq_decode_attention_window(A, P(k), P(k), A, 8, 0.0, 16, 0, A, 0, A, 1 << 40, None, None) == 2


def test_append_refusals(L):
    k, ch = _cache(), _chunk()
    call = lambda kn=A, vn=A, sr=256, sh=128, c=P(ch), a=P(k), b=P(k): L.kvq_append_chunk(kn, vn, sr, sh, c, a, b,
                                                                                         None, None)
    assert call(kn=None) == 1 and call(vn=None) == 1 and call(a=None) == 1 and call(b=None) == 1 and call(c=None) == 1
    assert call(kn=A + 8) == 1 and call(vn=A + 2) == 1
    assert call(sr=257) == 1 and call(sh=100) == 1 and call(sr=-256) == 1
    assert call(b=P(_cache((8, 4)))) == 1 and call(b=P(_cache(Tcap=64))) == 1
    assert call(a=P(_cache(codes=None))) == 1 and call(b=P(_cache(sz=A + 4))) == 1
    assert call(a=P(_cache(D=96)), b=P(_cache(D=96))) == 2
    pool, bt = _cache(B=9, Tcap=64), _table()
    paged = lambda t, p=pool: L.kvq_append_chunk_paged(A, A, 256, 128, P(ch), P(p), P(p), t, None, None)
    assert paged(None) == 1 and paged(P(_table(pages=None))) == 1 and paged(P(_table(pages=A + 1))) == 1
    assert paged(P(_table(max_pages=0))) == 1 and paged(P(_table(B=3))) == 1
    assert paged(P(bt), k) == 1                                 # not a pool of 64-token pages


def test_dequantize_refusals(L):
    k, ch = _cache(), _chunk()
    call = lambda s=P(k), c=P(ch), o=A, dt=0: L.kvq_dequantize(s, c, o, dt, None, None)
    assert call(s=None) == 1 and call(c=None) == 1 and call(o=None) == 1 and call(o=A + 8) == 1 and call(dt=2) == 1
    assert call(s=P(_cache(D=96))) == 2 and call(s=P(_cache((8, 5)))) == 1
    assert L.kvq_dequantize_paged(P(k), P(ch), None, A, 0, None, None) == 1


def test_chunk_attention_refusals(L):
    k, ch = _cache(), _chunk()
    need = L.kvq_chunk_workspace_bytes(10, 2, 8, 2, 128)
    assert need > 0
    call = lambda q=A, sr=1024, sh=128, c=P(ch), a=P(k), b=P(k), Hq=8, w=0, s=0, o=A, dt=0, ws=A, n=need: \
        L.kvq_chunk_attention(q, sr, sh, c, a, b, Hq, 0.0, w, s, o, dt, ws, n, None, None)
    assert call(q=None) == 1 and call(o=None) == 1 and call(c=None) == 1 and call(a=None) == 1 and call(b=None) == 1
    assert call(q=A + 8) == 1 and call(o=A + 4) == 1 and call(sr=1023) == 1 and call(sh=-128) == 1
    assert call(Hq=7) == 1 and call(Hq=0) == 1 and call(Hq=258) == 2
    assert call(w=-1) == 1 and call(s=-1) == 1 and call(dt=3) == 1
    assert call(b=P(_cache((8, 4)))) == 1
    assert call(ws=None) == 4 and call(n=need - 1) == 4 and call(ws=A + 8) == 4
    assert L.kvq_chunk_attention_paged(A, 1024, 128, P(ch), P(k), P(k), None, 8, 0.0, 0, 0, A, 0, A, need, None,
                                       None) == 1


def test_chunk_workspace_bytes_of_bad_shapes(L):
    f = L.kvq_chunk_workspace_bytes
    assert f(-1, 2, 8, 2, 128) == 0 and f(10, 0, 8, 2, 128) == 0 and f(10, 2, 7, 2, 128) == 0
    assert f(10, 2, 8, 2, 96) == 0 and f(10, 2, 300, 2, 128) == 0 and f(10, 5000, 8, 2, 128) == 0
    assert f(0, 2, 8, 2, 128) > 0
    assert f(1 << 28, 2, 8, 2, 128) == 0


def test_windowed_decode_refusals(L):
    k = _cache()
    call = lambda q=A, lens=A, Hq=8, w=16, s=0, o=A, dt=0, b=P(k): L.kvq_decode_attention_window(
        q, P(k), b, lens, Hq, 0.0, w, s, o, dt, A, 1 << 30, None, None)
    assert call(q=None) == 1 and call(lens=None) == 1 and call(o=None) == 1 and call(q=A + 8) == 1
    assert call(w=-1) == 1 and call(s=-1) == 1 and call(dt=9) == 1 and call(Hq=7) == 1 and call(Hq=32) == 2
    assert call(b=P(_cache((8, 4)))) == 1
    pool = _cache(B=9, Tcap=64)
    assert L.kvq_decode_attention_window_paged(A, P(pool), P(pool), None, A, 8, 0.0, 16, 0, A, 0, A, 1 << 30, None,
                                               None) == 1


def test_binding_refuses_tensors_that_do_not_fit():
    torch = pytest.importorskip("torch")
    mk = lambda dt, *s: torch.zeros(s, dtype=dt)
    k = kvq.QuantCache(mk(torch.uint8, 1 << 16), mk(torch.int32, 1 << 12), np.array([8, 8], np.int8), 2, 2, 128, 128)
    start, lens = mk(torch.int32, 3), mk(torch.int32, 2)
    row = mk(torch.bfloat16, 4, 2, 128)
    q = mk(torch.bfloat16, 4, 8, 128)
    with pytest.raises(kvq.KvqError) as e:
        kvq.append_chunk(row.float(), row, k, k, start, lens)
    assert e.value.status == 1
    for bad in (row[:, :1], mk(torch.bfloat16, 4, 2, 64), row.transpose(1, 2)):
        with pytest.raises(kvq.KvqError):
            kvq.append_chunk(bad, row, k, k, start, lens)
    with pytest.raises(kvq.KvqError):                            # CPU tensors
        kvq.append_chunk(row, row, k, k, start, lens)
    with pytest.raises(kvq.KvqError):
        kvq.chunk_attention(q, k, k, start, lens)
    with pytest.raises(kvq.KvqError):
        kvq.dequantize(k, start, lens, 4)
    with pytest.raises(kvq.KvqError):
        kvq.decode_attention_window(q[:2], k, k, lens, 16)
    with pytest.raises(kvq.KvqError):
        kvq.decode_attention_window(q, k, k, lens, 16)           # four query rows, two sequences
