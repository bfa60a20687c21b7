"""CPU-only checks of the rotated append, the block calls and the page calls: what they refuse on the host, before any
device work, and what the binding refuses of tensors."""
import ctypes
import os

import numpy as np
import pytest

from attention_group_quantized_gb300 import kvq

torch = pytest.importorskip("torch")
P = ctypes.byref
A = 0x10000                                                         # a well-aligned address (never read)


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(kvq.LIB_PATH):
        from attention_group_quantized_gb300 import build
        build.build()
    return kvq.lib()


def _cache(bits=(8, 4), B=2, Tcap=128, D=128, codes=A, sz=A):
    hb = np.asarray(bits, np.int8)
    c = kvq.CCache(codes, sz, hb.ctypes.data, B, len(hb), Tcap, D)
    c._keep = hb
    return c


def _chunk(rows=4, B=2, start=A, lens=A, most=0):
    return kvq._pack_chunk(start, lens, B, rows, most)


def _rotation(table=A, qw=A, kw=A, positions=100, rot=128, inter=0, eps=1e-6):
    return kvq._pack_rotation(table, qw, kw, positions, rot, inter, eps)


def test_the_structs_have_the_headers_sizes(L):
    assert len(_rotation()) == 40 and len(kvq._pack_bounds(A, A)) == 16 and len(kvq._pack_page_table(A, A, A, 1, 1, 1)) == 40


def test_rotate_append_refusals(L):
    k, v = _cache(), _cache()
    def call(q=A, sq=(1280, 128), kn=A, vn=A, s=(1280, 128), chunk=None, rot=None, Hq=4, k=k, v=v, out=A, dtype=1):
        return L.kvq_rotate_append(q, sq[0], sq[1], kn, vn, s[0], s[1], _chunk() if chunk is None else chunk,
                                   _rotation() if rot is None else rot, Hq, P(k), P(v), out, dtype, None, None)
    assert call(chunk=_chunk(rows=0), q=None, kn=None, vn=None, out=None) == 0
    for bad in (dict(q=None), dict(kn=None), dict(vn=None), dict(out=None), dict(q=A + 8), dict(out=A + 8),
                dict(sq=(1284, 128)), dict(sq=(-8, 128)), dict(s=(1280, 4)), dict(Hq=0), dict(Hq=-1), dict(dtype=5),
                dict(v=_cache((8, 8))), dict(k=_cache(codes=None)), dict(chunk=_chunk(B=3)), dict(chunk=_chunk(rows=-1)),
                dict(chunk=_chunk(start=0)), dict(chunk=_chunk(lens=A + 2)), dict(rot=_rotation(rot=8)), dict(rot=_rotation(rot=136)),
                dict(rot=_rotation(rot=40)), dict(rot=_rotation(positions=0)), dict(rot=_rotation(table=A + 4)),
                dict(rot=_rotation(qw=A + 2)), dict(rot=_rotation(inter=2)), dict(rot=_rotation(eps=0.0)),
                dict(rot=_rotation(eps=float("nan"))), dict(rot=_rotation(eps=2.0))):
        assert call(**bad) == 1, bad
    assert call(dtype=0) == 2                                       # queries come in bf16
    assert call(k=_cache(D=96), v=_cache(D=96)) == 2
    assert call(chunk=_chunk(rows=2 ** 28)) == 2                    # rows x heads past 2^31
    assert L.kvq_rotate_append(A, 1280, 128, A, A, 1280, 128, _chunk(), None, 4, P(k), P(v), A, 1, None, None) == 1
    assert L.kvq_rotate_append_paged(A, 1280, 128, A, A, 1280, 128, _chunk(), _rotation(), 4, P(k), P(v), None, A, 1,
                                     None, None) == 1


def test_bounds_refusals(L):
    k = _cache()
    assert L.kvq_bounds_bytes(P(k), 0) == 2 * 2 * 2 * 4 * 64 and L.kvq_bounds_bytes(P(k), 1) == 2 * 2 * 2 * 4 * 4
    assert L.kvq_bounds_bytes(P(k), 2) == -1 and L.kvq_bounds_bytes(None, 0) == -1
    b = kvq._pack_bounds(A, A)
    assert L.kvq_block_bounds(P(k), _chunk(rows=0), b, None, None) == 0
    for bounds in (None, kvq._pack_bounds(0, A), kvq._pack_bounds(A, 0), kvq._pack_bounds(A + 4, A)):
        assert L.kvq_block_bounds(P(k), _chunk(), bounds, None, None) == 1
        assert L.kvq_bounds_values(P(k), bounds, A, 1, A, None, None) == 1
    assert L.kvq_block_bounds(P(k), _chunk(B=1), b, None, None) == 1
    assert L.kvq_block_bounds_paged(P(k), _chunk(), None, b, None, None) == 1
    assert L.kvq_bounds_values(P(k), b, None, 0, None, None, None) == 0
    assert L.kvq_bounds_values(P(k), b, A, -1, A, None, None) == 1
    assert L.kvq_bounds_values(P(k), b, None, 1, A, None, None) == 1
    assert L.kvq_bounds_values(P(k), b, A, 1, None, None, None) == 1
    assert L.kvq_bounds_values(P(k), b, A, 1, A + 4, None, None) == 1


def test_select_and_attend_refusals(L):
    k, v = _cache(), _cache()
    b = kvq._pack_bounds(A, A)
    n = int(L.kvq_select_workspace_bytes(2, 2, 128))
    assert n > 0
    for bad in ((-1, 2, 128), (4097, 2, 128), (2, 0, 128), (2, 65, 128), (2, 2, 0)):
        assert L.kvq_select_workspace_bytes(*bad) == 0
    def pick(q=A, k=k, bounds=b, seq=None, lens=A, rows=2, Hq=8, take=4, first=1, last=1, out=A, ws=A, ws_n=n):
        return L.kvq_select_blocks(q, P(k), bounds, seq, lens, rows, Hq, take, first, last, out, ws, ws_n, None, None)
    def look(q=A, k=k, v=v, seq=None, lens=A, rows=2, Hq=8, take=4, blocks=A, out=A, dtype=0, ws=A):
        return L.kvq_decode_attention_blocks(q, P(k), P(v), blocks, take, seq, lens, rows, Hq, 0.0, out, dtype, ws,
                                             1 << 40, None, None)
    assert pick(rows=0, q=None) == 0 and look(rows=0, q=None, out=None) == 0
    for bad in (dict(q=None), dict(q=A + 8), dict(lens=None), dict(lens=A + 2), dict(seq=A + 1), dict(rows=-1),
                dict(rows=3), dict(Hq=7), dict(Hq=0), dict(take=0)):
        assert pick(**bad) == 1, bad
        assert look(**bad) == 1, bad
    for bad in (dict(rows=4097, seq=A), dict(Hq=18), dict(take=65537), dict(k=_cache(D=96))):
        assert pick(**bad) == 2, bad
    for bad in (dict(rows=4097, seq=A), dict(Hq=18), dict(take=65537), dict(k=_cache(D=96), v=_cache(D=96))):
        assert look(**bad) == 2, bad
    for bad in (dict(first=-1), dict(last=-1), dict(first=3, last=2), dict(first=2 ** 31 - 1, last=2 ** 31 - 1),
                dict(out=None), dict(bounds=None)):
        assert pick(**bad) == 1, bad
    assert pick(ws=None) == 4 and pick(ws_n=n - 1) == 4 and pick(ws=A + 8) == 4
    for bad in (dict(out=None), dict(out=A + 8), dict(dtype=2), dict(blocks=None), dict(v=_cache((8, 8))), dict(ws=A + 8)):
        assert look(**bad) == 1, bad
    # 2^29 tokens a sequence at most: tile numbers stay within the kernel's fields
    one = _cache((4,), B=1, Tcap=2 ** 29 + 64, D=64)
    assert pick(k=one, rows=1, Hq=1, ws_n=1 << 40) == 2
    assert look(k=one, v=_cache((4,), B=1, Tcap=2 ** 29 + 64, D=64), rows=1, Hq=1) == 2


def test_page_refusals(L):
    def pt(refs=A, table=A, lens=A, n=10, slots=4, most=3):
        return kvq._pack_page_table(refs, table, lens, n, slots, most)
    k, v = _cache(B=10, Tcap=64), _cache(B=10, Tcap=64)
    ws = int(L.kvq_pages_workspace_bytes(10, 4))
    assert ws > 0 and L.kvq_pages_workspace_bytes(0, 4) == 0 and L.kvq_pages_workspace_bytes(10, 65537) == 0
    reserve = lambda t=pt(), add=A, w=A, n=ws: L.kvq_pages_reserve(t, add, w, n, None, None)
    fork = lambda t=pt(), k=k, v=v, b=None, f=A, to=A, n=4, w=A, wn=ws: L.kvq_pages_fork(t, P(k), P(v), b, f, to, n, w, wn, None, None)
    free = lambda t=pt(), s=A, n=4: L.kvq_pages_free(t, s, n, None, None)
    compact = lambda t=pt(), k=k, v=v, b=None, live=None, w=A, wn=ws: L.kvq_pages_compact(t, P(k), P(v), b, live, w, wn, None, None)
    copy = lambda k=k, v=v, b=None, s=A, d=A, n=2: L.kvq_copy_pages(P(k), P(v), b, s, d, n, None, None)
    assert fork(n=0, f=None, to=None) == 0 and free(n=0, s=None) == 0 and copy(n=0, s=None, d=None) == 0
    for t in (None, pt(refs=0), pt(table=0), pt(lens=0), pt(refs=A + 2), pt(n=0), pt(slots=0), pt(most=0)):
        assert reserve(t) == fork(t) == free(t) == compact(t) == 1, t
    for t in (pt(n=2 ** 24 + 1), pt(slots=65537), pt(most=2 ** 25), pt(slots=65536, most=2 ** 15)):
        assert reserve(t) == free(t) == 2
    assert reserve(add=None) == 1 and reserve(w=None) == 4 and reserve(n=ws - 1) == 4 and reserve(w=A + 4) == 4
    assert fork(f=None) == 1 and fork(to=A + 2) == 1 and fork(n=5) == 1 and fork(n=-1) == 1 and fork(wn=ws - 1) == 4
    assert compact(live=A + 2) == 1 and compact(w=None) == 4
    wide, other, pool9 = _cache(B=10, Tcap=128), _cache((8, 8), B=10, Tcap=64), _cache(B=9, Tcap=64)
    for kk, vv in ((wide, wide), (k, other), (_cache(B=10, Tcap=64, sz=None), v)):
        assert fork(k=kk, v=vv) == compact(k=kk, v=vv) == copy(k=kk, v=vv) == 1
    assert fork(k=pool9, v=pool9) == 1 and compact(k=pool9, v=pool9) == 1
    assert fork(b=kvq._pack_bounds(A + 4, A)) == compact(b=kvq._pack_bounds(0, A)) == copy(b=kvq._pack_bounds(A, 0)) == 1
    assert copy(n=-1) == 1 and copy(s=None) == 1 and copy(d=None) == 1
    x = _cache(B=10, Tcap=64, D=96)
    assert fork(k=x, v=x) == copy(k=x, v=x) == 2


def test_binding_refusals_of_tensors(L):
    """Wrong types and shapes, and tensors that are not on a GPU, before the library is called."""
    c = lambda: kvq.empty_cache([8, 8], 2, 64, 64, device="cpu")
    k, v = c(), c()
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)
    q, kn = torch.zeros(3, 4, 64, dtype=torch.bfloat16), torch.zeros(3, 2, 64, dtype=torch.bfloat16)
    bounds = kvq.empty_bounds(k)
    assert tuple(bounds.codes.shape) == (2, 2, 2, 2, 32)
    pages = kvq.empty_page_table(4, 2, 3, device="cpu")
    for call in (lambda: kvq.rotate_append(q, kn, kn, k, v, i32(3), i32(2)),
                 lambda: kvq.rotate_append(q[0], kn, kn, k, v, i32(3), i32(2)),
                 lambda: kvq.rotate_append(q.float(), kn, kn, k, v, i32(3), i32(2)),
                 lambda: kvq.rotate_append(q, kn[:2], kn[:2], k, v, i32(3), i32(2)),
                 lambda: kvq.block_bounds(k, bounds, i32(3), i32(2), 3),
                 lambda: kvq.bounds_values(bounds, i32(2)),
                 lambda: kvq.bounds_values(bounds, i32(2, 2)),
                 lambda: kvq.select_blocks(q, k, bounds, i32(3), 2),
                 lambda: kvq.select_blocks(q, k, bounds, i32(2), 2),
                 lambda: kvq.select_blocks(q.transpose(0, 1), k, bounds, i32(4), 2),
                 lambda: kvq.decode_attention_blocks(q, k, v, i32(3, 2, 2), i32(3)),
                 lambda: kvq.decode_attention_blocks(q, k, v, i32(3, 3, 2), i32(3)),
                 lambda: kvq.pages_reserve(pages, i32(2)),
                 lambda: kvq.pages_free(pages, i32(2)),
                 lambda: kvq.pages_fork(pages, k, v, i32(1), i32(1)),
                 lambda: kvq.pages_compact(pages, k, v),
                 lambda: kvq.copy_pages(k, v, i32(1), i32(1))):
        with pytest.raises(kvq.KvqError):
            call()
