"""CPU checks of the largest numbers of packed rows: refused before any launch."""
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


@pytest.mark.parametrize("rows", [2 ** 31 - 1, 2 ** 31 - 33, 2 ** 31 - 256])
def test_rows_whose_runs_pass_32_bits_are_refused(L, rows):
    """The kernels take rows in runs of up to 32 and number those of a run in 32 bits."""
    hb = np.array([8], np.int8)
    k, ch = kvq.CCache(A, A, hb.ctypes.data, 2, 1, 128, 64), kvq.CChunk(A, A, 2, rows, 0)
    assert L.kvq_append_chunk(A, A, 0, 0, P(ch), P(k), P(k), None, None) == 2
    assert L.kvq_dequantize(P(k), P(ch), A, 1, None, None) == 2
    assert L.kvq_chunk_attention(A, 64, 64, P(ch), P(k), P(k), 1, 0.0, 0, 0, A, 0, A, 1 << 40, None, None) == 2


def test_capacities_whose_tiles_pass_32_bits_are_refused(L):
    """A 128-token tile that begins below 2^31 has to end there."""
    hb = np.array([4], np.int8)
    ch = kvq.CChunk(A, A, 1, 5, 0)
    for tokens in (2 ** 31 - 64, 2 ** 31 - 128):
        k = kvq.CCache(A, A, hb.ctypes.data, 1, 1, tokens, 64)
        assert L.kvq_append_chunk(A, A, 64, 64, P(ch), P(k), P(k), None, None) == 2
        assert L.kvq_dequantize(P(k), P(ch), A, 1, None, None) == 2
        assert L.kvq_chunk_attention(A, 64, 64, P(ch), P(k), P(k), 1, 0.0, 0, 0, A, 0, A, 1 << 40, None, None) == 2
        pool, bt = kvq.CCache(A, A, hb.ctypes.data, 9, 1, 64, 64), kvq.CBlockTable(A, 1, tokens // 64)
        assert L.kvq_chunk_attention_paged(A, 64, 64, P(ch), P(pool), P(pool), P(bt), 1, 0.0, 0, 0, A, 0, A, 1 << 40, None,
                                           None) == 2
