"""CPU checks of the out_dtype flag of the chunk calls: taken by the calls that say so, refused by the others."""
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


def test_zero_rest_is_a_flag_of_the_read_back_and_of_chunk_attention(L):
    hb = np.array([8, 8], np.int8)
    k, ch = kvq.CCache(A, A, hb.ctypes.data, 2, 2, 128, 128), kvq.CChunk(A, A, 2, 0, 0)
    for dt, want in ((0, 0), (1, 0), (0x100, 0), (0x101, 0), (0x102, 1), (0x200, 1), (0x300, 1), (-1, 1)):
        assert L.kvq_dequantize(P(k), P(ch), A, dt, None, None) == want
        assert L.kvq_chunk_attention(A, 1024, 128, P(ch), P(k), P(k), 8, 0.0, 0, 0, A, dt, A, 1 << 40, None, None) == want
    for dt in (0x100, 0x101):
        assert L.kvq_decode_attention_window(A, P(k), P(k), A, 8, 0.0, 16, 0, A, dt, A, 1 << 40, None, None) == 1
        assert L.kvq_decode_attention(A, P(k), P(k), A, 8, 0.0, A, dt, A, 1 << 40, None, None) == 1
