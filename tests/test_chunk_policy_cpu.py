"""CPU checks of chunk attention with a policy: what is refused before any launch."""
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


def test_chunk_policies_are_checked(L):
    hb = np.array([8, 8], np.int8)
    flat, pool = (kvq.CCache(A, A, hb.ctypes.data, B, 2, T, 128) for B, T in ((2, 128), (9, 64)))
    bt = kvq.CBlockTable(A, 2, 3)

    def call(policy, rows=10, cache=flat, table=None, ws=1 << 40, window=0):
        ch = kvq.CChunk(A, A, 2, rows, 0)
        return L.kvq_chunk_attention_ex(A, 1024, 128, P(ch), P(cache), P(cache), table, 8, 0.0, window, 0, A, 0, A, ws,
                                        policy, None, None)

    for bad in (dict(wait_limit_us=0), dict(wait_limit_us=60_000_001), dict(decode_ring_tiles=3),
                dict(decode_l2_warm_tiles=17)):
        assert call(P(kvq.policy(**bad))) == 1
        assert call(P(kvq.policy(**bad)), cache=pool, table=P(bt)) == 1
    good = P(kvq.policy(wait_limit_us=1))
    for pol in (None, good):
        assert call(pol, rows=0) == 0
        assert call(pol, rows=0, cache=pool, table=P(bt)) == 0
        assert call(pol, ws=16) == 4
        assert call(pol, window=-1) == 1
        assert call(pol, table=P(bt)) == 1                       # not a pool of 64-token pages
