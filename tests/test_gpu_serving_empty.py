"""Calls with nothing to do: a step without decode rows passes through selection and attention, and a rotary table
without positions or channels is refused rather than taken for none."""
import numpy as np
import pytest

from tests import kvq_testutil as U

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def kvq():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from attention_group_quantized_gb300 import kvq as K
    K.lib()
    return K


@pytest.mark.parametrize("paged", [False, True])
@pytest.mark.parametrize("own", [False, True])
def test_no_rows(kvq, paged, own):
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")
    q = torch.empty((0, 8, 64), dtype=torch.bfloat16, device="cuda")
    k, v = ((kvq.empty_page_pool([8, 4], 4, 64) if paged else kvq.empty_cache([8, 4], 2, 128, 64)) for _ in range(2))
    b = kvq.empty_bounds(k)
    at, sfx = ((i32(2, 2),), "_paged") if paged else ((), "")
    ws = (kvq.select_workspace(2, 2, 128), kvq.decode_workspace(2, 8, 2, 64)) if own else (None, None)
    for seq in (None, i32(0)):
        sel = getattr(kvq, "select_blocks" + sfx)(q, k, b, *at, i32(0), 3, row_seq=seq, workspace=ws[0])
        assert sel.shape == (0, 2, 3)
        for dt in (kvq.OUT_F32, kvq.OUT_BF16):
            out = getattr(kvq, "decode_attention_blocks" + sfx)(q, k, v, *at, sel, i32(0), row_seq=seq, out_dtype=dt,
                                                                workspace=ws[1])
            assert out.shape == (0, 8, 64)


@pytest.mark.parametrize("shape", [(0, 64), (0, 0), (100, 0)])
def test_an_empty_rotary_table_is_refused(kvq, shape):
    k, v = kvq.empty_cache([8], 1, 64, 64), kvq.empty_cache([8], 1, 64, 64)
    x = torch.randn((3, 4, 64), device="cuda").bfloat16()
    start, lens = (torch.tensor(a, dtype=torch.int32, device="cuda") for a in ([0, 3], [3]))
    codes = k.codes.clone()
    with pytest.raises(kvq.KvqError):
        kvq.rotate_append(x[:, :2], x[:, 2:3], x[:, 3:], k, v, start, lens, rotary=torch.empty(shape, device="cuda"))
    assert torch.equal(k.codes, codes)
