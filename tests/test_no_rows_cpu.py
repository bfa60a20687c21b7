"""Packed rows that are none, without a device: an array without elements has strides of 0, which no index uses."""
import numpy as np
import pytest

from attention_group_quantized_gb300 import kvq

torch = pytest.importorskip("torch")


def _bf16(a):
    return torch.from_numpy(a.view(np.int16)).view(torch.bfloat16)


def test_the_strides_of_no_rows_do_not_matter():
    x = _bf16(np.zeros((2, 0, 4, 64), np.uint16)[0])
    assert x.stride(2) == 0
    kvq._packed(x, 4, 64, "rows")


def test_the_strides_of_rows_do():
    x = _bf16(np.zeros((3, 4, 64, 2), np.uint16))[..., 0]
    with pytest.raises(kvq.KvqError):
        kvq._packed(x, 4, 64, "rows")
    for shape in ((0, 5, 64), (0, 4, 128), (0, 64)):
        with pytest.raises(kvq.KvqError):
            kvq._packed(torch.empty(shape, dtype=torch.bfloat16), 4, 64, "rows")


def test_strides_that_no_index_uses_count_as_zero():
    make = lambda *shape: torch.zeros(shape, dtype=torch.bfloat16)
    assert kvq._strides(make(0, 4, 64)) == kvq._strides(_bf16(np.zeros((2, 0, 4, 64), np.uint16)[0])) == (0, 0)
    assert kvq._strides(make(1, 4, 64)) == (0, 64) and kvq._strides(make(3, 1, 64)) == (64, 0)
    assert kvq._strides(make(3, 4, 64)) == (256, 64)
