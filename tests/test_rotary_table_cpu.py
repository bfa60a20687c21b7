"""What the binding makes of a rotary table's shape, without a device: an empty tensor has no address, and no address
means no rotation to the library."""
import pytest

from attention_group_quantized_gb300 import kvq

torch = pytest.importorskip("torch")


@pytest.mark.parametrize("shape", [(0, 64), (0, 0), (100, 0)])
def test_empty_tables_are_refused(shape):
    kvq._torch()
    with pytest.raises(kvq.KvqError):
        kvq._rotation(torch.empty(shape), None, None, 1e-6, False, 64, -1)


def test_no_table_and_a_table():
    kvq._torch()
    assert kvq._rotation(None, None, None, 1e-6, False, 64, -1)[:8] == bytes(8)
    assert kvq._rotation(torch.empty((1, 16)), None, None, 1e-6, False, 64, -1)[:8] != bytes(8)
