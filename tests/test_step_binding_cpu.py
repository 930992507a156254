"""The binding's objects of a decoding step, without a GPU."""
import pytest

from lossless_bit_weight_02_amd import w12


@pytest.mark.parametrize("cls,names", [(w12.KVCache, ("k", "v", "k_scale", "v_scale")),
                                       (w12.KVBatch, ("table", "lens", "q_start", "positions", "tree"))])
def test_tensors_are_read_only(cls, names):
    """A tensor whose address the library has cannot be replaced unnoticed."""
    obj = object.__new__(cls)
    obj._tensors = {n: object() for n in names}
    for n in names:
        assert getattr(obj, n) is obj._tensors[n]
        with pytest.raises(AttributeError):
            setattr(obj, n, None)
