"""The native check of a call's tensors (CPU tensors here: their device number is -1): the address of a tensor
that fits, and the explanation's error for one that does not."""
import pytest
import torch

from hybrid_gated_deltanet_gb300 import binding as gb
from hybrid_gated_deltanet_gb300 import build as gbuild


@pytest.fixture()
def marshal():
    gbuild.build()
    from hybrid_gated_deltanet_gb300 import _marshal
    told = []

    def explain(*args):
        told.append(args)
        raise ValueError(args[1])

    _marshal.explain(explain)
    yield _marshal, told
    _marshal.explain(gb._explain)


def test_addresses_of_tensors_that_fit(marshal):
    m, told = marshal
    for t in (torch.zeros(2, 3), torch.zeros(4, dtype=torch.int64), torch.zeros(2, 0, 5, dtype=torch.bfloat16),
              torch.zeros(6, 4)[2:], torch.zeros(()), torch.zeros(3, 1, 2).transpose(0, 1).contiguous()):
        assert m.ptr(t, "t", t.dtype, t.shape, -1) == t.data_ptr()
        assert m.ptr(t, "t", t.dtype, tuple(t.shape), -1) == t.data_ptr()
    assert not told


def test_what_does_not_fit_is_explained(marshal):
    m, told = marshal
    t = torch.zeros(2, 3)
    for args in ((t, "dtype", torch.int32, (2, 3), -1), (t, "shape", torch.float32, (3, 2), -1),
                 (t, "dims", torch.float32, (2, 3, 1), -1), (t, "device", torch.float32, (2, 3), 0),
                 (t.t(), "strides", torch.float32, (3, 2), -1), (None, "none", torch.float32, (2, 3), -1),
                 (t, "a dtype by name", "float32", (2, 3), -1), (t, "a list", torch.float32, [2, 3], -1),
                 (t, "no number", torch.float32, (2, None), -1), (t, "no device", torch.float32, (2, 3), None),
                 (t, "past 64 bits", torch.float32, (2, 1 << 70), -1),
                 (torch.zeros(2, 3, device="meta"), "meta", torch.int8, (2, 3), -1),
                 (torch.eye(3).to_sparse(), "sparse", torch.float32, (3, 3), -1)):
        with pytest.raises(ValueError, match=args[1]):
            m.ptr(*args)
        assert told[-1] == args or told[-1][1] == args[1]
    with pytest.raises(TypeError):
        m.ptr(t, "t", torch.float32, (2, 3))


def test_references_are_returned(marshal):
    """A call keeps no reference to its arguments."""
    import sys
    m, _ = marshal
    t, shape = torch.zeros(5), (5,)
    before = sys.getrefcount(t), sys.getrefcount(shape)
    for _ in range(100):
        m.ptr(t, "t", torch.float32, shape, -1)
    assert (sys.getrefcount(t), sys.getrefcount(shape)) == before
