"""Lists of tensors as the arrays that the C entry points take."""
import pytest
import torch

import adamw_hybrid_optimizer_muon_b200 as ma

TENSORS = [torch.zeros(5), torch.zeros((3, 4), dtype=torch.bfloat16)[1:], torch.nn.Parameter(torch.zeros(())),
           torch.zeros((0, 7)), torch.zeros((6, 6)).t()[2:, 1:], torch.zeros(9)[4:5]]


@pytest.fixture(params=["module", "methods"])
def marshal(request, monkeypatch):
    if request.param == "methods":
        monkeypatch.setattr(ma, "_MARSHAL", ma._Methods)
    else:
        assert ma._marshal() is not ma._Methods  # built beside the library
    return request.param


@pytest.mark.parametrize("kind", [list, tuple])
@pytest.mark.parametrize("n", [0, 1, 6])
def test_addresses_and_counts(marshal, kind, n):
    xs = kind(TENSORS[:n])
    ptrs, counts = ma._ptr_array(xs), ma._numel_array(xs)
    assert [p or 0 for p in ptrs] == ([x.data_ptr() for x in xs] or [0])
    assert list(counts) == ([x.numel() for x in xs] or [0])


def test_plain_addresses_and_none(marshal):
    assert list(ma._ptr_array([4096, None, TENSORS[0]])) == [4096, None, TENSORS[0].data_ptr()]
    assert list(ma._ptr_array([1 << 63])) == [1 << 63]


@pytest.mark.parametrize("bad", [[object()], ["x"], [TENSORS[0], 1.5]])
def test_what_has_no_address(marshal, bad):
    with pytest.raises((AttributeError, TypeError)):
        ma._ptr_array(bad)
    with pytest.raises((AttributeError, TypeError)):
        ma._numel_array(bad)


def test_not_a_sequence():
    with pytest.raises(TypeError):
        ma._marshal().pointers(7)
    with pytest.raises(TypeError):
        ma._marshal().numels([TENSORS[0], None])
