"""The descriptors of lq.Norm follow their tensors. No GPU is used: host tensors stand in, whose
addresses are compared and never read."""
import pytest
import torch

import fractional_bit_weight_b200 as lq

HOST = -1       # get_device() of a host tensor


@pytest.fixture(autouse=True)
def host_tensors(monkeypatch):
    monkeypatch.setattr(lq, "_device_of", lambda t, name: t.get_device())


def desc(norm, K):
    return norm._arg(K, HOST)._obj


def check(norm, K):
    d = desc(norm, K)
    for t, at in ((norm.weight, d.weight), (norm.bias, d.bias)):
        assert at == (None if t is None else t.data_ptr())
    t = norm.weight if norm.weight is not None else norm.bias
    assert d.dtype == lq._DTYPES[t.dtype]


@pytest.mark.parametrize("bias", [False, True])
def test_new_storage(bias):
    w = torch.nn.Parameter(torch.ones(64))
    b = torch.nn.Parameter(torch.zeros(64)) if bias else None
    norm = lq.Norm("layer", w, b)
    check(norm, 64)
    first = norm._arg(64, HOST)
    assert norm._arg(64, HOST) is first         # nothing new, nothing made
    w.data = torch.full((64,), 2.0)
    check(norm, 64)
    if bias:
        b.data = torch.full((64,), 3.0)
        check(norm, 64)
    module = torch.nn.LayerNorm(64, bias=bias)
    norm = lq.Norm("layer", module.weight, module.bias)
    module.to(torch.bfloat16)                   # the same Parameter objects
    assert norm.weight.dtype == torch.bfloat16
    check(norm, 64)


def test_other_tensors_and_numbers():
    norm = lq.Norm("rms", torch.ones(64))
    norm.weight = torch.ones(64, dtype=torch.float16)
    norm.eps = 1e-3
    check(norm, 64)
    assert desc(norm, 64).eps == pytest.approx(1e-3)
    norm.weight = None
    assert desc(norm, 100).weight is None       # no tensors: rows of any length


def test_what_no_longer_fits_is_refused():
    w, b = torch.ones(64), torch.zeros(64)
    norm = lq.Norm("layer", w, b)
    w.data = torch.ones(64, dtype=torch.bfloat16)
    with pytest.raises(TypeError, match="one dtype"):
        norm._arg(64, HOST)
    b.data = torch.zeros(64, dtype=torch.bfloat16)
    check(norm, 64)
    w.data = torch.ones(128, dtype=torch.bfloat16)[::2]
    with pytest.raises(ValueError, match="contiguous"):
        norm._arg(64, HOST)
    w.data = torch.ones(63, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="shape"):
        norm._arg(64, HOST)
    w.data, b.data = torch.ones(63), torch.zeros(63)
    with pytest.raises(ValueError, match="norm over 63"):
        norm._arg(64, HOST)
    norm.kind = "batch"
    with pytest.raises(ValueError, match="norm kind"):
        norm._arg(63, HOST)
