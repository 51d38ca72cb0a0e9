"""The serving calls' native binding on the host: what it reads off tensors before any kernel is launched."""
from __future__ import annotations

import pytest
import torch

import __graft_entry__
from gated_delta_rule_sm_gb300 import _lib


@pytest.fixture(scope="module")
def ops():
    __graft_entry__.build()
    return _lib._native()


@pytest.mark.parametrize("shape,lead", [((1, 50, 4), 2), ((3, 50, 4), 2), ((3, 50, 4, 8), 2), ((3, 1, 4), 2), ((3, 4), 1), ((3, 4, 8), 1)])
def test_expanded_tokens_have_no_stride(ops, shape, lead):
    """A stride of 0 is "contiguous" to the C entries, which would read past the one token there is."""
    one = torch.zeros(*[1] * lead, *shape[lead:])
    with pytest.raises(ValueError):
        ops.token_stride(one.expand(*shape), lead)
    assert ops.token_stride(one.expand(*shape).contiguous(), lead) == one.numel()
    assert ops.token_stride(one.expand(*one.shape), lead) == one.numel()


def test_overlapping_tokens_have_no_stride(ops):
    flat = torch.zeros(64)
    with pytest.raises(ValueError):
        ops.token_stride(flat.as_strided((1, 10, 8), (0, 3, 1)), 2)
    with pytest.raises(ValueError):
        ops.token_stride(torch.zeros(1, 5, 4).expand(3, 5, 4), 2)       # each row of tokens the same memory
    assert ops.token_stride(flat.as_strided((1, 6, 8), (0, 9, 1)), 2) == 9


def test_a_call_runs_on_its_tensors_device(ops):
    """Whatever device is current.  (Fake tensors: a device's number without the device.)"""
    fake = pytest.importorskip("torch._subclasses.fake_tensor").FakeTensorMode
    with fake():
        here, there = torch.empty(2, 3, device="cuda:0"), torch.empty(2, 3, device="cuda:1")
    host = torch.zeros(2)
    assert ops.device_of(there) == 1 and ops.device_of(here) == 0
    assert ops.device_of(None, 3, host, there) == 1          # the first CUDA tensor decides
    assert ops.device_of() == ops.device_of(None, host, [1]) == -1
