"""What the training entries' binding takes for a device buffer, on the CPU."""
import enum

import numpy as np
import pytest

import mixture_experts_layer_tcgen05_b200 as moe


class Address(enum.IntEnum):
    A = 0x7F0000000000


@pytest.mark.parametrize("what", [np.zeros(64, np.uint16), np.int64(1 << 40), "0x7f0000000000", 1.5, [1, 2]])
def test_no_device_buffers_are_refused_as_types(what):
    with pytest.raises(TypeError, match="address"):
        moe.moe_orthogonalize(what, 1, 8, 8, moe.MOE_GRAD_F32, 1, (1.0, 0.0, 0.0), 0.0, 1.0, 1 << 41, 1 << 42, 1 << 20, 0)
    with pytest.raises(TypeError, match="address"):
        moe.moe_combine_backward(1 << 40, what, 1 << 41, 1 << 42, (16, 128, 128, 4, 2), 1 << 43, 1 << 44, stream=0)


def test_any_int_is_an_address(monkeypatch):
    monkeypatch.setenv("MOE_FAKE_CC", "90")  # past the checks of arguments, refused before a launch
    with pytest.raises(moe.MoeError, match="sm_100a"):
        moe.moe_orthogonalize(Address.A, 1, 8, 8, moe.MOE_GRAD_F32, 1, (1.0, 0.0, 0.0), 0.0, 1.0, 1 << 41, 1 << 42,
                              1 << 20, 0)
