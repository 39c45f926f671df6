"""Arrays of another type than the library reads are refused before it is
called (it takes addresses, and would copy bytes that are not there)."""

import types

import numpy as np
import pytest
import torch

from flow_matching_action_dm0_b200 import ActionExpert
from flow_matching_action_dm0_b200 import _lib as L


@pytest.fixture
def ex(monkeypatch):
    for name in ("rtv_denoise", "rtv_denoise_shared", "rtv_verify"):
        monkeypatch.setattr(L, name, lambda *a: pytest.fail("the library was called"))
    e = object.__new__(ActionExpert)
    e.device, e.h = 0, None
    e.cfg = types.SimpleNamespace(chunk_len=5, action_dim=3, state_dim=4)
    return e


OTHERS = [np.float64, np.float16, np.int32, torch.bfloat16, torch.float16, torch.float64, torch.int32]


def array(shape, dtype):
    return torch.zeros(shape, dtype=dtype) if isinstance(dtype, torch.dtype) else np.zeros(shape, dtype)


@pytest.mark.parametrize("dtype", OTHERS, ids=str)
@pytest.mark.parametrize("which", ["noise", "state", "out"])
def test_denoise_calls_take_fp32_alone(ex, which, dtype):
    given = {"noise": (2, 5, 3), "state": (4,), "out": (2, 5, 3)}
    given = {k: array(v, dtype if k == which else np.float32) for k, v in given.items()}
    with pytest.raises(TypeError):
        ex.denoise_shared(given["noise"], given["state"], 2, out=given["out"])
    with pytest.raises(TypeError):
        ex.denoise(given["noise"], given["state"], 2, out=given["out"])


@pytest.mark.parametrize("dtype", OTHERS, ids=str)
def test_a_result_is_not_allocated_in_the_type_of_the_noise(ex, dtype):
    with pytest.raises(TypeError):
        ex.denoise_shared(array((2, 5, 3), dtype), np.zeros(4, np.float32), 2)


@pytest.mark.parametrize("dtype", OTHERS, ids=str)
def test_verify_takes_fp32_alone(ex, dtype):
    for which in range(3):
        a = [np.zeros((5, 3), np.float32), np.zeros((5, 3), np.float32), np.zeros(4, np.float32)]
        a[which] = array(a[which].shape, dtype)
        with pytest.raises(TypeError):
            ex.verify(*a, (0.5,), 0.1, 0)
