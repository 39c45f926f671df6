"""What a failing install leaves of the prefix, on stand-in GPUs: the rows and
the tensor-core tiles are two launches, and calls read one or the other."""

import ctypes as C

import numpy as np
import pytest

from flow_matching_action_dm0_b200 import ActionExpert, RtvError
from flow_matching_action_dm0_b200 import _lib as L
from synthetic import get_config, make_noise, make_prefix_kv, make_state, make_weights
from tests.fake_gpu import gpus, host_library_path  # noqa: F401

CFG = get_config("pi0-bf16", n_layers=1, width=256, mlp_dim=512, prefix_len=70)


def device_array(lib, n):
    p = C.c_void_p()
    assert lib.cudaMalloc(C.byref(p), C.c_size_t(n)) == 0
    return p.value


@pytest.fixture
def ex(gpus):  # noqa: F811
    e = ActionExpert(CFG, max_batch=2)
    e.load(make_weights(CFG))
    assert e.path == "tcgen05"
    yield e
    e.close()


def install(ex, lib, how, batch):
    kv = np.ascontiguousarray(make_prefix_kv(CFG, batch=batch))
    if how == "rows":
        ex.set_prefix_kv(kv)
    else:
        rows = kv.size // CFG.head_dim
        codes, scales = device_array(lib, rows * CFG.head_dim), device_array(lib, rows * 4)
        L.rtv_set_prefix_kv_quantized(ex.h, codes, scales, CFG.prefix_len, batch)


def calls(ex):
    noise, state = np.ascontiguousarray(make_noise(CFG, batch=2)), np.ascontiguousarray(make_state(CFG, batch=2))
    yield lambda: ex.denoise(noise, state, 2)
    yield lambda: ex.denoise_shared(noise, state[0], 2)
    yield lambda: L.rtv_get_prefix_kv_quantized(ex.h, 256, 256, CFG.prefix_len, 1)


@pytest.mark.parametrize("how", ["rows", "codes"])
def test_an_install_that_fails_between_rows_and_tiles_leaves_no_prefix(ex, gpus, how):  # noqa: F811
    install(ex, gpus, "rows", 1)
    for call in list(calls(ex))[:2]:
        call()
    gpus.fake_fail_launch(C.c_long(2))
    with pytest.raises(RtvError) as e:
        install(ex, gpus, how, 2)
    assert e.value.status == L.RTV_ERR_CUDA
    for call in calls(ex):
        with pytest.raises(RtvError) as e:
            call()
        assert e.value.status == L.RTV_ERR_STATE
    install(ex, gpus, how, 2)
    for call in list(calls(ex))[:2]:
        call()


@pytest.mark.parametrize("how", ["rows", "codes"])
def test_an_install_that_writes_nothing_leaves_the_prefix_it_found(ex, gpus, how):  # noqa: F811
    install(ex, gpus, "rows", 1)
    gpus.fake_fail_launch(C.c_long(1))
    with pytest.raises(RtvError):
        install(ex, gpus, how, 2)
    for call in list(calls(ex))[:2]:
        call()
    with pytest.raises(RtvError) as e:          # of batch 1 still
        L.rtv_get_prefix_kv_quantized(ex.h, 256, 256, CFG.prefix_len, 2)
    assert e.value.status == L.RTV_ERR_SHAPE
