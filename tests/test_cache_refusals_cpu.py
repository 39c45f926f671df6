"""Calls of the cache operators that are refused, on stand-in GPUs."""

import ctypes as C

import pytest

from flow_matching_action_dm0_b200 import RtvError
from flow_matching_action_dm0_b200 import _lib as L
from tests.fake_gpu import gpus, host_library_path  # noqa: F401


@pytest.fixture
def ops(gpus):  # noqa: F811
    h = L.rtv_ops_create(0)
    yield h
    L.rtv_ops_destroy(h)


def memory(lib, n):
    p = C.c_void_p()
    assert lib.cudaMalloc(C.byref(p), C.c_size_t(n)) == 0
    return p.value


def test_keys_and_values_are_not_written_to_one_place(ops, gpus):  # noqa: F811
    a, b, c, d, e, f = (memory(gpus, 2 * 8 * 64 * 4) for _ in range(6))
    rows = lambda k, v: L.rtv_kv(k, v, None, None, L.RTV_BF16, 2, 8, 1, 64, 512, 64, 64)  # noqa: E731
    cache = lambda k, v, ks, vs: L.rtv_kv(k, v, ks, vs, L.RTV_FP8_E4M3, 2, 8, 1, 64, 512, 64, 64, 8, 1, 1)  # noqa: E731

    def refused(call, *args):
        before = gpus.fake_launches()
        with pytest.raises(RtvError) as err:
            call(ops, *args)
        assert err.value.status == L.RTV_ERR_ARG and "same place" in str(err.value)
        assert gpus.fake_launches() == before

    refused(L.rtv_kv_write, rows(a, b), cache(c, c, e, f), None, 0, None)
    refused(L.rtv_kv_write, rows(a, b), cache(c, d, e, e), None, 0, None)
    refused(L.rtv_kv_read, cache(c, d, e, f), 0, None, rows(a, a))
    # the same array may be keys and values where it is only read
    L.rtv_kv_write(ops, rows(a, a), cache(c, d, e, f), None, 0, None)
    L.rtv_kv_read(ops, cache(c, c, e, e), 0, None, rows(a, b))


def test_calls_run_on_the_handles_gpu_and_leave_the_current_one(gpus):  # noqa: F811
    h = L.rtv_ops_create(1)
    assert gpus.cudaSetDevice(1) == 0
    a, b, c, d, e, f, w = (memory(gpus, 1 << 16) for _ in range(7))
    assert gpus.cudaSetDevice(0) == 0
    here = memory(gpus, 1 << 16)
    rows = lambda k, v: L.rtv_kv(k, v, None, None, L.RTV_BF16, 2, 8, 1, 64, 512, 64, 64)  # noqa: E731
    cache = L.rtv_kv(c, d, e, f, L.RTV_FP8_E4M3, 2, 8, 1, 64, 512, 64, 64, 8, 1, 1)
    q = lambda x, o: L.rtv_queries(x, o, None, L.RTV_BF16, 2, 1, 4, 64, 256, 256, 64, 256, 256, 64, 0.125)  # noqa: E731
    now = C.c_int(-1)
    need = L.rtv_cross_attention_workspace(h, q(a, b), rows(c, d))
    for call in (lambda: L.rtv_kv_write(h, rows(a, b), cache, None, 0, None),
                 lambda: L.rtv_kv_read(h, cache, 0, None, rows(a, b)),
                 lambda: L.rtv_cross_attention(h, q(a, b), rows(c, d), None, None, 0, w if need else None, need)):
        gpus.fake_launched_on.restype = C.c_int
        before = gpus.fake_launches()
        call()
        assert gpus.fake_launches() > before and gpus.fake_launched_on() == 1
        assert gpus.cudaGetDevice(C.byref(now)) == 0 and now.value == 0
    with pytest.raises(RtvError) as err:      # memory of another GPU than the handle's
        L.rtv_kv_write(h, rows(here, b), cache, None, 0, None)
    assert err.value.status == L.RTV_ERR_ARG
    L.rtv_ops_destroy(h)
