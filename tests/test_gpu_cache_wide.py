"""Places whose element offset passes 2^32: tokens, elements or heads of every
array lie gigabytes apart, in each kernel of the operators over key/value
caches, against their fp64 statement."""

import numpy as np
import pytest
import torch

from oracle import cache_ops as O
from tests.test_gpu_cache_ops import DEV, T, check_attention, f64, gen, ints, rand, visible
from tests.test_gpu_cache_ops import ops  # noqa: F401

pytestmark = pytest.mark.gpu

FAR = 2 ** 32
SPACE = 1 << 20                     # bytes of an array beside the others of its store
SIZES = {torch.float32: 4, torch.bfloat16: 2, torch.uint8: 1}


@pytest.fixture(scope="module")
def stores(cuda_ok):
    """Three buffers of 17 GB and a little: keys and values, queries, results."""
    held = [torch.empty(4 * FAR + (1 << 26), dtype=torch.uint8, device=DEV) for _ in range(3)]
    yield held
    held.clear()
    torch.cuda.empty_cache()


def wide(store, nth, dtype, shape, axis):
    """The nth array of a store, `axis` with a stride that brings its last
    index past 2^32 elements, the other indexes dense; its holes hold what they may."""
    n = shape[axis]
    far = (FAR // (n - 1) // 256 + 1) * 256        # elements; a multiple for every type, so that arrays do not meet
    stride, step = [0] * len(shape), 1
    for i in reversed(range(len(shape))):
        if i != axis:
            stride[i], step = step, step * shape[i]
    stride[axis] = far
    size = SIZES[dtype]
    assert step * size <= SPACE < far
    flat = store[nth * SPACE:nth * SPACE + ((n - 1) * far + step) * size].view(dtype)
    a = flat.as_strided(shape, stride)
    assert sum((x - 1) * s for x, s in zip(shape, stride)) > FAR
    return a


def put(store, nth, x, axis):
    a = wide(store, nth, x.dtype, tuple(x.shape), axis)
    a.copy_(x)
    assert bool(torch.equal(a, x))
    return a


def wide_cache(store, b, h, cap, d, axis):
    """A QuantizedKV with a far batch (0), head (1) or token (2) index."""
    from flow_matching_action_dm0_b200 import QuantizedKV
    k, v = (wide(store, i, torch.uint8, (b, h, cap, d), axis).view(torch.float8_e4m3fn) for i in (0, 1))
    ks, vs = (wide(store, i, torch.float32, (b, h, cap), axis) for i in (2, 3))
    return QuantizedKV(k, v, ks, vs)


AXES = {"batch": 0, "token": 1, "head": 2}          # of [B][N][H][D]
CACHE_AXES = {"batch": 0, "token": 2, "head": 1}    # of [B][H][capacity][D]


@pytest.mark.parametrize("axis", AXES)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_write_and_read(ops, stores, dtype, axis):  # noqa: F811
    g = gen(41)
    b, n, h, d, cap = 3, 40, 3, 128, 65
    k, v = rand(g, b, n, h, d, dtype=dtype), rand(g, b, n, h, d, dtype=dtype, size=30.0)
    cache = wide_cache(stores[0], b, h, cap, d, CACHE_AXES[axis])
    start = [25, 0, 13]
    ops.write(cache, put(stores[1], 0, k, AXES[axis]), put(stores[1], 1, v, AXES[axis]), start=ints(start))
    out = tuple(wide(stores[2], i, T[dtype], (b, cap - 1, h, d), AXES[axis]) for i in (0, 1))
    ops.read(cache, first=1, n=cap - 1, dtype=dtype, out=out)
    for x, codes, scales, back in ((k, cache.k, cache.k_scale, out[0]), (v, cache.v, cache.v_scale, out[1])):
        want, size = O.quantize_rows(f64(x))
        for i, at in enumerate(start):
            np.testing.assert_array_equal(f64(codes[i, :, at:at + n].contiguous()), want[i].transpose(1, 0, 2))
            np.testing.assert_array_equal(f64(scales[i, :, at:at + n].contiguous()), size[i].T)
            got = f64(back[i, max(at - 1, 0):at - 1 + n].contiguous())
            np.testing.assert_array_equal(got, (want[i] * size[i][..., None])[max(1 - at, 0):])
    assert ops.status() == (0, 0)


KINDS = [("bf16", "bf16"), ("bf16", "fp8"), ("f32", "f32"), ("f32", "fp8")]


@pytest.mark.parametrize("axis", AXES)
@pytest.mark.parametrize("tq", [2, 40])             # few rows of a key/value head (4), and many (80)
@pytest.mark.parametrize("dtype,cache", KINDS)
@pytest.mark.parametrize("d", [128, 256])
def test_cross_attention(ops, stores, dtype, cache, tq, axis, d):  # noqa: F811
    g = gen(42 + d + tq)
    b, n, hkv, hq = 3, 65, 3, 6
    q = rand(g, b, tq, hq, d, dtype=dtype)
    k, v = rand(g, b, n, hkv, d, dtype=dtype), rand(g, b, n, hkv, d, dtype=dtype)
    if cache == "fp8":
        kv = wide_cache(stores[0], b, hkv, n, d, CACHE_AXES[axis])
        ops.write(kv, k, v)
        k, v = ops.read(kv, dtype="f32")
    else:
        kv = put(stores[0], 0, k, AXES[axis]), put(stores[0], 1, v, AXES[axis])
    out = wide(stores[2], 0, T[dtype], (b, tq, hq, d), AXES[axis])
    lens = [65, 64, 9]
    _, lse = ops.cross_attention(put(stores[1], 0, q, AXES[axis]), kv, lens=ints(lens), out=out, lse=True)
    kn, vn = f64(k), f64(v)
    check_attention(q, lambda i: [(kn[i], vn[i], visible(n, lens, None, i))], d ** -0.5, out.contiguous(), lse)


@pytest.mark.parametrize("tq", [1, 20])
@pytest.mark.parametrize("dtype,cache", KINDS)
def test_shared_attention(ops, stores, dtype, cache, tq):  # noqa: F811
    g = gen(43 + tq)
    b, p, m, hkv, hq, d = 3, 130, 40, 2, 8, 128
    q, own = rand(g, b, tq, hq, d, dtype=dtype), [rand(g, b, m, hkv, d, dtype=dtype) for _ in range(2)]
    pk, pv = rand(g, p, hkv, d, dtype=dtype), rand(g, p, hkv, d, dtype=dtype)
    if cache == "fp8":
        pre = wide_cache(stores[0], 1, hkv, p, d, 2)
        ops.write(pre, pk[None], pv[None])
        pk, pv = (x[0] for x in ops.read(pre, dtype="f32"))
    else:
        pre = put(stores[0], 0, pk, 0), put(stores[0], 1, pv, 0)
    mine = put(stores[1], 0, own[0], 0), put(stores[1], 1, own[1], 0)
    out, lse = ops.shared_attention(q, pre, mine, lse=True, out=wide(stores[2], 0, T[dtype], (b, tq, hq, d), 0))
    parts, on = (f64(pk), f64(pv), np.ones(p, bool)), [f64(x) for x in own]
    check_attention(q, lambda i: [parts, (on[0][i], on[1][i], np.ones(m, bool))], d ** -0.5, out.contiguous(), lse)


@pytest.mark.parametrize("tq", [1, 40])
def test_masks_lie_far_apart_too(ops, tq):  # noqa: F811
    """A key mask's rows are gigabytes apart (offsets past 2^32 bytes), the same for every element (stride 0), or
    parts of longer rows."""
    g = gen(44 + tq)
    b, n, hq, d = 3, 200, 4, 128
    q, k, v = rand(g, b, tq, hq, d), rand(g, b, n, 1, d), rand(g, b, n, 1, d)
    one = torch.rand((b, n), generator=g, device=DEV) < 0.5
    store = torch.empty(2 * (FAR // 2 + 64) + n, dtype=torch.bool, device=DEV)
    far = store.as_strided((b, n), (FAR // 2 + 64, 1))
    far.copy_(one)
    longer = torch.ones((b, n + 77), dtype=torch.bool, device=DEV)
    longer[:, 5:5 + n] = one
    kn, vn = f64(k), f64(v)
    for mask in (far, longer[:, 5:5 + n], one[1:2].expand(b, n)):
        seen = mask.cpu().numpy()
        out, lse = ops.cross_attention(q, (k, v), mask=mask, lse=True)
        check_attention(q, lambda i: [(kn[i], vn[i], seen[i])], d ** -0.5, out, lse)
