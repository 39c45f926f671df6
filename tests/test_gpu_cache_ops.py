"""The operators over key/value caches against their fp64 statement
(oracle/cache_ops.py): the E4M3 cache bit for bit, attention within bounds
derived from its roundings."""

import numpy as np
import pytest
import torch

from oracle import cache_ops as O

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
T = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(scope="module")
def ops(cuda_ok):
    from flow_matching_action_dm0_b200 import CacheOps
    h = CacheOps(device=0)
    yield h
    assert h.status() == (0, 0)
    h.close()


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def rand(g, *shape, dtype="bf16", size=1.0):
    return (torch.randn(shape, generator=g, device=DEV) * size).to(T[dtype])


def f64(t):
    return t.detach().double().cpu().numpy()


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def empty_cache(b, cap, h, d):
    from flow_matching_action_dm0_b200 import QuantizedKV
    return QuantizedKV.empty(b, cap, h, d, device=0)


# --------------------------------------------------------------------------- cache


def check_write(ops, k, v, cap, start=None, count=None):
    """Writes into a cache of marked bytes and compares every byte of it."""
    b, n, h, d = k.shape
    cache = empty_cache(b, cap, h, d)
    for t in (cache.k, cache.v):
        t.view(torch.uint8).fill_(0x2B)
    for t in (cache.k_scale, cache.v_scale):
        t.fill_(-3.0)
    ops.write(cache, k, v, start=ints(start) if isinstance(start, list) else start,
              count=None if count is None else ints(count))
    for x, codes, scales in ((k, cache.k, cache.k_scale), (v, cache.v, cache.v_scale)):
        want, size = O.quantize_rows(f64(x))
        wc = np.full((b, h, cap, d), float(torch.tensor(0x2B, dtype=torch.uint8).view(torch.float8_e4m3fn).float()))
        ws = np.full((b, h, cap), -3.0)
        for i in range(b):
            at = start[i] if isinstance(start, list) else (start or 0)
            for t in range(n if count is None else min(max(count[i], 0), n)):
                if 0 <= at + t < cap:
                    wc[i, :, at + t], ws[i, :, at + t] = want[i, t], size[i, t]
        np.testing.assert_array_equal(f64(codes), wc)
        np.testing.assert_array_equal(f64(scales), ws)
    return cache


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("b,n,h,d", [(1, 1, 1, 64), (3, 1, 2, 256), (2, 37, 1, 128), (1, 130, 4, 64), (2, 65, 3, 256)])
def test_write(ops, dtype, b, n, h, d):
    g = gen(b * n + d)
    k, v = rand(g, b, n, h, d, dtype=dtype), rand(g, b, n, h, d, dtype=dtype, size=300.0)
    check_write(ops, k, v, n + 5, start=3)
    check_write(ops, k, v, n)


def test_write_at_positions_and_counts(ops):
    g = gen(5)
    k, v = rand(g, 4, 9, 2, 128), rand(g, 4, 9, 2, 128)
    check_write(ops, k, v, 40, start=[0, 31, 7, 20], count=[9, 4, 0, 1])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_write_values_at_the_edges(ops, dtype):
    rows = [[0.0] * 64, [-0.0] * 63 + [1.0], [448.0] * 64, [449.0] + [17.0] * 63, [2.0 ** -126] * 64, [2.0 ** -133] * 64,
            [3.0e38] + [1.0] * 63, [1.0] * 63 + [float("nan")], [float("inf")] + [2.0] * 63, [-float("inf")] * 64,
            [448.0] + [2.0 ** -9, 2.0 ** -10, 3 * 2.0 ** -10, 2.0 ** -11] + [1.0 + i / 64 for i in range(59)]]
    k = torch.tensor(rows, device=DEV).to(T[dtype])[None, :, None, :].contiguous()
    check_write(ops, k, k.flip(1).contiguous(), len(rows))


def test_write_strided_source_and_cache(ops):
    from flow_matching_action_dm0_b200 import QuantizedKV
    g = gen(6)
    qkv = rand(g, 2, 7, 6, 128)                        # packed heads: keys are 2..3, values 4..5
    k, v = qkv[:, :, 2:4], qkv[:, :, 4:6]
    big = torch.zeros((2, 2, 9, 2, 128), dtype=torch.uint8, device=DEV).view(torch.float8_e4m3fn)   # token-major
    scales = torch.zeros((2, 2, 9, 2), device=DEV)
    cache = QuantizedKV(big[0].transpose(1, 2), big[1].transpose(1, 2), scales[0].transpose(1, 2),
                        scales[1].transpose(1, 2))
    ops.write(cache, k, v, start=1)
    for x, c, s in ((k, cache.k, cache.k_scale), (v, cache.v, cache.v_scale)):
        want, size = O.quantize_rows(f64(x))
        np.testing.assert_array_equal(f64(c)[:, :, 1:8], want.transpose(0, 2, 1, 3))
        np.testing.assert_array_equal(f64(s)[:, :, 1:8], size.transpose(0, 2, 1))


def test_write_outside_the_cache_is_reported_and_not_done(ops):
    g = gen(7)
    k, v = rand(g, 3, 6, 1, 64), rand(g, 3, 6, 1, 64)
    check_write(ops, k, v, 10, start=[-3, 8, 2], count=[6, 6, 9])
    assert ops.status() == (0, 4)      # RTV_DEV_BOUNDS, cleared by the read
    assert ops.status() == (0, 0)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("b,cap,h,d,first,n", [(1, 1, 1, 64, 0, 1), (2, 50, 3, 128, 7, 43), (3, 33, 1, 256, 0, 20)])
def test_read(ops, dtype, b, cap, h, d, first, n):
    g = gen(cap)
    x = rand(g, b, cap, h, d, size=3.0), rand(g, b, cap, h, d, size=0.01)
    cache = empty_cache(b, cap, h, d)
    ops.write(cache, *x)
    for lens in (None, [0, first + 1, cap][:b]):
        got = ops.read(cache, n=n, first=first, lens=None if lens is None else ints(lens), dtype=dtype)
        for y, out in zip(x, got):
            codes, scale = O.quantize_rows(f64(y))
            want = (codes * scale[..., None])[:, first:first + n]      # exact in bf16 and fp32
            for i, m in enumerate(lens or []):
                want[i, max(0, m - first):] = 0
            assert out.dtype == T[dtype] and tuple(out.shape) == (b, n, h, d)
            np.testing.assert_array_equal(f64(out), want)


def test_read_scales_of_any_size_round_once(ops):
    g = gen(8)
    cache = empty_cache(1, 12, 1, 64)
    ops.write(cache, rand(g, 1, 12, 1, 64), rand(g, 1, 12, 1, 64))
    cache.k_scale.uniform_(0.1, 3.0, generator=g)
    cache.k_scale[0, 0, 3] = float("nan")
    k, _ = ops.read(cache, dtype="bf16")
    exact = f64(cache.k) * f64(cache.k_scale)[..., None]
    once = torch.from_numpy(exact).float().to(torch.bfloat16)     # fp32 rounds first: a tie of that is no tie
    got = f64(k)[0, :, 0]
    assert np.isnan(got[3]).all()
    keep = np.arange(12) != 3
    # one fp32 product, one bf16 rounding: half a bf16 step and half an fp32 one
    assert np.all(np.abs(got - exact[0, 0])[keep] <= (2.0 ** -8 + 2.0 ** -23) * np.abs(exact[0, 0])[keep])
    assert np.mean(got[keep] == once.double().numpy()[0, 0][keep]) > 0.99


# ----------------------------------------------------------------------- attention


def visible(n, lens, mask, i):
    w = np.ones(n, bool) if lens is None else np.arange(n) < lens[i]
    return w if mask is None else w & mask[i]


def check_attention(q, sources, scale, got, lse=None):
    """got (and lse) against the oracle.  sources(i): the parts [(k [N][Hkv][D], v, visible)] of element i.

    A score carries at most ds = (D + 4) 2^-24 sum|q k| scale + 2^-22 max|s|
    (fp32 sums in any order, the scale, the base-2 exponent's argument).  A
    weight is then off by 2 ds + 2^-21 (exponential, running rescales), its
    bf16 form by 2^-8 more; sums over n keys add (n + 16) 2^-23; the division
    and the rounding of the result add half a step of its type."""
    qn = f64(q)
    b, t, h, d = qn.shape
    step = 2.0 ** -8 if q.dtype == torch.bfloat16 else 2.0 ** -24
    p_step = 2.0 ** -8 if q.dtype == torch.bfloat16 else 0.0
    gn, ln = f64(got), None if lse is None else f64(lse)
    for i in range(b):
        parts = sources(i)
        group = h // parts[0][0].shape[1]
        for j in range(h):
            hk = j // group
            mine = [(k[:, hk], v[:, hk], w) for k, v, w in parts]
            out, want_lse, size = O.attention(qn[i, :, j], mine, scale)
            n = sum(int(w.sum()) for _, _, w in parts)
            if n == 0:
                assert np.all(gn[i, :, j] == 0)
                assert ln is None or np.all(ln[i, :, j] == -np.inf)
                continue
            ka = np.concatenate([k[w] for k, _, w in mine])
            mag = abs(scale) * np.abs(qn[i, :, j]) @ np.abs(ka).T
            top = np.abs(scale * qn[i, :, j] @ ka.T).max(1)
            ds = (d + 4) * 2.0 ** -24 * mag.max(1) + 2.0 ** -22 * top
            tol = size * (p_step + 2 * ds + 2.0 ** -21 + (n + 16) * 2.0 ** -23)[:, None] + step * np.abs(out)
            bad = ~(np.abs(gn[i, :, j] - out) <= tol * (1 + 2.0 ** -6) + 1e-30)
            assert not bad.any(), (i, j, np.argwhere(bad)[:3], gn[i, :, j][bad][:3], out[bad][:3], tol[bad][:3])
            if ln is not None:
                lt = ds + (n + 16) * 2.0 ** -23 + 2.0 ** -21 + 2.0 ** -22 * np.abs(want_lse)
                assert np.all(np.abs(ln[i, :, j] - want_lse) <= lt)


def cross_case(ops, dtype, cache, b, tq, tk, hq, hkv, d, lens=None, masked=False, seed=0, scale=None, size=1.0):
    g = gen(seed + tq * 7 + tk)
    q = rand(g, b, tq, hq, d, dtype=dtype, size=size)
    k, v = rand(g, b, tk, hkv, d, dtype=dtype), rand(g, b, tk, hkv, d, dtype=dtype)
    if cache == "fp8":
        kv = empty_cache(b, tk, hkv, d)
        ops.write(kv, k, v)
        k, v = ops.read(kv, dtype="f32")
    else:
        kv = (k, v)
    mask = torch.rand((b, tk), generator=g, device=DEV) < 0.5 if masked else None
    out, lse = ops.cross_attention(q, kv, lens=None if lens is None else ints(lens), mask=mask, scale=scale, lse=True)
    kn, vn, mn = f64(k), f64(v), None if mask is None else mask.cpu().numpy()
    check_attention(q, lambda i: [(kn[i], vn[i], visible(tk, lens, mn, i))], d ** -0.5 if scale is None else scale, out,
                    lse)
    return q, kv, out


KINDS = [("f32", "f32"), ("f32", "fp8"), ("bf16", "bf16"), ("bf16", "fp8")]


@pytest.mark.parametrize("dtype,cache", KINDS)
@pytest.mark.parametrize("tq,tk,hq,hkv,d", [
    (1, 1, 1, 1, 64), (1, 816, 8, 1, 256), (51, 63, 8, 1, 256), (9, 64, 4, 1, 64), (17, 65, 4, 4, 128),
    (130, 127, 2, 1, 128), (3, 128, 6, 2, 64), (64, 129, 2, 2, 256), (128, 257, 1, 1, 64), (129, 300, 3, 3, 128),
    (2, 1000, 16, 2, 128), (33, 561, 4, 2, 256)])
def test_cross_attention(ops, dtype, cache, tq, tk, hq, hkv, d):
    cross_case(ops, dtype, cache, 2, tq, tk, hq, hkv, d)


@pytest.mark.parametrize("dtype,cache", KINDS)
@pytest.mark.parametrize("d", [64, 128, 256])
def test_cross_attention_lengths_and_masks(ops, dtype, cache, d):
    cross_case(ops, dtype, cache, 5, 7, 300, 8, 2, d, lens=[0, 1, 128, 129, 300])
    cross_case(ops, dtype, cache, 5, 7, 300, 8, 2, d, lens=[0, 1, 131, 256, 300], masked=True)
    cross_case(ops, dtype, cache, 2, 40, 700, 8, 1, d, masked=True)
    cross_case(ops, dtype, cache, 1, 1, 2500, 2, 1, d, lens=[2200], masked=True)   # many ranges of keys


@pytest.mark.parametrize("dtype,cache", KINDS)
def test_cross_attention_peaked_scores(ops, dtype, cache):
    # growing maxima: the running maximum is raised many times
    cross_case(ops, dtype, cache, 1, 65, 600, 2, 1, 64, scale=3.0, seed=4)
    cross_case(ops, dtype, cache, 1, 65, 600, 2, 1, 256, scale=-0.5, size=8.0, seed=4)


@pytest.mark.parametrize("dtype,cache", KINDS)
def test_hidden_keys_may_hold_anything(ops, dtype, cache):
    g = gen(9)
    b, tq, tk, d = 3, 5, 200, 128
    q, k, v = rand(g, b, tq, 4, d, dtype=dtype), rand(g, b, tk, 2, d, dtype=dtype), rand(g, b, tk, 2, d, dtype=dtype)
    mask = torch.rand((b, tk), generator=g, device=DEV) < 0.6
    lens = [150, 0, 64]
    seen = mask & (torch.arange(tk, device=DEV)[None] < ints(lens)[:, None])

    def run(fill):
        kk, vv = k.clone(), v.clone()
        kk[~seen], vv[~seen] = fill, -fill
        kv = (kk, vv)
        if cache == "fp8":
            kv = empty_cache(b, tk, 2, d)
            ops.write(kv, kk, vv)
        return ops.cross_attention(q, kv, lens=ints(lens), mask=mask, lse=True)

    want = run(0.5)
    assert torch.isfinite(want[0]).all()
    for fill in (float("nan"), float("inf"), -float("inf"), 1e30):
        got = run(fill)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("dtype,cache", KINDS)
def test_a_nan_stays_with_its_query_and_element(ops, dtype, cache):
    g = gen(10)
    q, k, v = rand(g, 3, 6, 4, 64, dtype=dtype), rand(g, 3, 90, 1, 64, dtype=dtype), rand(g, 3, 90, 1, 64, dtype=dtype)

    def run():
        kv = (k, v)
        if cache == "fp8":
            kv = empty_cache(3, 90, 1, 64)
            ops.write(kv, k, v)
        return ops.cross_attention(q, kv)

    want = run()
    q[0, 2, 1] = float("nan")
    v[1, 30] = float("nan")
    k[2, 88] = float("nan")
    got = run()
    assert torch.isnan(got[0, 2, 1]).all()
    keep = torch.ones((6, 4), dtype=torch.bool, device=DEV)
    keep[2, 1] = False
    assert torch.equal(got[0][keep], want[0][keep])
    assert torch.isnan(got[1]).all() and torch.isnan(got[2]).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_strides_and_orders(ops, dtype):
    g = gen(11)
    b, tq, tk, d = 2, 21, 140, 128
    packed = rand(g, b, tq, 12, d, dtype=dtype)
    q = packed[:, :, 2:10]                                                  # heads of a packed projection
    kv = rand(g, 2, b, 2, tk, d, dtype=dtype)                               # head-major, as a cache holds them
    k, v = kv[0].transpose(1, 2), kv[1].transpose(1, 2)
    out = torch.full((b, 8, tq, d), 7.0, dtype=T[dtype], device=DEV).transpose(1, 2)
    got = ops.cross_attention(q, (k, v), out=out)
    assert got is out
    kn, vn = f64(k), f64(v)
    check_attention(q, lambda i: [(kn[i], vn[i], np.ones(tk, bool))], d ** -0.5, out)
    one = ops.cross_attention(q, (k[:1].expand(b, tk, 2, d), v[:1].expand(b, tk, 2, d)))    # one element's keys for all
    check_attention(q, lambda i: [(kn[0], vn[0], np.ones(tk, bool))], d ** -0.5, one)
    heads = ops.cross_attention(q, (k[:, :, :1].expand(b, tk, 2, d), v[:, :, :1].expand(b, tk, 2, d)))
    check_attention(q, lambda i: [(kn[i][:, [0, 0]], vn[i][:, [0, 0]], np.ones(tk, bool))], d ** -0.5, heads)


def shared_case(ops, dtype, cache, b, tq, p, m, hq, hkv, d, lens=None, masked=False, seed=0, scale=None):
    g = gen(seed + tq * 7 + p + (m or 0))
    q = rand(g, b, tq, hq, d, dtype=dtype)
    pk, pv = rand(g, p, hkv, d, dtype=dtype), rand(g, p, hkv, d, dtype=dtype)
    own = None if m is None else (rand(g, b, m, hkv, d, dtype=dtype), rand(g, b, m, hkv, d, dtype=dtype))
    pre = (pk, pv)
    if cache == "fp8":
        pre = empty_cache(1, p, hkv, d)
        ops.write(pre, pk[None], pv[None])
        pk, pv = (x[0] for x in ops.read(pre, dtype="f32"))
    mask = torch.rand((p,), generator=g, device=DEV) < 0.5 if masked else None
    if masked and lens is None:
        mask[:] = False
    out, lse = ops.shared_attention(q, pre, own, prefix_mask=mask, own_lens=None if lens is None else ints(lens),
                                    scale=scale, lse=True)
    pkn, pvn = f64(pk), f64(pv)
    pw = np.ones(p, bool) if mask is None else mask.cpu().numpy()
    on = None if own is None else [f64(x) for x in own]

    def sources(i):
        parts = [(pkn, pvn, pw)]
        return parts if on is None else parts + [(on[0][i], on[1][i], visible(m, lens, None, i))]

    check_attention(q, sources, d ** -0.5 if scale is None else scale, out, lse)


@pytest.mark.parametrize("dtype,cache", KINDS)
@pytest.mark.parametrize("b,tq,p,m,hq,hkv,d", [
    (3, 9, 64, 9, 4, 1, 64), (1, 1, 1, 1, 1, 1, 64), (5, 1, 300, 3, 8, 1, 256), (40, 1, 129, 1, 8, 2, 128),
    (2, 51, 816, 51, 8, 1, 256), (3, 5, 130, 200, 2, 2, 128), (2, 70, 127, 1, 2, 1, 64), (17, 2, 65, None, 4, 1, 128),
    (1, 33, 257, None, 8, 4, 64), (4, 130, 1, 129, 1, 1, 256)])
def test_shared_attention(ops, dtype, cache, b, tq, p, m, hq, hkv, d):
    shared_case(ops, dtype, cache, b, tq, p, m, hq, hkv, d)


@pytest.mark.parametrize("dtype,cache", KINDS)
@pytest.mark.parametrize("tq", [1, 60])
def test_shared_attention_lengths_and_masks(ops, dtype, cache, tq):
    shared_case(ops, dtype, cache, 5, tq, 200, 140, 4, 2, 128, lens=[0, 1, 64, 129, 140], masked=True)
    shared_case(ops, dtype, cache, 4, tq, 90, 3, 4, 1, 256, lens=[0, 3, 1, 2])
    shared_case(ops, dtype, cache, 3, tq, 150, 0, 4, 1, 64, masked=True)     # nothing to see: zeros
    shared_case(ops, dtype, cache, 3, tq, 0, 5, 4, 1, 64)                    # an empty prefix


@pytest.mark.parametrize("dtype,cache", KINDS)
def test_shared_attention_elements_do_not_touch_each_other(ops, dtype, cache):
    g = gen(12)
    q = rand(g, 6, 1, 8, 128, dtype=dtype)
    pk, pv = rand(g, 1, 100, 1, 128, dtype=dtype), rand(g, 1, 100, 1, 128, dtype=dtype)
    k, v = rand(g, 6, 30, 1, 128, dtype=dtype), rand(g, 6, 30, 1, 128, dtype=dtype)
    pre = (pk[0], pv[0])
    if cache == "fp8":
        pre = empty_cache(1, 100, 1, 128)
        ops.write(pre, pk, pv)
    want = ops.shared_attention(q, pre, (k, v))
    q[1] = float("nan")
    v[3, 4] = float("inf")
    k[4, 29] = float("nan")
    got = ops.shared_attention(q, pre, (k, v))
    for i in (0, 2, 5):
        assert torch.equal(got[i], want[i])
    assert torch.isnan(got[1]).all() and torch.isnan(got[4]).all()
    assert not torch.isfinite(got[3]).any()


# ------------------------------------------------------------------ runs of them together


@pytest.mark.parametrize("d", [64, 256])
def test_decode_over_a_growing_quantised_cache(ops, d):
    """Prompts of different lengths, then tokens appended one by one, each followed by attention over the cache."""
    g = gen(13)
    b, hq, hkv, cap = 3, 8, 2, 160
    lens = [120, 1, 127]
    cache = empty_cache(b, cap, hkv, d)
    k, v = rand(g, b, 127, hkv, d), rand(g, b, 127, hkv, d)
    ops.write(cache, k, v, count=ints(lens))
    for _ in range(5):
        kt, vt, q = rand(g, b, 1, hkv, d), rand(g, b, 1, hkv, d), rand(g, b, 1, hq, d)
        ops.write(cache, kt, vt, start=ints(lens))
        lens = [n + 1 for n in lens]
        out, lse = ops.cross_attention(q, cache, lens=ints(lens), lse=True)
        kn, vn = (f64(x) for x in ops.read(cache, dtype="f32"))
        check_attention(q, lambda i: [(kn[i], vn[i], np.arange(cap) < lens[i])], d ** -0.5, out, lse)
        # the bf16 form of the cache is exact, so attention over it is the same mathematics
        out2 = ops.cross_attention(q, ops.read(cache, dtype="bf16"), lens=ints(lens))
        check_attention(q, lambda i: [(kn[i], vn[i], np.arange(cap) < lens[i])], d ** -0.5, out2)


@pytest.mark.parametrize("dtype,cache", KINDS)
def test_repeat_calls_are_bitwise_identical(ops, dtype, cache):
    q, kv, out = cross_case(ops, dtype, cache, 2, 3, 1500, 8, 1, 128, lens=[1500, 700])
    for _ in range(3):
        assert torch.equal(ops.cross_attention(q, kv, lens=ints([1500, 700])), out)


def test_captured_calls_replay_on_new_inputs_beside_another_graph(ops):
    g = gen(14)
    q, own = rand(g, 16, 1, 8, 128), (rand(g, 16, 40, 1, 128), rand(g, 16, 40, 1, 128))
    pre = (rand(g, 2000, 1, 128), rand(g, 2000, 1, 128))
    cache = empty_cache(16, 50, 1, 128)
    at = ints([40] * 16)

    def step():
        out = ops.shared_attention(q, pre, own)
        ops.write(cache, own[0], own[1])
        return out, ops.cross_attention(q, cache, lens=at)

    step()
    torch.cuda.synchronize()
    graphs = [torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()]
    outs = []
    for gr in graphs:
        with torch.cuda.graph(gr):
            outs.append(step())
    for seed in (1, 2):
        q.copy_(rand(gen(seed), 16, 1, 8, 128))
        own[0].copy_(rand(gen(seed + 10), 16, 40, 1, 128))
        torch.cuda.synchronize()
        streams = [torch.cuda.Stream(), torch.cuda.Stream()]
        for gr, s in zip(graphs, streams):      # both at once: each has a workspace of its own
            with torch.cuda.stream(s):
                gr.replay()
        torch.cuda.synchronize()
        want = step()
        for o in outs:
            assert torch.equal(o[0], want[0]) and torch.equal(o[1], want[1])


def test_calls_on_two_streams_at_once(ops):
    g = gen(15)
    sets = [(rand(g, 2, 4, 8, 256), rand(g, 2, 3000, 1, 256), rand(g, 2, 3000, 1, 256)) for _ in range(2)]
    want = [ops.cross_attention(q, (k, v)) for q, k, v in sets]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(20):
        got = [ops.cross_attention(q, (k, v), stream=s if i else s.cuda_stream)
               for i, (s, (q, k, v)) in enumerate(zip(streams, sets))]
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(got, want))


def test_offsets_past_32_bits(ops):
    """Keys 5 GB apart: element strides whose product with the index passes 2^31 and 2^32."""
    g = gen(16)
    n, gap = 300, 9_000_000
    store = torch.zeros(n * gap // 2 + 256, dtype=torch.bfloat16, device=DEV)
    wide = store.as_strided((1, n // 2, 1, 128), (0, gap, 128, 1))
    v = store.as_strided((1, n // 2, 1, 128), (0, gap, 128, 1), 128)
    k0, v0 = rand(g, 1, n // 2, 1, 128), rand(g, 1, n // 2, 1, 128)
    wide.copy_(k0)
    v.copy_(v0)
    q = rand(g, 1, 3, 2, 128)
    assert torch.equal(ops.cross_attention(q, (wide, v)), ops.cross_attention(q, (k0, v0)))


def test_lengths_out_of_range_are_clamped_and_reported(ops):
    g = gen(17)
    q, k, v = rand(g, 3, 2, 4, 64), rand(g, 3, 30, 1, 64), rand(g, 3, 30, 1, 64)
    want = ops.cross_attention(q, (k, v), lens=ints([30, 0, 5]))
    assert ops.status() == (0, 0)
    got = ops.cross_attention(q, (k, v), lens=ints([31, -2, 5]))
    assert torch.equal(got, want)
    assert ops.status() == (0, 4)


# ------------------------------------------------------------------------- refusals


def test_refusals(ops):
    from flow_matching_action_dm0_b200 import QuantizedKV, RtvError
    g = gen(18)
    q, k, v = rand(g, 2, 3, 4, 64), rand(g, 2, 10, 2, 64), rand(g, 2, 10, 2, 64)
    cache = empty_cache(2, 10, 2, 64)

    def refused(status, call, *a, **kw):
        with pytest.raises(RtvError) as e:
            call(*a, **kw)
        assert e.value.status == status, str(e.value)

    refused(8, ops.cross_attention, rand(g, 1, 1, 1, 96), (rand(g, 1, 2, 1, 96), rand(g, 1, 2, 1, 96)))
    refused(2, ops.cross_attention, q[:, :, :3].contiguous(), (k, v))                    # 3 heads on 2
    refused(2, ops.cross_attention, q[:1], (k, v))                                       # another batch
    refused(1, ops.cross_attention, q.float(), (k, v))                                   # mixed types
    refused(1, ops.cross_attention, q, (k, v), scale=float("nan"))
    refused(2, ops.write, cache, k, v, start=1)                                          # past the end
    refused(2, ops.write, cache, k, v, start=-1)
    refused(2, ops.read, cache, n=5, first=6)
    refused(2, ops.write, cache, k[:1], v[:1])
    refused(8, ops.shared_attention, rand(g, 1, 1, 1, 80), (rand(g, 4, 1, 80), rand(g, 4, 1, 80)))
    odd = torch.zeros(2 * 10 * 2 * 64 + 4, dtype=torch.bfloat16, device=DEV)[4:].view(2, 10, 2, 64)   # 8 bytes off
    refused(1, ops.cross_attention, q, (odd, odd))
    thin = torch.zeros((2, 10, 2, 68), dtype=torch.bfloat16, device=DEV)[..., :64]       # rows of 136 bytes
    refused(1, ops.cross_attention, q, (thin, thin))
    still = k[:, :1].expand(2, 10, 2, 64)                                                # token stride 0
    refused(1, ops.cross_attention, q, (still, still))
    with pytest.raises(ValueError):
        ops.cross_attention(q, (k, v.transpose(1, 2).contiguous().transpose(1, 2)))      # other strides
    with pytest.raises(ValueError):
        ops.cross_attention(q, (k, v), lens=ints([1, 2, 3]))
    with pytest.raises(ValueError):
        ops.cross_attention(q, (k.cpu(), v.cpu()))
    with pytest.raises(TypeError):
        ops.cross_attention(q.half(), (k, v))
    with pytest.raises(TypeError):
        ops.write(cache, k.half(), v.half())
    with pytest.raises(TypeError):
        ops.cross_attention(q, QuantizedKV(cache.k.view(torch.uint8), cache.v, cache.k_scale, cache.v_scale))
    assert ops.status() == (0, 0)


def test_empty_calls(ops):
    g = gen(19)
    k, v = rand(g, 2, 10, 2, 64), rand(g, 2, 10, 2, 64)
    assert ops.cross_attention(rand(g, 2, 0, 4, 64), (k, v)).shape == (2, 0, 4, 64)
    out, lse = ops.cross_attention(rand(g, 2, 3, 4, 64), (k[:, :0], v[:, :0]), lse=True)
    assert (out == 0).all() and (lse == -float("inf")).all()
    cache = empty_cache(2, 10, 2, 64)
    ops.write(cache, k[:, :0], v[:, :0])
    assert (cache.k_scale == 0).all()
    assert ops.read(cache, n=0)[0].shape == (2, 0, 2, 64)


def test_host_pointers_are_refused_before_anything_runs(ops):
    import ctypes as C

    from flow_matching_action_dm0_b200 import _lib as L
    host = torch.zeros((1, 4, 1, 64), dtype=torch.bfloat16)
    dev = host.cuda()
    kv = lambda t: L.rtv_kv(t.data_ptr(), t.data_ptr(), None, None, L.RTV_BF16, 1, 4, 1, 64, 256, 64, 64)  # noqa: E731
    qs = lambda t, o: L.rtv_queries(t.data_ptr(), o.data_ptr(), None, L.RTV_BF16, 1, 4, 1, 64, 256, 64, 64, 256, 64, 64, 0.1)  # noqa: E731
    lib = L.load_library()
    for q, k in ((qs(host, dev), kv(dev)), (qs(dev, host), kv(dev)), (qs(dev, dev), kv(host))):
        assert lib.rtv_cross_attention(ops.h, C.byref(q), C.byref(k), None, None, 0, None, 0, None) == L.RTV_ERR_ARG
        assert b"GPU" in lib.rtv_ops_last_error(ops.h) or b"device" in lib.rtv_ops_last_error(ops.h)


@pytest.mark.parametrize("b,tq,d", [(1, 1, 64), (2, 3, 128), (1, 2, 256), (2, 30, 64)])
def test_value_rows_of_very_different_sizes(ops, b, tq, d):
    """Every other key's values are 2^17 times the others', in dims of their own: the small ones still count in
    theirs, to the weights' step."""
    g = gen(31 + d)
    n, half = 40, d // 2
    q, k = rand(g, b, tq, 4, d, size=0.1), rand(g, b, n, 1, d)
    v = rand(g, b, n, 1, d)
    v[:, 0::2, :, half:] = 0
    v[:, 1::2, :, :half] = 0
    v[:, 0::2] *= 2.0 ** 9
    v[:, 1::2] *= 2.0 ** -8
    cache = empty_cache(b, n, 1, d)
    ops.write(cache, k, v)
    kr, vr = (f64(x) for x in ops.read(cache, dtype="f32"))
    out, lse = ops.cross_attention(q, cache, lse=True)
    check_attention(q, lambda i: [(kr[i], vr[i], np.ones(n, bool))], d ** -0.5, out, lse)


def test_outputs_whose_rows_overlap_are_refused(ops):
    from flow_matching_action_dm0_b200 import QuantizedKV, RtvError
    g = gen(32)
    q, k, v = rand(g, 2, 3, 4, 64), rand(g, 2, 10, 2, 64), rand(g, 2, 10, 2, 64)
    flat = torch.zeros(4096, dtype=torch.bfloat16, device=DEV)
    for shape, stride in (((2, 3, 4, 64), (768, 64, 64, 1)), ((2, 3, 4, 64), (64, 256, 64, 1)), ((2, 3, 4, 64), (768, 256, 56, 1)),
                          ((2, 3, 4, 64), (0, 256, 64, 1))):
        with pytest.raises(RtvError) as e:
            ops.cross_attention(q, (k, v), out=flat.as_strided(shape, stride))
        assert e.value.status == 1
    cache = empty_cache(2, 10, 2, 64)
    with pytest.raises(RtvError) as e:
        ops.write(QuantizedKV(cache.k, cache.v, cache.k_scale[:, :1].expand(2, 2, 10), cache.v_scale[:, :1].expand(2, 2, 10)), k, v)
    assert e.value.status == 1
    with pytest.raises(RtvError) as e:
        ops.write(QuantizedKV(cache.k[:1].expand(2, 2, 10, 64), cache.v[:1].expand(2, 2, 10, 64), cache.k_scale, cache.v_scale), k, v)
    assert e.value.status == 1
    with pytest.raises(RtvError) as e:
        ops.read(cache, out=(flat.as_strided((2, 10, 2, 64), (64, 128, 64, 1)),) * 2)
    assert e.value.status == 1
    assert not flat.any() and (cache.k_scale == 0).all()


def test_places_and_sizes_that_do_not_fit_are_refused(ops):
    g = gen(33)
    k = rand(g, 1, 4, 1, 64)
    cache = empty_cache(1, 8, 1, 64)
    for call in (lambda: ops.write(cache, k, k, start=2 ** 32), lambda: ops.read(cache, n=1, first=2 ** 32),
                 lambda: ops.read(cache, n=3, out=(k, k)), lambda: ops.read(cache, n=-1)):
        with pytest.raises(ValueError):
            call()
    assert (cache.k_scale == 0).all()


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("tk", [130, 260, 520, 1000, 1500, 4000])
def test_key_ranges_join(ops, d, tk):
    """Few units over many keys: two to eight ranges of a unit that join in a cluster, and more by a second launch;
    an element's lengths leave some of them empty, or all."""
    cross_case(ops, "bf16", "bf16", 3, 40, tk, 8, 1, d, lens=[tk, 70, 0], masked=True)
    cross_case(ops, "bf16", "bf16", 1, 17, tk, 1, 1, d)
    cross_case(ops, "bf16", "fp8", 2, 3, tk, 8, 1, d, lens=[1, tk])
    shared_case(ops, "bf16", "bf16", 3, 20, tk, None, 8, 1, d, masked=tk == 1000)
    shared_case(ops, "bf16", "bf16", 2, 40, tk, 130, 8, 1, d, lens=[0, 130], masked=True)


def test_a_nan_in_one_key_range_reaches_its_rows_alone(ops):
    g = gen(34)
    q, k, v = rand(g, 2, 40, 8, 256), rand(g, 2, 1000, 1, 256), rand(g, 2, 1000, 1, 256)
    q[0, 5, 3] = float("nan")
    k[1, 900] = float("inf")
    out, lse = ops.cross_attention(q, (k, v), lens=ints([1000, 900]), lse=True)
    bad = torch.isnan(out).any(-1)
    assert bad[0, 5, 3] and bad.sum() == 1 and torch.isnan(lse[0, 5, 3]) and torch.isfinite(lse).sum() == lse.numel() - 1


@pytest.mark.parametrize("dtype,cache", KINDS)
@pytest.mark.parametrize("tq", [2, 40])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_values_near_the_least_exponents(ops, dtype, cache, tq, d):
    """Values of 2^-112 (E4M3 scales of 2^-120) weigh like any others: 2^112 times them is compared.  The results'
    step near 2^-126 (2^-134 at most) is under 2^-6 of the bound, 2^-8 times the mean of |v|."""
    g = gen(35 + d + tq)
    b, n, shrink = 2, 700, 2.0 ** -112
    q, k = rand(g, b, tq, 8, d, dtype=dtype), rand(g, b, n, 2, d, dtype=dtype)
    v = ((torch.rand((b, n, 2, d), generator=g, device=DEV) * 2 - 1) * shrink).to(T[dtype])
    kv = (k, v)
    if cache == "fp8":
        kv = empty_cache(b, n, 2, d)
        ops.write(kv, k, v)
        assert float(kv.v_scale.max()) <= 2.0 ** -120
        k, v = ops.read(kv, dtype="f32")
    lens = [n, 33]
    out, lse = ops.cross_attention(q, kv, lens=ints(lens), lse=True)
    kn, vn = f64(k), f64(v) / shrink
    check_attention(q, lambda i: [(kn[i], vn[i], visible(n, lens, None, i))], d ** -0.5, out.double() / shrink, lse)


def test_tensors_given_with_a_stream_may_be_released_at_once(ops):
    g = gen(36)
    made = [rand(g, 2, 3, 8, 128), rand(g, 2, 500, 1, 128), rand(g, 2, 500, 1, 128), ints([500, 77])]
    want = ops.cross_attention(made[0], made[1:3], lens=made[3])
    side = torch.cuda.Stream()
    for stream in (side, side.cuda_stream):
        given = [t.clone() for t in made]
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            torch.cuda._sleep(20_000_000)                 # the call waits some 10 ms
        got = ops.cross_attention(given[0], given[1:3], lens=given[3], stream=stream)
        del given
        for t in made:
            torch.empty_like(t).fill_(1)                  # what was released serves again
        torch.cuda.synchronize()
        assert torch.equal(got, want)
