"""Pins of the cache operators' oracle: the E4M3 grid against torch's float8
cast and worked rows, attention against torch's fp64 attention and closed
forms."""

import numpy as np
import pytest
import torch

from oracle import cache_ops as O


def test_worked_rows():
    codes, scale = O.quantize_rows([[448.0, -1.0, 0.0, 2.0 ** -9], [449.0, 16.0, 17.0, 18.0], [0.0, 0.0, 0.0, 0.0]])
    assert scale.tolist() == [1.0, 2.0, 2.0 ** -126]
    assert codes[0].tolist() == [448.0, -1.0, 0.0, 2.0 ** -9]
    # 224.5 -> 224 (step 16); 8, 8.5 (tie of 8 and 9) -> 8, 9
    assert codes[1].tolist() == [224.0, 8.0, 8.0, 9.0]
    assert codes[2].tolist() == [0.0, 0.0, 0.0, 0.0]


@pytest.mark.parametrize("bad", [np.nan, np.inf, -np.inf])
def test_a_row_that_is_not_finite(bad):
    codes, scale = O.quantize_rows([[1.0, bad], [1.0, 2.0]])
    assert np.isnan(scale[0]) and codes[0].tolist() == [0.0, 0.0]
    assert np.isfinite(scale[1])


def test_every_e4m3_value_is_its_own_code():
    c = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    c = c[np.isfinite(c)]
    codes, scale = O.quantize_rows(c[None])   # holds 448: scale 1
    assert scale[0] == 1.0
    np.testing.assert_array_equal(codes[0], c)


@pytest.mark.parametrize("size", [1e-30, 1e-3, 1.0, 37.0, 1e30])
def test_codes_match_torch_float8(size):
    x = np.random.default_rng(0).standard_normal((64, 128)).astype(np.float32) * np.float32(size)
    codes, scale = O.quantize_rows(x)
    y = torch.from_numpy(x.astype(np.float64) / scale[:, None]).float()   # exact: a power of two
    np.testing.assert_array_equal(codes, y.to(torch.float8_e4m3fn).double().numpy())
    assert np.all(np.abs(x).max(1) <= 448 * scale) and np.all(np.abs(x).max(1) > 224 * scale)
    # half a step of four significand bits, or of the subnormal grid
    assert np.all(np.abs(codes * scale[:, None] - x) <= np.maximum(2.0 ** -4 * np.abs(x), 2.0 ** -10 * scale[:, None]))


def test_attention_matches_torch():
    r = np.random.default_rng(1)
    q, k, v = r.standard_normal((5, 16)), r.standard_normal((11, 16)), r.standard_normal((11, 16))
    w = r.random(11) < 0.6
    out, lse, _ = O.attention(q, [(k[:4], v[:4], w[:4]), (k[4:], v[4:], w[4:])], 0.3)
    t = torch.nn.functional.scaled_dot_product_attention(
        *(torch.from_numpy(x)[None] for x in (q, k, v)), attn_mask=torch.from_numpy(w)[None, None, :].expand(1, 5, 11),
        scale=0.3)[0]
    np.testing.assert_allclose(out, t.numpy(), rtol=0, atol=1e-13)
    np.testing.assert_allclose(lse, torch.logsumexp(0.3 * torch.from_numpy(q) @ torch.from_numpy(k[w]).T, 1).numpy(),
                               rtol=0, atol=1e-13)


def test_attention_without_visible_keys():
    k = np.full((3, 4), np.nan)
    out, lse, size = O.attention(np.ones((2, 4)), [(k, k, np.zeros(3, bool))], 1.0)
    assert np.all(out == 0) and np.all(size == 0) and np.all(lse == -np.inf)
