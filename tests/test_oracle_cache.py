"""Pins of the oracle's key/value cache to things other than itself: hand-worked
rows, the quantizer's error interval, the transform's inverse, library softmax."""

import numpy as np
import pytest

import oracle as O


def test_hand_row():
    # range [-3, 12] in 15 steps of 1: z = 3, halves round up
    x = np.array([[-3.0, 12.0, 0.5, -0.5, 2.49, -2.5, 0.0, 11.5]])
    q, s, z = O.cache_quantize(x, 4, False)
    assert s[0] == 1.0 and z[0] == 3.0
    assert q[0].tolist() == [0, 15, 4, 3, 5, 1, 3, 15]
    assert O.cache_dequantize(q, s, z, False)[0].tolist() == [-3, 12, 1, 0, 2, -2, 0, 12]


def test_the_range_includes_zero():
    q, s, z = O.cache_quantize(np.array([[10.0, 20.0, 30.0, 15.0]]), 4, False)
    assert s[0] == 2.0 and z[0] == 0.0 and q[0].tolist() == [5, 10, 15, 8]
    q, s, z = O.cache_quantize(np.array([[-10.0, -20.0, -30.0, -15.0]]), 4, False)
    assert s[0] == 2.0 and z[0] == 15.0 and q[0].tolist() == [10, 5, 0, 8]


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("rotate", [False, True])
def test_zero_and_tiny_rows_store_zeros(bits, rotate):
    for x in (np.zeros((2, 64)), np.full((2, 64), 1e-42)):
        q, s, z = O.cache_quantize(x, bits, rotate)
        assert not q.any() and not s.any() and not z.any()
        assert not O.cache_dequantize(q, s, z, rotate).any()


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("n", [64, 128, 256])
def test_error_interval_and_inverse(bits, n):
    x = np.random.default_rng(n + bits).standard_normal((50, n)).astype(np.float32)
    q, s, z = O.cache_quantize(x, bits, False)
    err = O.cache_dequantize(q, s, z, False) - x
    # half a step either way, and half more where the range's end and the zero
    # point are both rounded
    assert np.abs(err).max() <= 1.0 * s.max() + 1e-6
    assert np.mean(np.abs(err) <= 0.5 * s[:, None] * (1 + 1e-5)) > 0.9
    # through the transform: the inverse of x H / n is v H
    q, s, z = O.cache_quantize(x, 8, True)
    err = O.cache_dequantize(q, s, z, True) - x
    assert np.linalg.norm(err) <= 0.02 * np.linalg.norm(x)


def test_the_transform_spreads_a_channel_that_stands_out():
    x = np.random.default_rng(1).standard_normal((200, 128))
    x[:, 17] *= 30
    e = []
    for rotate in (False, True):
        q, s, z = O.cache_quantize(x, 4, rotate)
        d = np.delete(O.cache_dequantize(q, s, z, rotate) - x, 17, axis=1)
        e.append(np.linalg.norm(d))
    assert e[1] < e[0]


def test_attend_matches_the_library():
    torch = pytest.importorskip("torch")
    rng = np.random.default_rng(3)
    q, k, v = rng.standard_normal((6, 64)), rng.standard_normal((9, 2, 64)), rng.standard_normal((9, 2, 64))
    got = O.attend(q, k, v, 0.3)
    kk, vv = (torch.from_numpy(a).permute(1, 0, 2).repeat_interleave(3, 0) for a in (k, v))
    a = torch.softmax(0.3 * (kk @ torch.from_numpy(q)[:, :, None])[..., 0], -1)
    assert np.allclose(got, (a[:, None] @ vv)[:, 0].numpy(), rtol=1e-12, atol=1e-13)
    assert not O.attend(q, k[:0], v[:0], 0.3).any()
