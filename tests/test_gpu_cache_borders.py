"""Codes of the key/value cache beside a border, at steps whose half is no fp32
number: steps in [2^-126, 2^-125) that are an odd multiple of 2^-149, fp32's
smallest number. Every quantity here is a whole number of 2^-149 units, so the
oracle's fp64 quotients tell the two sides of a border apart."""

import numpy as np
import pytest

import oracle as O
from tests.test_gpu_cache import DEV, host, pack, q, say, to_dev, torch  # noqa: F401

pytestmark = pytest.mark.gpu


def border_rows(bits, n, rng):
    """Rows whose step is an odd number of units, and values on either side of
    its borders."""
    unit, qmax = 2.0 ** -149, 2 ** bits - 1
    rows = []
    tops = [125829136] if bits == 4 else []
    while len(rows) < 6:
        hi = tops.pop() if tops else int(rng.integers(2 ** 23 * qmax, 2 ** 24 * qmax))
        hi = int(np.float32(hi))
        s = int(np.float32(hi * unit) / np.float32(qmax) / unit)
        if s % 2 == 0 or not 2 ** 23 <= s < 2 ** 24:
            continue
        k = rng.integers(0, qmax, n)
        x = np.float32(k * s + s // 2 + rng.integers(0, 2, n)).astype(np.float64)
        x[0], x[1], x[2], x[3] = 0, hi, s // 2, s // 2 + 1
        rows.append(np.float32(np.minimum(x, hi) * unit))
    x = np.stack(rows)
    x[3:] = -x[3:]
    return x[:, None, :]


@pytest.mark.parametrize("bits", [4, 8])
def test_write_where_half_a_step_is_no_fp32_number(q, bits):
    say("borders of tiny steps", bits)
    x = border_rows(bits, 64, np.random.default_rng(bits))
    arrays = q.qwha_cache_empty(1, 1, 8, 64, bits, DEV)
    t = to_dev(x)
    q.qwha_cache_write(t, t, to_dev(np.arange(6, dtype=np.int32)), *arrays, bits, rotate=False)
    torch.cuda.synchronize()
    qc, ss, zz = O.cache_quantize(x, bits, False)
    assert (ss > 0).all()
    want = np.zeros((2, 1, 1, 8, 64), dtype=np.uint8)
    want[:, 0, 0, :6] = qc[:, 0]
    assert np.array_equal(host(arrays[1])[0, 0, 0, :6], ss[:, 0])
    assert np.array_equal(host(arrays[2])[1, 0, 0, :6], zz[:, 0])
    assert torch.equal(arrays[0], pack(want, bits))
