"""What is not finite stays visible: a NaN or an infinity among the values that a
call uses gives NaN in the rows that depend on it, and leaves every other row as
it was, bit for bit."""

import numpy as np
import pytest

import oracle as O
import synth
from tests.test_gpu_cache import DEV, draw, host, pack, pool, q, say, to_dev, torch  # noqa: F401

pytestmark = pytest.mark.gpu

NAN, INF = float("nan"), float("inf")


def odd_nan(dtype):
    """A NaN whose upper mantissa bits are zero but for the type's last one."""
    if dtype == torch.bfloat16:
        return torch.tensor([0x7F81], dtype=torch.int16).view(torch.bfloat16)[0]
    return torch.tensor([0x7F800001], dtype=torch.int32).view(torch.float32)[0]


# ---------------------------------------------------------------- written rows
@pytest.mark.parametrize("act", ["bf16", "f32"])
@pytest.mark.parametrize("dim,bits,rotate", [(64, 4, True), (64, 8, False), (128, 4, False),
                                             (128, 8, True), (256, 4, True), (256, 8, False)])
def test_written_rows(q, dim, bits, rotate, act):
    say("cache write, not finite", dim, bits, rotate, act)
    rng = np.random.default_rng(dim + bits)
    T, heads, page = 24, 3, 16
    (kt, k), (vt, _) = draw(rng, (T, heads, dim), act), draw(rng, (T, heads, dim), act)
    bad = np.zeros((T, heads), dtype=bool)
    for i, what in enumerate([NAN, INF, -INF, odd_nan(kt.dtype)]):
        for j, at in enumerate((0, 17, dim - 1)):       # one in each of a row's lanes
            t, h = 3 * i + j, (i + j) % heads
            kt[t, h, at] = what
            bad[t, h] = True
    kt[12, 1, 5], kt[12, 1, dim - 2] = INF, -INF        # infinities that cancel
    kt[13, 2, :] = NAN
    bad[12, 1] = bad[13, 2] = True
    if not rotate:                                      # a range past the type's
        top = torch.finfo(kt.dtype).max
        kt[14, 0, 0], kt[14, 0, 1] = top, -top
        bad[14, 0] = True
    slots = np.arange(T, dtype=np.int32) + 3
    arrays = q.qwha_cache_empty(2, heads, page, dim, bits, DEV)
    q.qwha_cache_write(kt, vt, to_dev(slots), *arrays, bits, rotate=rotate)
    back = {dt: q.qwha_cache_read(*arrays, to_dev(slots), bits, dim, rotate=rotate, out_dtype=dt)
            for dt in (torch.float32, torch.bfloat16)}
    torch.cuda.synchronize()
    for k_back, v_back in back.values():
        assert np.isnan(host(k_back)[bad]).all()
        assert np.isfinite(host(k_back)[~bad]).all()
        assert np.isfinite(host(v_back)).all()
    # the rows beside them hold what they hold without them
    qc, s, z = O.cache_quantize(np.where(bad[..., None], 0.0, k), bits, rotate)
    want_s, want_z = (np.zeros((2, heads, page), np.float32) for _ in range(2))
    want_c = np.zeros((2, heads, page, dim), np.uint8)
    want_c[slots // page, :, slots % page] = qc
    want_s[slots // page, :, slots % page] = np.where(bad, np.nan, s)
    want_z[slots // page, :, slots % page] = z
    assert np.array_equal(host(arrays[1][0]), want_s, equal_nan=True)
    assert np.array_equal(host(arrays[2][0]), want_z)
    assert torch.equal(arrays[0][0], pack(want_c, bits))

