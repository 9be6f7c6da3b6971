"""What is not finite stays visible: a NaN or an infinity among the values that a
call uses gives NaN in the rows that depend on it, and leaves every other row as
it was, bit for bit. An empty sequence stays a row of zeros."""

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


# ---------------------------------------------------------------- attention
FORMS = [  # heads, per, dim, page, lens, bits, rotate, act
    (2, 4, 128, 16, [100, 0, 33, 1], 4, True, "f32"),           # one workgroup, 4 waves
    (2, 5, 64, 64, [1999, 0, 700], 8, False, "bf16"),           # slices
    (1, 4, 256, 32, [3000, 5], 4, False, "f32"),
    (20, 2, 128, 8, [900, 0, 1, 700, 31, 32, 33], 8, True, "bf16"),   # many waves
    (40, 1, 64, 32, [1500, 0, 2, 40], 4, False, "f32")]         # many waves


class Case:
    def __init__(self, heads, per, dim, page, lens, bits, rotate, act, seed):
        rng = np.random.default_rng(seed)
        self.need = [-(-n // page) for n in lens]
        n_pages = sum(self.need) + 1
        self.arrays, _ = pool(rng, n_pages, heads, page, dim, bits)
        order = rng.permutation(n_pages).astype(np.int32)
        self.table = np.zeros((len(lens), max(self.need)), np.int32)
        at = 0
        for b, n in enumerate(self.need):
            self.table[b, :n] = order[at:at + n]
            at += n
        self.q = draw(rng, (len(lens), heads * per, dim), act)[0]
        self.lens, self.bits, self.rotate, self.page = lens, bits, rotate, page
        self.heads, self.per, self.rng = heads, per, rng

    def run(self, q, qt=None, arrays=None):
        out = q.qwha_cache_attn(self.q if qt is None else qt, *(arrays or self.arrays),
                                to_dev(self.table), to_dev(np.array(self.lens, np.int32)),
                                self.bits, rotate=self.rotate)
        torch.cuda.synchronize()
        return out


@pytest.mark.parametrize("what", [NAN, INF, -INF, "odd"])
@pytest.mark.parametrize("form", range(len(FORMS)))
def test_queries(q, form, what):
    say("cache attn, query not finite", form, what)
    c = Case(*FORMS[form], seed=form)
    want = c.run(q)
    assert torch.isfinite(want).all()
    bad = torch.zeros(want.shape[:2], dtype=torch.bool, device=DEV)
    qt = c.q.clone()
    for b in range(len(c.lens)):
        i = int(c.rng.integers(qt.shape[1]))
        qt[b, i, int(c.rng.integers(qt.shape[2]))] = odd_nan(qt.dtype) if what == "odd" else what
        bad[b, i] = c.lens[b] > 0          # a query without tokens is not used
    got = c.run(q, qt=qt)
    assert torch.isnan(got[bad]).all()
    assert torch.equal(got[~bad], want[~bad])


@pytest.mark.parametrize("what", [NAN, INF, -INF])
@pytest.mark.parametrize("form", range(len(FORMS)))
def test_steps_and_zeros(q, form, what):
    # one step or zero of one row of one key/value head, at either end of a
    # sequence and in its middle: every query head that reads it, and no other
    say("cache attn, row not finite", form, what)
    c = Case(*FORMS[form], seed=10 + form)
    want = c.run(q)
    assert torch.isfinite(want).all()
    b = 0
    for kind in (1, 2):                    # steps, zeros
        for part in (0, 1):
            for t in (0, c.lens[b] // 2, c.lens[b] - 1):
                arrays = [a.clone() for a in c.arrays]
                h = int(c.rng.integers(c.heads))
                arrays[kind][part, c.table[b, t // c.page], h, t % c.page] = what
                got = c.run(q, arrays=arrays)
                bad = torch.zeros(want.shape[:2], dtype=torch.bool, device=DEV)
                bad[b, h * c.per:(h + 1) * c.per] = True
                if part == 0:
                    assert torch.isnan(got[bad]).all(), (kind, t)
                else:
                    assert not torch.isfinite(got[bad]).any(), (kind, t)
                assert torch.equal(got[~bad], want[~bad]), (kind, part, t)


def test_a_row_written_from_a_nan(q):
    # through the cache: the sequence that holds the row shows it, the other does not
    say("nan through the cache")
    rng = np.random.default_rng(1)
    heads, dim, page = 2, 64, 16
    arrays = q.qwha_cache_empty(8, heads, page, dim, 4, DEV)
    (kt, _), (vt, _) = draw(rng, (64, heads, dim), "bf16"), draw(rng, (64, heads, dim), "bf16")
    kt[40, 1, 7] = NAN
    slots = to_dev(np.arange(64, dtype=np.int32))
    q.qwha_cache_write(kt, vt, slots, *arrays, 4)
    table = to_dev(np.array([[0, 1], [2, 3]], np.int32))
    lens = to_dev(np.array([32, 32], np.int32))
    qt, _ = draw(rng, (2, 4, dim), "bf16")
    out = host(q.qwha_cache_attn(qt, *arrays, table, lens, 4))
    torch.cuda.synchronize()
    assert np.isfinite(out[0]).all() and np.isfinite(out[1, :2]).all()
    assert np.isnan(out[1, 2:]).all()


def test_scores_past_fp32_range_weigh_nothing_below_and_show_above(q):
    # finite inputs whose scores pass fp32's range: -inf weighs nothing beside a
    # finite score, +inf shows as NaN
    say("scores past the range")
    dim, page = 64, 8
    codes = np.zeros((2, 1, 1, page, dim), np.uint8)
    codes[0, 0, 0, 0], codes[0, 0, 0, 1] = 15, 0
    s = np.full((2, 1, 1, page), 1.0, np.float32)
    s[0, 0, 0, 0] = 2.0 ** 120
    codes[1, 0, 0, 1] = 3
    z = np.zeros((2, 1, 1, page), np.float32)
    arrays = [pack(codes, 4), to_dev(s), to_dev(z)]
    table, lens = to_dev(np.zeros((1, 1), np.int32)), to_dev(np.array([2], np.int32))
    for sign in (-1.0, 1.0):
        qt = torch.full((1, 1, dim), sign * 2.0 ** 10, device=DEV)
        out = host(q.qwha_cache_attn(qt, *arrays, table, lens, 4, rotate=False))
        torch.cuda.synchronize()
        if sign < 0:
            assert (out == 3.0).all()
        else:
            assert np.isnan(out).all()
