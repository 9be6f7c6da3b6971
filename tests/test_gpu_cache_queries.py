"""How queries are held in the cache's attention: as whole numbers of 2^(e - 31),
2^e the power of two from the largest component of q' = scale log2(e) q (turned
with rotate) on, or the next one where that component is within 1 % of it. Each
component is off by half a unit at most, 1.02 * 2^-31 of the largest; the sums
over the columns, zeros taken off, are exact until they are joined in fp32.

Bar: half a unit u / 2 at most, with errors of either sign u / sqrt(12) each, of
which 8 standard deviations over the columns' codes; the joined sum and the
products with step and scale round five times at 2^-24 of the score, and fp32 q'
itself once. Softmax and the sums over tokens as in attn_bar: an error d of the
scores moves the output by 2 d max|v|, and 8 (sqrt(L) + sqrt(n)) 2^-24 of max|v|."""

import numpy as np
import pytest

import oracle as O
from tests.test_gpu_cache import DEV, U, draw, host, pack, pool, q, say, to_dev, torch  # noqa: F401

pytestmark = pytest.mark.gpu


def bar(qv, codes, z, s, vabs, scale, L):
    c = codes.astype(np.float64) - z[:, None]
    unit = 2.05 * np.abs(qv).max(-1)[:, None] * 2.0 ** -31
    held = 8 * unit / np.sqrt(12) * np.sqrt((c ** 2).sum(-1))[None]
    size = np.abs(qv[:, None, :] * c[None]).sum(-1)
    d = (abs(scale) * s[None] * (held + 6 * U * size)).max()
    return vabs * (2 * d + 8 * U * (np.sqrt(L) + np.sqrt(qv.shape[-1])))


@pytest.mark.parametrize("L,heads,per", [(40, 2, 4), (700, 1, 7), (300, 20, 2)])
@pytest.mark.parametrize("bits,dim", [(4, 64), (4, 128), (4, 256), (8, 64), (8, 128), (8, 256)])
@pytest.mark.parametrize("above", [1.0, 64.0, 4096.0])
def test_a_channel_that_stands_out(q, L, heads, per, bits, dim, above):
    # the keys hold nothing in the query's largest channel, where every code is the
    # zero point: what the score is made of are the small channels
    say("query channels", L, heads, per, bits, dim, above)
    rng = np.random.default_rng(L + dim + bits)
    page = 16
    n_pages = -(-L // page)
    _, (codes, s, z) = pool(rng, n_pages, heads, page, dim, bits)
    zero = 2 ** bits // 2
    z[:] = zero
    codes[0, ..., 11] = zero
    s[0] = np.float32(3 / (np.sqrt(dim) * 2 ** bits * 0.3) * np.sqrt(dim))   # scores of 3
    arrays = [pack(codes, bits), to_dev(s), to_dev(z)]
    qt, _ = draw(rng, (1, heads * per, dim), "f32")
    qt[..., 3] /= 8
    qt[..., 11] = above * torch.sign(qt[..., 11])
    qv = host(qt)[0]
    table = to_dev(np.arange(n_pages, dtype=np.int32)[None])
    out = q.qwha_cache_attn(qt, *arrays, table, to_dev(np.array([L], np.int32)), bits,
                            rotate=False)
    torch.cuda.synchronize()
    got = host(out)[0]
    t = np.arange(L)
    rows = [[a[p, t // page, :, t % page] for a in (codes, s, z)] for p in (0, 1)]
    k, v = (O.cache_dequantize(*r, False) for r in rows)
    sc = dim ** -0.5
    ref = O.attend(qv, k, v, sc)
    for i in range(heads * per):
        h = i // per
        b = bar(qv[i:i + 1], rows[0][0][:, h], rows[0][2][:, h], rows[0][1][:, h].astype(np.float64),
                np.abs(v[:, h]).max(), sc, L)
        assert np.abs(got[i] - ref[i]).max() <= b, (i, np.abs(got[i] - ref[i]).max(), b)


@pytest.mark.parametrize("up", [-110, -60, 60])
def test_queries_far_from_one(q, up):
    # tiny queries beside large steps and the reverse: the scores are ordinary,
    # and a power of two moves from one to the other without a change
    say("queries of 2^", up)
    rng = np.random.default_rng(9)
    heads, per, dim, page, bits, L = 2, 4, 128, 16, 8, 90
    arrays, _ = pool(rng, 6, heads, page, dim, bits)
    qt, _ = draw(rng, (1, heads * per, dim), "f32")
    table, lens = to_dev(np.arange(6, dtype=np.int32)[None]), to_dev(np.array([L], np.int32))
    want = q.qwha_cache_attn(qt, *arrays, table, lens, bits, rotate=False)
    steps = arrays[1].clone()
    steps[0] *= 2.0 ** -up
    got = q.qwha_cache_attn(qt * 2.0 ** up, arrays[0], steps, arrays[2], table, lens, bits,
                            rotate=False)
    torch.cuda.synchronize()
    assert torch.equal(got, want)
