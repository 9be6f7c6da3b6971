"""The quantized key/value cache (qwha_cache_write, qwha_cache_read,
qwha_cache_attn) against the fp64 oracle, and a decoding step made of them and
qwha_layer_decode.

Bars. What is written is compared exactly: codes, steps and zeros follow from
fp32 numbers by exact rules. Rows read back: without the transform s (q - z) is
rounded once, 2^-24 of the value; with it each of the log2 n stages and the
product round once, (log2 n + 1) 2^-24 of the sum of magnitudes. Outputs in bf16
add 2^-8 of the value, half a step.

Attention: see attn_bar."""

import numpy as np
import pytest

import oracle as O
import synth

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

DEV = "cuda:0"
U = 2.0 ** -24


@pytest.fixture(scope="module")
def q():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import quantization_aware_sparse_amd as qq
    return qq


def say(*a):
    print(*a, flush=True)


def to_dev(a):
    if a.dtype == np.uint16:
        return torch.from_numpy(a.view(np.int16).copy()).to(DEV).view(torch.bfloat16)
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


def host(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def draw(rng, shape, act):
    x = rng.standard_normal(shape).astype(np.float32)
    x[..., 3] *= 8                       # a channel that stands out
    if act == "bf16":
        bits = synth.f32_to_bf16_bits(x)
        return to_dev(bits), synth.bf16_bits_to_f32(bits).astype(np.float64)
    return to_dev(x), x.astype(np.float64)


def pool(rng, n_pages, heads, page, dim, bits):
    """A cache whose every row holds something, on the device and as codes,
    steps and zeros."""
    codes = rng.integers(0, 2 ** bits, (2, n_pages, heads, page, dim)).astype(np.uint8)
    s = rng.uniform(0.01, 0.2, codes.shape[:-1]).astype(np.float32)
    z = rng.integers(0, 2 ** bits, codes.shape[:-1]).astype(np.float32)
    return [pack(codes, bits), to_dev(s), to_dev(z)], [codes, s, z]


def pack(codes, bits):
    w = synth.pack_codes(codes.reshape(-1, codes.shape[-1]), bits)
    return to_dev(w.view(np.int32).reshape(*codes.shape[:-1], -1))


def rows_of(cache, part, slots, page):
    return [a[part, slots // page, :, slots % page] for a in cache]


WRITES = [  # T, heads, dim, page, pages, bits, rotate, act
    (1, 1, 64, 8, 1, 4, True, "bf16"), (1, 8, 128, 16, 3, 4, True, "bf16"),
    (5, 3, 128, 32, 2, 8, True, "f32"), (37, 2, 256, 16, 5, 4, True, "f32"),
    (64, 5, 64, 64, 2, 8, False, "bf16"), (33, 1, 256, 8, 9, 8, False, "f32"),
    (100, 7, 64, 128, 1, 4, False, "f32"), (200, 8, 128, 16, 40, 4, False, "bf16"),
    (3, 16, 256, 1024, 1, 8, True, "bf16"), (19, 5, 64, 16, 4, 4, True, "f32")]


@pytest.mark.parametrize("T,heads,dim,page,pages,bits,rotate,act", WRITES)
def test_write(q, T, heads, dim, page, pages, bits, rotate, act):
    say("cache write", T, heads, dim, page, pages, bits, rotate, act)
    rng = np.random.default_rng(T + dim + bits)
    arrays, (codes, s, z) = pool(rng, pages, heads, page, dim, bits)
    slots = rng.permutation(pages * page)[:T].astype(np.int32)
    if T > 4:   # padding, and slots outside the cache on either side
        slots[[1, 3]] = -1
        slots[2] = pages * page
        slots[4] = np.iinfo(np.int32).min
    live = (slots >= 0) & (slots < pages * page)
    (kt, k), (vt, v) = draw(rng, (T, heads, dim), act), draw(rng, (T, heads, dim), act)
    k[0, 0] = 0.0                         # a row of zeros
    kt[0, 0] = 0.0
    q.qwha_cache_write(kt, vt, to_dev(slots), *arrays, bits, rotate=rotate)
    torch.cuda.synchronize()
    at = slots[live]
    for part, x in enumerate((k, v)):
        qc, ss, zz = O.cache_quantize(x[live], bits, rotate)
        codes[part, at // page, :, at % page] = qc
        s[part, at // page, :, at % page] = ss
        z[part, at // page, :, at % page] = zz
    # the whole cache: rows that no token was written to are as they were
    assert torch.equal(arrays[1].cpu(), torch.from_numpy(s))
    assert torch.equal(arrays[2].cpu(), torch.from_numpy(z))
    assert torch.equal(arrays[0], pack(codes, bits))


@pytest.mark.parametrize("bits", [4, 8])
def test_write_on_the_border_between_two_codes(q, bits):
    # steps of exactly 1 and 2^-k: values on halves round up, one unit in the
    # last place below them rounds down; and steps that are no fp32 fraction
    say("borders", bits)
    rng = np.random.default_rng(7)
    n, qmax = 64, 2 ** bits - 1
    x = rng.integers(0, qmax, (6, 1, n)).astype(np.float32) + np.float32(0.5)
    x[:, :, 0], x[:, :, 1] = 0, qmax
    x[1] = np.nextafter(x[1], np.float32(-1e9))
    x[2] = x[2] * np.float32(2 ** -9)
    x[3] = -x[3]
    x[4] = x[4] * np.float32(0.1)
    x[5] = np.nextafter(x[5] * np.float32(1 / 3), np.float32(1e9))
    arrays = q.qwha_cache_empty(1, 1, 8, n, bits, DEV)
    t = to_dev(x)
    q.qwha_cache_write(t, t, to_dev(np.arange(6, dtype=np.int32)), *arrays, bits, rotate=False)
    torch.cuda.synchronize()
    qc, ss, zz = O.cache_quantize(x, bits, False)
    want = np.zeros((2, 1, 1, 8, n), dtype=np.uint8)
    want[:, 0, 0, :6] = qc[:, 0]
    assert torch.equal(arrays[0], pack(want, bits))
    assert np.array_equal(host(arrays[1])[0, 0, 0, :6], ss[:, 0])
    assert np.array_equal(host(arrays[2])[1, 0, 0, :6], zz[:, 0])


@pytest.mark.parametrize("dim,bits", [(64, 4), (128, 8), (256, 4)])
def test_write_and_read_at_the_ends_of_fp32(q, dim, bits):
    # rows whose sums pass fp32's range though their mean does not, and rows
    # beside its lowest normal numbers. Read back s times a whole number below
    # 2^24 is rounded once, so it is the oracle's value, rounded
    say("ends of fp32", dim, bits)
    rng = np.random.default_rng(dim + bits)
    x = rng.uniform(-1, 1, (6, 1, dim)).astype(np.float32)
    x[0] = 1.0
    x[1] = -1.0
    x[:3] *= np.float32(1.9 * 2.0 ** 126)
    x[3] *= np.float32(2.0 ** -118)
    x[4] *= np.float32(2.0 ** -122)
    x[5] *= np.float32(2.0 ** -140)
    arrays = q.qwha_cache_empty(1, 1, 8, dim, bits, DEV)
    t, slots = to_dev(x), to_dev(np.arange(6, dtype=np.int32))
    q.qwha_cache_write(t, t, slots, *arrays, bits)
    k, _ = q.qwha_cache_read(*arrays, slots, bits, dim, out_dtype=torch.float32)
    torch.cuda.synchronize()
    qc, ss, zz = O.cache_quantize(x, bits, True)
    want = np.zeros((2, 1, 1, 8, dim), dtype=np.uint8)
    want[:, 0, 0, :6] = qc[:, 0]
    assert np.array_equal(host(arrays[1])[0, 0, 0, :6], ss[:, 0])
    assert np.array_equal(host(arrays[2])[1, 0, 0, :6], zz[:, 0])
    assert torch.equal(arrays[0], pack(want, bits))
    assert np.array_equal(host(k), O.cache_dequantize(qc, ss, zz, True).astype(np.float32))


READS = [  # T, heads, dim, page, pages, bits, rotate, act
    (1, 1, 64, 8, 1, 4, True, "bf16"), (1, 8, 128, 16, 3, 8, True, "f32"),
    (77, 3, 128, 32, 2, 4, True, "f32"), (130, 2, 256, 16, 7, 8, True, "bf16"),
    (64, 5, 64, 64, 1, 8, False, "bf16"), (333, 1, 256, 8, 30, 4, False, "f32"),
    (41, 16, 128, 1024, 1, 4, True, "bf16"), (9, 5, 64, 16, 2, 8, True, "f32")]


@pytest.mark.parametrize("T,heads,dim,page,pages,bits,rotate,act", READS)
def test_read(q, T, heads, dim, page, pages, bits, rotate, act):
    say("cache read", T, heads, dim, page, pages, bits, rotate, act)
    rng = np.random.default_rng(T + dim + bits)
    arrays, cache = pool(rng, pages, heads, page, dim, bits)
    slots = rng.integers(0, pages * page, T).astype(np.int32)       # repeated, in any order
    if T > 4:
        slots[[0, 3]] = -1
        slots[T - 1] = pages * page
        slots[4] = np.iinfo(np.int32).max
    dt = torch.bfloat16 if act == "bf16" else torch.float32
    out = q.qwha_cache_read(*arrays, to_dev(slots), bits, dim, rotate=rotate, out_dtype=dt)
    torch.cuda.synchronize()
    live = (slots >= 0) & (slots < pages * page)
    for part, got in enumerate(out):
        assert got.dtype == dt and got.shape == (T, heads, dim)
        got = host(got)
        assert not got[~live].any()
        qc, s, z = rows_of(cache, part, slots[live], page)
        ref = O.cache_dequantize(qc, s, z, rotate)
        size = np.abs((qc - z[..., None].astype(np.float64)) * s[..., None])
        bar = (np.log2(dim) + 1) * U * size.sum(-1, keepdims=True) if rotate else U * np.abs(ref)
        if act == "bf16":
            bar = bar * (1 + 2.0 ** -8) + 2.0 ** -8 * np.abs(ref)
        assert (np.abs(got[live] - ref) <= bar).all()


@pytest.mark.parametrize("act", ["bf16", "f32"])
@pytest.mark.parametrize("T,dim,bits,rotate", [(2051, 64, 4, True), (2050, 64, 8, True),
                                               (1027, 128, 4, False), (1031, 128, 8, True),
                                               (515, 256, 4, True), (517, 256, 8, False)])
def test_read_of_many_rows(q, T, dim, bits, rotate, act):
    # four rows a lane, written past the caches where an instruction fills lines
    assert T * 2 * 16 * dim >= 1 << 22
    test_read(q, T, 16, dim, 16, 5, bits, rotate, act)


@pytest.mark.parametrize("bits,rotate", [(4, True), (8, False)])
def test_offsets_past_32_bits(q, bits, rotate):
    # more than 2^31 words of codes in each part: the last slots
    say("long cache", bits, rotate)
    heads, page, dim = 8, 1024, 128
    n_pages = 2 ** 31 // (heads * page * dim * bits // 32) + 3
    arrays = q.qwha_cache_empty(n_pages, heads, page, dim, bits, DEV)
    assert arrays[0][0].numel() > 2 ** 31
    rng = np.random.default_rng(5)
    last = n_pages * page - 1
    slots = np.array([last, last - 1, last - 1500, 7, last // 2], dtype=np.int32)
    (kt, k), (vt, v) = draw(rng, (5, heads, dim), "bf16"), draw(rng, (5, heads, dim), "bf16")
    q.qwha_cache_write(kt, vt, to_dev(slots), *arrays, bits, rotate=rotate)
    got = q.qwha_cache_read(*arrays, to_dev(slots), bits, dim, rotate=rotate,
                            out_dtype=torch.float32)
    table = to_dev(np.array([[n_pages - 1]], dtype=np.int32))
    lens = to_dev(np.array([page], dtype=np.int32))
    qt, qv = draw(rng, (1, heads, dim), "f32")
    out = q.qwha_cache_attn(qt, *arrays, table, lens, bits, rotate=rotate)
    torch.cuda.synchronize()
    rows = []
    for x, y in zip((k, v), got):
        qc, s, z = O.cache_quantize(x, bits, rotate)
        ref = O.cache_dequantize(qc, s, z, rotate)
        assert np.abs(host(y) - ref).max() <= 1e-5 * np.abs(ref).max()
        full = np.zeros((page, heads, dim))        # slots not written read as zeros
        full[[page - 1, page - 2]] = ref[:2]
        rows.append(full)
    ref = O.attend(qv[0], rows[0], rows[1], dim ** -0.5)
    assert np.abs(host(out)[0] - ref).max() <= 1e-5 * np.abs(ref).max()
    del arrays


def attn_bar(qv, kq, ks, vabs, L, bits, rotate, scale, act, ref):
    """A score is scale * s * sum_j q'_j code_j with codes offset by up to 2^bits
    each way, every product exact and every addition rounded at 2^-24 of its
    partial sum: errors of either sign give sqrt(n) 2^-24 times the root of the
    products' squares, of which 8 standard deviations. An error d of the scores
    moves the weights by a factor of at most exp(2 d) in total, and the output by
    2 d max|v|; the sums over L tokens and the transform add 8 (sqrt(L) + n^1/2)
    2^-24 of max|v|."""
    n = qv.shape[-1]
    turned = qv @ O.sylvester(n) if rotate else qv
    top = abs(scale) * ks.max() * 2 ** (bits + 1) * np.sqrt((turned ** 2).sum(-1).max())
    d = 8 * U * np.sqrt(n) * top / np.sqrt(3)
    bar = vabs * (2 * d + 8 * U * (np.sqrt(L) + np.sqrt(n)))
    return bar + (2.0 ** -8 * np.abs(ref) if act == "bf16" else 0.0)


def attn_case(q, B, heads, per, dim, page, lens, bits, rotate, act, seed, scale=None, extra=0,
              spoil=False):
    """Runs one case: sequences of the given lengths in shuffled pages; `extra`
    more table columns than the longest needs. With spoil everything that no
    sequence uses is NaN or out of range."""
    rng = np.random.default_rng(seed)
    need = [-(-n // page) for n in lens]
    n_pages = max(1, sum(need)) + 2
    arrays, cache = pool(rng, n_pages, heads, page, dim, bits)
    order = rng.permutation(n_pages)
    width = max(1, max(need)) + extra
    table = np.full((B, width), -7 if spoil else 0, dtype=np.int32)
    used = np.zeros((n_pages, page), dtype=bool)
    at = 0
    for b in range(B):
        table[b, :need[b]] = order[at:at + need[b]]
        for t in range(lens[b]):
            used[table[b, t // page], t % page] = True
        at += need[b]
    if spoil:
        for a in arrays[1:]:
            a[:, to_dev(~used)[:, None, :].expand(n_pages, heads, page)] = float("nan")
    qt, qv = draw(rng, (B, heads * per, dim), act)
    out = q.qwha_cache_attn(qt, *arrays, to_dev(table), to_dev(np.array(lens, dtype=np.int32)),
                            bits, rotate=rotate, scale=scale)
    torch.cuda.synchronize()
    assert out.dtype == qt.dtype and out.shape == qt.shape
    got = host(out)
    sc = dim ** -0.5 if scale is None else scale
    for b in range(B):
        if lens[b] == 0:
            assert not got[b].any()
            continue
        t = np.arange(lens[b])
        slots = table[b, t // page].astype(np.int64) * page + t % page
        k, v = (O.cache_dequantize(*rows_of(cache, part, slots, page), rotate) for part in (0, 1))
        ref = O.attend(qv[b], k, v, sc)
        ks = rows_of(cache, 0, slots, page)[1]
        bar = attn_bar(qv[b], None, ks, np.abs(v).max(), lens[b], bits, rotate, sc, act, ref)
        assert (np.abs(got[b] - ref) <= bar).all(), (b, np.abs(got[b] - ref).max(), np.min(bar))


ATTN = [  # heads, per, dim, page, lens, bits, rotate, act
    (1, 1, 64, 8, [1], 4, True, "f32"), (2, 4, 128, 16, [1, 15, 16, 17, 0, 33], 4, True, "bf16"),
    (8, 4, 128, 16, [777], 4, True, "f32"), (1, 3, 64, 32, [31, 32, 33, 63, 64, 65], 8, True, "f32"),
    (3, 5, 128, 64, [200, 0, 1, 64], 8, False, "f32"), (2, 8, 256, 16, [130, 2], 4, True, "f32"),
    (1, 12, 128, 128, [300, 129], 4, False, "bf16"), (2, 16, 64, 8, [9, 8, 7, 100], 4, True, "f32"),
    (16, 1, 64, 32, [501, 0, 3], 8, False, "f32"), (4, 2, 256, 1024, [1025, 5], 8, True, "bf16"),
    (1, 71, 64, 16, [40], 4, True, "f32"), (5, 6, 128, 8, [255, 256, 257], 4, True, "f32"),
    (1, 4, 128, 64, [9001], 4, True, "f32"), (2, 7, 256, 32, [2100, 2048], 8, False, "f32")]


@pytest.mark.parametrize("heads,per,dim,page,lens,bits,rotate,act", ATTN)
def test_attn(q, heads, per, dim, page, lens, bits, rotate, act):
    say("cache attn", heads, per, dim, page, lens, bits, rotate, act)
    attn_case(q, len(lens), heads, per, dim, page, lens, bits, rotate, act,
              seed=heads + per + dim + page)


@pytest.mark.parametrize("bits,dim", [(4, 64), (4, 128), (4, 256), (8, 64), (8, 128), (8, 256)])
def test_attn_of_what_lies_behind_the_sequences(q, bits, dim):
    # NaN steps and zeros in every slot that no sequence uses, table entries out
    # of range behind the last page, a table much wider than needed
    say("spoilt surroundings", bits, dim)
    attn_case(q, 7, 2, 4, dim, 16, [0, 1, 16, 17, 100, 31, 333], bits, True, "f32", seed=bits,
              extra=40, spoil=True)


# short tables and many of them: one workgroup of many waves a sequence and head
ATTN_ALONE = [  # heads, per, dim, page, lens, bits, rotate, act
    (16, 4, 128, 16, [1000, 0, 1, 513, 512, 511, 33, 900, 2, 777], 4, True, "bf16"),
    (8, 1, 128, 64, [250], 8, True, "f32"), (2, 8, 64, 8, [249, 256, 1], 8, False, "f32"),
    (1, 2, 256, 32, [129, 250], 4, True, "bf16"), (1, 1, 64, 1024, [1000] * 130, 4, False, "f32"),
    (40, 1, 64, 16, [1999, 16, 15, 1025, 0], 4, True, "f32"),
    (16, 3, 256, 32, [1500, 31, 32, 33, 700, 0, 1, 2, 257, 255, 256, 1024], 8, True, "bf16"),
    (20, 5, 128, 8, [700, 9, 8, 7, 0, 699], 8, False, "f32")]


@pytest.mark.parametrize("heads,per,dim,page,lens,bits,rotate,act", ATTN_ALONE)
def test_attn_of_short_sequences(q, heads, per, dim, page, lens, bits, rotate, act):
    say("cache attn, short", heads, per, dim, page, lens[:12], bits, rotate, act)
    attn_case(q, len(lens), heads, per, dim, page, lens, bits, rotate, act,
              seed=heads + per + dim + page, spoil=True)


def test_attn_scale_and_extreme_scores(q):
    say("scales")
    # with a large scale one token takes all the weight, exp of the rest underflows
    for scale in (0.0, -0.5, 3.0):
        attn_case(q, 2, 2, 2, 64, 16, [50, 7], 8, False, "f32", seed=3, scale=scale)


def test_attn_missing_pages_and_lengths_past_the_table(q):
    say("missing pages")
    rng = np.random.default_rng(2)
    heads, per, dim, page, bits = 2, 3, 128, 16, 4
    arrays, cache = pool(rng, 6, heads, page, dim, bits)
    table = np.array([[2, -1, 4, 99], [5, 0, 1, 3], [-5, 6, 2 ** 30, -1]], dtype=np.int32)
    lens = np.array([60, 1000, 64], dtype=np.int32)
    qt, qv = draw(rng, (3, heads * per, dim), "f32")
    out = host(q.qwha_cache_attn(qt, *arrays, to_dev(table), to_dev(lens), bits))
    torch.cuda.synchronize()
    for b in range(2):
        t = np.arange(min(lens[b], 64))
        t = t[(table[b, t // page] >= 0) & (table[b, t // page] < 6)]
        slots = table[b, t // page] * page + t % page
        k, v = (O.cache_dequantize(*rows_of(cache, part, slots, page), True) for part in (0, 1))
        ref = O.attend(qv[b], k, v, dim ** -0.5)
        ks = rows_of(cache, 0, slots, page)[1]
        bar = attn_bar(qv[b], None, ks, np.abs(v).max(), len(t), bits, True, dim ** -0.5, "f32", ref)
        assert (np.abs(out[b] - ref) <= bar).all()
    assert not out[2].any()
    neg = q.qwha_cache_attn(qt, *arrays, to_dev(table), to_dev(np.array([-3, 0, 0], np.int32)), bits)
    torch.cuda.synchronize()
    assert not host(neg).any()


def test_empty_calls(q):
    arrays = q.qwha_cache_empty(2, 3, 16, 64, 4, DEV)
    none = torch.empty(0, 3, 64, device=DEV)
    slots = torch.empty(0, dtype=torch.int32, device=DEV)
    q.qwha_cache_write(none, none, slots, *arrays, 4)
    k, v = q.qwha_cache_read(*arrays, slots, 4, 64)
    assert k.shape == v.shape == (0, 3, 64)
    table = torch.empty(0, 4, dtype=torch.int32, device=DEV)
    assert q.qwha_cache_attn(none, *arrays, table, slots, 4).shape == (0, 3, 64)


def test_attn_graph_with_growing_lengths(q):
    say("attn graph")
    rng = np.random.default_rng(4)
    heads, per, dim, page, bits, B = 2, 4, 128, 16, 4, 3
    arrays, _ = pool(rng, 90, heads, page, dim, bits)
    table = to_dev(rng.permutation(90).reshape(3, 30).astype(np.int32))
    lens = torch.tensor([1, 100, 479], dtype=torch.int32, device=DEV)
    qt, _ = draw(rng, (B, heads * per, dim), "bf16")
    out = torch.empty_like(qt)
    need = q.lib.qwha_cache_attn_workspace_bytes(B, heads * per, heads, dim, 30, page)
    ws = q.workspace(need, DEV)
    q.qwha_cache_attn(qt, *arrays, table, lens, bits, out=out, ws=ws)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        q.qwha_cache_attn(qt, *arrays, table, lens, bits, out=out, ws=ws)
    for i in range(5):
        out.zero_()
        g.replay()
        want = q.qwha_cache_attn(qt, *arrays, table, lens, bits)
        torch.cuda.synchronize()
        assert torch.equal(out, want), i
        lens += torch.tensor([7, 90, -60], dtype=torch.int32, device=DEV)
        qt.copy_(draw(rng, tuple(qt.shape), "bf16")[0])


def test_attn_on_two_streams(q):
    say("attn on two streams")
    rng = np.random.default_rng(6)
    arrays, _ = pool(rng, 64, 2, 32, 64, 8)
    table = to_dev(rng.permutation(64).reshape(2, 32).astype(np.int32))
    lens = [to_dev(np.array(n, np.int32)) for n in ([1024, 3], [500, 900])]
    qs = [draw(rng, (2, 8, 64), "f32")[0] for _ in range(2)]
    want = [q.qwha_cache_attn(a, *arrays, table, n, 8) for a, n in zip(qs, lens)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in qs]
    got = [[], []]
    for _ in range(10):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(q.qwha_cache_attn(qs[i], *arrays, table, lens[i], 8))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(y, want[i]) for y in got[i])


def test_decoding_steps_of_an_attention_block(q):
    """q, k and v projections with their adapters, the cache, attention and the o
    projection, captured once and replayed while the sequences grow; every stage
    against the oracle's on what the stage before it gave."""
    from tests.test_gpu_decode import adapter, close, layer, weights
    say("decoding steps")
    B, hidden, heads, q_heads, dim, page, bits = 3, 256, 2, 8, 64, 8, 4
    rng = np.random.default_rng(8)
    Ls = {n: layer(o, i, 4, 64, 3000, seed=ord(n)) for n, o, i in
          (("q", q_heads * dim, hidden), ("k", heads * dim, hidden), ("v", heads * dim, hidden),
           ("o", hidden, q_heads * dim))}
    dev = {n: (weights(L), adapter(L)) for n, L in Ls.items()}
    arrays = q.qwha_cache_empty(12, heads, page, dim, bits, DEV)
    table = rng.permutation(12).reshape(3, 4).astype(np.int32)
    x = torch.zeros(B, hidden, dtype=torch.bfloat16, device=DEV)
    slots, lens = (torch.zeros(B, dtype=torch.int32, device=DEV) for _ in range(2))
    tab = to_dev(table)
    got = {}

    def step():
        for n in "qkv":
            got[n] = q.qwha_layer_decode(x, *dev[n][0], *dev[n][1])
        k, v = (got[n].view(B, heads, dim) for n in "kv")
        q.qwha_cache_write(k, v, slots, *arrays, bits)
        got["a"] = q.qwha_cache_attn(got["q"].view(B, q_heads, dim), *arrays, tab, lens, bits)
        got["o"] = q.qwha_layer_decode(got["a"].view(B, q_heads * dim), *dev["o"][0], *dev["o"][1])

    slots.fill_(-1)
    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    have = np.array([0, 5, 20])                 # tokens so far: none written for the first ones
    cache = [np.zeros((2, 12, heads, page, dim), np.uint8), np.zeros((2, 12, heads, page), np.float32),
             np.zeros((2, 12, heads, page), np.float32)]
    for i in range(6):
        bits16 = synth.f32_to_bf16_bits(rng.standard_normal((B, hidden)).astype(np.float32))
        x.copy_(to_dev(bits16))
        at = table[np.arange(B), have // page] * page + have % page
        slots.copy_(to_dev(at.astype(np.int32)))
        have = have + 1
        lens.copy_(to_dev(have.astype(np.int32)))
        g.replay()
        torch.cuda.synchronize()
        for n in "qkv":
            close(got[n], bits16, Ls[n], "bf16")
        for part, n in enumerate("kv"):
            qc, s, z = O.cache_quantize(host(got[n]).reshape(B, heads, dim), bits, True)
            for a, b in zip(cache, (qc, s, z)):
                a[part, at // page, :, at % page] = b
        assert torch.equal(arrays[0], pack(cache[0], bits))
        a = host(got["a"])
        qv = host(got["q"]).reshape(B, q_heads, dim)
        for b in range(B):
            t = np.arange(have[b])
            sl = table[b, t // page].astype(np.int64) * page + t % page
            k, v = (O.cache_dequantize(*rows_of(cache, part, sl, page), True) for part in (0, 1))
            ref = O.attend(qv[b], k, v, dim ** -0.5)
            ks = rows_of(cache, 0, sl, page)[1]
            bar = attn_bar(qv[b], None, ks, np.abs(v).max(), have[b], bits, True, dim ** -0.5,
                           "bf16", ref)
            assert (np.abs(a[b].reshape(q_heads, dim) - ref) <= bar).all()
        at_bits = got["a"].view(torch.int16).cpu().numpy().view(np.uint16).reshape(B, -1)
        close(got["o"], at_bits, Ls["o"], "bf16")
