"""The quantized layer for a decoding step's few tokens (qwha_layer_decode)
against the fp64 oracle.

Bars (tests/bars.py): fp32 outputs normwise 1e-5 of the largest; bf16 outputs
element by element 2^-8 |b|, half a step, twice what rounding once costs at
most, and the same 1e-5 of the largest for the fp32 sums. What the fp32 sums
cost: a group's partial sums are of codes offset by up to 2^(b-1) + z, about
six times the centred codes of 4 bits, and each of a row's K products and p
nonzeros rounds at 2^-24 of the partial sum at most: over K = 16384 columns
with errors of either sign 6 * 2^-24 * sqrt(16384) = 4.6e-5 of a typical
product's share, against a row's sum of sqrt(16384) of them: 3.6e-7 of it."""

import numpy as np
import pytest

import oracle as O
import synth
from tests.bars import assert_act_close

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

DEV = "cuda:0"


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
    if a.dtype == np.uint32:
        return torch.from_numpy(a.view(np.int32).copy()).to(DEV)
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


def host(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def positions(rng, d_out, d_in, p, skew):
    """p distinct positions; with skew some rows are empty and some are full."""
    if skew:
        n = np.zeros(d_out, dtype=np.int64)
        left = p
        for at, i in enumerate(rng.permutation(d_out)):
            n[i] = min(left, d_in if at == 0 or rng.random() < 0.3 else rng.integers(0, d_in + 1))
            left -= n[i]
        assert left == 0
        E = np.concatenate([np.stack([np.full(n[i], i), np.sort(rng.choice(d_in, n[i], False))], 1)
                            for i in range(d_out)])
    else:
        at = np.sort(rng.choice(d_out * d_in, p, replace=False))
        E = np.stack([at // d_in, at % d_in], 1)
    row_ptr = np.zeros(d_out + 1, dtype=np.int32)
    np.add.at(row_ptr[1:], E[:, 0], 1)
    return np.cumsum(row_ptr, dtype=np.int64).astype(np.int32), E.astype(np.int32)


def layer(d_out, d_in, bits, group, p, seed, skew=False):
    rng = np.random.default_rng(seed)
    w0 = (0.02 * rng.standard_normal((d_out, d_in))).astype(np.float32)
    qc, s, z = synth.rtn_codes(w0, bits, group)
    row_ptr, E = positions(rng, d_out, d_in, p, skew)
    c = (0.5 * rng.standard_normal(p)).astype(np.float32)
    return dict(words=synth.pack_codes(qc, bits), s=s, z=z, W_Q=synth.rtn_quantize(w0, bits, group),
                E=E, c=c, row_ptr=row_ptr, bits=bits, group=group)


def weights(L):
    return [to_dev(L["words"]), to_dev(L["s"]), to_dev(L["z"]), L["bits"], L["group"]]


def adapter(L):
    return [to_dev(L["row_ptr"]), to_dev(L["E"]), to_dev(L["c"])]


def tokens(T, d_in, act, seed):
    x = np.random.default_rng(seed).standard_normal((T, d_in)).astype(np.float32)
    return synth.f32_to_bf16_bits(x) if act == "bf16" else x


def close(y, x, L, act, alpha=1.0):
    ref = O.layer_forward(synth.act_to_f64(x), L["W_Q"], L["E"], L["c"], alpha)
    assert_act_close(host(y), ref, act, "y")


SHAPES = [  # T, d_out, d_in, bits, group, p
    (1, 37, 64, 4, 32, 40), (1, 1, 64, 4, 64, 1), (1, 256, 256, 4, 64, 2048),
    (1, 300, 4096, 4, 128, 9000), (2, 33, 128, 4, 128, 300), (3, 100, 14336, 4, 128, 5000),
    (5, 200, 64, 2, 64, 700), (7, 130, 320, 4, 64, 2000), (4, 65, 192, 4, 32, 1000),
    (16, 129, 1024, 3, 128, 1500), (17, 257, 1024, 3, 32, 4000), (9, 64, 4096, 8, 128, 3000),
    (31, 70, 448, 8, 64, 900), (33, 96, 512, 4, 64, 0), (64, 300, 128, 4, 32, 300 * 128),
    (64, 128, 2048, 4, 256, 5000), (63, 1, 128, 4, 32, 1), (48, 90, 8192, 2, 64, 9000),
    (1, 50, 16384, 4, 1024, 3000), (15, 20, 16384, 2, 16384, 1000), (1, 5000, 128, 4, 128, 4000),
    (8, 2050, 960, 4, 32, 50000), (6, 2049, 64, 3, 64, 0), (32, 700, 1216, 2, 64, 8000)]


@pytest.mark.parametrize("act", ["bf16", "f32"])
@pytest.mark.parametrize("T,d_out,d_in,bits,group,p", SHAPES)
def test_layer_decode(q, T, d_out, d_in, bits, group, p, act):
    say("layer decode", T, d_out, d_in, bits, group, p, act)
    L = layer(d_out, d_in, bits, group, p, seed=T + d_out + d_in + bits)
    x = tokens(T, d_in, act, T)
    y = q.qwha_layer_decode(to_dev(x), *weights(L), *adapter(L), alpha=0.8)
    torch.cuda.synchronize()
    assert y.shape == (T, d_out)
    close(y, x, L, act, 0.8)


# two tiles of rows a workgroup beside one, the largest transforms in LDS, long
# rows of F beside few rows
LARGE = [  # T, d_out, d_in, bits, group, p
    (1, 4097, 8192, 4, 128, 30000), (1, 4096, 16384, 8, 128, 40000), (1, 4200, 16384, 2, 128, 900),
    (3, 4100, 2048, 2, 32, 20000), (4, 4097, 1024, 3, 64, 9000), (2, 9000, 256, 4, 128, 5000),
    (8, 4085, 4096, 4, 128, 7000), (16, 4000, 192, 8, 64, 9000), (4, 520, 256, 4, 64, 520 * 200),
    (2, 500, 2048, 4, 128, 500 * 600), (1, 8193, 4096, 4, 128, 8193)]


@pytest.mark.parametrize("act", ["bf16", "f32"])
@pytest.mark.parametrize("T,d_out,d_in,bits,group,p", LARGE)
def test_layer_decode_of_many_rows(q, T, d_out, d_in, bits, group, p, act):
    test_layer_decode(q, T, d_out, d_in, bits, group, p, act)


# many tokens of many rows: K split over workgroups
WIDE = [  # T, d_out, d_in, bits, group, p
    (64, 2100, 320, 4, 64, 9000), (33, 2751, 192, 8, 32, 20000), (17, 4130, 128, 3, 64, 0),
    (64, 2065, 1024, 2, 128, 30000), (40, 2750, 4096, 4, 128, 8000), (64, 2049, 64, 4, 32, 5000),
    (63, 1600, 16384, 3, 32, 4000), (50, 2800, 960, 8, 64, 0), (18, 4100, 448, 2, 32, 5000)]


@pytest.mark.parametrize("act", ["bf16", "f32"])
@pytest.mark.parametrize("T,d_out,d_in,bits,group,p", WIDE)
def test_layer_decode_of_many_tokens(q, T, d_out, d_in, bits, group, p, act):
    test_layer_decode(q, T, d_out, d_in, bits, group, p, act)


@pytest.mark.parametrize("act", ["bf16", "f32"])
@pytest.mark.parametrize("T,d_out,d_in,p", [(1, 40, 256, 3000), (3, 19, 1024, 9000),
                                            (20, 64, 128, 4000), (64, 33, 512, 8000)])
def test_rows_without_nonzeros_and_full_rows(q, T, d_out, d_in, p, act):
    say("skewed rows", T, d_out, d_in, p, act)
    L = layer(d_out, d_in, 4, 64, p, seed=T, skew=True)
    assert (np.diff(L["row_ptr"]) == 0).any() and (np.diff(L["row_ptr"]) == d_in).any()
    x = tokens(T, d_in, act, 5)
    y = q.qwha_layer_decode(to_dev(x), *weights(L), *adapter(L), alpha=-1.25)
    torch.cuda.synchronize()
    close(y, x, L, act, -1.25)


@pytest.mark.parametrize("T", [1, 5, 40])
def test_without_an_adapter_and_without_tokens(q, T):
    say("base layer alone", T)
    L = layer(130, 512, 4, 128, 0, seed=4)
    x = tokens(T, 512, "bf16", 6)
    y = torch.full((T, 130), 7.0, dtype=torch.bfloat16, device=DEV)
    got = q.qwha_layer_decode(to_dev(x), *weights(L), y=y)
    torch.cuda.synchronize()
    assert got is y
    close(y, x, L, "bf16")
    none = q.qwha_layer_decode(to_dev(x)[:0], *weights(L))
    assert none.shape == (0, 130)
    with pytest.raises(q.QwhaError, match="qwha_layer_fwd"):
        q.qwha_layer_decode(torch.zeros(65, 512, dtype=torch.bfloat16, device=DEV), *weights(L))


@pytest.mark.parametrize("bits", [2, 3, 4, 8])
def test_any_zero_point(q, bits):
    # zeros outside the codes' range: the groups do not span zero
    say("zero points", bits)
    rng = np.random.default_rng(bits)
    d_out, d_in, group = 75, 256, 64
    codes = rng.integers(0, 2 ** bits, (d_out, d_in)).astype(np.uint8)
    z = rng.integers(-90, 2 ** bits + 90, (d_out, d_in // group)).astype(np.float32)
    s = rng.uniform(1e-3, 1e-2, z.shape).astype(np.float32)
    W = O.dequantize(codes, s, z, group)
    x = tokens(3, d_in, "f32", 1)
    y = q.qwha_layer_decode(to_dev(x), to_dev(synth.pack_codes(codes, bits)), to_dev(s),
                            to_dev(z), bits, group)
    torch.cuda.synchronize()
    # |q - z| reaches a hundred steps, so y's largest entry is far above one
    # product; the fp32 sums' error is relative to it
    assert_act_close(host(y), synth.act_to_f64(x) @ W.astype(np.float64).T, "f32", "y")


def test_agrees_with_the_layer_of_many_tokens(q):
    say("decode against layer_fwd")
    L = layer(384, 1024, 4, 128, 6000, seed=9)
    x = tokens(64, 1024, "bf16", 2)
    a = q.qwha_layer_fwd(to_dev(x), *weights(L), *adapter(L), 1.0)
    for T in (1, 16, 64):
        b = q.qwha_layer_decode(to_dev(x)[:T], *weights(L), *adapter(L), 1.0)
        torch.cuda.synchronize()
        # two roundings to bf16 of fp32 values that differ by 2 * 1e-5 of the
        # largest at most: each is off by half a step, 2^-8 of the larger of the
        # two, so they are apart by a step, 2^-7 |b| (1 + 2^-8), and that
        ref, got = host(a[:T]), host(b)
        bar = 2.0 ** -7 * (1 + 2.0 ** -7) * np.abs(ref) + 2e-5 * np.abs(ref).max()
        assert (np.abs(got - ref) <= bar).all(), T


def test_a_token_does_not_depend_on_the_others(q):
    # a row of x spoilt by infinities leaves the other rows' results alone
    say("independent tokens")
    L = layer(200, 512, 4, 128, 4000, seed=11)
    for act in ("bf16", "f32"):
        for T in (2, 5, 16, 40):
            x = to_dev(tokens(T, 512, act, T))
            a = q.qwha_layer_decode(x, *weights(L), *adapter(L))
            bad = x.clone()
            bad[T // 2] = float("inf")
            b = q.qwha_layer_decode(bad, *weights(L), *adapter(L))
            torch.cuda.synchronize()
            keep = [t for t in range(T) if t != T // 2]
            assert torch.equal(a[keep], b[keep]), (act, T)


@pytest.mark.parametrize("T", [1, 3, 24])
def test_replayed_graph(q, T):
    say("decode graph", T)
    L = layer(520, 768, 4, 64, 9000, seed=13)
    w, a = weights(L), adapter(L)
    x = to_dev(tokens(T, 768, "bf16", 1))
    ws = q.workspace(q.lib.qwha_layer_decode_workspace_bytes(T, 768, 520, 9000), DEV)
    y = torch.empty(T, 520, dtype=torch.bfloat16, device=DEV)
    q.qwha_layer_decode(x, *w, *a, y=y, ws=ws)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        q.qwha_layer_decode(x, *w, *a, y=y, ws=ws)
    for i in range(4):
        x.copy_(to_dev(tokens(T, 768, "bf16", 20 + i)))
        y.zero_()
        g.replay()
        want = q.qwha_layer_decode(x, *w, *a)       # eager, its own workspace
        torch.cuda.synchronize()
        assert torch.equal(y, want), i


def test_two_streams_at_once(q):
    say("decode on two streams")
    L = layer(1024, 1024, 4, 128, 20000, seed=15)
    w, a = weights(L), adapter(L)
    xs = [to_dev(tokens(T, 1024, "bf16", T)) for T in (1, 20)]
    want = [q.qwha_layer_decode(x, *w, *a) for x in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in xs]
    got = [[], []]
    for _ in range(10):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(q.qwha_layer_decode(xs[i], *w, *a))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(y, want[i]) for y in got[i])


def test_workspace_refusal(q):
    # 20 tokens: their transforms go through memory
    L = layer(64, 256, 4, 64, 500, seed=1)
    x = to_dev(tokens(20, 256, "bf16", 2))
    with pytest.raises(q.QwhaError, match="workspace"):
        q.qwha_layer_decode(x, *weights(L), *adapter(L), ws=q.workspace(16, DEV))
