"""qwha_layer_decode with more nonzeros a workgroup than it fetches at once (4096):
every form of the walk over F's nonzeros takes several rounds. Bars as in
test_gpu_decode."""

import numpy as np
import pytest

import synth
from tests.test_gpu_decode import adapter, close, q, say, to_dev, tokens, torch, weights  # noqa: F401

pytestmark = pytest.mark.gpu

ROUND = 4096


def layer_of(counts, d_in, bits, group, seed):
    """A layer whose rows of F have these many nonzeros."""
    rng = np.random.default_rng(seed)
    counts = np.asarray(counts, dtype=np.int64)
    d_out = counts.size
    w0 = (0.02 * rng.standard_normal((d_out, d_in))).astype(np.float32)
    qc, s, z = synth.rtn_codes(w0, bits, group)
    order = np.argsort(rng.random((d_out, d_in)), axis=1) if d_out * d_in < 1 << 22 else None
    cols = [np.sort(order[i, :n] if order is not None else rng.choice(d_in, n, replace=False))
            for i, n in enumerate(counts)]
    E = np.stack([np.repeat(np.arange(d_out), counts), np.concatenate(cols)], 1).astype(np.int32)
    c = (0.1 * rng.standard_normal(E.shape[0])).astype(np.float32)
    row_ptr = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    return dict(words=synth.pack_codes(qc, bits), s=s, z=z, W_Q=synth.rtn_quantize(w0, bits, group),
                E=E, c=c, row_ptr=row_ptr, bits=bits, group=group)


def run(q, counts, rows, T, d_in, act, bits=4, group=128):
    counts = np.asarray(counts)
    pad = np.zeros(-counts.size % rows, dtype=counts.dtype)
    assert np.concatenate([counts, pad]).reshape(-1, rows).sum(1).max() > ROUND
    say("long rows of F", counts.size, rows, T, d_in, act)
    L = layer_of(counts, d_in, bits, group, seed=T + d_in + counts.size)
    x = tokens(T, d_in, act, T)
    y = q.qwha_layer_decode(to_dev(x), *weights(L), *adapter(L), alpha=0.6)
    torch.cuda.synchronize()
    close(y, x, L, act, 0.6)


@pytest.mark.parametrize("act", ["bf16", "f32"])
@pytest.mark.parametrize("T", [1, 3, 20, 64])
def test_a_row_over_a_workgroup(q, T, act):
    run(q, [9000, 0, 16384, 4097, 4096, 8193], 1, T, 16384, act)


@pytest.mark.parametrize("act", ["bf16", "f32"])
@pytest.mark.parametrize("T", [5, 40])
def test_eight_rows_a_workgroup(q, T, act):
    counts = np.full(1100, 700)
    counts[[8, 9, 10]] = [2048, 0, 2048]          # a round that ends inside a row
    counts[16:24] = 0
    run(q, counts, 8, T, 2048, act)


@pytest.mark.parametrize("act", ["bf16", "f32"])
@pytest.mark.parametrize("T", [6, 33])
def test_sixteen_rows_a_workgroup(q, T, act):
    counts = np.full(4100, 290)
    counts[32:48] = 512                           # two rounds to the last entry
    run(q, counts, 16, T, 512, act, bits=2, group=64)


@pytest.mark.parametrize("act", ["bf16", "f32"])
@pytest.mark.parametrize("T,d_in,group", [(1, 4096, 128), (4, 1024, 32), (2, 2048, 64)])
def test_tokens_transformed_by_every_workgroup(q, T, d_in, group, act):
    # short rows on the average, as that form asks for, and a few full ones together
    counts = np.full(800, 8)
    counts[33:40] = d_in
    assert 16 * T * (counts.sum() // counts.size) <= ROUND
    run(q, counts, 16, T, d_in, act, group=group)


@pytest.mark.parametrize("act", ["bf16", "f32"])
def test_tokens_transformed_by_every_workgroup_of_two_tiles(q, act):
    counts = np.full(4130, 8)
    counts[40:60] = 512
    run(q, counts, 32, 3, 512, act)
