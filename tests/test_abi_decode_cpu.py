"""The decoding calls on the CPU: what their host-side checks refuse, with the
documented status, before anything reaches the GPU; and what the binding
refuses. No compute call is made."""

import os

import pytest

from tests.conftest import ROOT

LIB = os.path.join(ROOT, "quantization_aware_sparse_amd", "libqwha.so")
OK, INVALID, SHAPE, BUDGET, DTYPE, ALIGN, WORKSPACE, HIP = range(8)
FAKE = 0x10000          # aligned, never dereferenced (validation fails first)


@pytest.fixture(scope="module")
def q():
    if not os.path.exists(LIB):
        pytest.fail("libqwha.so is not built (run __graft_entry__.build())")
    from quantization_aware_sparse_amd import _lib
    return _lib.lib


def test_layer_decode_validation(q):
    def call(**kw):
        a = dict(x=FAKE, act=1, T=20, d_in=256, d_out=64, codes=FAKE, s=FAKE, z=FAKE, bits=4,
                 group=128, p=500, row_ptr=FAKE, E=FAKE, c=FAKE, alpha=1.0, y=FAKE, ws=FAKE,
                 wsb=0)
        a.update(kw)
        return q.qwha_layer_decode(a["x"], a["act"], a["T"], a["d_in"], a["d_out"], a["codes"],
                                   a["s"], a["z"], a["bits"], a["group"], a["p"], a["row_ptr"],
                                   a["E"], a["c"], a["alpha"], a["y"], a["ws"], a["wsb"], None)
    need = q.qwha_layer_decode_workspace_bytes(20, 256, 64, 500)
    assert need > 0
    assert call() == WORKSPACE
    assert call(wsb=need - 1) == WORKSPACE
    assert call(ws=FAKE + 16, wsb=need) == ALIGN
    assert call(T=65) == SHAPE and call(T=-1) == SHAPE
    assert b"qwha_layer_fwd" in (call(T=65), q.qwha_last_error())[1]
    assert call(d_in=32, group=32) == SHAPE
    assert call(d_in=100) == SHAPE
    assert call(d_out=0) == SHAPE
    assert call(group=16) == INVALID and call(group=96) == INVALID and call(group=512) == INVALID
    assert call(d_in=320, group=128) == INVALID
    assert call(bits=5) == INVALID
    assert call(act=2) == DTYPE
    assert call(p=-1) == BUDGET and call(p=64 * 256 + 1) == BUDGET
    assert call(alpha=float("inf")) == INVALID
    assert call(codes=None) == INVALID and call(codes=FAKE + 4) == ALIGN
    assert call(c=None) == INVALID and call(row_ptr=FAKE + 2) == ALIGN
    assert call(x=FAKE + 2) == ALIGN and call(y=None) == INVALID
    assert call(T=0, x=None, y=None, ws=None) == OK
    assert q.qwha_layer_decode_workspace_bytes(65, 256, 64, 1) == 0
    assert q.qwha_layer_decode_workspace_bytes(-1, 256, 64, 1) == 0


def _cache(**kw):
    a = dict(k=FAKE, v=FAKE, act=1, T=5, slots=FAKE, heads=8, dim=128, bits=4, rotate=1,
             n_pages=10, page=16, codes=FAKE, s=FAKE, z=FAKE)
    a.update(kw)
    return a


CACHE_REFUSALS = [
    (dict(heads=0), SHAPE), (dict(heads=4097), SHAPE), (dict(dim=96), SHAPE),
    (dict(dim=512), SHAPE), (dict(bits=3), INVALID), (dict(rotate=2), INVALID),
    (dict(page=4), SHAPE), (dict(page=24), SHAPE), (dict(page=2048), SHAPE),
    (dict(n_pages=0), SHAPE), (dict(n_pages=2 ** 31 // 16), SHAPE), (dict(act=7), DTYPE),
    (dict(codes=None), INVALID), (dict(codes=FAKE + 8), ALIGN), (dict(s=FAKE + 2), ALIGN),
    (dict(z=None), INVALID)]


@pytest.mark.parametrize("kw,status", CACHE_REFUSALS + [
    (dict(T=-1), SHAPE), (dict(T=2 ** 28), SHAPE), (dict(k=None), INVALID),
    (dict(v=FAKE + 8), ALIGN), (dict(slots=FAKE + 1), ALIGN), (dict(T=0, k=None, v=None), OK)])
def test_cache_write_and_read_validation(q, kw, status):
    a = _cache(**kw)
    assert q.qwha_cache_write(a["k"], a["v"], a["act"], a["T"], a["slots"], a["heads"], a["dim"],
                              a["bits"], a["rotate"], a["n_pages"], a["page"], a["codes"], a["s"],
                              a["z"], None) == status
    assert q.qwha_cache_read(a["codes"], a["s"], a["z"], a["heads"], a["dim"], a["bits"],
                             a["rotate"], a["n_pages"], a["page"], a["slots"], a["T"], a["act"],
                             a["k"], a["v"], None) == status


@pytest.mark.parametrize("kw,status", CACHE_REFUSALS + [
    (dict(B=-1), SHAPE), (dict(B=65536), SHAPE), (dict(q_heads=12), SHAPE),
    (dict(q_heads=0), SHAPE), (dict(width=0), SHAPE), (dict(width=2 ** 31 // 16), SHAPE),
    (dict(scale=float("nan")), INVALID), (dict(q=None), INVALID), (dict(q=FAKE + 4), ALIGN),
    (dict(table=None), INVALID), (dict(lens=FAKE + 2), ALIGN), (dict(out=None), INVALID),
    (dict(B=0, q=None, out=None, table=None), OK)])
def test_cache_attn_validation(q, kw, status):
    a = _cache(B=3, q_heads=32, q=FAKE, table=FAKE, width=4, lens=FAKE, scale=0.1, out=FAKE)
    a.update(kw)
    assert q.qwha_cache_attn(a["q"], a["act"], a["B"], a["q_heads"], a["codes"], a["s"], a["z"],
                             a["heads"], a["dim"], a["bits"], a["rotate"], a["n_pages"], a["page"],
                             a["table"], a["width"], a["lens"], a["scale"], a["out"], FAKE,
                             1 << 40, None) == status


def test_cache_attn_workspace(q):
    need = q.qwha_cache_attn_workspace_bytes
    assert need(65536, 32, 8, 128, 4, 16) == 0
    assert need(1, 12, 8, 128, 4, 16) == 0
    assert need(1, 8, 8, 96, 4, 16) == 0
    big = need(1, 32, 8, 128, 1 << 16, 16)
    if big:
        a = _cache(q=FAKE, table=FAKE, lens=FAKE, out=FAKE)
        def call(ws, wsb):
            return q.qwha_cache_attn(FAKE, 1, 1, 32, FAKE, FAKE, FAKE, 8, 128, 4, 1, a["n_pages"],
                                     16, FAKE, 1 << 16, FAKE, 0.1, FAKE, ws, wsb, None)
        assert call(None, 0) == WORKSPACE
        assert call(FAKE, big - 1) == WORKSPACE
        assert call(FAKE + 16, big) == ALIGN


def test_binding_refusals():
    torch = pytest.importorskip("torch")
    import quantization_aware_sparse_amd as lib
    x = torch.zeros(2, 256, dtype=torch.bfloat16)
    codes = torch.zeros(64, 32, dtype=torch.int32)
    s = torch.zeros(64, 2)
    with pytest.raises(ValueError, match="GPU"):        # no CPU path
        lib.qwha_layer_decode(x, codes, s, s, 4, 128)
    with pytest.raises(ValueError, match="codes"):
        lib.qwha_layer_decode(x, codes[:, :31], s, s, 4, 128)
    with pytest.raises(TypeError, match="codes"):
        lib.qwha_layer_decode(x, codes.long(), s, s, 4, 128)
    with pytest.raises(ValueError, match="groups of"):
        lib.qwha_layer_decode(x, codes, s, s, 4, 64)
    with pytest.raises(ValueError, match="bits"):
        lib.qwha_layer_decode(x, codes, s, s, 5, 128)
    with pytest.raises(ValueError, match="contiguous"):
        lib.qwha_layer_decode(x, torch.zeros(32, 64, dtype=torch.int32).t(), s, s, 4, 128)
    with pytest.raises(TypeError):
        lib.qwha_layer_decode(x.half(), codes, s, s, 4, 128)

    cache = lib.qwha_cache_empty(4, 2, 16, 64, 4, "cpu")
    assert [tuple(t.shape) for t in cache] == [(2, 4, 2, 16, 8), (2, 4, 2, 16), (2, 4, 2, 16)]
    k = torch.zeros(3, 2, 64)
    slots = torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError, match="GPU"):
        lib.qwha_cache_write(k, k, slots, *cache, 4)
    with pytest.raises(ValueError, match="codes"):
        lib.qwha_cache_write(k, k, slots, *cache, 8)
    with pytest.raises(TypeError, match="slots"):
        lib.qwha_cache_write(k, k, slots.long(), *cache, 4)
    with pytest.raises(ValueError, match="v must"):
        lib.qwha_cache_write(k, k[:2], slots, *cache, 4)
    with pytest.raises(ValueError, match="GPU"):
        lib.qwha_cache_read(*cache, slots, 4, 64)
    with pytest.raises(TypeError, match="dtype"):
        lib.qwha_cache_read(*cache, slots, 4, 64, out_dtype=torch.float16)
    table = torch.zeros(3, 2, dtype=torch.int32)
    with pytest.raises(ValueError, match="GPU"):
        lib.qwha_cache_attn(k, *cache, table, slots, 4)
    with pytest.raises(ValueError, match="lens"):
        lib.qwha_cache_attn(k, *cache, table, slots[:2], 4)
    with pytest.raises(TypeError, match="table"):
        lib.qwha_cache_attn(k, *cache, table.long(), slots, 4)
