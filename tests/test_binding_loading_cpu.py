"""The package without the compiled binding of the decoding calls, or with one
that does not load: everything else works, the decoding calls say what to do."""

import os
import shutil
import subprocess
import sys

import pytest

from tests.conftest import ROOT

PKG = "quantization_aware_sparse_amd"

PROGRAM = """
import torch
import quantization_aware_sparse_amd as q
assert q.__file__.startswith({at!r}), q.__file__
assert q.lib.qwha_version() == 100
codes, s, z = q.qwha_cache_empty(4, 2, 16, 64, 4, "cpu")
x = torch.zeros(2, 256, dtype=torch.bfloat16)
k = torch.zeros(3, 2, 64)
slots, table = torch.zeros(3, dtype=torch.int32), torch.zeros(3, 2, dtype=torch.int32)
calls = [lambda: q.qwha_layer_decode(x, codes, s, z, 4, 128),
         lambda: q.qwha_cache_write(k, k, slots, codes, s, z, 4),
         lambda: q.qwha_cache_read(codes, s, z, slots, 4, 64),
         lambda: q.qwha_cache_attn(k, codes, s, z, table, slots, 4)]
for call in calls * 2:
    try:
        call()
    except ImportError as e:
        assert "build.py" in str(e), e
    else:
        raise AssertionError("no ImportError")
print("fine")
"""


@pytest.mark.parametrize("binding", [None, b"not a library"])
def test_everything_else_works_without_it(tmp_path, binding):
    at = tmp_path / PKG
    at.mkdir()
    for name in ("__init__.py", "_lib.py"):
        shutil.copy(os.path.join(ROOT, PKG, name), at / name)
    os.symlink(os.path.join(ROOT, PKG, "libqwha.so"), at / "libqwha.so")
    if binding is not None:
        (at / "_binding.so").write_bytes(binding)
    r = subprocess.run([sys.executable, "-c", PROGRAM.format(at=str(at))], cwd=tmp_path,
                       env=dict(os.environ, PYTHONPATH=str(tmp_path)), capture_output=True,
                       text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip().endswith("fine"), r.stdout + r.stderr


def test_with_it_the_calls_are_the_compiled_ones():
    import quantization_aware_sparse_amd as q
    with pytest.raises(TypeError, match="x must be a tensor"):
        q.qwha_layer_decode(None, None, None, None, 4, 128)
    assert q._decoding.__name__ == PKG + "._binding"     # looked up once
