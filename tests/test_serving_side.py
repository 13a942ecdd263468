"""The torch side of the serving calls fits one PyTorch; the rest of the binding does without it."""
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PKG = "bit_quantized_attention_sa_b200"


@pytest.mark.parametrize("what", ["missing", "unfit"])
def test_the_binding_without_its_torch_side(libsa, tmp_path, what):
    """Import, calls by ctypes and the serving calls' host-only one work; a serving call says what to do."""
    os.makedirs(tmp_path / PKG)
    for f in os.listdir(os.path.join(ROOT, PKG)):
        if f.endswith(".py") or f == "libsa.so":
            os.symlink(os.path.join(ROOT, PKG, f), tmp_path / PKG / f)
    if what == "unfit":
        (tmp_path / PKG / "_sa_torch.so").write_bytes(b"of another PyTorch")
    code = f"""
import torch
from {PKG} import binding as sa
assert sa.library_path().startswith({str(tmp_path)!r})
assert sa.sa_status_string(0) == "SA_OK" and sa.padded_len(129) == 256
assert sa.sa_rope_frequencies(64, device="cpu")[0].shape == (32,)
try:
    sa.sa_rope(torch.zeros(1, 1, 64), None, torch.zeros(1, dtype=torch.int32), torch.zeros(32, dtype=torch.float64))
except ImportError as e:
    assert "{PKG}.build" in str(e)
else:
    raise SystemExit("no error")
"""
    r = subprocess.run([sys.executable, "-c", code], cwd=tmp_path, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr


def test_another_pytorch_has_it_rebuilt(libsa, tmp_path, monkeypatch):
    from bit_quantized_attention_sa_b200 import build

    built = []
    monkeypatch.setattr(build, "build_torch_ext", built.append)
    build.build()
    assert not built                                     # fresh, as the fixture left it
    note = tmp_path / "fits"
    monkeypatch.setattr(build, "TORCH_EXT_FITS", str(note))
    build.build()
    assert len(built) == 1                               # nobody knows what it was built against
    note.write_text(build._torch_ext_for())
    build.build()
    assert len(built) == 1
    monkeypatch.setattr("importlib.metadata.version", lambda name: "1.0.0")
    build.build()
    assert len(built) == 2
