"""The compiled binding is a file of its own: the calls that do without it work without it, and one
made for another torch or Python is never loaded."""
import glob
import os
import shutil
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PKG = os.path.join(ROOT, "bit_weight_gemv_gb300")

PROBE = """
import torch, bit_weight_gemv_gb300 as lb
assert lb.__file__.startswith({home!r}), lb.__file__
assert lb.lowbit_int4_packed_bytes(256, 512) > 0
t = torch.zeros(4, dtype=torch.int8)
try:
    lb.lowbit_pack_int4(t, t, 1, 128, t)
except TypeError as e:
    print("int4:", e)
for call in (lambda: lb.lowbit_sample(t, t, t), lambda: lb.lowbit_paged_attention(t, C, t, t, t, t, t),
             lambda: lb.lowbit_kv_append(t, t, t, t, t, t, t, C, t)):
    class C:
        address, head_dim = 0, 64
    try:
        call()
    except ImportError as e:
        print("no binding:", e)
"""


@pytest.fixture(scope="module")
def built():
    from bit_weight_gemv_gb300 import build
    build.build()
    return build


@pytest.fixture
def copy(built, tmp_path):
    """The package's Python files and library in a place of their own."""
    home = tmp_path / "bit_weight_gemv_gb300"
    home.mkdir()
    for f in glob.glob(os.path.join(PKG, "*.py")) + [built.LIB]:
        shutil.copy(f, home)
    return home


def probe(home):
    r = subprocess.run([sys.executable, "-c", PROBE.format(home=str(home))], capture_output=True, text=True, timeout=300,
                       cwd=home.parent, env={**os.environ, "PYTHONPATH": str(home.parent)})
    return r.stdout.splitlines(), r.stderr


def test_other_calls_do_without_the_binding(copy):
    out, err = probe(copy)
    assert len(out) == 4 and out[0].startswith("int4:"), (out, err)
    for line in out[1:]:
        assert "is missing" in line and "bit_weight_gemv_gb300.build" in line


def test_a_binding_for_another_torch_is_not_loaded(built, copy):
    own = os.path.basename(built.binding_path())
    for name in ("_binding.so", own.replace("torch", "torch0."), own.replace("cpython-", "cpython-9")):
        assert name != own
        (copy / name).write_bytes(b"not for this torch")   # loading it would fail
    out, err = probe(copy)
    assert len(out) == 4 and all("is missing" in line for line in out[1:]), (out, err)


def test_a_binding_that_does_not_load_says_so(built, copy):
    (copy / os.path.basename(built.binding_path())).write_bytes(b"no module")
    out, err = probe(copy)
    assert len(out) == 4 and all("does not load" in line for line in out[1:]), (out, err)


def test_the_name_is_that_of_this_torch(built, monkeypatch):
    import torch
    mine = built.binding_path()
    assert torch.__version__ in mine and f"cpython-{sys.version_info[0]}{sys.version_info[1]}" in mine
    assert os.path.exists(mine)
    monkeypatch.setattr(torch, "__version__", "99.0.0")
    assert built.binding_path() != mine and not os.path.exists(built.binding_path())
