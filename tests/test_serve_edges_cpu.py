"""The decode-step operators where their tests on a GPU cannot show a fault (no GPU needed)."""
import glob
import os
import re
import subprocess
import sys

import pytest

from latency_barrier_free_gb300 import build_ext, rra
from test_serve_cpu import FAKE, fields, serve  # noqa: F401

torch = pytest.importorskip("torch")


def source(name):
    text = open(name).read()
    return re.sub(r"//[^\n]*|/\*.*?\*/", "", text, flags=re.S)


def test_no_operator_reads_through_the_non_coherent_path():
    """A grid that is launched before its predecessor has ended may hold on to what that path read of a buffer; the operators
    read each other's results."""
    names = glob.glob(os.path.join(build_ext.CSRC, "serve*.cu*"))
    assert len(names) >= 6
    for name in names:
        text = source(name)
        for word in ("__ldg(", "ld.global.nc", "ld_nc", "__restrict__"):
            assert word not in text, (name, word)


@pytest.fixture
def be(tmp_path, monkeypatch):
    """The build with one small unit, into a folder of its own."""
    monkeypatch.setattr(build_ext, "SOURCES", ["rra_static.cu"])
    monkeypatch.setattr(build_ext, "BUILD", str(tmp_path / "_build"))
    for name, file in (("LIB", "librra.so"), ("NATIVE", "_serve.so"), ("NATIVE_STAMP", "_build/_serve.torch")):
        monkeypatch.setattr(build_ext, name, str(tmp_path / file), raising=False)
    return build_ext


def test_the_library_builds_without_torch(be, tmp_path):
    """In a Python that has none."""
    code = """
import sys
class Hidden:
    def find_spec(self, name, path=None, target=None):
        if name.split(".")[0] == "torch":
            raise ModuleNotFoundError("No module named 'torch'", name="torch")
sys.meta_path.insert(0, Hidden())
sys.path.insert(0, %r)
from latency_barrier_free_gb300 import build_ext as be
be.SOURCES, be.BUILD, be.LIB, be.NATIVE, be.NATIVE_STAMP = ["rra_static.cu"], %r, %r, %r, %r
print(be.build())
assert "torch" not in sys.modules
""" % (build_ext.ROOT, be.BUILD, be.LIB, be.NATIVE, getattr(be, "NATIVE_STAMP", ""))
    p = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True)
    assert p.returncode == 0, p.stderr
    assert os.path.exists(be.LIB) and not os.path.exists(be.NATIVE) and p.stdout.strip() == be.LIB


def test_a_binding_that_does_not_compile_leaves_the_library(be, monkeypatch):
    bad = os.path.join(os.path.dirname(be.LIB), "bad.cpp")
    open(bad, "w").write("#error not today\n")
    monkeypatch.setattr(be, "_native_command", lambda out: ["g++", "-c", bad, "-o", out])
    with pytest.raises(RuntimeError, match="not today"):
        be.build()
    assert os.path.exists(be.LIB) and not os.path.exists(be.NATIVE)


def test_the_binding_is_built_again_for_another_torch(be, monkeypatch):
    built = []
    monkeypatch.setattr(be, "_native_command", lambda out: built.append(out) or ["touch", out])
    be.build()
    be.build()
    assert len(built) == 1 and os.path.exists(be.NATIVE)
    before = os.path.getmtime(be.LIB)
    monkeypatch.setattr(be, "_torch", lambda: "another")
    be.build()
    be.build()
    assert len(built) == 2 and os.path.getmtime(be.LIB) == before
    monkeypatch.setattr(be, "_torch", lambda: "")
    be.build(force=True)
    assert len(built) == 2 and os.path.getmtime(be.LIB) > before


def test_attention_refuses_a_scale_beyond_binary32(serve):  # noqa: F811
    """Scores are binary32 and in units of log2."""
    names = fields("rra_kv_attention_args_t")
    good = [FAKE, 100, 16, 2, 128, 0] + [FAKE] * 7 + [1024, 128] * 2 + [8, 0, 0.1, 0, 8, 8, 1, 100, 1, 0, 0]
    assert len(names) == len(good)
    call = lambda scale: serve._lib().rra_kv_attention(  # noqa: E731
        serve._ATTN.pack(*good[:names.index("scale")], scale, *good[names.index("scale") + 1:]), 0)
    for scale in (0.1, -0.1, 0.0, 2.3e38, -2.3e38, 1e-300):  # no tokens, no requests: nothing is launched
        assert call(scale) == rra.OK
    for scale in (2.4e38, -2.4e38, 1e39, 1e300, float("inf"), float("nan")):
        assert call(scale) == rra.ERR_INVALID_ARG
